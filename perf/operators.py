"""What is measured of the cache append and of the attention over page scales.

The operators: writing a step's keys and values into the paged fp8 cache with
the rotation of their positions (one scale per tensor, or one scale per page
and KV head that grows with the page), and the block scorer, the attention over
listed pages, its prefill form and dense decode over a cache with page scales.

Layouts are the library's: q [T, Hq, 128], cache fp8 e4m3 [NB, Hkv, 128, 256]
(K in bytes 0-127 of a row, V in 128-255), block_table int32 [B, S], seq_lens
int32 [B], page scales fp32 [NB, Hkv, 2] (K's, then V's), Hq = 16 Hkv."""
import math

import torch

own = False

D, PAGE, TOPK, GROUP = 128, 128, 16, 16
F8 = torch.float8_e4m3fn
TOP = 448.0          # the largest e4m3 value
SM = D ** -0.5
BASE = 10000.0       # base of the rotation's frequencies


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token for each of 16 requests on one KV head (a tensor-parallel
        # shard): the smallest append, all latency
        dict(name="append_b16_q1_h16kv1", op="append", batch=16, qlen=1, hkv=1, lo=2048, hi=3000,
             chunk=0, scaled=False, rot=128, pairs=False, q8=False, pad=False),
        # a decode batch of 128 requests, a tenth of them padding, page scales,
        # the query handed on as fp8
        dict(name="append_scaled_b128_q1_h64kv4", op="append", batch=128, qlen=1, hkv=4, lo=1024,
             hi=65536, chunk=0, scaled=True, rot=64, pairs=False, q8=True, pad=True),
        # chunked prefill: four chunks of 1k-2k tokens
        dict(name="append_prefill_b4_1k-2k", op="append", batch=4, qlen=0, hkv=4, lo=8192,
             hi=32768, chunk=1500, scaled=False, rot=64, pairs=True, q8=False, pad=False),
        # prompts of up to 8k tokens into fresh and begun pages, page scales
        dict(name="append_scaled_prefill_b8_4k", op="append", batch=8, qlen=0, hkv=4, lo=4200,
             hi=8193, chunk=4097, scaled=True, rot=64, pairs=False, q8=False, pad=False),
        # the scorer on the batch-16 step, four speculative tokens a request
        dict(name="score_b16_q4_8k-32k", op="score", batch=16, qlen=4, hkv=4, lo=8192, hi=32768,
             q8=False, pad=False),
        # the scorer where it is bound by the tensor cores: 32 tokens at 256k
        dict(name="score_b2_q32_256k", op="score", batch=2, qlen=32, hkv=4, lo=262144, hi=262144,
             q8=False, pad=False),
        # two short requests, one token each: attend latency
        dict(name="sparse_b2_q1_h16kv1", op="sparse", batch=2, qlen=1, hkv=1, lo=2048, hi=3000,
             q8=False, pad=False),
        # the batch-16 step's attend over its 16 pages a token and head
        dict(name="sparse_b16_q4_8k-32k", op="sparse", batch=16, qlen=4, hkv=4, lo=8192, hi=32768,
             q8=False, pad=False),
        # a short prefill batch beside decode, odd lengths, fp8 query
        dict(name="prefill_b5_short", op="prefill", batch=5, qlen=0, hkv=1, lo=129, hi=5000,
             chunk=37, q8=True, pad=False),
        # chunks of a few hundred tokens, a list for every token
        dict(name="prefill_b4_384", op="prefill", batch=4, qlen=0, hkv=4, lo=8192, hi=32768,
             chunk=384, q8=False, pad=False),
        # the model's dense layers on the batch-16 step
        dict(name="dense_b16_q4_8k-32k", op="dense", batch=16, qlen=4, hkv=4, lo=8192, hi=32768,
             q8=False, pad=False),
        # one request, one token, the longest context dense decode takes
        dict(name="dense_b1_q1_256k", op="dense", batch=1, qlen=1, hkv=4, lo=262144, hi=262144,
             q8=False, pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "score", "sparse", "prefill", "dense"])
    c = dict(op=op, hkv=rng.choice([1, 2, 4]), q8=rng.random() < 0.4, pad=rng.random() < 0.3,
             qlen=0)
    if op == "append":
        c.update(scaled=rng.random() < 0.6, rot=rng.choice([0, 16, 32, 64, 96, 128]),
                 pairs=rng.random() < 0.4, chunk=0)
        if rng.random() < 0.5:
            c.update(qlen=rng.choice([1, 1, 2, 3, 4, 7, 8, 16, 32]), batch=_log(rng, 1, 200))
            c["lo"] = _log(rng, 40, 8000)
            c["hi"] = c["lo"] + _log(rng, 1, 30000)
        else:
            c.update(batch=_log(rng, 1, 24), chunk=_log(rng, 1, 1300))
            c["lo"] = 2 * c["chunk"] + _log(rng, 1, 4000)
            c["hi"] = c["lo"] + _log(rng, 1, 8000)
        return c
    if op == "prefill":
        c.update(batch=_log(rng, 1, 12), chunk=_log(rng, 1, 120))
        c["lo"] = 2 * c["chunk"] + _log(rng, 1, 8000)
        c["hi"] = c["lo"] + _log(rng, 1, 24000)
        return c
    c.update(qlen=rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 13, 16, 32]), batch=_log(rng, 1, 32))
    if op == "sparse":
        c["batch"] = _log(rng, 1, max(1, 512 // c["qlen"]))
    c["lo"] = _log(rng, 40, 8000)
    c["hi"] = c["lo"] + _log(rng, 1, 24000)
    if op != "sparse":      # no more keys times tokens than the largest listed case
        c["batch"] = max(1, min(c["batch"], (1 << 23) // (c["qlen"] * c["hi"])))
    return c


def _lens(c):
    """(seq_lens, query lengths), from the case alone: lengths spread over
    [lo, hi] in an order that is not sorted; of a prefill batch, chunks around
    `chunk`; every tenth request of a padded batch is empty."""
    B = c["batch"]
    at = [(k * 7 + 3) % B if B % 7 else k for k in range(B)]
    lens = [c["lo"] + (c["hi"] - c["lo"]) * k // max(1, B - 1) for k in at]
    if c["pad"]:
        lens = [0 if k % 10 == 4 else n for k, n in enumerate(lens)]
    if c.get("chunk"):
        q = [min(n, max(1, c["chunk"] * (2 + (3 * k) % 5) // 4)) for k, n in enumerate(lens)]
    else:
        q = [c["qlen"]] * B
    return lens, q


def _pages(n):
    return (n + PAGE - 1) // PAGE


# ---------------------------------------------------------------------------
# inputs


def _codes(shape, gen):
    """Random e4m3 codes with the values' spread of a quantised activation."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).mul_(110.0)
    return x.clamp_(-TOP, TOP).to(F8).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, q_lens = _lens(case)
    B, hkv, T = case["batch"], case["hkv"], sum(q_lens)
    hq = GROUP * hkv
    pages = [_pages(n) for n in lens]
    S, NB = max(max(pages), 1), sum(pages) + 1
    perm = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(B)], device="cuda")
    n_pg = torch.tensor(pages, device="cuda")
    at = torch.arange(S, device="cuda")
    table = torch.where(at < n_pg[:, None], perm[(first[:, None] + at).clamp(max=NB - 1)], 0)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s = dict(case=case, qlen=case["qlen"], T=T, hkv=hkv, table=table.to(torch.int32).contiguous(),
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             kv=_codes((NB, hkv, PAGE, 2 * D), gen))
    # page scales around 2^-8, as keys and values of a spread of a half have
    s["scales"] = torch.exp2(torch.randn((NB, hkv, 2), generator=gen, device="cuda") * 0.7 - 8.0)
    if case["op"] == "append":
        s["scales"] = torch.exp2(torch.log2(s["scales"]).round())   # as appends leave them
        # q, k and v are slices of one projection's output
        s["qkv"] = torch.randn((T, (hq + 2 * hkv) * D), generator=gen, device="cuda",
                               dtype=torch.bfloat16).mul_(0.7)
        s["k_scale"], s["v_scale"] = (1.0, 1.0) if case["scaled"] else (0.0071, 0.0068)
        s["q_scale"] = 0.0086
        s["cos_sin"] = None
        if case["rot"]:
            freq = BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
                            / case["rot"])
            ang = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        s["q_out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        if case["q8"]:
            s["q_out"] = s["q_out"].to(F8)
        return s
    q = torch.randn((T, hq, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["q_scale"] = 1.0
    if case["q8"]:
        s["q_scale"] = 0.0123
        q = (q.float() / s["q_scale"]).clamp(-TOP, TOP).to(F8)
    s["q"], s["out"] = q, torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "score":
        s["scores"] = torch.zeros((hkv, T, S), device="cuda")
    if case["op"] in ("sparse", "prefill"):
        s["topk"] = _lists(s, S, gen)
    # room for the parts of a split step, kept by a serving program for its largest batch
    s["work"] = torch.empty(16 * min(T, 320) * hq * (D + 2) * 4, dtype=torch.uint8, device="cuda")
    return s


def _token(s):
    """(request, position) of every token; positions below 0 are padding."""
    b = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(s["T"], dtype=torch.int32, device="cuda"),
                           right=True)
    i = torch.arange(s["T"], device="cuda")
    q_len = (s["cu"][1:] - s["cu"][:-1])[b]
    return b, (s["lens"][b] - q_len + i - s["cu"][b]).long()


def _lists(s, S, gen):
    """Each token's own block and up to 15 distinct earlier ones, ascending."""
    b, pos = _token(s)
    cur = torch.div(pos, PAGE, rounding_mode="floor")
    r = torch.rand((s["T"], s["hkv"], S), generator=gen, device="cuda")
    n = torch.arange(S, device="cuda")
    r = torch.where(n < cur[:, None, None], r, torch.where(n == cur[:, None, None], 2.0, -1.0))
    k = min(S, TOPK)
    val, idx = r.topk(k, dim=2)
    idx = torch.where(val >= 0, idx, 1 << 30).sort(dim=2).values
    out = torch.full((s["T"], s["hkv"], TOPK), -1, dtype=torch.int32, device="cuda")
    out[:, :, :k] = torch.where(idx < (1 << 30), idx, -1).to(torch.int32)
    return out


# ---------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "append":
        return _plain_append(s)
    if op in ("sparse", "prefill"):
        return _plain_listed(s)
    return _plain_every(s)


def _run_own(s):
    import block_sparse_gqa_score_gb300 as msa
    c = s["case"]
    if c["op"] == "append":
        hq, hkv = GROUP * s["hkv"], s["hkv"]
        q, k, v = s["qkv"].view(s["T"], -1, D).split([hq, hkv, hkv], dim=1)
        kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"],
                  kv_scales=s["scales"] if c["scaled"] else None, cos_sin=s["cos_sin"],
                  interleaved=c["pairs"], q=q, q_out=s["q_out"], q_scale=s["q_scale"])
        if c["chunk"]:
            msa.append_kv_prefill(k, v, s["kv"], s["table"], s["lens"], s["cu"], **kw)
        else:
            msa.append_kv(k, v, s["kv"], s["table"], s["lens"], c["qlen"], **kw)
        return _state(s)
    kw = dict(kv_scales=s["scales"], q_scale=s["q_scale"])
    if c["op"] == "score":
        return msa.score(s["q"], s["kv"], s["table"], s["lens"], c["qlen"], SM, scores=s["scores"], **kw)
    if c["op"] == "sparse":
        return msa.sparse_decode(s["q"], s["kv"], s["table"], s["lens"], s["topk"], c["qlen"], SM,
                                 out=s["out"], workspace=s["work"], **kw)
    if c["op"] == "prefill":
        return msa.sparse_prefill(s["q"], s["kv"], s["table"], s["lens"], s["cu"], s["topk"], SM,
                                  out=s["out"], workspace=s["work"], **kw)
    return msa.dense_decode(s["q"], s["kv"], s["table"], s["lens"], c["qlen"], SM, out=s["out"],
                            workspace=s["work"], **kw)


def _state(s):
    """The outputs of an append: the cache's values, its scales, the query."""
    return [s["kv"].view(F8), s["scales"] if s["case"]["scaled"] else None, s["q_out"]]


def _e4m3(x):
    """fp32 -> e4m3, nearest even, saturating."""
    return x.clamp(-TOP, TOP).to(F8)


def _rotate(x, cs, pairs):
    """x [T, H, 128]: its first dims rotated by the table rows cs [T, rot]."""
    h = cs.shape[1] // 2
    c, sn = cs[:, None, :h], cs[:, None, h:]
    if pairs:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    return torch.cat([y, x[..., 2 * h:]], dim=-1)


def _power(amax):
    """The smallest power of two s >= 2^-40 with amax <= 448 s, at most 2^40."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -40).clamp(-40, 40)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append(s):
    c, hkv = s["case"], s["hkv"]
    hq = GROUP * hkv
    b, pos = _token(s)
    live = pos >= 0
    at = pos.clamp(min=0)
    page, row = s["table"][b, at // PAGE].long(), at % PAGE
    x = s["qkv"].view(s["T"], -1, D).float()
    q, k, v = x.split([hq, hkv, hkv], dim=1)
    if c["rot"]:
        cs = s["cos_sin"][at]
        q, k = _rotate(q, cs, c["pairs"]), _rotate(k, cs, c["pairs"])
    q = torch.where(live[:, None, None], q, 0.0)
    s["q_out"].copy_(_e4m3(q * (1.0 / s["q_scale"])) if c["q8"] else q.to(torch.bfloat16))
    x = torch.stack([k, v], dim=2)[live]                               # [T', Hkv, 2, 128]
    page, row = page[live], row[live]
    per = torch.tensor([s["k_scale"], s["v_scale"]], device="cuda")
    if c["scaled"]:
        sc, NB = s["scales"], s["scales"].shape[0]
        amax = torch.zeros_like(sc).index_reduce_(0, page, x.abs().amax(dim=3), "amax")
        start = torch.full((NB,), PAGE, device="cuda").index_reduce_(0, page, row, "amin")
        old = sc.clone()
        new = torch.where(start[:, None, None] > 0, torch.maximum(old, _power(amax)), _power(amax))
        sc.copy_(torch.where((start < PAGE)[:, None, None], new, old))
        # the rows before a request's first token, in the one page it had begun
        at0 = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).clamp(min=0)
        p0 = s["table"][torch.arange(at0.shape[0], device="cuda"), at0 // PAGE].long()[s["lens"] > 0]
        ratio = (old[p0] / sc[p0]).repeat_interleave(D, dim=2)[:, :, None]      # [B', Hkv, 1, 256]
        was = s["kv"][p0].view(F8).float()
        before = torch.arange(PAGE, device="cuda")[:, None] < start[p0][:, None, None, None]
        s["kv"][p0] = _e4m3(torch.where(before, was * ratio, was)).view(torch.uint8)
        x = x * (1.0 / sc[page])[..., None]
    else:
        x = x * (1.0 / per)[:, None]
    s["kv"][page, :, row] = _e4m3(x).view(torch.uint8).flatten(2)
    return _state(s)


def _attend(logits, seen, v):
    """softmax(logits) v over the seen keys; rows that see none give 0."""
    z = torch.where(seen, logits, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(m > -math.inf, m, 0.0))
    den = p.sum(dim=-1, keepdim=True)
    return (p / torch.where(den > 0, den, 1.0)) @ v


def _plain_listed(s):
    hkv, T = s["hkv"], s["T"]
    b, pos = _token(s)
    blk = s["topk"].long()                                             # [T, Hkv, 16]
    page = s["table"][b[:, None, None], blk.clamp(min=0)].long()
    g = torch.arange(hkv, device="cuda")[:, None]
    kv = s["kv"][page, g].view(F8).float()                             # [T, Hkv, 16, 128, 256]
    sc = s["scales"][page, g]
    k = (kv[..., :D] * sc[..., 0, None, None]).flatten(2, 3)
    v = (kv[..., D:] * sc[..., 1, None, None]).flatten(2, 3)
    t = (blk[..., None] * PAGE + torch.arange(PAGE, device="cuda"))
    seen = ((blk[..., None] >= 0) & (t <= pos[:, None, None, None])).flatten(2)[:, :, None]
    q = (s["q"].float() * s["q_scale"]).view(T, hkv, GROUP, D)
    return _attend(q @ k.transpose(2, 3) * SM, seen, v).view(T, -1, D).to(torch.bfloat16)


def _plain_every(s):
    hkv, Q, (B, S) = s["hkv"], s["qlen"], s["table"].shape
    pos = (s["lens"][:, None] - Q + torch.arange(Q, device="cuda"))    # [B, Q]
    page = s["table"].long()[:, None]                                  # [B, 1, S]
    g = torch.arange(hkv, device="cuda")[:, None]
    seen = torch.arange(S * PAGE, device="cuda") <= pos[..., None]     # [B, Q, keys]
    seen = seen[:, None, :, None]                                      # [B, 1, Q, 1, keys]
    sc = s["scales"][page, g]                                          # [B, Hkv, S, 2]
    k = (s["kv"][..., :D][page, g].view(F8).float() * sc[..., 0, None, None]).flatten(2, 3)
    q = (s["q"].float() * s["q_scale"]).view(B, Q, hkv, GROUP, D).transpose(1, 2)
    z = (q.flatten(2, 3) @ k.transpose(2, 3) * SM).view(B, hkv, Q, GROUP, -1)
    if s["case"]["op"] == "score":
        z = torch.where(seen, z, -math.inf).view(B, hkv, Q, GROUP, S, PAGE).amax(dim=(3, 5))
        return z.permute(1, 0, 2, 3).reshape(hkv, B * Q, S)
    v = (s["kv"][..., D:][page, g].view(F8).float() * sc[..., 1, None, None]).flatten(2, 3)
    o = _attend(z.flatten(2, 3), seen.expand(-1, -1, -1, GROUP, -1).flatten(2, 3), v)
    return o.view(B, hkv, Q, GROUP, D).transpose(1, 2).reshape(B * Q, -1, D).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# work


def work(case):
    lens, q_lens = _lens(case)
    hkv, T = case["hkv"], sum(q_lens)
    hq = GROUP * hkv
    live = sum(min(n, q) for n, q in zip(lens, q_lens))
    qb = 1 if case["q8"] else 2
    if case["op"] == "append":
        bytes_ = live * ((hq + 2 * hkv) * D * 2 + 4 * case["rot"] + 2 * hkv * D) + T * hq * D * qb
        return {"bytes": bytes_, "flops": live * (hq + hkv) * 3 * case["rot"] + live * (hq + 2 * hkv) * D}
    rows = T * hq * D * (qb + 2)      # the query in, the output out
    if case["op"] == "score":
        pg = sum(map(_pages, lens))
        return {"bytes": hkv * pg * PAGE * D + T * hq * D * qb + 4 * hkv * T * max(1, max(map(_pages, lens))),
                "flops": 2 * D * hq * sum(n * q for n, q in zip(lens, q_lens))}
    if case["op"] == "dense":
        return {"bytes": hkv * sum(map(_pages, lens)) * PAGE * 2 * D + rows,
                "flops": 4 * D * hq * sum(n * q for n, q in zip(lens, q_lens))}
    distinct, keys = 0.0, 0
    for n, q in zip(lens, q_lens):
        p = _pages(n)
        # each token lists 15 earlier blocks drawn from p - 1 beside its own
        share = min(1.0, 15 / max(1, p - 1))
        distinct += max(0, p - 1) * (1 - (1 - share) ** q) + (p > 0)
        keys += q * min(n, TOPK * PAGE)
    return {"bytes": int(hkv * distinct) * PAGE * 2 * D + rows + T * hkv * TOPK * 4, "flops": 4 * D * hq * keys}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, request by request


def exact(case, seed):
    s = prepare(case, seed)
    lens, q_lens = _lens(case)
    hkv, f = s["hkv"], torch.float64
    if case["op"] == "append":
        return _exact_append(s, case, lens, q_lens)
    out = torch.zeros((s["T"], GROUP * hkv, D), dtype=f, device="cuda")
    scores = torch.full((hkv, s["T"], s["table"].shape[1]), -math.inf, dtype=f, device="cuda")
    i0 = 0
    for b, (n, ql) in enumerate(zip(lens, q_lens)):
        pages = s["table"][b, :_pages(n)].long()
        key = torch.arange(len(pages) * PAGE, device="cuda")
        where = n - ql + torch.arange(ql, device="cuda")
        causal = key[None, :] <= where[:, None]                        # [ql, keys]
        for g in range(hkv if n else 0):
            c = s["kv"][pages, g].view(F8).to(f)
            sc = s["scales"][pages, g].to(f)
            k = (c[:, :, :D] * sc[:, :1, None]).reshape(-1, D)
            q = s["q"][i0:i0 + ql, GROUP * g:GROUP * (g + 1)].to(f) * s["q_scale"]
            ok = causal
            if "topk" in s:
                hit = torch.zeros((ql, len(pages) + 1), dtype=torch.bool, device="cuda")
                hit.scatter_(1, s["topk"][i0:i0 + ql, g].long() % (len(pages) + 1), True)
                ok = ok & hit[:, :-1].repeat_interleave(PAGE, dim=1)
            z = torch.einsum("jhd,kd->jhk", q, k).mul_(SM).masked_fill_(~ok[:, None], -math.inf)
            if case["op"] == "score":
                scores[g, i0:i0 + ql, :len(pages)] = z.view(ql, GROUP, -1, PAGE).amax(dim=3).amax(dim=1)
                continue
            v = (c[:, :, D:] * sc[:, 1:, None]).reshape(-1, D)
            p = torch.softmax(z, dim=2).nan_to_num_(0.0)
            out[i0:i0 + ql, GROUP * g:GROUP * (g + 1)] = torch.einsum("jhk,kd->jhd", p, v)
        i0 += ql
    return scores if case["op"] == "score" else out


def _exact_append(s, case, lens, q_lens):
    """The values before they are rounded to e4m3 or bf16, from complex
    rotations; a page's scale from the exponent of its largest value."""
    hkv, f = s["hkv"], torch.float64
    hq, h = GROUP * hkv, case["rot"] // 2
    cache, scales = s["kv"].view(F8).to(f), s["scales"].to(f)
    rows = s["qkv"].view(s["T"], -1, D).to(f)
    q_out = torch.zeros((s["T"], hq, D), dtype=f, device="cuda")
    i0 = 0
    for b, (n, ql) in enumerate(zip(lens, q_lens)):
        x = rows[i0 + max(0, ql - n):i0 + ql].clone()                  # the tokens that are there
        start, live = max(0, n - ql), min(n, ql)
        if h and live:
            turn = torch.complex(*(t.contiguous() for t in s["cos_sin"][start:n].to(f).split(h, dim=1)))
            r = x[:, :hq + hkv]
            a, d = (r[..., 0:2 * h:2], r[..., 1:2 * h:2]) if case["pairs"] else (r[..., :h], r[..., h:2 * h])
            y = torch.complex(a.contiguous(), d.contiguous()) * turn[:, None]
            if case["pairs"]:
                r[..., 0:2 * h:2], r[..., 1:2 * h:2] = y.real, y.imag
            else:
                r[..., :h], r[..., h:2 * h] = y.real, y.imag
        q_out[i0 + ql - live:i0 + ql] = x[:, :hq] / (s["q_scale"] if case["q8"] else 1.0)
        k, v = x[:, hq:hq + hkv] / s["k_scale"], x[:, hq + hkv:] / s["v_scale"]
        at = start
        while at < n:                                                  # page by page
            page, r0 = int(s["table"][b, at // PAGE]), at % PAGE
            m = min(PAGE - r0, n - at)
            for side, t in enumerate((k, v)):
                t = t[at - start:at - start + m]
                cells = cache[page, :, :, D * side:D * (side + 1)]
                if case["scaled"]:
                    want = torch.tensor([2.0 ** min(40, max(-40, math.ceil(math.log2(a / TOP)) if a else -40))
                                         for a in t.abs().amax(dim=(0, 2)).tolist()], dtype=f, device="cuda")
                    had = scales[page, :, side].clone()
                    grown = torch.maximum(want, had) if r0 else want
                    scales[page, :, side] = grown
                    cells[:, :r0] *= (had / grown)[:, None, None]
                    t = t / grown[:, None]
                cells[:, r0:r0 + m] = t.transpose(0, 1)
            at += m
        i0 += ql
    return [cache.clamp(-TOP, TOP), scales if case["scaled"] else None, q_out]
