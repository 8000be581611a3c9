"""What is measured of chunked prefill over the paged cache and of the cache's pages.

The operators: dense attention of a chunk of new tokens over the paged fp8 cache
(dense_prefill), the block scorer and the block selector of prefill batches, whose
requests have one query length each (score_prefill, topk_prefill), and the pages of
a cache: rows forked, reordered, freed and grown (fork_pages), pages moved together
(compact_pages), each with the copies of the pages' bytes.

Layouts are the library's: q [T, Hq, 128], cache fp8 e4m3 [NB, Hkv, 128, 256] (K in
bytes 0-127 of a row, V in 128-255) or K-only [NB, Hkv, 128, 128], block_table int32
[B, S], seq_lens int32 [B], cu_seqlens_q int32 [B + 1], page scales fp32 [NB, Hkv, 2]
(K's, then V's; [NB, Hkv, 1] of a K-only cache), scores fp32 [Hkv, T, S], refs int32
[NB] (how many rows of tables hold a page), Hq = 16 Hkv."""
import math

import numpy as np
import torch

own = False

D, PAGE, TOPK, GROUP = 128, 128, 16, 16
F8 = torch.float8_e4m3fn
TOP = 448.0          # the largest e4m3 value
SM = D ** -0.5
K_SCALE, V_SCALE, Q_SCALE = 0.0071, 0.0068, 0.0123   # one scale per tensor


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # two short chunks on one KV head (a tensor-parallel shard): latency
        dict(name="dense_b2_q24_h16kv1", op="dense", batch=2, hkv=1, lo=2048, hi=3000, chunk=24,
             q8=False, scaled=False),
        # chunked prefill in the model's dense layers: four chunks of up to 1k tokens
        dict(name="dense_b4_1k_h64kv4", op="dense", batch=4, hkv=4, lo=4096, hi=16384, chunk=820,
             q8=False, scaled=False),
        # chunks of odd lengths, an fp8 query, page scales
        dict(name="dense_b5_odd_fp8q", op="dense", batch=5, hkv=2, lo=701, hi=5003, chunk=301,
             q8=True, scaled=True),
        # one chunk of a long document on one KV head, page scales
        dict(name="dense_b1_1k_128k", op="dense", batch=1, hkv=1, lo=131072, hi=131072, chunk=1400,
             q8=False, scaled=True),
        # the sparse layers' scorer on short chunks on one KV head: latency
        dict(name="score_b3_q40_h16kv1", op="score", batch=3, hkv=1, lo=2048, hi=5000, chunk=40,
             q8=False, scaled=False, konly=False),
        # the scorer on the four chunks of up to 1k tokens, page scales
        dict(name="score_b4_1k_h64kv4", op="score", batch=4, hkv=4, lo=4096, hi=16384, chunk=820,
             q8=False, scaled=True, konly=False),
        # selection for short chunks: latency
        dict(name="topk_b4_q50", op="topk", batch=4, hkv=1, lo=2500, hi=4000, chunk=50),
        # selection for four chunks of 1k-2k tokens over up to 512 blocks
        dict(name="topk_b4_1k-2k", op="topk", batch=4, hkv=4, lo=8192, hi=65536, chunk=1500),
        # beam search on one KV head: two requests of four beams, one cache
        dict(name="fork_2x4_h16kv1", op="fork", requests=2, width=4, hkv=1, lo=2048, hi=3000,
             tail=200, grow=1, caches=1),
        # parallel sampling: 48 requests of four rows, a K|V and an index-K cache with
        # page scales, some requests replaced by new prompts
        dict(name="fork_48x4_h64kv4", op="fork", requests=48, width=4, hkv=4, lo=1024, hi=8192,
             tail=700, grow=4, caches=4),
        # a small pool, one cache
        dict(name="compact_8_h16kv1", op="compact", requests=8, width=1, hkv=1, lo=1000, hi=8000,
             tail=0, fill=60, caches=1),
        # a pool of thousands of pages, half of it holes: K|V and index-K, page scales
        dict(name="compact_64x2_h64kv4", op="compact", requests=64, width=2, hkv=4, lo=1024,
             hi=8192, tail=300, fill=55, caches=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dense", "dense", "score", "topk", "fork", "compact"])
    c = dict(op=op, hkv=rng.choice([1, 2, 4]))
    if op in ("fork", "compact"):
        c.update(width=rng.choice([1, 2, 3, 4, 5, 8]), tail=_log(rng, 1, 900),
                 caches=rng.choice([1, 2, 3, 4]))
        c["requests"] = _log(rng, 1, max(1, 160 // c["width"]))
        c["lo"] = _log(rng, 1, 3000)
        c["hi"] = c["lo"] + _log(rng, 1, 5000)
        if op == "fork":
            c["grow"] = rng.choice([0, 1, 1, 2, 4, 7, 32, 150])
        else:
            c["fill"] = rng.randint(20, 97)
            c["requests"] = min(c["requests"], 40)
        return c
    c.update(batch=_log(rng, 1, 12), chunk=_log(rng, 1, 820))
    c["lo"] = 2 * c["chunk"] + _log(rng, 1, 6000)
    c["hi"] = c["lo"] + _log(rng, 1, 12000)
    if op == "topk":        # more than 16 blocks, so that there is something to select
        c["lo"] += 2200
        c["hi"] = c["lo"] + _log(rng, 1, 50000)
        return c
    c.update(q8=rng.random() < 0.4, scaled=rng.random() < 0.5)
    if op == "score":
        c["konly"] = rng.random() < 0.4
    # no more keys times tokens, padded, than the largest listed case
    c["batch"] = max(1, min(c["batch"], (1 << 27) // (c["hkv"] * c["chunk"] * c["hi"])))
    return c


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _lens(c):
    """(seq_lens, query lengths), from the case alone: lengths spread over
    [lo, hi] in an order that is not sorted, chunks of 3/4 to 5/4 of `chunk`."""
    B = c["batch"]
    at = [(k * 7 + 3) % B if B % 7 else k for k in range(B)]
    lens = [c["lo"] + (c["hi"] - c["lo"]) * k // max(1, B - 1) for k in at]
    return lens, [min(n, max(1, c["chunk"] * (6 + (3 * k) % 5) // 8)) for k, n in enumerate(lens)]


def _rows(c):
    """Of a pool, from the case alone: per row of the table its length and how many
    leading pages its request's rows share; the rows of a request have a prompt in
    common and up to `tail` tokens of their own."""
    lens, shared = [], []
    R, W = c["requests"], c["width"]
    for i in range(R):
        prompt = c["lo"] + (c["hi"] - c["lo"]) * ((i * 7 + 3) % R if R % 7 else i) // max(1, R - 1)
        for k in range(W):
            lens.append(prompt + (37 * k + 11 * i) % (c["tail"] + 1))
            shared.append(prompt // PAGE if W > 1 else 0)
    return lens, shared


def _parents(c):
    """(parents, growth) of the next step's rows: beams that follow beams of their
    request, some of them twice and some not at all; every seventh request is over, and
    every fourteenth row is a new prompt in its place."""
    W, parents, grow = c["width"], [], []
    for b in range(c["requests"] * W):
        i, k = divmod(b, W)
        over = i % 7 == 5
        parents.append(-1 if over else i * W + (k * k + i) % W)
        grow.append((300 if b % 2 else 0) if over else c["grow"])
    return parents, grow


def _fork_need(c):
    """(copies (rows of tokens), fresh pages, columns) of a fork, from the case alone."""
    lens, _ = _rows(c)
    parents, grow = _parents(c)
    seen, copies, need, cols = set(), [], 0, 1
    for p, g in zip(parents, grow):
        n = lens[p] if p >= 0 else 0
        need += _pages(n + g) - _pages(n)
        cols = max(cols, _pages(n + g))
        if p >= 0 and p in seen and n % PAGE:
            copies.append(n % PAGE)
            need += 1
        seen.add(p)
    return copies, need, cols


# ---------------------------------------------------------------------------
# inputs


def _codes(shape, gen):
    """Random e4m3 codes with the values' spread of a quantised activation."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).mul_(110.0)
    return x.clamp_(-TOP, TOP).to(F8).view(torch.uint8)


def _scales(shape, gen):
    """Page scales around 2^-8, as keys and values of a spread of a half have."""
    return torch.exp2(torch.randn(shape, generator=gen, device="cuda") * 0.7 - 8.0)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("fork", "compact"):
        return _prepare_pool(case, gen)
    lens, q_lens = _lens(case)
    B, hkv, T = case["batch"], case["hkv"], sum(q_lens)
    hq = GROUP * hkv
    pages = [_pages(n) for n in lens]
    S, NB = max(pages), sum(pages) + 1
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s = dict(case=case, T=T, hkv=hkv, S=S, lens=_int(lens), cu=_int(cu), qmax=max(q_lens))
    if case["op"] == "topk":
        # scores as a scorer leaves them: most rows without ties, a quarter on a coarse
        # grid with many, blocks that a token does not see at -inf
        x = torch.randn((hkv, T, S), generator=gen, device="cuda") * 2.0 + 3.0
        coarse = torch.rand((hkv, T, 1), generator=gen, device="cuda") < 0.25
        x = torch.where(coarse, (x * 4.0).round() / 4.0, x)
        _, pos = _token(s)
        late = torch.arange(S, device="cuda") > torch.div(pos, PAGE, rounding_mode="floor")[:, None]
        s["scores"] = torch.where(late, -math.inf, x)
        s["out"] = torch.zeros((T, hkv, TOPK), dtype=torch.int32, device="cuda")
        return s
    perm = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(B)], device="cuda")
    n_pg = torch.tensor(pages, device="cuda")
    at = torch.arange(S, device="cuda")
    table = torch.where(at < n_pg[:, None], perm[(first[:, None] + at).clamp(max=NB - 1)], 0)
    s["table"] = table.to(torch.int32).contiguous()
    sides = 1 if case.get("konly") else 2
    s["kv"] = _codes((NB, hkv, PAGE, D * sides), gen)
    scales = _scales((NB, hkv, sides), gen)
    s["scales"] = scales if case["scaled"] else None
    s["k_scale"], s["v_scale"] = (1.0, 1.0) if case["scaled"] else (K_SCALE, V_SCALE)
    q = torch.randn((T, hq, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["q_scale"] = 1.0
    if case["q8"]:
        s["q_scale"] = Q_SCALE
        q = (q.float() / s["q_scale"]).clamp(-TOP, TOP).to(F8)
    s["q"] = q
    if case["op"] == "score":
        s["scores"] = torch.zeros((hkv, T, S), device="cuda")
    else:
        s["out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        # room for the parts of rows that several blocks share, kept by a serving program
        s["work"] = torch.empty(48 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_pool(case, gen):
    lens, shared = _rows(case)
    B, W, hkv = len(lens), case["width"], case["hkv"]
    cols = max(map(_pages, lens))
    if case["op"] == "fork":
        _, need, c = _fork_need(case)
        cols = max(cols, c)
    at, table = 0, np.zeros((B, cols), dtype=np.int64)
    for b, (n, sh) in enumerate(zip(lens, shared)):
        if b % W == 0:
            table[b, :sh] = at + np.arange(sh)
            at += sh
        else:
            table[b, :sh] = table[b - 1, :sh]
        m = _pages(n) - sh
        table[b, sh:sh + m] = at + np.arange(m)
        at += m
    refs = np.zeros(at, dtype=np.int64)
    for b, n in enumerate(lens):
        refs[table[b, :_pages(n)]] += 1
    if case["op"] == "fork":
        NB = at + need + max(2, at // 4)
        kept = at // 20                      # pages that a prefix cache alone holds
        NB += kept
    else:
        kept = at // 10
        NB = max(at + kept + 1, (at + kept) * 100 // case["fill"])
    perm = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32)
    all_refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    all_refs[perm[:at].long()] = _int(refs)
    all_refs[perm[at:at + kept].long()] = 1
    s = dict(case=case, refs=all_refs, lens=_int(lens),
             table=perm[torch.from_numpy(table).cuda()].contiguous())
    caches = [_codes((NB, hkv, PAGE, 2 * D), gen), _scales((NB, hkv, 2), gen),
              _codes((NB, hkv, PAGE, D), gen), _scales((NB, hkv, 1), gen)]
    s["caches"] = caches[:case["caches"]]
    s["table_out"], s["refs_out"] = torch.zeros_like(s["table"]), torch.zeros_like(all_refs)
    if case["op"] == "fork":
        parents, grow = _parents(case)
        s["parents"], s["grow"] = _int(parents), _int(grow)
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["copies"] = torch.zeros((B, 3), dtype=torch.int32, device="cuda")
    else:
        s["copies"] = torch.zeros((NB // 2, 3), dtype=torch.int32, device="cuda")
    return s


def _token(s):
    """(request, position) of every token."""
    b = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(s["T"], dtype=torch.int32, device="cuda"),
                           right=True)
    i = torch.arange(s["T"], device="cuda")
    q_len = (s["cu"][1:] - s["cu"][:-1])[b]
    return b, (s["lens"][b] - q_len + i - s["cu"][b]).long()


# ---------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "topk":
        return _plain_topk(s)
    if op == "fork":
        return _plain_fork(s)
    if op == "compact":
        return _plain_compact(s)
    return _plain_every(s)


def _run_own(s):
    import block_sparse_gqa_score_gb300 as msa
    op = s["case"]["op"]
    if op == "topk":
        return msa.topk_prefill(s["scores"], s["lens"], s["cu"], out=s["out"])
    if op == "fork":
        msa.fork_pages(s["table"], s["lens"], s["parents"], s["refs"], s["caches"], grow=s["grow"],
                       block_table_out=s["table_out"], seq_lens_out=s["lens_out"],
                       refs_out=s["refs_out"], copies=s["copies"])
        return _pool(s)
    if op == "compact":
        msa.compact_pages(s["table"], s["lens"], s["refs"], s["caches"],
                          block_table_out=s["table_out"], refs_out=s["refs_out"], copies=s["copies"])
        return _pool(s)
    kw = dict(kv_scales=s["scales"], q_scale=s["q_scale"])
    if op == "score":
        return msa.score_prefill(s["q"], s["kv"], s["table"], s["lens"], s["cu"], SM, s["k_scale"],
                                 scores=s["scores"], **kw)
    return msa.dense_prefill(s["q"], s["kv"], s["table"], s["lens"], s["cu"], SM, s["k_scale"],
                             s["v_scale"], out=s["out"], workspace=s["work"], **kw)


def _pool(s):
    """The outputs of a fork or a compaction: tables, counts, what was copied, and the
    caches' values."""
    out = [s["table_out"], s["refs_out"], s["copies"]]
    if s["case"]["op"] == "fork":
        out.append(s["lens_out"])
    return out + [x.view(F8) if x.dtype == torch.uint8 else x for x in s["caches"]]


def _padded(s):
    """[B, qmax] token of each place of the padded batch and whether it is one."""
    j = torch.arange(s["qmax"], device="cuda")
    n = (s["cu"][1:] - s["cu"][:-1])[:, None]
    return (s["cu"][:-1, None] + j).clamp(max=s["T"] - 1).long(), j < n


def _plain_every(s):
    """Scores or attention over every visible key of the requests, padded to the
    longest chunk."""
    hkv, (B, S), Q = s["hkv"], s["table"].shape, s["qmax"]
    tok, there = _padded(s)
    pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(Q, device="cuda")
    pos = torch.where(there, pos, -1)                                  # [B, Q]
    page = s["table"].long()[:, None]                                  # [B, 1, S]
    g = torch.arange(hkv, device="cuda")[:, None]
    kv = s["kv"][page, g].view(F8).float()                             # [B, Hkv, S, 128, .]
    sc = s["scales"][page, g] if s["scales"] is not None else torch.ones((1, 1, 1, 2), device="cuda")
    k = (kv[..., :D] * (sc[..., 0, None, None] * s["k_scale"])).flatten(2, 3)
    q = (s["q"][tok].float() * s["q_scale"]).view(B, Q, hkv, GROUP, D).transpose(1, 2)
    z = (q.flatten(2, 3) @ k.transpose(2, 3)).mul_(SM).view(B, hkv, Q, GROUP, S * PAGE)
    hid = (torch.arange(S * PAGE, device="cuda") > pos[..., None])[:, None, :, None]
    z.masked_fill_(hid, -math.inf)
    if s["case"]["op"] == "score":
        z = z.view(B, hkv, Q, GROUP, S, PAGE).amax(dim=(3, 5))
        s["scores"].copy_(z.transpose(0, 1)[:, there])
        return s["scores"]
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp_(z.sub_(torch.where(m > -math.inf, m, 0.0)))
    den = p.sum(dim=-1, keepdim=True)
    v = (kv[..., D:] * (sc[..., 1, None, None] * s["v_scale"])).flatten(2, 3)
    o = (p.flatten(2, 3) @ v).view(B, hkv, Q, GROUP, D) / torch.where(den > 0, den, 1.0)
    s["out"].copy_(o.transpose(1, 2)[there].flatten(1, 2))
    return s["out"]


def _plain_topk(s):
    """The current block and the 15 best before it, ties to the lower index, ascending."""
    hkv, T, S = s["hkv"], s["T"], s["S"]
    _, pos = _token(s)
    cur = torch.div(pos, PAGE, rounding_mode="floor")[:, None]         # [T, 1]
    n = torch.arange(S, device="cuda")
    x = torch.where(n < cur, s["scores"], torch.where(n == cur, math.inf, -math.inf))
    val, idx = x.sort(dim=2, descending=True, stable=True)
    idx = torch.nn.functional.pad(idx[..., :TOPK], (0, max(0, TOPK - S)), value=S)
    rank = torch.arange(TOPK, device="cuda")
    idx = torch.where(rank <= cur, idx, S).sort(dim=2).values
    s["out"].copy_(torch.where(idx < S, idx, -1).transpose(0, 1))
    return s["out"]


def _plain_fork(s):
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    parents, grow = s["parents"].long(), s["grow"].long()
    (B, S), NB = table.shape, refs.shape[0]
    e = torch.arange(S, device="cuda")
    has = parents >= 0
    p = parents.clamp(min=0)
    n = torch.where(has, lens[p], 0)
    r = n % PAGE
    row = torch.arange(B, device="cuda")
    first = torch.full((B,), B, device="cuda").scatter_reduce_(0, p, torch.where(has, row, B), "amin")
    copy = has & (r > 0) & (first[p] != row)
    held = (n + PAGE - 1) // PAGE - copy.long()            # entries taken over
    want = (n + grow + PAGE - 1) // PAGE
    fresh = (e >= held[:, None]) & (e < want[:, None])
    free = torch.argsort((refs != 0).int(), stable=True)   # the free pages first, ascending
    rank = fresh.flatten().cumsum(0).view(B, S) - 1
    new = torch.where(e < held[:, None], table[p], torch.where(fresh, free[rank.clamp(min=0)], -1))
    s["table_out"].copy_(new)
    s["lens_out"].copy_(n + grow)
    old = (e < ((lens + PAGE - 1) // PAGE)[:, None])
    count = refs.clone()
    count.index_add_(0, table.flatten(), -old.flatten().long())
    count.index_add_(0, new.clamp(min=0).flatten(), (new >= 0).flatten().long())
    s["refs_out"].copy_(count)
    last = held.clamp(max=S - 1)[:, None]
    move = torch.cat([table[p].gather(1, last), new.gather(1, last), r[:, None]], dim=1)
    s["copies"].copy_(torch.where(copy[:, None], move, torch.tensor([-1, -1, 0], device="cuda")))
    _plain_copy(s)
    return _pool(s)


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"].long()
    NB = refs.shape[0]
    page = torch.arange(NB, device="cuda")
    live = refs != 0
    L = live.sum()
    hole, mover = ~live & (page < L), live & (page >= L)
    holes = torch.argsort((~hole).int(), stable=True)      # the holes first, ascending
    movers = torch.argsort((~mover).int(), stable=True)
    k = torch.arange(NB // 2, device="cuda")
    there = (k < mover.sum())[:, None]
    move = torch.stack([movers[:NB // 2], holes[:NB // 2], torch.full_like(k, PAGE)], dim=1)
    s["copies"].copy_(torch.where(there, move, torch.tensor([-1, -1, 0], device="cuda")))
    to = torch.where(mover, holes[(mover.long().cumsum(0) - 1).clamp(min=0)], page)
    s["table_out"].copy_(torch.where(
        torch.arange(table.shape[1], device="cuda") < ((s["lens"] + PAGE - 1) // PAGE)[:, None], to[table], -1))
    s["refs_out"].copy_(torch.zeros_like(refs).index_add_(0, to, refs))
    _plain_copy(s)
    return _pool(s)


def _plain_copy(s):
    c = s["copies"]
    src, dst, rows = c[c[:, 1] >= 0].long().unbind(1)
    row = (torch.arange(PAGE, device="cuda") < rows[:, None])[:, None, :, None]
    kv = s["caches"][0]
    kv[dst] = torch.where(row, kv[src], kv[dst])
    if len(s["caches"]) > 2:
        ik = s["caches"][2]
        ik[dst] = torch.where(row, ik[src], ik[dst])
    if len(s["caches"]) > 1:
        s["caches"][1][dst] = s["caches"][1][src]
    if len(s["caches"]) > 3:
        s["caches"][3][dst] = s["caches"][3][src]


# ---------------------------------------------------------------------------
# work


def work(case):
    hkv = case["hkv"]
    if case["op"] in ("fork", "compact"):
        lens, shared = _rows(case)
        pages = sum(map(_pages, lens))
        token = hkv * (2 * D + (D if case["caches"] > 2 else 0))
        per_page = hkv * (8 * (case["caches"] > 1) + 4 * (case["caches"] > 3))
        live = pages - sum(sh for b, sh in enumerate(shared) if b % case["width"])
        if case["op"] == "fork":
            copies, need, cols = _fork_need(case)
            cols = max(cols, max(map(_pages, lens)))
            moved = 2 * (sum(copies) * token + len(copies) * per_page)
            NB = live + live // 20 + need + max(2, live // 4)
            return {"bytes": moved + 4 * (pages + len(lens) * (cols + 7) + 2 * NB), "flops": 0}
        live += live // 10
        NB = max(live + 1, live * 100 // case["fill"])
        moved = int(live * (1 - live / NB)) * 2 * (PAGE * token + per_page)
        return {"bytes": moved + 4 * (pages + len(lens) * max(map(_pages, lens)) + 2 * NB + 3 * (NB // 2)),
                "flops": 0}
    lens, q_lens = _lens(case)
    T, hq = sum(q_lens), GROUP * hkv
    seen = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, q_lens))   # keys of all tokens
    if case["op"] == "topk":
        blocks = sum((n - q + j) // PAGE for n, q in zip(lens, q_lens) for j in range(q))
        return {"bytes": 4 * hkv * (blocks + TOPK * T), "flops": hkv * blocks}
    keys, qb = sum(lens), 1 if case["q8"] else 2
    if case["op"] == "score":
        return {"bytes": hkv * keys * D + T * hq * D * qb + 4 * hkv * T * max(map(_pages, lens)),
                "flops": 2 * D * hq * seen}
    return {"bytes": hkv * keys * 2 * D + T * hq * D * (qb + 2), "flops": 4 * D * hq * seen}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, request by request


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return _exact_pool(s, case)
    lens, q_lens = s["lens"].tolist(), s["cu"].diff().tolist()
    hkv, f = s["hkv"], torch.float64
    if case["op"] == "topk":
        return _exact_topk(s, lens, q_lens)
    out = torch.zeros((s["T"], GROUP * hkv, D), dtype=f, device="cuda")
    scores = torch.full((hkv, s["T"], s["S"]), -math.inf, dtype=f, device="cuda")
    i0 = 0
    for b, (n, ql) in enumerate(zip(lens, q_lens)):
        pages = s["table"][b, :_pages(n)].long()
        key = torch.arange(len(pages) * PAGE, device="cuda")
        for g in range(hkv):
            c = s["kv"][pages, g].view(F8).to(f)
            one = torch.ones((len(pages), 2), dtype=f, device="cuda")
            sc = s["scales"][pages, g].to(f) if s["scales"] is not None else one
            k = (c[:, :, :D] * sc[:, :1, None]).reshape(-1, D) * s["k_scale"]
            for j0 in range(0, ql, 256):                               # 256 tokens at a time
                j1 = min(ql, j0 + 256)
                ok = key[None, :] <= (n - ql + torch.arange(j0, j1, device="cuda"))[:, None]
                q = s["q"][i0 + j0:i0 + j1, GROUP * g:GROUP * (g + 1)].to(f) * s["q_scale"]
                z = torch.einsum("jhd,kd->jhk", q, k).mul_(SM).masked_fill_(~ok[:, None], -math.inf)
                if case["op"] == "score":
                    scores[g, i0 + j0:i0 + j1, :len(pages)] = \
                        z.view(j1 - j0, GROUP, -1, PAGE).amax(dim=3).amax(dim=1)
                    continue
                v = (c[:, :, D:] * sc[:, 1:, None]).reshape(-1, D) * s["v_scale"]
                out[i0 + j0:i0 + j1, GROUP * g:GROUP * (g + 1)] = \
                    torch.einsum("jhk,kd->jhd", torch.softmax(z, dim=2), v)
        i0 += ql
    return scores if case["op"] == "score" else out


def _exact_topk(s, lens, q_lens):
    x = s["scores"].double().cpu().numpy()
    out = np.full((s["T"], s["hkv"], TOPK), -1, dtype=np.int32)
    i0 = 0
    for n, ql in zip(lens, q_lens):
        for j in range(ql):
            cur = (n - ql + j) // PAGE
            best = np.argsort(-x[:, i0 + j, :cur], axis=1, kind="stable")[:, :TOPK - 1]
            kept = np.concatenate([np.sort(best, axis=1), np.full((s["hkv"], 1), cur)], axis=1)
            out[i0 + j, :, :kept.shape[1]] = kept
        i0 += ql
    return torch.from_numpy(out)


def _exact_pool(s, case):
    """Page by page on the host, from the meaning: what each row holds, who else does,
    and the lowest free pages in turn."""
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    caches = [x.clone() for x in s["caches"]]
    S = len(table[0])
    rows = [t[:_pages(n)] for t, n in zip(table, lens)]
    copies, lens_out = [], None
    if case["op"] == "fork":
        free = [p for p, r in enumerate(refs) if r == 0]
        lens_out, new, taken = [], [], set()
        for p, g in zip(s["parents"].tolist(), s["grow"].tolist()):
            got = list(rows[p]) if p >= 0 else []
            n = lens[p] if p >= 0 else 0
            copies.append((-1, -1, 0))
            if n % PAGE and p in taken:
                copies[-1] = (got[-1], free[0], n % PAGE)
                got[-1] = free.pop(0)
            taken.add(p)
            while len(got) < _pages(n + g):
                got.append(free.pop(0))
            new.append(got)
            lens_out.append(n + g)
        for pages in rows:
            for p in pages:
                refs[p] -= 1
        for pages in new:
            for p in pages:
                refs[p] += 1
    else:
        live = [p for p, r in enumerate(refs) if r]
        holes = [p for p in range(len(live)) if not refs[p]]
        move = dict(zip([p for p in live if p >= len(live)], holes))
        copies = [(a, b, PAGE) for a, b in move.items()]
        new = [[move.get(p, p) for p in pages] for pages in rows]
        for a, b in move.items():
            refs[b], refs[a] = refs[a], 0
        copies += [(-1, -1, 0)] * (len(refs) // 2 - len(copies))
    at = [c for c in copies if c[0] >= 0]
    for a, b, r in at:
        for x in caches:
            if x.dim() == 4:
                x[b, :, :r] = x[a, :, :r]
            else:
                x[b] = x[a]
    out = [_int([t + [-1] * (S - len(t)) for t in new]), _int(refs), _int(copies)]
    if lens_out is not None:
        out.append(_int(lens_out))
    return out + [x.view(F8).half().double() if x.dtype == torch.uint8 else x.double() for x in caches]
