"""Plain 64-bit forms of the cache append and of attention over page scales, and
the inputs their tests share.  Written from the definitions (include/msa.h) with
elementary torch operations, token by token where that is clearest."""
from __future__ import annotations

import math

import torch

D, PAGE, GROUP, TOPK = 128, 128, 16, 16
F8 = torch.float8_e4m3fn
TOP = 448.0
HALF_BF16, HALF_E4M3, U32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def table(max_pos: int, rot: int, device="cuda", base: float = 10000.0) -> torch.Tensor:
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float().to(device)


def layout(seq_lens, gen, spare: int = 2, min_cols: int = 1):
    """(block_table [B, S], pages): every request's pages scattered over a pool
    with `spare` pages that belong to nobody."""
    n = [-(-max(L, 0) // PAGE) for L in seq_lens]
    nb = sum(n) + spare
    perm = torch.randperm(nb, generator=gen).to(torch.int32)
    bt = torch.zeros((len(seq_lens), max(n + [min_cols])), dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        bt[b, :m] = perm[at:at + m]
        at += m
    return bt, nb


def codes(shape, gen, nan: float = 0.0) -> torch.Tensor:
    """uint8 e4m3 codes of N(0, 110^2), a share of them NaN."""
    c = (torch.randn(shape, generator=gen) * 110).clamp(-TOP, TOP).to(F8).view(torch.uint8)
    if nan:
        c[torch.rand(shape, generator=gen) < nan] = 0x7F
    return c


def rotate64(x, pos, cs, interleaved):
    """(rotated x, |terms|) of x [H, 128] in 64 bits at position pos."""
    x = x.double()
    rot = cs.shape[1] if cs is not None else 0
    y, size = x.clone(), x.abs()
    if rot:
        c, s = cs[pos, :rot // 2].double(), cs[pos, rot // 2:].double()
        i = torch.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        size[:, a] = (x[:, a] * c).abs() + (x[:, b] * s).abs()
        size[:, b] = (x[:, b] * c).abs() + (x[:, a] * s).abs()
    return y, size


def power_for(amax: float) -> float:
    """The smallest power of two s in [2^-40, 2^40] with amax <= 448 s."""
    if amax <= 0:
        return 2.0 ** -40
    e = math.ceil(math.log2(amax / TOP))
    if 2.0 ** (e - 1) * TOP >= amax:
        e -= 1
    if 2.0 ** e * TOP < amax:
        e += 1
    return 2.0 ** max(-40, min(40, e))


class Append:
    """The append in 64 bits on host copies: `want` holds each written element's
    value before its rounding to e4m3 and `slack` how far 32-bit arithmetic may
    be off it; `mask` marks the written elements, all others keep their bytes."""

    def __init__(self, kv, scales, block_table, seq_lens, k_scale=1.0, v_scale=1.0):
        self.kv, self.bt, self.lens = kv.cpu().clone(), block_table.cpu(), list(seq_lens)
        self.scales = None if scales is None else scales.cpu().double()
        self.per = (float(torch.tensor(k_scale)), float(torch.tensor(v_scale)))
        self.want = self.kv.view(F8).double()
        self.slack = torch.zeros_like(self.want)
        self.mask = torch.zeros(self.kv.shape, dtype=torch.bool)

    def run(self, k, v, q, q_lens, cs=None, interleaved=False):
        k, q = k.cpu(), None if q is None else q.cpu()
        v = None if v is None else v.cpu()
        cs = None if cs is None else cs.cpu()
        T = k.shape[0]
        qv = qs = None
        if q is not None:
            qv, qs = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
        i = 0
        for b, n in enumerate(q_lens):
            L = self.lens[b]
            groups = {}      # (page) -> [(row, token)]
            for j in range(n):
                pos = L - n + j
                tok, i = i, i + 1
                if pos < 0:
                    continue
                if qv is not None:
                    qv[tok], qs[tok] = rotate64(q[tok], pos, cs, interleaved)
                groups.setdefault(int(self.bt[b, pos // PAGE]), []).append((pos % PAGE, tok, pos))
            for page, rows in groups.items():
                for side, x in ((0, k), (1, v)):
                    if x is not None:
                        self._page(page, side, rows, x, cs if side == 0 else None, interleaved)
        assert i <= T
        return qv, qs

    def _page(self, page, side, rows, x, cs, interleaved):
        vals, sizes = zip(*[rotate64(x[t], pos, cs, interleaved) for _, t, pos in rows])
        val = torch.stack(vals) / self.per[side]               # [n, Hkv, 128]
        size = torch.stack(sizes) / self.per[side]
        r0, at = rows[0][0], [r for r, _, _ in rows]
        lo, hi = D * side, D * side + D
        if self.scales is not None:
            for g in range(val.shape[1]):
                fin = val[:, g][torch.isfinite(val[:, g])].abs()
                s = power_for(float(fin.max()) if fin.numel() else 0.0)
                old = float(self.scales[page, g, side])
                if r0 > 0:
                    s = max(s, old)
                    if s > old:
                        self.want[page, g, :r0, lo:hi] = (
                            self.kv.view(F8)[page, g, :r0, lo:hi].double() * (old / s))
                        # the ratio and the product in 32 bits
                        self.slack[page, g, :r0, lo:hi] = (
                            2 * U32 * self.want[page, g, :r0, lo:hi].abs().nan_to_num(0.0))
                        self.mask[page, g, :r0, lo:hi] = True
                self.scales[page, g, side] = s
                val[:, g] /= s
                size[:, g] /= s
        self.want[page, :, at, lo:hi] = val.transpose(0, 1)
        # the rotation: two products and a sum; the tensor scale's reciprocal and
        # its product; the page scale's (exact, a power of two)
        self.slack[page, :, at, lo:hi] = 6 * U32 * size.transpose(0, 1)
        self.mask[page, :, at, lo:hi] = True

    def settle(self, kv):
        """Takes the codes written so far as the state before the next append."""
        self.kv = kv.cpu().clone()
        self.want = self.kv.view(F8).double()
        self.mask.zero_(), self.slack.zero_()

    def check(self, kv, scales=None):
        got = kv.cpu()
        assert torch.equal(got[~self.mask], self.kv[~self.mask]), "bytes that were not written changed"
        check_e4m3(got.view(F8).float()[self.mask], self.want[self.mask], self.slack[self.mask])
        if self.scales is not None:
            assert torch.equal(scales.cpu().double().nan_to_num(-7.0), self.scales.nan_to_num(-7.0))


def check_e4m3(code, want, slack):
    """Codes within half an e4m3 step (and the slack of the value before it) of
    the value, saturated at 448; NaN where the value is NaN."""
    got = code.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    got, want, slack = got[~nan], want[~nan].clamp(-TOP, TOP), slack[~nan]
    slack = torch.where(torch.isfinite(slack), slack, 0.0)
    # steps are 2^(e - 3) of a value of exponent e, 2^-9 below 2^-6
    e = torch.floor(torch.log2((want.abs() + slack).clamp(min=2.0 ** -6)))
    bound = torch.exp2(e - 3) / 2 + slack
    bad = (got - want).abs() > bound
    assert not bad.any(), (got[bad][:4], want[bad][:4])


def check_bf16(got, want, size):
    """bf16 values within half a step of the value and its 32-bit error."""
    err = (got.double() - want).abs()
    assert (err <= HALF_BF16 * want.abs() + 6 * U32 * size + 1e-38).all(), err.max()


def attend64(q, kv, scales, block_table, seq_lens, q_lens, sm, k_scale, v_scale, lists=None):
    """(out, bound, scores) in 64 bits on the tensors' device: softmax attention
    of every token over its listed (or all) visible blocks with page scales, and
    the error the kernels' arithmetic allows each output element:
      P as fp16 and two e4m3 parts: 2^-8 + 2^-11 of each term.  hi is at most 2^-4 P
        off, so |lo| <= 2^-4 P, and lo is off by 2^-4 |lo| <= 2^-8 P or, as an e4m3
        subnormal (steps of 2^-9), by 2^-10, which is more only where P < 2^-2.  P is
        2^6.5 at the row's largest term when the reference is set there and never less
        than that at a largest seen later, so P < 2^-2 is a term below 2^-8.5 of the
        largest and 2^-10 is 2^-16.5 of it (or all of the term);
      logits in 32 bits: |z| 2^-19 or so in the exponent;
      the bf16 query's hi + lo parts: 2^-18 of the row's largest element;
      the output's rounding to bf16: 2^-8.
    scores[g, i, n]: the largest visible logit of block n over g's heads."""
    dev = q.device
    T, Hq, _ = q.shape
    Hkv = kv.shape[1]
    S = block_table.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    scores = torch.full((Hkv, T, S), -math.inf, dtype=torch.float64, device=dev)
    sides = scales.shape[2]
    i = 0
    for b, n in enumerate(q_lens):
        L = int(seq_lens[b])
        for j in range(n):
            pos, tok, i = L - n + j, i, i + 1
            if pos < 0:
                continue
            for g in range(Hkv):
                blocks = list(range(pos // PAGE + 1)) if lists is None else \
                    [x for x in lists[tok, g].tolist() if x >= 0]
                if not blocks:
                    continue
                pages = block_table[b, blocks].long()
                kk = kv[pages, g, :, :D].view(F8).double() * (scales[pages, g, 0].double() * k_scale)[:, None, None]
                h = slice(GROUP * g, GROUP * (g + 1))
                qq = q[tok, h].double()
                z = torch.einsum("hd,nkd->hnk", qq, kk) * sm
                t = torch.tensor(blocks, device=dev)[:, None] * PAGE + torch.arange(PAGE, device=dev)
                z = torch.where(t <= pos, z, -math.inf)
                scores[g, tok, blocks] = z.amax(dim=(0, 2))
                if sides == 1 or kv.shape[3] == D:
                    continue
                vs = scales[pages, g, 1].double() * v_scale
                v8 = torch.where((t <= pos)[..., None], kv[pages, g, :, D:].view(F8).double(), 0.0)
                v = (v8 * vs[:, None, None]).flatten(0, 1)
                p = torch.softmax(z.flatten(1), dim=1)
                out[tok, h] = p @ v
                size = p @ v.abs()
                zmax = z[z > -math.inf].abs().max()
                seen = torch.where(t <= pos, kk.abs().sum(dim=2), 0.0)
                qerr = 2.0 ** -18 * qq.abs().max() * seen.max() * sm
                # weights of the product with V8, and the largest of each row
                w = p * vs.repeat_interleave(PAGE)
                top = w.amax(dim=1, keepdim=True)
                small = torch.where(w < 2.0 ** -8.5 * top, torch.minimum(2 * w, 2.0 ** -16.5 * top), 0.0)
                floor = small @ v8.flatten(0, 1).abs()
                bound[tok, h] = ((2.0 ** -8 + 2.0 ** -11 + 2 * (zmax * 2.0 ** -19 + qerr)) * size
                                 + floor + HALF_BF16 * out[tok, h].abs())
    return out, bound, scores


def check_attend(got, out, bound):
    assert torch.isfinite(got.float()).all()
    err = (got.double() - out).abs()
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()))


def draw_lists(seq_lens, q_lens, Hkv, gen):
    """Each token's own block and up to 15 earlier ones, in random order with
    unused slots between them."""
    rows = []
    for L, n in zip(seq_lens, q_lens):
        for j in range(n):
            pos = L - n + j
            for _ in range(Hkv):
                row = torch.full((TOPK,), -1, dtype=torch.int32)
                if pos >= 0:
                    cur = pos // PAGE
                    pick = torch.randperm(cur, generator=gen)[:TOPK - 1].tolist() + [cur]
                    at = torch.randperm(TOPK, generator=gen)[:len(pick)]
                    row[at] = torch.tensor(pick, dtype=torch.int32)
                rows.append(row)
    return torch.stack(rows).view(-1, Hkv, TOPK)
