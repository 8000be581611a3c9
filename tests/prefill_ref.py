"""Plain 64-bit forms of dense attention and block scores of prefill batches, and the
error bounds that their tests use.  Written from the definitions (include/msa.h), request
by request, with elementary torch operations."""
from __future__ import annotations

import math

import torch

from tests.page_cache import D, F8, GROUP, PAGE, codes, layout

# Bounds of the kernels' roundings.
#  - a dot product: 128 products, fp8 parts summed in fp32 in two halves, 2^8 sums of at
#    most 2^-24 of the absolute sum: 2^-16 of sum |q k|; the query's parts lose at most
#    2^-18 of the rows' largest |q| an element (bf16; fp8 nothing)
#  - a weight: fp16, 2^-11 of itself; ex2.approx and fp32 sums over a page and over
#    pages are far below another 2^-11: 2^-10 of sum p |v|, and both sides of the
#    quotient carry the logits' error: twice dz (p moves by the factor e^dz)
#  - a weight below 2^-21 of the largest (times V scales): fp16's step ends at 2^-24, the
#    largest is at least 2^7: at most 2^-32 of it, for each key, times |V8| <= 448
#  - the result: bf16, 2^-8 of itself
DOT, PART, WEIGHT, HALF_BF16 = 2.0 ** -16, 2.0 ** -18, 2.0 ** -10, 2.0 ** -8


def cu(q_lens, device="cuda"):
    c = [0]
    for n in q_lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


class Batch:
    """A drawn batch on the GPU: cache, table, lengths, query, page scales."""

    def __init__(self, seq_lens, q_lens, Hkv, seed, *, q8=False, scaled=False, sides=2, nan=0.0,
                 min_cols=1, spare=2, std=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.seq_lens, self.q_lens, self.Hkv = list(seq_lens), list(q_lens), Hkv
        bt, self.NB = layout(seq_lens, gen, spare=spare, min_cols=min_cols)
        T = sum(q_lens)
        self.kv = codes((self.NB, Hkv, PAGE, D * sides), gen, nan).cuda()
        self.scales = None
        self.k_scale, self.v_scale = 0.0071, 0.0068
        if scaled:
            self.scales = torch.exp2(torch.randn((self.NB, Hkv, sides), generator=gen) * 1.5 - 8.0).cuda()
            self.k_scale, self.v_scale = 1.0, 1.0
        q = torch.randn((T, GROUP * Hkv, D), generator=gen) * std
        self.q_scale = 1.0
        if q8:
            self.q_scale = 0.0123
            self.q = (q / self.q_scale).clamp(-448, 448).to(F8).cuda()
        else:
            self.q = q.to(torch.bfloat16).cuda()
        self.bt, self.lens = bt.cuda(), torch.tensor(seq_lens, dtype=torch.int32).cuda()
        self.cu = cu(q_lens)
        self.S, self.T, self.sm = self.bt.shape[1], T, D ** -0.5

    def args(self):
        return self.q, self.kv, self.bt, self.lens, self.cu, self.sm, self.k_scale

    def kw(self):
        return dict(q_scale=self.q_scale, kv_scales=self.scales)


def _logits(x: Batch, b, g, j0, j1, f=torch.float64):
    """(logits [j, 16, keys], bound on their error, V [keys, 128], pages)."""
    n = x.seq_lens[b]
    pages = x.bt[b, :-(-n // PAGE)].long()
    c = x.kv[pages, g].view(F8).to(f)
    sc = (x.scales[pages, g].to(f) if x.scales is not None
          else torch.ones((len(pages), 2), dtype=f, device=x.kv.device))
    k = (c[..., :D] * sc[:, :1, None]).reshape(-1, D) * float(torch.tensor(x.k_scale))
    v = ((c[..., D:] * sc[:, 1:, None]).reshape(-1, D) * float(torch.tensor(x.v_scale))
         if c.shape[2] == 2 * D else None)
    i0 = int(sum(x.q_lens[:b]))
    q = x.q[i0 + j0:i0 + j1, GROUP * g:GROUP * (g + 1)].to(f) * float(torch.tensor(x.q_scale))
    z = torch.einsum("jhd,kd->jhk", q, k) * x.sm
    dz = torch.einsum("jhd,kd->jhk", q.abs(), k.abs()) * (x.sm * DOT)
    if x.q.dtype == torch.bfloat16:
        dz += q.abs().amax(dim=(1, 2), keepdim=True) * k.abs().sum(dim=1) * (x.sm * PART)
    return z, dz, v, pages


def every(x: Batch, scores=False, step=64):
    """(output [T, Hq, 128], bound) or, with scores, (scores [Hkv, T, S], bound)."""
    f, dev = torch.float64, x.kv.device
    if scores:
        out = torch.full((x.Hkv, x.T, x.S), -math.inf, dtype=f, device=dev)
    else:
        out = torch.zeros((x.T, GROUP * x.Hkv, D), dtype=f, device=dev)
    tol = torch.zeros_like(out)
    i0 = 0
    for b, (n, ql) in enumerate(zip(x.seq_lens, x.q_lens)):
        for g in range(x.Hkv if ql else 0):
            for j0 in range(0, ql, step):
                j1 = min(ql, j0 + step)
                z, dz, v, pages = _logits(x, b, g, j0, j1)
                key = torch.arange(z.shape[2], device=dev)
                seen = (key <= (n - ql + torch.arange(j0, j1, device=dev))[:, None])[:, None]
                z = z.masked_fill(~seen, -math.inf)
                at = slice(i0 + j0, i0 + j1)
                if scores:
                    blocks = (j1 - j0, GROUP, len(pages), PAGE)
                    out[g, at, :len(pages)] = z.view(blocks).amax(dim=(1, 3))
                    tol[g, at, :len(pages)] = dz.view(blocks).amax(dim=(1, 3)) + \
                        out[g, at, :len(pages)].abs().nan_to_num(0.0, 0.0, 0.0) * 2.0 ** -21
                    continue
                p = torch.softmax(z, dim=2)
                h = slice(GROUP * g, GROUP * (g + 1))
                # (keys that are not seen have no part in it, whatever their values are)
                v = torch.where(seen.any(dim=0).any(dim=0)[:, None], v, 0.0)
                out[at, h] = torch.einsum("jhk,kd->jhd", p, v)
                size = torch.einsum("jhk,kd->jhd", p, v.abs())
                worst = torch.where(seen, dz, 0.0).amax(dim=2, keepdim=True)
                vs = x.v_scale * (float(x.scales[pages, g, 1].max()) if x.scales is not None else 1.0)
                tol[at, h] = (WEIGHT + 2 * worst) * size + len(key) * 2.0 ** -32 * 448 * vs
        i0 += ql
    if not scores:
        tol += HALF_BF16 * out.abs()
    return out, tol


def check(got, want, tol):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))
    off = ((got - want).abs() - tol)[fin]
    if off.numel():
        assert bool((off <= 0).all()), (float(off.max()), int((off > 0).sum()))
