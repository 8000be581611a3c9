"""The block scorer and the block selector of prefill batches (score_prefill,
topk_prefill) against their definitions in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import D, GROUP, PAGE, TOPK
from tests.prefill_ref import Batch, check, cu, every

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def score(x, **kw):
    out = torch.full((x.Hkv, x.T, x.S), 5.0, device="cuda")
    assert msa.score_prefill(*x.args(), scores=out, **x.kw(), **kw) is out
    return out


CASES = [
    # seq_lens, q_lens, Hkv
    ([1], [1], 1),
    ([128], [128], 2),
    ([300, 17, 0, 700], [300, 5, 0, 130], 2),
    ([127, 128, 129, 130], [8, 9, 16, 17], 1),
    ([2100, 1, 640, 256, 255], [33, 1, 0, 256, 24], 4),
    ([5003], [37], 1),
    ([20000], [3], 1),
    ([2500, 901], [1100, 450], 4),
    ([3] * 700, [2] * 700, 1),
]


@pytest.mark.parametrize("seq_lens,q_lens,Hkv", CASES)
@pytest.mark.parametrize("q8,scaled,sides", [(False, False, 2), (True, True, 2), (False, True, 1),
                                             (True, False, 1)])
def test_score_prefill(seq_lens, q_lens, Hkv, q8, scaled, sides):
    x = Batch(seq_lens, q_lens, Hkv, 200 + len(seq_lens), q8=q8, scaled=scaled, sides=sides)
    check(score(x), *every(x, scores=True))
    assert msa.get_error() == 0


def test_same_as_score():
    """Requests of one query length: msa_score's scores, within both bounds."""
    x = Batch([800, 300, 5000, 0], [4, 4, 4, 0], 2, 16)
    got = score(x)
    want = msa.score(x.q, x.kv, x.bt[:3], x.lens[:3], 4, x.sm, x.k_scale)
    _, tol = every(x, scores=True)
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))
    seen = ~torch.isneginf(got)
    assert bool(((got - want).abs()[seen] <= 2 * tol[seen]).all())


def test_wide_table_is_filled():
    x = Batch([300, 90], [40, 90], 2, 3, min_cols=700)
    got = score(x)
    assert got.shape[2] == 700
    check(got, *every(x, scores=True))


def test_bad_pages_scales_and_requests():
    x = Batch([700, 300, 260], [40, 300, 20], 2, 4, scaled=True)
    want, tol = every(x, scores=True)
    x.bt[0, 2] = x.NB
    want[:, :40, 2] = -math.inf
    x.scales[int(x.bt[0, 4]), 1, 0] = float("nan")
    want[1, :40, 4] = -math.inf
    x.scales[int(x.bt[1, 0]), 0, 1] = float("nan")      # V's: the scorer does not read it
    x.lens[2] = 19
    want[:, 340:] = -math.inf
    check(score(x), want, tol)
    assert msa.get_error() == _native.ERR_PAGE_RANGE | _native.ERR_SCALE | _native.ERR_SEQ_RANGE


def test_masked_keys_may_be_anything():
    """NaN and large codes in keys that a token does not see."""
    x = Batch([300], [50], 1, 5)
    want, tol = every(x, scores=True)
    x.kv[int(x.bt[0, 2]), :, 44:] = 0x7F
    x.kv[int(x.bt[0, 2]), :, 60:] = 0x7E
    check(score(x), want, tol)


# ---------------------------------------------------------------------------


def select(scores, seq_lens, q_lens):
    """topk by the definition, on the host."""
    x = scores.double().cpu().numpy()
    x = np.where(np.isnan(x), -math.inf, x)
    Hkv, T, _ = x.shape
    out = np.full((T, Hkv, TOPK), -1, dtype=np.int32)
    i0 = 0
    for n, ql in zip(seq_lens, q_lens):
        for j in range(ql):
            cur = (n - ql + j) // PAGE
            for g in range(Hkv):
                best = np.argsort(-x[g, i0 + j, :cur], kind="stable")[:TOPK - 1]
                kept = sorted(best.tolist()) + [cur]
                out[i0 + j, g, :len(kept)] = kept
        i0 += ql
    return torch.from_numpy(out)


TOPK_CASES = [
    # seq_lens, q_lens, Hkv, S
    ([1], [1], 1, 1),
    ([2048, 2049, 2176, 2177], [5, 9, 128, 130], 2, 18),
    ([300, 0, 9000], [300, 0, 21], 3, 71),
    ([40000, 33000], [33, 7], 2, 400),
    ([70000], [9], 1, 600),
    ([140000], [9], 1, 1100),
    ([300000], [3], 1, 2400),
    ([2300] * 200, [1, 2] * 100, 1, 18),
]


@pytest.mark.parametrize("seq_lens,q_lens,Hkv,S", TOPK_CASES)
@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "infinite"])
def test_topk_prefill(seq_lens, q_lens, Hkv, S, kind):
    gen = torch.Generator().manual_seed(S + len(kind))
    T = sum(q_lens)
    x = torch.randn((Hkv, T, S), generator=gen)
    if kind == "ties":
        x = (x * 2).round() / 2
    elif kind == "equal":
        x = torch.zeros_like(x)
    elif kind == "infinite":
        x = torch.where(x > 1, math.inf, torch.where(x < 0, -math.inf, x))
    lens = torch.tensor(seq_lens, dtype=torch.int32, device="cuda")
    want = select(x, seq_lens, q_lens)
    got = msa.topk_prefill(x.cuda(), lens, cu(q_lens))
    assert torch.equal(got.cpu(), want)
    strided = x.permute(0, 2, 1).contiguous().cuda().transpose(1, 2)     # [Hkv, T, S], S outermost but one
    out = torch.full_like(got, 99)
    assert msa.topk_prefill(strided, lens, cu(q_lens), out=out) is out
    assert torch.equal(out.cpu(), want)
    assert msa.get_error() == 0


def test_topk_prefill_bad_requests_and_nan():
    x = torch.randn((1, 60, 30), generator=torch.Generator().manual_seed(0)).cuda()
    lens = torch.tensor([3000, 29, 2800], dtype=torch.int32, device="cuda")
    at = cu([20, 30, 10])
    got = msa.topk_prefill(x, lens, at)
    want = select(x, [3000, 3000, 2800], [20, 30, 10])
    want[20:50] = -1
    assert torch.equal(got.cpu(), want)
    assert msa.get_error() == _native.ERR_SEQ_RANGE
    x[0, 3, 7] = float("nan")
    lens[1] = 3000
    assert torch.equal(msa.topk_prefill(x, lens, at).cpu(), select(x, lens.tolist(), [20, 30, 10]))
    assert msa.get_error() == _native.ERR_SCORE_NAN


def test_refusals():
    x = Batch([300], [20], 1, 17)
    s = torch.zeros((1, 20, 3), device="cuda")
    none = torch.empty((0, 16, D), dtype=torch.bfloat16, device="cuda")
    assert msa.score_prefill(none, x.kv, x.bt[:0], x.lens[:0], cu([]), x.sm).shape == (1, 0, 3)
    for kw in (dict(scores=torch.zeros((1, 20, 4), device="cuda")), dict(cu_seqlens_q=x.cu[:1]),
               dict(kv_scales=torch.ones((x.NB, 1, 1), device="cuda")), dict(sm_scale=0.0),
               dict(q=x.q.to(torch.float16))):
        a = dict(q=x.q, kv=x.kv, block_table=x.bt, seq_lens=x.lens, cu_seqlens_q=x.cu, sm_scale=x.sm)
        a.update(kw)
        with pytest.raises((ValueError, TypeError, msa.MSAError)):
            msa.score_prefill(**a)
    for a in ((s, x.lens, x.cu[:1]), (s[0], x.lens, x.cu), (s.half(), x.lens, x.cu),
              (s, x.lens.cpu(), x.cu)):
        with pytest.raises((ValueError, TypeError)):
            msa.topk_prefill(*a)
    with pytest.raises((ValueError, msa.MSAError)):
        msa.topk_prefill(s, x.lens, x.cu, k=8)
    assert msa.get_error() == 0


@pytest.mark.parametrize("n,S", [(130, 200), (500, 512), (900, 1024), (2000, 2048)])
@pytest.mark.parametrize("lanes", [1, 3, 14, 15, 31])
def test_topk_prefill_keys_in_few_columns(n, S, lanes):
    """The best blocks all at indices that are the same modulo 32: many keys above the
    15th largest of the 32 columns' maxima, or none."""
    gen = torch.Generator().manual_seed(n + lanes)
    x = torch.randn((2, 12, S), generator=gen)
    col = torch.arange(S) % 32 < lanes
    x[:, :6] = torch.where(col, x[:, :6] + 100, x[:, :6])
    x[:, 6:9] = torch.where(col, 7.0, x[:, 6:9])                        # and all alike
    x[:, 9:] = torch.where(col, (x[:, 9:] * 2).round() + 100, x[:, 9:])  # and with ties
    lens = torch.tensor([n * PAGE + 60], dtype=torch.int32, device="cuda")
    got = msa.topk_prefill(x.cuda(), lens, cu([12]))
    assert torch.equal(got.cpu(), select(x, lens.tolist(), [12]))
    assert torch.equal(msa.topk(x.cuda(), lens, 12).cpu(), got.cpu())


@pytest.mark.parametrize("op", ["score", "dense"])
def test_requests_out_of_order_stay_in_bounds(op):
    """cu_seqlens_q that does not ascend: the error is set, and tokens of a request that is
    in order are right."""
    x = Batch([300, 200, 100], [20, 30, 10], 1, 12)
    x.cu = torch.tensor([0, 20, 5, 60], dtype=torch.int32, device="cuda")
    x.lens[2] = 100                                   # tokens 5 .. 59 of 100
    if op == "score":
        got = score(x)
        want, tol = every(Batch([300, 200, 100], [20, 30, 10], 1, 12), scores=True)
        check(got[:, :5], want[:, :5], tol[:, :5])
    else:
        got = msa.dense_prefill(*x.args(), x.v_scale, **x.kw())
        want, tol = every(Batch([300, 200, 100], [20, 30, 10], 1, 12))
        check(got[:5], want[:5], tol[:5])
    assert msa.get_error() == _native.ERR_SEQ_RANGE
    x.cu = torch.tensor([-7, 20, 1 << 30, 60], dtype=torch.int32, device="cuda")
    (score(x) if op == "score" else msa.dense_prefill(*x.args(), x.v_scale, **x.kw()))
    assert msa.get_error() == _native.ERR_SEQ_RANGE


def test_overlapped_calls_keep_their_order():
    """With input overlap on, append, scorer, selector, sparse and dense attention back to
    back give what they give one by one."""
    x = Batch([1500, 700, 2600], [130, 700, 64], 2, 21, scaled=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((x.T, 2, D), device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    x.scales.copy_(torch.exp2(torch.log2(x.scales).round()))
    kv0, sc0 = x.kv.clone(), x.scales.clone()

    def run(sync):
        x.kv.copy_(kv0)
        x.scales.copy_(sc0)
        torch.cuda.synchronize()
        out = []
        for f in (lambda: msa.append_kv_prefill(k, v, x.kv, x.bt, x.lens, x.cu, kv_scales=x.scales),
                  lambda: out.append(score(x)),
                  lambda: out.append(msa.topk_prefill(out[0], x.lens, x.cu)),
                  lambda: out.append(msa.sparse_prefill(x.q, x.kv, x.bt, x.lens, x.cu, out[1], x.sm,
                                                        kv_scales=x.scales)),
                  lambda: out.append(msa.dense_prefill(*x.args(), **x.kw())),
                  lambda: out.append(msa.score_prefill(*x.args(), **x.kw()))):
            f()
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out

    want = run(True)
    was = msa.set_input_overlap(True)
    try:
        for _ in range(3):
            for a, b in zip(run(False), want):
                assert torch.equal(a, b)
    finally:
        msa.set_input_overlap(was)
    assert msa.get_error() == 0


def test_scores_past_four_billion_bytes():
    """The widest table: scores and lists whose offsets pass 2^31 elements."""
    wide, narrow = (Batch([300], [300], 16, 22, min_cols=m) for m in (1 << 19, 1))
    s, want = score(wide), score(narrow)
    assert s.numel() > 1 << 31 and torch.equal(s[:, :, :narrow.S], want)
    assert bool(torch.isneginf(s[15, :, narrow.S:]).all()) and bool(torch.isneginf(s[0, 299, narrow.S:]).all())
    lists = msa.topk_prefill(s, wide.lens, wide.cu)
    assert torch.equal(lists, msa.topk_prefill(want, narrow.lens, narrow.cu))
    assert msa.get_error() == 0


@pytest.mark.parametrize("n,S", [(2048, 2049), (2049, 2060), (2079, 2080), (5000, 5003), (70001, 70010)])
@pytest.mark.parametrize("lanes", [0, 1, 15, 31])
def test_long_rows(n, S, lanes):
    """Rows of more blocks than a warp holds, beside shorter ones: drawn, with ties, alike, in
    few columns, with NaN and with -inf."""
    gen = torch.Generator().manual_seed(n + lanes)
    x = torch.randn((2, 14, S), generator=gen)
    if lanes:
        x[:, ::2] = torch.where(torch.arange(S) % 32 < lanes, x[:, ::2] + 100, x[:, ::2])
    x[0, 3] = 1.0
    x[:, 4:6] = (x[:, 4:6] * 2).round()
    x[:, 6, 20:] = -math.inf
    x[1, 7] = -math.inf
    x[:, 8, ::3] = float("nan")
    lens = torch.tensor([n * PAGE + 60, 3000], dtype=torch.int32, device="cuda")
    at = cu([12, 2])
    got = msa.topk_prefill(x.cuda(), lens, at)
    assert torch.equal(got.cpu(), select(x, lens.tolist(), [12, 2]))
    assert msa.get_error() == _native.ERR_SCORE_NAN
    clean = x[:, :12].nan_to_num(nan=-math.inf, neginf=-math.inf).cuda()
    assert torch.equal(msa.topk(clean, lens[:1], 12), got[:12])
    wide = torch.empty((2, 12, S, 2), device="cuda")
    wide[..., 1] = clean
    assert torch.equal(msa.topk(wide[..., 1], lens[:1], 12), got[:12])
    assert msa.get_error() == 0
