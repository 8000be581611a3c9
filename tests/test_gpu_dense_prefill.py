"""Dense attention of prefill batches (dense_prefill) against its definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import D, F8, GROUP, PAGE
from tests.prefill_ref import Batch, check, cu, every

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def run(x, **kw):
    out = torch.full((x.T, GROUP * x.Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = msa.dense_prefill(*x.args(), x.v_scale, out=out, **x.kw(), **kw)
    assert got is out
    return out


CASES = [
    # seq_lens, q_lens, Hkv
    ([1], [1], 1),
    ([5], [5], 2),
    ([128], [128], 1),
    ([129], [1], 1),
    ([257], [130], 3),
    ([300, 17, 0, 700], [300, 5, 0, 130], 2),
    ([127, 128, 129, 130], [8, 9, 16, 17], 1),
    ([1000, 1, 640, 256, 255], [33, 1, 0, 256, 24], 4),
    ([5003], [37], 1),                    # a few units: every one cut over many CTAs
    ([20000], [3], 1),
    ([2500, 901], [1100, 450], 4),        # more units than CTAs
    ([3] * 700, [2] * 700, 1),            # more requests than threads of a block
    ([200, 30] * 300, [7, 0] * 300, 2),
]


@pytest.mark.parametrize("seq_lens,q_lens,Hkv", CASES)
@pytest.mark.parametrize("q8,scaled", [(False, False), (True, True), (False, True), (True, False)])
def test_dense_prefill(seq_lens, q_lens, Hkv, q8, scaled):
    x = Batch(seq_lens, q_lens, Hkv, 100 + len(seq_lens), q8=q8, scaled=scaled)
    check(run(x), *every(x))
    assert msa.get_error() == 0


@pytest.mark.parametrize("scaled", [False, True])
def test_growing_maxima(scaled):
    """Keys whose logits grow along the row: the reference moves again and again, inside
    pages and between them, by less and by more than its headroom."""
    x = Batch([1500], [40], 1, 7, scaled=scaled)
    x.q[:] = 0
    x.q[..., 0] = 4.0
    at = torch.arange(1500, device="cuda")
    level = (at.double() / 1500 * 440).float()
    k = x.kv.view(F8)
    for n, page in enumerate(x.bt[0].tolist()):
        rows = level[n * PAGE:(n + 1) * PAGE]
        k[page, 0, :len(rows), 0] = rows.to(F8)
    x.k_scale = 0.5 if not scaled else 1.0
    if scaled:
        x.scales[..., 0] = 0.5
    check(run(x), *every(x))


def test_a_dominant_key_and_a_long_tail():
    """One key of half the weight and 32767 that share the rest: what is small is not lost."""
    n = 32768
    x = Batch([n], [20], 1, 8)
    x.q[:] = 0
    x.q[..., 0] = 1.0
    k = x.kv.view(F8)
    k[..., 0] = 0
    x.k_scale = 0.25
    first = int(x.bt[0, 3])
    k[first, 0, 5, 0] = 448.0            # logit 448 / 4 * D^-1/2 = 9.9, e^9.9 = 19930
    check(run(x), *every(x))


def test_scales_far_apart():
    """Pages whose V scales differ by powers up to 2^40 and whose keys compensate."""
    x = Batch([900, 400], [21, 400], 2, 9, scaled=True)
    e = torch.randint(-20, 20, x.scales.shape[:2], generator=torch.Generator().manual_seed(1))
    x.scales[..., 1] = torch.exp2(e.float()).cuda()
    got = run(x)
    want, tol = every(x)
    check(got, want, tol)


@pytest.mark.parametrize("scaled", [False, True])
def test_nan_reaches_who_sees_it(scaled):
    """NaN in rows behind the sequence, in keys and in values of the chunk itself."""
    x = Batch([300, 200], [50, 200], 2, 10, scaled=scaled)
    kv = x.kv
    for b, n in enumerate(x.seq_lens):       # rows that belong to no token yet
        kv[int(x.bt[b, n // PAGE]), :, n % PAGE:] = 0x7F
    for b, key, side, d, g in [(0, 270, 1, 5, 0), (0, 299, 1, 127, 1), (0, 255, 1, 0, 1),
                               (0, 256, 1, 77, 0), (1, 0, 1, 3, 1), (1, 130, 1, 64, 0),
                               (1, 150, 0, 9, 1), (0, 290, 0, 0, 0), (0, 20, 1, 33, 0)]:
        kv[int(x.bt[b, key // PAGE]), g, key % PAGE, side * D + d] = 0xFF
    got = run(x)
    want, tol = every_with_nan(x)
    check(got, want, tol)
    assert bool(torch.isnan(want).any()) and not bool(torch.isnan(want).all())


def every_with_nan(x):
    """The definition where codes are NaN: a key takes part for the tokens that see it
    and not at all for the others."""
    clean = Batch(x.seq_lens, x.q_lens, x.Hkv, 10, scaled=x.scales is not None)
    clean.q, clean.bt, clean.scales = x.q, x.bt, x.scales
    clean.kv = torch.where((x.kv & 0x7F) == 0x7F, torch.zeros_like(x.kv), x.kv)
    want, tol = every(clean)
    i0 = 0
    for b, (n, ql) in enumerate(zip(x.seq_lens, x.q_lens)):
        c = (x.kv[x.bt[b, :-(-n // PAGE)].long()] & 0x7F) == 0x7F     # [pages, Hkv, 128, 256]
        c = c.transpose(1, 2).flatten(0, 1)                            # [keys, Hkv, 256]
        for j in range(ql):
            seen = c[:n - ql + j + 1]
            for g in range(x.Hkv):
                rows = slice(GROUP * g, GROUP * (g + 1))
                if bool(seen[:, g, :D].any()):
                    want[i0 + j, rows] = float("nan")
                want[i0 + j, rows][:, seen[:, g, D:].any(dim=0)] = float("nan")
        i0 += ql
    return want, tol


def test_bad_pages_and_scales_are_skipped():
    x = Batch([700, 300], [40, 300], 2, 11, scaled=True)
    y = Batch([700, 300], [40, 300], 2, 11, scaled=True)
    x.bt[0, 2] = x.NB + 5
    x.bt[1, 1] = -3
    x.scales[int(x.bt[0, 4]), 1, 0] = 2.0 ** 41
    x.scales[int(x.bt[0, 0]), 0, 1] = float("nan")
    got = run(x)
    assert msa.get_error() == _native.ERR_PAGE_RANGE | _native.ERR_SCALE
    # the same without those keys: their K so far below the others that they have no weight
    want, tol = [], []
    for g in range(2):
        gone = {(0, 2), (1, 1)} | ({(0, 4)} if g == 1 else {(0, 0)})
        o, t = every_without(y, gone)
        want.append(o[:, GROUP * g:GROUP * (g + 1)])
        tol.append(t[:, GROUP * g:GROUP * (g + 1)])
    check(got, torch.cat(want, 1), torch.cat(tol, 1))


def every_without(x, gone):
    """The definition without the pages (b, n) in `gone`."""
    f = torch.float64
    out = torch.zeros((x.T, GROUP * x.Hkv, D), dtype=f, device="cuda")
    tol = torch.zeros_like(out)
    from tests.prefill_ref import WEIGHT, HALF_BF16, _logits
    i0 = 0
    for b, (n, ql) in enumerate(zip(x.seq_lens, x.q_lens)):
        for g in range(x.Hkv):
            z, dz, v, pages = _logits(x, b, g, 0, ql)
            key = torch.arange(z.shape[2], device="cuda")
            off = torch.tensor([(b, m) in gone for m in range(len(pages))], device="cuda")
            seen = (key <= (n - ql + torch.arange(ql, device="cuda"))[:, None]) & ~off.repeat_interleave(PAGE)
            z = z.masked_fill(~seen[:, None], float("-inf"))
            p = torch.softmax(z, dim=2).nan_to_num(0.0)
            h = slice(GROUP * g, GROUP * (g + 1))
            out[i0:i0 + ql, h] = torch.einsum("jhk,kd->jhd", p, v)
            tol[i0:i0 + ql, h] = (WEIGHT + 2 * dz.amax()) * torch.einsum("jhk,kd->jhd", p, v.abs()) + 1e-9
        i0 += ql
    return out, tol + HALF_BF16 * out.abs()


def test_rows_that_see_nothing_are_zero():
    """A request all of whose pages are bad; requests with bad lengths; tokens of nobody."""
    x = Batch([300, 200, 100], [20, 30, 10], 1, 12)
    x.bt[1] = -1
    got = run(x)
    assert msa.get_error() == _native.ERR_PAGE_RANGE
    want, tol = every(Batch([300, 200, 100], [20, 30, 10], 1, 12))
    want[20:50], tol[20:50] = 0, 0
    check(got, want, tol)

    for change in ("too long", "negative", "past the table", "before", "behind"):
        x = Batch([300, 200, 100], [20, 30, 10], 1, 12)
        want, tol = every(x)
        zero = slice(20, 50)
        if change == "too long":
            x.lens[1] = 29
        elif change == "negative":
            x.lens[1] = -1
        elif change == "past the table":
            x.lens[1] = x.S * PAGE + 1
        elif change == "before":
            x.cu = torch.tensor([4, 20, 50, 60], dtype=torch.int32, device="cuda")
            x.lens[0] = 300                      # its tokens are the last 16 of 300
            zero = slice(0, 4)
        else:
            x.cu = torch.tensor([0, 20, 50, 57], dtype=torch.int32, device="cuda")
            x.lens[2] = 97
            zero = slice(57, 60)
        want[zero], tol[zero] = 0, 0
        check(run(x), want, tol)
        assert msa.get_error() == _native.ERR_SEQ_RANGE, change


def test_past_two_gigabytes():
    """Pages whose bytes lie past 2^31 and 2^32."""
    NB = 140000
    x = Batch([700], [60], 1, 13)
    kv = torch.zeros((NB, 1, PAGE, 2 * D), dtype=torch.uint8, device="cuda")
    far = torch.tensor([NB - 1 - 7919 * i for i in range(x.S)], dtype=torch.int32, device="cuda")
    kv[far.long()] = x.kv[x.bt[0].long()]
    want, tol = every(x)
    x.kv, x.bt = kv, far[None].contiguous()
    check(run(x), want, tol)


def test_same_bits_whatever_runs_beside_it():
    """The parts' places and order go by the shapes: the bits are the same again, in a
    graph, on another stream and beside another call with its own workspace."""
    x, y = Batch([3000, 700], [50, 300], 2, 14), Batch([9000], [100], 1, 15, scaled=True)
    want_x, want_y = run(x).clone(), run(y).clone()
    ws = [torch.full((msa.dense_prefill_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    assert torch.equal(run(x, workspace=ws[0]), want_x)
    outs = [torch.empty_like(want_x), torch.empty_like(want_y)]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for z, o, w, s in zip((x, y), outs, ws, side):
            msa.dense_prefill(*z.args(), z.v_scale, out=o, workspace=w, stream=s, **z.kw())
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want_x) and torch.equal(outs[1], want_y)
    g = torch.cuda.CUDAGraph()
    outs[0].zero_()
    with torch.cuda.graph(g):
        msa.dense_prefill(*x.args(), x.v_scale, out=outs[0], workspace=ws[0], **x.kw())
    x.q.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], run(x)) and not torch.equal(outs[0], want_x)


def test_same_as_dense_decode():
    """Requests of one query length: what dense_decode gives on page scales, within both
    bounds."""
    x = Batch([800, 300, 5000], [4, 4, 4], 2, 16, scaled=True)
    want, tol = every(x)
    got = run(x)
    check(got, want, tol)
    dec = msa.dense_decode(x.q, x.kv, x.bt, x.lens, 4, x.sm, kv_scales=x.scales)
    assert float((dec.double() - got.double()).abs().max()) <= float((2 * tol).max()) + 2.0 ** -7


def test_empty_batches_and_refusals():
    x = Batch([300], [20], 1, 17)
    none = torch.empty((0, 16, D), dtype=torch.bfloat16, device="cuda")
    assert msa.dense_prefill(none, x.kv, x.bt[:0], x.lens[:0], cu([]), x.sm).shape == none.shape
    for kw in (dict(cu_seqlens_q=x.cu[:1]), dict(out=torch.empty((20, 16, 64), dtype=torch.bfloat16, device="cuda")),
               dict(kv_scales=torch.ones((x.NB, 1, 1), device="cuda")), dict(q=x.q[0]),
               dict(kv=x.kv[..., :D].contiguous()), dict(seq_lens=x.lens.cpu()), dict(q=x.q[:, ::2])):
        a = dict(q=x.q, kv=x.kv, block_table=x.bt, seq_lens=x.lens, cu_seqlens_q=x.cu)
        a.update(kw)
        with pytest.raises((ValueError, TypeError, msa.MSAError)):
            msa.dense_prefill(**a, sm_scale=x.sm)
    with pytest.raises(msa.MSAError):
        msa.dense_prefill(*x.args(), float("nan"))
    with pytest.raises(msa.MSAError):
        msa.dense_prefill(x.q, x.kv, x.bt, x.lens, x.cu, -1.0)
    assert msa.get_error() == 0


def test_nan_reaches_across_parts():
    """A row that many CTAs share, with NaN in keys and values whose parts weigh nothing
    beside the rest: 0 times NaN is NaN however the row was cut."""
    n = 9000
    x = Batch([n], [20], 2, 17)
    x.q[:] = 0
    x.q[..., 0] = 2048.0
    k = x.kv.view(F8)
    k[..., :D] = 0
    for page in x.bt[0, :-(-n // PAGE)].tolist():
        k[page, :, :, 0] = -448.0
    k[int(x.bt[0, 60]), :, 7, 0] = 448.0      # 448 * 2048 * 0.0071 / D^1/2 = 576 against -576
    for key, g, d in [(3, 0, D + 5), (2000, 0, D + 9), (4100, 1, D + 127), (8999, 1, D)]:
        x.kv[int(x.bt[0, key // PAGE]), g, key % PAGE, d] = 0x7F
    want, tol = every_with_nan(x)
    assert 0 < int(torch.isnan(want).sum()) < want.numel() // 16
    check(run(x), want, tol)
    x.kv[int(x.bt[0, 2]), 1, 44, 17] = 0xFF   # a key: the whole of its heads
    got = run(x)
    assert bool(torch.isnan(got[:, GROUP:]).all())
    assert torch.equal(torch.isnan(got[:, :GROUP]), torch.isnan(want[:, :GROUP]))


@pytest.mark.parametrize("sm,k_scale", [(1e-25, 1e-25), (1e-30, 1e-12)])
def test_scales_that_vanish(sm, k_scale):
    """Logits that are all 0 in fp32, the factors' product too: every visible key counts alike."""
    x = Batch([300, 130], [50, 130], 1, 18)
    x.sm, x.k_scale = sm, k_scale
    x.q *= 2.0 ** -100
    check(run(x), *every(x))


def test_workspace_of_the_call_on_another_stream():
    """A call on a given stream without a workspace: its own is not handed to other tensors
    while that stream works with it."""
    x = Batch([9000, 300], [40, 300], 2, 19)
    want = run(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    need = msa.dense_prefill_workspace_bytes("cuda")
    for _ in range(4):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)
        out = msa.dense_prefill(*x.args(), x.v_scale, stream=side, **x.kw())
        junk = torch.full((need,), 0x55, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, want) and int(junk[0]) == 0x55
    wide = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need)
    with pytest.raises(ValueError):
        msa.dense_prefill(*x.args(), x.v_scale, workspace=wide, **x.kw())


def test_a_million_tokens():
    """As many requests as a call takes, rows of q and out past 2^31 elements: every copy of
    a batch of 4 gives what the batch gives."""
    x = Batch([17, 40, 130, 1], [17, 40, 20, 1], 1, 20)
    want, tol = every(x)
    n = 16368
    lens = list(x.q_lens) * n
    q = x.q.repeat(n, 1, 1)
    cus = cu(lens)
    bt, sl = x.bt.repeat(n, 1), x.lens.repeat(n)
    assert sl.numel() == 65472 and q.numel() > 1 << 31
    out = msa.dense_prefill(q, x.kv, bt, sl, cus, x.sm, x.k_scale, x.v_scale)
    for k in (0, 1, n // 2, n - 2, n - 1):
        check(out[k * x.T:(k + 1) * x.T], want, tol)
    s = msa.score_prefill(q, x.kv, bt, sl, cus, x.sm, x.k_scale)
    assert torch.equal(s.view(1, n, x.T, x.S), s[:, -x.T:].view(1, 1, x.T, x.S).expand(1, n, x.T, x.S))
    assert msa.get_error() == 0
