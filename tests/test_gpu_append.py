"""The cache append (append_kv, append_kv_prefill) against its definition in 64
bits: every written code within half an e4m3 step, every other byte as it was."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import (D, F8, GROUP, PAGE, Append, check_bf16, check_e4m3, codes, layout,
                              table)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def _case(seq_lens, q_lens, Hkv, seed, *, sides=2, scaled=False, rot=64, fused=True, std=1.0,
          min_cols=1):
    """Host draws: a cache of random codes, scales, and T new tokens whose rows
    are slices of one projection (fused) or tensors of their own."""
    gen = torch.Generator().manual_seed(seed)
    bt, nb = layout(seq_lens, gen, min_cols=min_cols)
    Hq, T = GROUP * Hkv, sum(q_lens)
    kv = codes((nb, Hkv, PAGE, D * sides), gen, nan=0.001)
    sc = torch.exp2(torch.randint(-9, -5, (nb, Hkv, sides), generator=gen).float()) if scaled else None
    x = (torch.randn((T, (Hq + 2 * Hkv) * D + 8), generator=gen) * std).to(torch.bfloat16)
    rows = x[:, :-8].reshape(T, -1, D) if not fused else x.to(DEV)[:, :-8].unflatten(1, (-1, D))
    q, k, v = rows.to(DEV).split([Hq, Hkv, Hkv], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if sides == 1:
        v = None
    cs = table(max(max(seq_lens), 1), rot) if rot else None
    return dict(bt=bt.to(DEV), lens=torch.tensor(seq_lens, dtype=torch.int32, device=DEV),
                kv=kv.to(DEV), sc=None if sc is None else sc.to(DEV), q=q, k=k, v=v, cs=cs,
                seq_lens=list(seq_lens), q_lens=list(q_lens))


def _check_q(q_out, want, size, q_scale=1.0):
    if q_out.dtype == torch.bfloat16:
        check_bf16(q_out.cpu(), want, size)
    else:
        s = float(torch.tensor(q_scale))
        check_e4m3(q_out.cpu().flatten(), (want / s).flatten(), (6 * 2.0 ** -24 * size / s).flatten())


DECODE = [
    # seq_lens, Q, Hkv, rot, interleaved, scaled
    ([1], 1, 1, 128, False, False),
    ([2048, 3000], 1, 1, 128, False, True),
    ([257, 513, 0, 129], 1, 4, 64, False, True),
    ([257, 513, 2, 0, 128, 129], 4, 4, 64, True, True),       # page borders, padding rows
    ([257, 513, 2, 0, 128, 129], 4, 4, 64, True, False),
    ([130, 1, 127, 256], 2, 3, 0, False, True),
    ([300, 15, 16, 17], 16, 2, 96, False, True),              # the most rows of one warp
    ([300, 15, 16, 17], 17, 2, 96, True, True),               # one more
    ([500, 31, 140, 0], 32, 1, 16, False, True),
    ([500, 31, 140, 0], 32, 2, 112, False, False),
    ([4000] * 70, 1, 2, 32, False, True),
]


@pytest.mark.parametrize("seq_lens,Q,Hkv,rot,inter,scaled", DECODE)
@pytest.mark.parametrize("fused", [True, False])
def test_decode_append(seq_lens, Q, Hkv, rot, inter, scaled, fused):
    c = _case(seq_lens, [Q] * len(seq_lens), Hkv, 11 + Q, scaled=scaled, rot=rot, fused=fused)
    ks, vs = (1.0, 1.0) if scaled else (0.011, 0.013)
    ref = Append(c["kv"], c["sc"], c["bt"], seq_lens, ks, vs)
    want, size = ref.run(c["k"], c["v"], c["q"], c["q_lens"], c["cs"], inter)
    out = msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], Q, ks, vs, kv_scales=c["sc"],
                        cos_sin=c["cs"], interleaved=inter, q=c["q"])
    ref.check(c["kv"], c["sc"])
    _check_q(out, want, size)
    assert msa.get_error() == 0


PREFILL = [
    # seq_lens, q_lens, Hkv, rot, interleaved, scaled
    ([1], [1], 1, 64, False, True),
    ([129, 5000, 128, 700], [129, 37, 128, 0], 1, 64, False, True),
    ([129, 5000, 128, 700], [129, 37, 128, 0], 4, 128, True, False),
    ([1000, 0, 513, 257], [400, 0, 513, 130], 2, 32, False, True),
    ([700] * 40, [3, 1, 0, 130, 2] * 8, 1, 64, True, True),
    ([3000, 126, 255, 384], [1500, 126, 128, 256], 4, 64, False, True),
]


@pytest.mark.parametrize("seq_lens,q_lens,Hkv,rot,inter,scaled", PREFILL)
@pytest.mark.parametrize("q8", [False, True])
def test_prefill_append(seq_lens, q_lens, Hkv, rot, inter, scaled, q8):
    c = _case(seq_lens, q_lens, Hkv, 31, scaled=scaled, rot=rot)
    cu = torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32, device=DEV)
    ks, vs = (0.5, 2.0) if scaled else (0.011, 0.013)
    ref = Append(c["kv"], c["sc"], c["bt"], seq_lens, ks, vs)
    want, size = ref.run(c["k"], c["v"], c["q"], q_lens, c["cs"], inter)
    qo = torch.full(c["q"].shape, 3.0, device=DEV).to(F8 if q8 else torch.bfloat16)
    out = msa.append_kv_prefill(c["k"], c["v"], c["kv"], c["bt"], c["lens"], cu, ks, vs,
                                kv_scales=c["sc"], cos_sin=c["cs"], interleaved=inter, q=c["q"],
                                q_out=qo, q_scale=0.0093)
    assert out is qo
    ref.check(c["kv"], c["sc"])
    _check_q(out, want, size, 0.0093)
    assert msa.get_error() == 0


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("Q", [1, 5])
def test_k_only_cache(scaled, Q):
    lens = [257, 130, 3]
    c = _case(lens, [Q] * 3, 2, 5, sides=1, scaled=scaled)
    ref = Append(c["kv"], c["sc"], c["bt"], lens, 0.01)
    ref.run(c["k"], None, None, c["q_lens"], c["cs"])
    assert msa.append_kv(c["k"], None, c["kv"], c["bt"], c["lens"], Q, 0.01, kv_scales=c["sc"],
                         cos_sin=c["cs"]) is None
    ref.check(c["kv"], c["sc"])
    assert msa.get_error() == 0


def test_query_in_place():
    c = _case([257, 40, 0], [4] * 3, 2, 6, fused=False)
    q = c["q"].clone()
    want = msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], 4, 0.01, 0.01,
                         cos_sin=c["cs"], q=q)
    assert msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], 4, 0.01, 0.01,
                         cos_sin=c["cs"], q=c["q"], q_out=c["q"]) is c["q"]
    assert torch.equal(c["q"], want)


def _one(x_rows, scales, kv, start, v_rows=None):
    """Appends rows [n, 128] at position `start` of a one-request, one-head cache."""
    n = x_rows.shape[0]
    L = torch.tensor([start + n], dtype=torch.int32, device=DEV)
    bt = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    k = x_rows[:, None].contiguous().to(DEV)
    v = (x_rows if v_rows is None else v_rows)[:, None].contiguous().to(DEV)
    msa.append_kv_prefill(k, v, kv, bt, L, cu, kv_scales=scales)


def test_a_page_scale_grows_and_requantises_the_rows_before():
    """Rows appended one by one: 100 of ones, then one of 10000; the scale is the
    power of two that holds the largest, and the earlier codes follow it."""
    kv = torch.full((2, 1, PAGE, 2 * D), 0x55, dtype=torch.uint8, device=DEV)
    sc = torch.full((2, 1, 2), float("nan"), device=DEV)        # a fresh page reads no old scale
    ones = torch.ones((1, D), dtype=torch.bfloat16)
    for r in range(100):
        _one(ones, sc, kv, r)
    assert sc[0].tolist() == [[2.0 ** -8, 2.0 ** -8]]           # 1 <= 448 / 256, not 448 / 512
    big = ones * 10000
    _one(big, sc, kv, 100, v_rows=ones)
    assert sc[0].tolist() == [[2.0 ** 5, 2.0 ** -8]]            # 10000 <= 448 * 32
    k = kv[0, 0, :101, :D].view(F8).float() * 2.0 ** 5
    assert (k[:100] == 1.0).all() and (k[100] == float(torch.tensor(10000.0 / 32).to(F8)) * 32).all()
    assert (kv[0, 0, :101, D:].view(F8).float() * 2.0 ** -8 == 1.0).all()
    assert (kv[0, 0, 101:] == 0x55).all() and (kv[1] == 0x55).all()
    assert torch.isnan(sc[1]).all()
    # the page started anew: row 0 sets the scale again, down too
    _one(ones, sc, kv, 0)
    assert sc[0].tolist() == [[2.0 ** -8, 2.0 ** -8]]
    assert msa.get_error() == 0


def test_page_scale_borders_and_extremes():
    """amax at, and just past, 448 s; zeros; values past both bounds of the
    scale; infinities saturate and take no part in the scale, NaN stays NaN."""
    for amax, want in [(448.0, 1.0), (450.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                       (0.0, 2.0 ** -40), (1e-30, 2.0 ** -40), (1e30, 2.0 ** 40),
                       (3.3895313892515355e38, 2.0 ** 40)]:
        x = torch.zeros((3, D), dtype=torch.bfloat16)
        x[1, 7], x[2, 100] = -amax, amax / 2
        assert float(x[1, 7]) == -amax or amax in (1e-30, 1e30)
        kv = torch.zeros((2, 1, PAGE, 2 * D), dtype=torch.uint8, device=DEV)
        sc = torch.zeros((2, 1, 2), device=DEV)
        _one(x, sc, kv, 0)
        assert sc[0, 0].tolist() == [want, want], amax
        got = kv[0, 0, :3, :D].view(F8).float().cpu()
        ref = (x.double() / want).clamp(-448, 448)
        check_e4m3(got.flatten(), ref.flatten(), torch.zeros(3 * D, dtype=torch.float64))
    x = torch.ones((1, D), dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 2] = float("inf"), float("-inf"), float("nan")
    kv = torch.zeros((2, 1, PAGE, 2 * D), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((2, 1, 2), device=DEV)
    _one(x, sc, kv, 0)
    assert sc[0, 0, 0] == 2.0 ** -8
    got = kv[0, 0, 0, :D].view(F8).float()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 256


@pytest.mark.parametrize("chunks", [[1] * 300, [130, 1, 125, 44], [300]])
def test_page_scales_do_not_depend_on_the_chunks(chunks):
    """However 300 tokens are cut into appends, a page's scale is that of its
    largest value; the codes of a page whose scale never grew afterwards are the
    single roundings."""
    gen = torch.Generator().manual_seed(9)
    x = (torch.randn((300, D), generator=gen) * torch.logspace(-1, 1, 300)[:, None]).to(torch.bfloat16)
    kv = torch.zeros((3, 1, PAGE, 2 * D), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((3, 1, 2), device=DEV)
    bt = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    at = 0
    for n in chunks:
        L = torch.tensor([at + n], dtype=torch.int32, device=DEV)
        k = x[at:at + n, None].contiguous().to(DEV)
        if n <= 32:
            msa.append_kv(k, k, kv, bt, L, n, kv_scales=sc)
        else:
            cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            msa.append_kv_prefill(k, k, kv, bt, L, cu, kv_scales=sc)
        at += n
    from tests.page_cache import power_for
    for n, page in enumerate((2, 0, 1)):
        rows = x[n * PAGE:(n + 1) * PAGE]
        s = power_for(float(rows.abs().max()))
        assert sc[page].tolist() == [[s, s]]
        got = kv[page, 0, :rows.shape[0], :D].view(F8).double().cpu()
        # a value requantised through k growths: half a step each time, at a
        # step no larger than the last one's
        v = rows.double() / s
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        most = 1 if len(chunks) == 1 else 8
        assert ((got - v).abs() <= most * torch.exp2(e - 3) / 2).all()


@pytest.mark.parametrize("scaled", [False, True])
def test_bad_entries_are_flagged_and_skipped(scaled):
    """A bad page, a bad length, a position past the table: flagged; the other
    tokens are written, nothing else is touched."""
    Q, lens = 2, [300, 300, 300, 300]
    c = _case(lens, [Q] * 4, 2, 8, scaled=scaled, rot=64)
    ref = Append(c["kv"], c["sc"], c["bt"], lens, 0.01, 0.01)
    nb = c["kv"].shape[0]
    c["bt"][1, 2] = nb                     # page past the cache
    c["bt"][2, 2] = -1
    c["lens"][3] = 128 * c["bt"].shape[1] + 1   # longer than the table
    # only request 0 is written; the padding of the other requests' q is 0 or rotated
    rows = slice(0, Q)
    ref.lens, ref.bt = [300], c["bt"].cpu()[:1]
    want, size = ref.run(c["k"][rows], c["v"][rows], c["q"][rows], [Q], c["cs"])
    out = msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], Q, 0.01, 0.01,
                        kv_scales=c["sc"], cos_sin=c["cs"], q=c["q"])
    assert msa.get_error() == _native.ERR_PAGE_RANGE | _native.ERR_SEQ_RANGE
    ref.check(c["kv"], c["sc"])
    _check_q(out[rows], want, size)
    assert (out[3 * Q:] == 0).all() and (out[Q:3 * Q] != 0).any()
    # positions past the rotation table: 299 is, 298 is not
    c = _case([300], [Q], 2, 8, scaled=scaled, rot=64)
    c["cs"] = c["cs"][:299].contiguous()
    ref = Append(c["kv"], c["sc"], c["bt"], [299], 0.01, 0.01)
    want, size = ref.run(c["k"][:1], c["v"][:1], c["q"][:1], [1], c["cs"])
    out = msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], Q, 0.01, 0.01,
                        kv_scales=c["sc"], cos_sin=c["cs"], q=c["q"])
    assert msa.get_error() == _native.ERR_POS_RANGE
    ref.check(c["kv"], c["sc"])
    _check_q(out[:1], want, size)
    assert (out[1:] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), 0.0, -1.0, 2.0 ** -41, 2.0 ** 41])
def test_a_begun_page_with_a_bad_scale_is_skipped(bad):
    c = _case([300], [1], 1, 8, scaled=True)
    page = int(c["bt"][0, 2])
    c["sc"][page, 0, 0] = bad              # K's; V's stays good
    kv, sc = c["kv"].clone(), c["sc"].clone()
    msa.append_kv(c["k"], c["v"], c["kv"], c["bt"], c["lens"], 1, kv_scales=c["sc"])
    assert msa.get_error() == _native.ERR_SCALE
    assert torch.equal(c["kv"][..., :D], kv[..., :D])
    assert not torch.equal(c["kv"][page, 0, 299 % PAGE, D:], kv[page, 0, 299 % PAGE, D:])
    assert torch.equal(c["sc"][:, :, 0].nan_to_num(7.0), sc[:, :, 0].nan_to_num(7.0))


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("cu", [[0, 3, 3, 6], [0, 5, 2, 8], [2, 4, 6, 8], [0, 0, 0, 0],
                                [-5, 3, 900, 8], [0, 8, 8, 8]])
def test_cu_seqlens_out_of_order_or_short(scaled, cu):
    """Tokens in no request, ranges out of order or out of the batch: flagged
    unless the ranges are ascending and cover the 8 tokens; nothing past the
    three requests' pages is touched and q rows without a request are 0."""
    lens = [200, 140, 9]
    c = _case(lens, [3, 3, 2], 1, 3, scaled=scaled, min_cols=2)
    before = c["kv"].clone()
    out = msa.append_kv_prefill(c["k"], c["v"], c["kv"], c["bt"], c["lens"],
                                torch.tensor(cu, dtype=torch.int32, device=DEV), 0.01, 0.01,
                                kv_scales=c["sc"], cos_sin=c["cs"], q=c["q"])
    err = msa.get_error()
    assert err & ~_native.ERR_SEQ_RANGE == 0
    assert err == (0 if cu == [0, 8, 8, 8] else _native.ERR_SEQ_RANGE)
    used = set(c["bt"].flatten().tolist())
    for page in range(before.shape[0]):
        if page not in used:
            assert torch.equal(c["kv"][page], before[page])
    if cu == [0, 3, 3, 6]:
        assert (out[6:] == 0).all() and (out[:6] != 0).any()
    if cu == [0, 0, 0, 0]:
        assert (out == 0).all() and torch.equal(c["kv"], before)


def test_empty_batches():
    kv = torch.zeros((2, 1, PAGE, 2 * D), dtype=torch.uint8, device=DEV)
    e = torch.empty((0, 1, D), dtype=torch.bfloat16, device=DEV)
    bt = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    sl = torch.empty((0,), dtype=torch.int32, device=DEV)
    assert msa.append_kv(e, e, kv, bt, sl, 4) is None
    cu = torch.zeros((1,), dtype=torch.int32, device=DEV)
    assert msa.append_kv_prefill(e, e, kv, bt, sl, cu) is None


def test_python_refusals():
    c = _case([300, 20], [2, 2], 2, 3, scaled=True)
    call = lambda **kw: msa.append_kv(**{**dict(  # noqa: E731
        k=c["k"], v=c["v"], kv=c["kv"], block_table=c["bt"], seq_lens=c["lens"], qlen=2,
        kv_scales=c["sc"], cos_sin=c["cs"], q=c["q"]), **kw})
    call()
    for kw in (dict(k=c["k"].float()), dict(q_out=c["q"].float()), dict(kv_scales=c["sc"].double()),
               dict(v="v")):
        with pytest.raises(TypeError):
            call(**kw)
    wide = torch.zeros((4, 2, 256), dtype=torch.bfloat16, device=DEV)
    for kw in (dict(qlen=3), dict(k=c["k"][:, :1]), dict(v=None), dict(k=wide[..., ::2]),
               dict(k=torch.zeros((4, 4, D), dtype=torch.bfloat16, device=DEV)[:, ::2]),
               dict(k=torch.zeros((4, 2 * D + 4), dtype=torch.bfloat16, device=DEV)[:, :2 * D]
                    .unflatten(1, (2, D))),
               dict(k=c["k"].cpu()), dict(kv_scales=c["sc"][:, :, :1].contiguous()),
               dict(kv_scales=c["sc"].transpose(0, 1)), dict(cos_sin=c["cs"][:, :24].contiguous()),
               dict(cos_sin=c["cs"].flatten()), dict(q=None, q_out=c["q"]),
               dict(q_out=torch.empty((4, 16, D), dtype=torch.bfloat16, device=DEV)),
               dict(q_out=torch.empty((4, 32, D), device=DEV).to(F8), q_scale=0.0)):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(msa.MSAError):
        call(k_scale=0.0)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for k, sl in ((None, c["lens"]), (c["k"], [300, 20])):
        with pytest.raises(TypeError):
            msa.append_kv_prefill(k, c["v"], c["kv"], c["bt"], sl, cu, kv_scales=c["sc"])
    assert msa.get_error() == 0
