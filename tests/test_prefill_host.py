"""Host-side refusals of the prefill scorer, selector and dense attention and of the calls
on pages: bad arguments are rejected before any CUDA call (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native, build

EINVAL = _native.EINVAL
A = ctypes.c_void_p(1 << 20)       # an aligned address; rejected calls never use it
OUT = ctypes.c_void_p(1 << 21)


def off(n):
    return ctypes.c_void_p((1 << 20) + n)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


BATCH = dict(q=A, q8=0.0, kv=A, sc=A, k_only=0, bt=A, sl=A, cu=A, ws=A, wb=1 << 30, out=OUT, B=3,
             T=505, Hq=64, Hkv=4, S=8, NB=100, sm=0.088, k_s=1.0, v_s=1.0)


def dense(lib, **kw):
    a = dict(BATCH, **kw)
    return lib.msa_dense_prefill(a["q"], a["q8"], a["kv"], a["sc"], a["bt"], a["sl"], a["cu"],
                                 a["ws"], a["wb"], a["out"], a["B"], a["T"], a["Hq"], a["Hkv"],
                                 a["S"], a["NB"], a["sm"], a["k_s"], a["v_s"], None)


def score(lib, **kw):
    a = dict(BATCH, **kw)
    return lib.msa_score_prefill(a["q"], a["q8"], a["kv"], a["sc"], a["k_only"], a["bt"], a["sl"],
                                 a["cu"], a["out"], a["B"], a["T"], a["Hq"], a["Hkv"], a["S"],
                                 a["NB"], a["sm"], a["k_s"], None)


def topk(lib, **kw):
    a = dict(BATCH, k=16, **kw)
    return lib.msa_topk_prefill(a["q"], 0, 0, 1, a["sl"], a["cu"], a["out"], a["B"], a["T"],
                                a["Hkv"], a["S"], a["k"], None)


BAD = [
    dict(q=None), dict(kv=None), dict(bt=None), dict(sl=None), dict(cu=None), dict(out=None),
    dict(q=off(8)), dict(kv=off(4)), dict(sc=off(4)), dict(bt=off(2)), dict(sl=off(1)),
    dict(cu=off(2)), dict(out=off(2)), dict(B=-1), dict(B=0), dict(T=0), dict(T=-1),
    dict(T=(1 << 31) - 1), dict(B=65536), dict(Hq=48), dict(Hkv=0), dict(S=0), dict(NB=0),
    dict(NB=(1 << 31) // 512), dict(sm=0.0), dict(sm=float("nan")), dict(k_s=-1.0),
    dict(k_s=float("inf")), dict(q8=-1.0), dict(q8=float("nan")), dict(q8=float("inf")),
]


@pytest.mark.parametrize("kw", BAD)
def test_prefill_rejects(lib, kw):
    assert dense(lib, **kw) == EINVAL
    assert score(lib, **kw) == EINVAL


def test_prefill_rejects_rows_longer_than_a_wait(lib):
    for f in (dense, score):
        assert f(lib, B=1, S=(1 << 19) + 1) == EINVAL
        if not torch.cuda.is_available():
            assert f(lib, B=1, S=1 << 19) == _native.ECUDA


def test_prefill_more_rejections(lib):
    assert dense(lib, v_s=float("nan")) == EINVAL and dense(lib, out=off(8)) == EINVAL
    assert score(lib, k_only=1, sc=off(2)) == EINVAL
    for kw in (dict(q=None), dict(sl=None), dict(cu=None), dict(out=None), dict(q=off(2)),
               dict(cu=off(1)), dict(k=8), dict(B=-1), dict(B=0), dict(T=0), dict(T=1 << 30),
               dict(Hkv=0), dict(S=0)):
        a = dict(BATCH, k=16)
        a.update(kw)
        assert lib.msa_topk_prefill(a["q"], 0, 0, 1, a["sl"], a["cu"], a["out"], a["B"], a["T"],
                                    a["Hkv"], a["S"], a["k"], None) == EINVAL, kw
    assert dense(lib, B=0, T=0) == 0 and score(lib, B=0, T=0) == 0 and topk(lib, B=0, T=0) == 0
    if not torch.cuda.is_available():
        for kw in (dict(), dict(sc=None), dict(q8=0.5)):
            assert dense(lib, **kw) == _native.ECUDA and score(lib, **kw) == _native.ECUDA
        assert score(lib, k_only=1, sc=off(4)) == _native.ECUDA and topk(lib) == _native.ECUDA


def test_dense_workspace(lib):
    per = 2 * 256 * (128 * 4 + 8) + 16       # two parts a CTA, and what its shared unit is
    assert lib.msa_dense_prefill_workspace_bytes(152) == 152 * per
    assert lib.msa_dense_prefill_workspace_bytes(1) == per
    assert lib.msa_dense_prefill_workspace_bytes(0) == 0
    assert lib.msa_dense_prefill_workspace_bytes(-3) == 0


POOL = dict(bt=A, sl=A, pa=A, gr=A, refs=A, bt2=OUT, sl2=OUT, refs2=OUT, co=OUT, B=4, rows=5, S=8,
            NB=100)


def caches(*c):
    out = (_native.Cache * max(1, len(c)))()
    for i, x in enumerate(c):
        out[i] = _native.Cache(*x)
    return out, len(c)


GOOD = caches((1 << 20, 4, 128, 256), ((1 << 20) + 4, 4, 1, 8))


def fork(lib, cs=GOOD, **kw):
    a = dict(POOL, **kw)
    return lib.msa_fork_pages(a["bt"], a["sl"], a["pa"], a["gr"], a["refs"], a["bt2"], a["sl2"],
                              a["refs2"], a["co"], a["B"], a["rows"], a["S"], a["NB"], *cs, None)


def compact(lib, cs=GOOD, **kw):
    a = dict(POOL, **kw)
    return lib.msa_compact_pages(a["bt"], a["sl"], a["refs"], a["bt2"], a["refs2"], a["co"], a["B"],
                                 a["S"], a["NB"], *cs, None)


def copy(lib, cs=GOOD, co=A, n=5, NB=100):
    return lib.msa_copy_pages(co, n, NB, *cs, None)


def test_pages_reject(lib):
    for kw in (dict(bt=None), dict(sl=None), dict(refs=None), dict(bt2=None), dict(refs2=None),
               dict(co=None), dict(bt=off(2)), dict(sl=off(1)), dict(refs=off(3)),
               dict(bt2=off(2)), dict(refs2=off(2)), dict(co=off(2)), dict(bt2=A), dict(refs2=A),
               dict(B=-1), dict(S=0), dict(S=1 << 30), dict(NB=0), dict(NB=1 << 31)):
        assert fork(lib, **kw) == EINVAL, kw
        assert compact(lib, **kw) == EINVAL, kw
    for kw in (dict(pa=None), dict(pa=off(2)), dict(gr=off(2)), dict(sl2=None), dict(sl2=A),
               dict(sl2=off(2)), dict(B=8193), dict(rows=8193), dict(rows=-1)):
        assert fork(lib, **kw) == EINVAL, kw
    for kw in (dict(co=None), dict(co=off(2)), dict(n=-1), dict(NB=0), dict(NB=1 << 31)):
        assert copy(lib, **kw) == EINVAL, kw
    for c in ((0, 4, 128, 256), ((1 << 20) + 8, 4, 128, 256), (1 << 20, 0, 128, 256),
              (1 << 20, 4, 64, 256), (1 << 20, 4, 128, 200), (1 << 20, 4, 128, 0),
              ((1 << 20) + 2, 4, 1, 8), (1 << 20, 4, 1, 6)):
        for f in (fork, compact, copy):
            assert f(lib, cs=caches(c)) == EINVAL, c
    for f in (fork, compact, copy):
        assert f(lib, cs=(None, 1)) == EINVAL and f(lib, cs=(GOOD[0], -1)) == EINVAL
    assert copy(lib, n=0, co=None) == 0
    if not torch.cuda.is_available():
        assert fork(lib) == _native.ECUDA and compact(lib) == _native.ECUDA
        assert copy(lib) == _native.ECUDA
        assert fork(lib, B=0, bt=None, sl=None) == _native.ECUDA
        assert fork(lib, gr=None, cs=(None, 0)) == _native.ECUDA
        assert compact(lib, NB=1, co=None) == _native.ECUDA


@pytest.mark.parametrize("f,outs,ins", [
    (fork, dict(bt2=5 * 8, sl2=5, refs2=100, co=15), dict(bt=4 * 8, sl=4, pa=5, gr=5, refs=100)),
    (compact, dict(bt2=4 * 8, refs2=100, co=150), dict(bt=4 * 8, sl=4, refs=100))])
def test_pages_reject_outputs_over_inputs(lib, f, outs, ins):
    """An output that begins at an input's last word or ends at its first; and, next to
    them, those that just do not."""
    apart = {k: ctypes.c_void_p((2 + i) << 20) for i, k in enumerate((*ins, *outs))}
    for o, n in outs.items():
        for k, m in ins.items():
            at = apart[k].value
            for x, y in ((at + 4 * (m - 1), at + 4 * m), (at - 4 * (n - 1), at - 4 * n)):
                assert f(lib, **dict(apart, **{o: ctypes.c_void_p(x)})) == EINVAL, (o, k)
                if not torch.cuda.is_available():
                    assert f(lib, **dict(apart, **{o: ctypes.c_void_p(y)})) == _native.ECUDA, (o, k)


def test_python_rejects_host_tensors():
    q = torch.zeros((2, 16, 128), dtype=torch.bfloat16)
    kv = torch.zeros((3, 1, 128, 256), dtype=torch.uint8)
    bt, sl = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cu = torch.zeros(3, dtype=torch.int32)
    for f in (lambda: msa.dense_prefill(q, kv, bt, sl, cu, 1.0),
              lambda: msa.score_prefill(q, kv, bt, sl, cu, 1.0),
              lambda: msa.fork_pages(bt, sl, sl, sl, [kv]),
              lambda: msa.compact_pages(bt, sl, sl, [kv]),
              lambda: msa.copy_pages(torch.zeros((1, 3), dtype=torch.int32), [kv])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        msa.topk_prefill(torch.zeros((1, 2, 1)), sl, cu)
