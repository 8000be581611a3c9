"""Host-side refusals of the cache append and of the page-scale entry points:
bad arguments are rejected before any CUDA call (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native, build

EINVAL = _native.EINVAL
A = ctypes.c_void_p(1 << 20)       # an aligned address; rejected calls never use it


def off(n):
    return ctypes.c_void_p((1 << 20) + n)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


APPEND = dict(k=A, ks=9216, v=A, vs=9216, q=A, qs=9216, cs=A, maxp=4096, rot=64, inter=0, kv=A,
              sc=A, qo=off(4096), q8=0.0, bt=A, sl=A, B=16, Q=4, Hq=64, Hkv=4, S=8, NB=100,
              k_s=1.0, v_s=1.0)


def _append(lib, **kw):
    a = dict(APPEND, **kw)
    return lib.msa_append_kv(a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["cs"], a["maxp"],
                             a["rot"], a["inter"], a["kv"], a["sc"], a["qo"], a["q8"], a["bt"],
                             a["sl"], a["B"], a["Q"], a["Hq"], a["Hkv"], a["S"], a["NB"],
                             a["k_s"], a["v_s"], None)


def _prefill(lib, **kw):
    a = dict(APPEND, cu=A, T=505, **kw)
    return lib.msa_append_kv_prefill(a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["cs"],
                                     a["maxp"], a["rot"], a["inter"], a["kv"], a["sc"], a["qo"],
                                     a["q8"], a["bt"], a["sl"], a["cu"], a["B"], a["T"], a["Hq"],
                                     a["Hkv"], a["S"], a["NB"], a["k_s"], a["v_s"], None)


BAD = [
    dict(k=None), dict(kv=None), dict(bt=None), dict(sl=None), dict(qo=None),
    dict(k=off(8)), dict(v=off(2)), dict(q=off(8)), dict(kv=off(4)), dict(qo=off(8)),
    dict(cs=off(8)), dict(sc=off(4)), dict(bt=off(2)), dict(sl=off(1)),
    dict(ks=9212), dict(ks=504), dict(vs=9220), dict(vs=0), dict(qs=8184), dict(qs=-8192),
    dict(rot=-16), dict(rot=8), dict(rot=72), dict(rot=144), dict(cs=None), dict(maxp=0),
    dict(Hq=48), dict(Hkv=0), dict(S=0), dict(NB=0), dict(B=-1), dict(NB=(1 << 31) // 512),
    dict(k_s=0.0), dict(k_s=-1.0), dict(k_s=float("nan")), dict(v_s=float("inf")),
    dict(q8=-1.0), dict(q8=float("nan")), dict(q8=float("inf")),
    dict(qo=A),                                   # in place with another stride than the output's
    dict(qo=A, qs=8192, q8=1.0),                  # in place with fp8 codes
]


@pytest.mark.parametrize("kw", BAD)
def test_append_rejects(lib, kw):
    assert _append(lib, **kw) == EINVAL
    assert _prefill(lib, **kw) == EINVAL


def test_append_query_length_and_batch_bounds(lib):
    assert _append(lib, Q=0) == EINVAL and _append(lib, Q=33) == EINVAL
    assert _append(lib, B=65536) == EINVAL
    assert _append(lib, B=0) == 0
    for kw in (dict(cu=None), dict(cu=off(2)), dict(T=-1), dict(T=(1 << 31) - 1), dict(B=0),
               dict(T=0)):
        a = dict(APPEND, cu=A, T=505)
        a.update(kw)
        st = lib.msa_append_kv_prefill(
            a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["cs"], a["maxp"], a["rot"],
            a["inter"], a["kv"], a["sc"], a["qo"], a["q8"], a["bt"], a["sl"], a["cu"], a["B"],
            a["T"], a["Hq"], a["Hkv"], a["S"], a["NB"], a["k_s"], a["v_s"], None)
        assert st == EINVAL, kw


def test_append_optional_parts_pass_the_host_checks(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for kw in (dict(), dict(v=None, vs=0, sc=off(4)), dict(q=None, qs=0, qo=None), dict(sc=None),
               dict(rot=0, cs=None, maxp=0), dict(qo=A, qs=8192), dict(q8=0.5), dict(inter=1)):
        assert _append(lib, **kw) == _native.ECUDA, kw


def test_scaled_entry_points_reject(lib):
    """A missing or misaligned kv_scales, a bad q_scale, and what the entry point
    without the suffix rejects."""
    tail = (64, 4, 8, 100, 0.088, 1.0)

    def score(q8=0.0, sc=A, k_only=0, q=A, out=A, Q=4):
        return lib.msa_score_scaled(q, q8, A, sc, k_only, A, A, out, 16, Q, *tail, None)

    def decode(q8=0.0, sc=A, tk=A, Q=4, splits=1, ws=None):
        return lib.msa_sparse_decode_scaled(A, q8, A, sc, A, A, tk, ws, 0, A, 16, Q, *tail, 1.0,
                                            splits, None)

    def select(q8=0.0, sc=A, scores=A, Q=4):
        return lib.msa_sparse_decode_select_scaled(A, q8, A, sc, A, A, scores, 0, 0, 1, A, None, 0,
                                                   A, 16, Q, *tail, 1.0, 1, None)

    def dense(q8=0.0, sc=A, S=8, Q=4):
        return lib.msa_dense_decode_scaled(A, q8, A, sc, A, A, A, 1 << 30, A, 16, Q, 64, 4, S, 100,
                                           0.088, 1.0, 1.0, None)

    def prefill(q8=0.0, sc=A, cu=A, T=505):
        return lib.msa_sparse_prefill_scaled(A, q8, A, sc, A, A, cu, A, None, 0, A, 3, T, *tail,
                                             1.0, 1, None)

    def prefill_select(q8=0.0, sc=A, cu=A, scores=A):
        return lib.msa_sparse_prefill_select_scaled(A, q8, A, sc, A, A, cu, scores, 0, 0, 1, A,
                                                    None, 0, A, 3, 505, *tail, 1.0, 1, None)

    def step(q8=0.0, sc=A, index=None, iks=0.0, isc=None):
        return lib.msa_decode_step_scaled(A, q8, A, sc, index, iks, isc, A, A, A, A, None, 0, A, 16,
                                          4, *tail, 1.0, 1, None)

    for f in (score, decode, select, dense, prefill, prefill_select, step):
        assert f(sc=None) == EINVAL
        assert f(sc=off(4)) == EINVAL
        for qs in (-1.0, float("nan"), float("inf")):
            assert f(q8=qs) == EINVAL
        if not torch.cuda.is_available():
            assert f() == _native.ECUDA and f(q8=0.5) == _native.ECUDA
    for f in (score, decode, select, dense):
        assert f(Q=33) == EINVAL
    assert score(out=None) == EINVAL and score(sc=off(2), k_only=1) == EINVAL
    assert decode(tk=None) == EINVAL and decode(splits=17) == EINVAL
    assert select(scores=None) == EINVAL and prefill_select(scores=None) == EINVAL
    assert dense(S=2049) == EINVAL
    assert prefill(cu=None) == EINVAL and prefill_select(cu=None) == EINVAL
    assert prefill(T=0) == EINVAL
    assert step(index=A, iks=0.0) == EINVAL


def test_python_rejects_host_tensors():
    k = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    kv = torch.zeros((3, 1, 128, 256), dtype=torch.uint8)
    bt, sl = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.append_kv(k, k, kv, bt, sl, 1)
    with pytest.raises(ValueError):
        msa.append_kv_prefill(k, k, kv, bt, sl, torch.zeros(3, dtype=torch.int32))
