"""The largest tables that the calls on pages take: their kernels' counters step by up to a
whole cluster's threads past the last entry."""
from __future__ import annotations

import ctypes

import pytest
import torch

from block_sparse_gqa_score_gb300 import _native, build

MOST = (1 << 31) - 1 - 8192


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def at(i):
    return ctypes.c_void_p((i + 1) << 40)


def fork(lib, B, rows, S):
    return lib.msa_fork_pages(*[at(i) for i in range(9)], B, rows, S, 100, None, 0, None)


def compact(lib, B, S):
    return lib.msa_compact_pages(*[at(i) for i in range(6)], B, S, 100, None, 0, None)


def test_tables_near_the_largest_int(lib):
    for n in (MOST + 1, MOST + 8160, MOST + 8192):
        assert fork(lib, 1, 1, n) == fork(lib, 0, 1, n) == fork(lib, 1, 0, n) == _native.EINVAL
        assert compact(lib, 1, n) == compact(lib, n, 1) == _native.EINVAL
    if not torch.cuda.is_available():
        assert fork(lib, 1, 1, MOST) == compact(lib, 1, MOST) == compact(lib, MOST, 1) == _native.ECUDA
