"""Prefill units of two halves of a query tile followed by long units of one, and the other
way round, with page scales that differ from page to page: each half's warps must have read
a page's factors before another page's take their place."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from tests.prefill_ref import Batch, check, every

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq_lens,q_lens", [([6000, 5000, 4100], [24, 24, 24]),
                                             ([5100, 70, 9000, 300], [20, 3, 17, 8]),
                                             ([3000] * 12, [8, 16] * 6)])
@pytest.mark.parametrize("q8", [False, True])
def test_units_of_one_half_behind_units_of_two(seq_lens, q_lens, q8):
    x = Batch(seq_lens, q_lens, 4, 40, q8=q8, scaled=True)
    msa.get_error(clear=True)
    want, tol = every(x, scores=True)
    first = msa.score_prefill(*x.args(), **x.kw())
    check(first, want, tol)
    dense = msa.dense_prefill(*x.args(), x.v_scale, **x.kw())
    check(dense, *every(x))
    for _ in range(20):
        assert torch.equal(msa.score_prefill(*x.args(), **x.kw()), first)
        assert torch.equal(msa.dense_prefill(*x.args(), x.v_scale, **x.kw()), dense)
    assert msa.get_error() == 0
