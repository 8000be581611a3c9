"""Outputs of the calls on pages that share memory with each other."""
from __future__ import annotations

import itertools

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from tests.test_sync_order_host import function, source


def test_outputs_apart():
    for order in itertools.permutations([(0, 8, "a"), (8, 20, "b"), (20, 24, "c"), (64, 68, "d")]):
        msa._apart(list(order))
    for extra in ((0, 8, "x"), (4, 8, "x"), (19, 21, "x"), (7, 9, "x"), (60, 65, "x"), (0, 100, "x")):
        for order in itertools.permutations([(0, 8, "a"), (8, 20, "b"), (64, 68, "d"), extra]):
            with pytest.raises(ValueError, match="share memory"):
                msa._apart(list(order))


def test_compaction_checks_the_moves_that_it_reads_back():
    """The moves and their numbers pass through outputs; if these share memory (the library
    cannot rule it out) no index of theirs may lead out of bounds."""
    body = function(source("msa_pages.cu"), "compact_kernel")
    back = body[body.index("const int moves"):]
    assert "p.refs_out[__ldcg(" not in back and "__ldcg(p.copies + 3 * static_cast<int64_t>(__ldcg(" not in back
    assert "dst >= 0 && dst < p.num_blocks" in back and "src >= 0 && src < p.num_blocks" in back
    assert "k >= 0 && k < moves" in back


@pytest.mark.gpu
def test_calls_refuse_outputs_over_each_other():
    i32 = dict(dtype=torch.int32, device="cuda")
    NB, B, S = 24, 2, 4
    bt, sl = torch.zeros((B, S), **i32), torch.zeros(B, **i32)
    refs, parents = torch.zeros(NB, **i32), torch.tensor([0, 1], **i32)
    one = torch.full((64,), 7, **i32)
    shapes = dict(block_table_out=(B, S), seq_lens_out=(B,), refs_out=(NB,), copies=(B, 3))
    at = lambda start, shape: one[start:start + torch.Size(shape).numel()].view(shape)
    for a, b in itertools.combinations(shapes, 2):
        for start in (0, torch.Size(shapes[a]).numel() - 1):
            with pytest.raises(ValueError, match="share memory"):
                msa.fork_pages(bt, sl, parents, refs, **{a: at(0, shapes[a]), b: at(start, shapes[b])})
        msa.fork_pages(bt, sl, parents, refs,
                       **{a: at(0, shapes[a]), b: at(torch.Size(shapes[a]).numel(), shapes[b])})
    one.fill_(7)
    shapes = dict(block_table_out=(B, S), refs_out=(NB,), copies=(NB // 2, 3))
    for a, b in itertools.combinations(shapes, 2):
        with pytest.raises(ValueError, match="share memory"):
            msa.compact_pages(bt, sl, refs, **{a: at(0, shapes[a]), b: at(2, shapes[b])})
    assert bool((one == 7).all())
    assert msa.get_error() == 0
