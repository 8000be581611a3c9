"""Outputs of the calls on pages that share memory with each other, and arrays that share it
with a cache."""
from __future__ import annotations

import itertools

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from tests.test_sync_order_host import function, source


def test_compaction_checks_the_moves_that_it_reads_back():
    """The moves and their numbers pass through outputs; whatever is in there, no index of
    theirs may lead out of bounds."""
    body = function(source("msa_pages.cu"), "compact_kernel")
    back = body[body.index("const int moves"):]
    assert "p.refs_out[__ldcg(" not in back and "__ldcg(p.copies + 3 * static_cast<int64_t>(__ldcg(" not in back
    assert "dst >= 0 && dst < p.num_blocks" in back and "src >= 0 && src < p.num_blocks" in back
    assert "k >= 0 && k < moves" in back


@pytest.mark.parametrize("call", ["msa_fork_pages", "msa_compact_pages", "msa_copy_pages"])
def test_arrays_are_compared_before_anything_is_enqueued(call):
    body = function(source("msa_api.cu"), call)
    assert body.index("arrays_meet(") < min(body.index(f) for f in ("launch_", "enqueue_copies(") if f in body)


i32 = dict(dtype=torch.int32, device="cuda")
NB, B, S = 24, 2, 4


def words(shape):
    return torch.Size(shape).numel()


@pytest.mark.gpu
@pytest.mark.parametrize("fork", [True, False])
def test_outputs_over_each_other(fork):
    bt, sl = torch.zeros((B, S), **i32), torch.zeros(B, **i32)
    refs, parents = torch.zeros(NB, **i32), torch.tensor([0, 1], **i32)
    one = torch.full((96,), 7, **i32)
    if fork:
        shapes = dict(block_table_out=(B, S), seq_lens_out=(B,), refs_out=(NB,), copies=(B, 3))
        call = lambda **kw: msa.fork_pages(bt, sl, parents, refs, **kw)
    else:
        shapes = dict(block_table_out=(B, S), refs_out=(NB,), copies=(NB // 2, 3))
        call = lambda **kw: msa.compact_pages(bt, sl, refs, **kw)

    def at(start, shape):
        return one[start:start + words(shape)].view(shape)

    for a, b in itertools.permutations(shapes, 2):
        for start in (0, words(shapes[a]) - 1):
            with pytest.raises(msa.MSAError):
                call(**{a: at(0, shapes[a]), b: at(start, shapes[b])})
    assert bool((one == 7).all())
    for a, b in itertools.permutations(shapes, 2):     # side by side
        call(**{a: at(0, shapes[a]), b: at(words(shapes[a]), shapes[b])})
    assert msa.get_error() == 0


@pytest.mark.gpu
def test_arrays_over_a_cache():
    """The last word of an array at a cache's first, and its first at the cache's last."""
    cache = torch.zeros((NB, 1, 128, 128), dtype=torch.uint8, device="cuda")
    room = torch.zeros(2 * 96 + 2 * NB, **i32)
    scales = room[96:96 + 2 * NB].view(torch.float32).view(NB, 1, 2)
    bt, sl = torch.zeros((B, S), **i32), torch.zeros(B, **i32)
    refs, parents = torch.zeros(NB, **i32), torch.tensor([0, 1], **i32)
    end = 96 + scales.numel()
    for name, shape in dict(block_table=(B, S), seq_lens=(B,), refs=(NB,), parents=(B,), grow=(B,),
                            block_table_out=(B, S), seq_lens_out=(B,), refs_out=(NB,),
                            copies=None).items():
        for f, args in ((msa.fork_pages, dict(block_table=bt, seq_lens=sl, parents=parents, refs=refs)),
                        (msa.compact_pages, dict(block_table=bt, seq_lens=sl, refs=refs))):
            if f is msa.compact_pages and name in ("parents", "grow", "seq_lens_out"):
                continue
            shape_f = shape or ((B, 3) if f is msa.fork_pages else (NB // 2, 3))
            n = words(shape_f)
            for start, ok in ((96 - n, True), (97 - n, False), (end - 1, False), (end, True)):
                a = dict(args)
                a[name] = room[start:start + n].view(shape_f)
                room.zero_()
                if ok:
                    f(caches=[cache, scales], **a)
                    continue
                with pytest.raises(msa.MSAError):
                    f(caches=[cache, scales], **a)
    torch.cuda.synchronize()
    msa.get_error(clear=True)
    for start, ok in ((93, True), (94, False), (end - 1, False), (end, True)):
        c = room[start:start + 3].view(1, 3)
        if ok:
            msa.copy_pages(c, [cache, scales])
            continue
        with pytest.raises(msa.MSAError):
            msa.copy_pages(c, [cache, scales])
    assert msa.get_error() == 0
