"""Buffers that a call makes for itself when it is given a stream: memory of that stream, so
that work which another stream has still queued on the same memory cannot reach them."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.prefill_ref import Batch, D, GROUP, cu

pytestmark = pytest.mark.gpu


class Spy:
    """The library, noting the arguments of its calls."""

    def __init__(self, lib, calls):
        self._at, self._calls = lib, calls

    def __getattr__(self, name):
        f = getattr(self._at, name)

        def call(*args):
            self._calls.append((name, args))
            return f(*args)
        return call


def owners():
    """[(first byte, past the last, stream)] of the allocator's memory."""
    return [(s["address"], s["address"] + s["total_size"], s["stream"])
            for s in torch.cuda.memory_snapshot()]


def calls(x):
    """Every call that takes a stream, without buffers of the caller's."""
    B, Hkv, S = len(x.q_lens), x.kv.shape[1], x.bt.shape[1]
    a = (x.q, x.kv, x.bt, x.lens)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    qd = x.q[:4 * B].contiguous()
    d = (qd, x.kv, x.bt, x.lens, 4)
    scores = torch.randn((Hkv, 4 * B, S), device="cuda")
    every = torch.randn((Hkv, x.T, S), device="cuda")
    lists = msa.topk(scores, x.lens, 4)
    long = msa.topk_prefill(every, x.lens, x.cu)
    ws = torch.zeros(msa.workspace_bytes(B, 4, GROUP * Hkv, 4), dtype=torch.uint8, device="cuda")
    refs = torch.zeros(x.kv.shape[0], dtype=torch.int32, device="cuda")
    for b in range(B):
        refs[x.bt[b, :-(-int(x.lens[b]) // D)].long()] = 1
    parents = torch.arange(B, dtype=torch.int32, device="cuda")
    k = torch.randn((B, Hkv, D), device="cuda").to(torch.bfloat16)
    kp = torch.randn((x.T, Hkv, D), device="cuda").to(torch.bfloat16)
    spare = x.kv.clone()
    keep = [a, d, one, scores, every, lists, long, ws, refs, parents, k, kp, spare, x.q[:B]]
    q1 = x.q[:B].contiguous()
    keep.append(q1)
    return keep, {
        "score": lambda s: msa.score(*d, x.sm, stream=s),
        "topk": lambda s: msa.topk(scores, x.lens, 4, stream=s),
        "sparse_decode": lambda s: msa.sparse_decode(qd, x.kv, x.bt, x.lens, lists, 4, x.sm,
                                                     num_splits=2, stream=s),
        "sparse_decode_select": lambda s: msa.sparse_decode_select(
            qd, x.kv, x.bt, x.lens, scores, 4, x.sm, num_splits=2, stream=s),
        "dense_decode": lambda s: msa.dense_decode(*d, x.sm, stream=s),
        "decode_step": lambda s: msa.decode_step(*d, x.sm, stream=s),
        "combine": lambda s: msa.combine(ws, 4 * B, GROUP * Hkv, 4, stream=s),
        "sparse_prefill": lambda s: msa.sparse_prefill(*a, x.cu, long, x.sm, num_splits=2, stream=s),
        "sparse_prefill_select": lambda s: msa.sparse_prefill_select(*a, x.cu, every, x.sm,
                                                                     num_splits=2, stream=s),
        "score_prefill": lambda s: msa.score_prefill(*a, x.cu, x.sm, stream=s),
        "topk_prefill": lambda s: msa.topk_prefill(every, x.lens, x.cu, stream=s),
        "dense_prefill": lambda s: msa.dense_prefill(*a, x.cu, x.sm, stream=s),
        "append_kv": lambda s: msa.append_kv(k, k, spare, x.bt, x.lens, 1, q=q1, stream=s),
        "append_kv_prefill": lambda s: msa.append_kv_prefill(kp, kp, spare, x.bt, x.lens, x.cu,
                                                             q=x.q, stream=s),
        "fork_pages": lambda s: msa.fork_pages(x.bt, x.lens, parents, refs, [spare], stream=s),
        "compact_pages": lambda s: msa.compact_pages(x.bt, x.lens, refs, [spare], stream=s),
    }


NAMES = ["score", "topk", "sparse_decode", "sparse_decode_select", "dense_decode", "decode_step",
         "combine", "sparse_prefill", "sparse_prefill_select", "score_prefill", "topk_prefill",
         "dense_prefill", "append_kv", "append_kv_prefill", "fork_pages", "compact_pages"]


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", NAMES)
def test_buffers_are_of_the_stream(name, monkeypatch):
    x = Batch([5000, 300, 2000], [40, 200, 7], 2, 31)
    keep, every = calls(x)
    want = tensors(every[name](None))
    want = [t.clone() for t in want]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ours = torch.cuda.current_stream().cuda_stream
    # memory of the current stream that is free on the host and still being written
    sizes = [t.numel() * t.element_size() for t in want] + [msa.dense_prefill_workspace_bytes()]
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    given = {(s, e) for s, e, st in owners() if st == ours}
    seen = []
    monkeypatch.setattr(_native, "_lib", Spy(_native._lib, seen))
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in late]
    torch.cuda._sleep(2000000)
    for t in late:
        t.fill_(0x7F)
    del late, t
    got = tensors(every[name](side))
    memory = owners()
    side.synchronize()
    assert given and seen
    for t in got:
        at = t.data_ptr()
        assert [st for s, e, st in memory if s <= at < e] == [side.cuda_stream]
    for f, args in seen:
        for p in args:
            if isinstance(p, int) and p > 1 << 20:
                assert not any(s <= p < e for s, e in spans), f
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("name", ["dense_prefill", "score_prefill", "fork_pages"])
def test_outputs_outlive_their_name(name):
    """An output made for a stream and read by the current one: its memory does not go to
    another tensor of that stream while the reading is queued."""
    x = Batch([5000, 300], [40, 200], 2, 32)
    keep, every = calls(x)
    want = tensors(every[name](None))[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        out = tensors(every[name](side))[0]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2000000)
        copy = out.clone()
        n = out.numel() * out.element_size()
        del out
        with torch.cuda.stream(side):
            junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(copy.view(torch.uint8), want.view(torch.uint8)) and len(junk) == 3


def test_capture_on_a_given_stream():
    """Calls on the stream that is captured, named or not, with buffers of their own."""
    x = Batch([5000, 300], [40, 200], 2, 33)
    a = (x.q, x.kv, x.bt, x.lens, x.cu, x.sm)
    want = msa.dense_prefill(*a), msa.score_prefill(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = msa.dense_prefill(*a, stream=side), msa.score_prefill(*a)
    for t in got:
        t.zero_()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip(got, want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    assert msa.get_error() == 0
