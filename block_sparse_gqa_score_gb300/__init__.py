"""GB300-native (sm_103a) block-sparse GQA decode over a paged fp8 KV cache.

One decode step of MiniMax-M3-style indexer-selected sparse attention, as the
vLLM MiniMax-M3 sparse attention pages and TensorRT-LLM PR #17171 describe it:

  score()          each block's largest visible scaled q.k over a KV head's query heads
  topk()           top-16 blocks (current block kept, ties to the lower index)
  sparse_decode()  split-K attention over the selected pages (+ merge)
  sparse_prefill() the same attend for prefill batches (one query length per
                   request, cu_seqlens_q)
  combine()        merge of split-K partials
  decode_step()    the three stages back to back on one stream
  append_kv()      the step before: new keys and values rotated, quantised and
                   written to the paged cache, the query rotated
                   (append_kv_prefill() for prefill batches)
  score_prefill(), topk_prefill()  the scorer and the selector for prefill batches
  dense_prefill()  attention over every visible block for prefill batches
  fork_pages(), compact_pages(), copy_pages()  the cache's pages: rows forked,
                   reordered, freed and grown, pages moved together

Every function here only checks and marshals torch tensors into the C ABI of
libmsa.so (include/msa.h); all arithmetic runs in that library's CUDA kernels.
There is no CPU fallback: if the library is missing, calls raise.

Tensor layouts (see include/msa.h): q bf16 [T, Hq, 128] with T = B * qlen
request-major; kv fp8 e4m3 [num_blocks, Hkv, 128, 256] (K bytes 0..127, V bytes
128..255), given as uint8 or float8_e4m3fn; block_table int32 [B, S];
seq_lens int32 [B]; scores fp32 [Hkv, T, S]; topk int32 [T, Hkv, 16].  Every
function that reads the cache takes kv_scales=, page scales fp32 [num_blocks,
Hkv, 2] (a page's K and V factor per KV head, as append_kv keeps them), which
multiply k_scale and v_scale (msa_*_scaled).
"""
from __future__ import annotations

import ctypes
import functools
import math
from dataclasses import dataclass

import torch

from . import _native
from ._native import MSAError  # noqa: F401

HEAD_DIM = 128
PAGE_SIZE = 128
TOPK = 16
GROUP = 16
MAX_QLEN = 32

__all__ = ["score", "topk", "sparse_decode", "sparse_decode_select", "sparse_prefill",
           "sparse_prefill_select", "dense_decode", "dense_splits",
           "combine", "decode_step", "append_kv", "append_kv_prefill", "score_prefill",
           "topk_prefill", "dense_prefill", "dense_prefill_workspace_bytes", "fork_pages",
           "compact_pages", "copy_pages",
           "fused_selection", "FUSED_MAX_BLOCKS", "workspace_bytes",
           "choose_splits", "get_error", "set_input_overlap", "set_union_tile", "DecodeBuffers",
           "MSAError"]


def _lib():
    return _native._lib or _native.load()


_devices = 0    # visible devices, once a call has asked


def _stream(device: torch.device, stream) -> int:
    """The handle of the stream of a call on tensors of `device`.  The library launches on the
    current device, so that has to be theirs (with one device it is: 0.4 us less a call)."""
    global _devices
    index = device.index
    if _devices != 1:
        _devices = _devices or torch.cuda.device_count()
        if index != torch._C._cuda_getDevice():
            raise ValueError(f"the tensors are on {device}, which is not the current device: "
                             f"call under torch.cuda.device({index})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device_index != index:
        raise ValueError(f"the stream is not one of {device}")
    return stream.cuda_stream


def _own(shape, dtype, device, stream):
    """A buffer that only a call's kernels use, memory of their stream (None: the current
    one): nothing that is still queued on another stream can write to it, and it goes to
    others of that stream alone."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream`: memory of that stream, which is not given away either
    before what the current stream does with it until it is freed."""
    t = _own(shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _need(t: torch.Tensor, name: str, dtypes, device=None):
    try:   # what every call passes; the checks below name what is wrong
        if (t.is_cuda and t.dtype in dtypes and t.is_contiguous()
                and (device is None or t.device == device)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


_KV_DTYPES = (torch.uint8, torch.float8_e4m3fn)


_FP8_Q = getattr(torch, "float8_e4m3fn", None)


def _geometry(q, kv, block_table, seq_lens, qlen: int | None, k_only_ok: bool = False):
    """Shapes of a step's inputs; q must hold B * qlen tokens (qlen None: any).
    k_only_ok: kv may also be a K-only cache [num_blocks, Hkv, 128, 128]."""
    _need(q, "q", (torch.bfloat16,) + ((_FP8_Q,) if _FP8_Q is not None else ()))
    dev = q.device
    _need(kv, "kv", _KV_DTYPES, dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    shape, rows, table = kv.shape, q.shape, block_table.shape
    if len(shape) != 4 or shape[2] != PAGE_SIZE or not (
            shape[3] == 2 * HEAD_DIM or (k_only_ok and shape[3] == HEAD_DIM)):
        raise ValueError("kv must be [num_blocks, Hkv, 128, 256]"
                         + (" (or a K-only [num_blocks, Hkv, 128, 128])" if k_only_ok else ""))
    if len(rows) != 3 or rows[2] != HEAD_DIM:
        raise ValueError("q must be [T, Hq, 128]")
    if len(table) != 2 or seq_lens.shape != table[:1]:
        raise ValueError("block_table must be [B, S] and seq_lens [B]")
    B, S = table
    Hkv = shape[1]
    Hq = rows[1]
    if qlen is not None and rows[0] != B * qlen:
        raise ValueError(f"q has {rows[0]} tokens, expected B*qlen = {B * qlen}")
    return dev, B, S, Hq, Hkv, shape[0]


def workspace_bytes(batch: int, qlen: int, num_q_heads: int, num_splits: int) -> int:
    return int(_lib().msa_workspace_bytes(batch, qlen, num_q_heads, num_splits))


def choose_splits(batch: int, qlen: int, num_kv_heads: int, sm_count: int | None = None) -> int:
    if sm_count is None:
        sm_count = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(_lib().msa_choose_splits(batch, qlen, num_kv_heads, sm_count))


def _fp8(q, q_scale: float) -> bool:
    """Whether q is an fp8 query (then its value is q * q_scale)."""
    if q.dtype == torch.bfloat16:
        return False
    if not (q_scale > 0 and math.isfinite(q_scale)):
        raise ValueError("an fp8 query needs a finite q_scale > 0")
    return True


def _page_scales(kv_scales, name: str, dev, num_blocks: int, num_kv_heads: int, sides: int):
    """Checks page scales fp32 [num_blocks, Hkv, sides] and returns their address."""
    _need(kv_scales, name, (torch.float32,), dev)
    if kv_scales.shape != (num_blocks, num_kv_heads, sides):
        raise ValueError(f"{name} must be [num_blocks, Hkv, {sides}]")
    return kv_scales.data_ptr()


def _parts(num_splits: int, kv_scales, batch: int, qlen: int, num_q_heads: int, num_kv_heads: int,
           workspace, dev, stream):
    """(split count, workspace, its address and bytes) of an attend on lists: with
    page scales the library cuts a row by itself and needs no workspace."""
    if num_splits <= 0 and kv_scales is not None:
        return 0, None, None, 0
    splits = num_splits if num_splits > 0 else choose_splits(batch, qlen, num_kv_heads)
    need = workspace_bytes(batch, qlen, num_q_heads, splits)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = _own(need, torch.uint8, dev, stream)
    if workspace is None:
        return splits, None, None, 0
    return splits, workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def score(q, kv, block_table, seq_lens, qlen: int, sm_scale: float, k_scale: float = 1.0,
          scores: torch.Tensor | None = None, stream=None, q_scale: float = 1.0,
          kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Block scores fp32 [Hkv, T, S] (msa_score; msa_score_q8 for an fp8 q of
    value q * q_scale).  `kv` may be the packed K|V cache [NB, Hkv, 128, 256]
    or a K-only (index-K) cache [NB, Hkv, 128, 128] (msa_score_kcache).
    kv_scales: page scales [NB, Hkv, 2] ([NB, Hkv, 1] of a K-only cache)."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, qlen, k_only_ok=True)
    if scores is None:
        scores = _empty((Hkv, B * qlen, S), torch.float32, dev, stream)
    _need(scores, "scores", (torch.float32,), dev)
    if tuple(scores.shape) != (Hkv, B * qlen, S):
        raise ValueError("scores must be [Hkv, T, S]")
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), scores.data_ptr(), B, qlen,
            Hq, Hkv, S, NB, float(sm_scale), float(k_scale), _stream(dev, stream))
    k_only = kv.shape[3] == HEAD_DIM
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 1 if k_only else 2)
        st = _lib().msa_score_scaled(q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0,
                                     args[0], sc, int(k_only), *args[1:])
    elif _fp8(q, q_scale):
        f = _lib().msa_score_kcache_q8 if k_only else _lib().msa_score_q8
        st = f(q.data_ptr(), float(q_scale), *args)
    else:
        f = _lib().msa_score_kcache if k_only else _lib().msa_score
        st = f(q.data_ptr(), *args)
    _native.check(st, "msa_score")
    return scores


def topk(scores: torch.Tensor, seq_lens: torch.Tensor, qlen: int, k: int = TOPK,
         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Selected blocks int32 [T, Hkv, 16] (msa_topk).  `scores` is indexed
    [g, i, n] and may be any strided view (e.g. a transpose of [Hkv, S, T])."""
    if not (isinstance(scores, torch.Tensor) and scores.is_cuda and scores.dtype == torch.float32):
        raise TypeError("scores must be a CUDA float32 tensor")
    dev = scores.device
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    Hkv, T, S = scores.shape
    B = seq_lens.shape[0]
    if T != B * qlen:
        raise ValueError("scores' token dim must be B*qlen")
    if out is None:
        out = _empty((T, Hkv, k), torch.int32, dev, stream)
    _need(out, "out", (torch.int32,), dev)
    sh, stt, sn = scores.stride()
    st = _lib().msa_topk(scores.data_ptr(), sh, stt, sn, seq_lens.data_ptr(), out.data_ptr(), B,
                         qlen, Hkv, S, k, _stream(dev, stream))
    _native.check(st, "msa_topk")
    return out


def sparse_decode(q, kv, block_table, seq_lens, topk_idx, qlen: int, sm_scale: float,
                  k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
                  num_splits: int = 0, workspace: torch.Tensor | None = None,
                  stream=None, q_scale: float = 1.0,
                  kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Attention over the selected pages, bf16 [T, Hq, 128] (msa_sparse_decode;
    with more than one split the merge runs on the same stream).  kv_scales:
    page scales [NB, Hkv, 2]."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, qlen)
    _need(topk_idx, "topk", (torch.int32,), dev)
    if tuple(topk_idx.shape) != (B * qlen, Hkv, TOPK):
        raise ValueError("topk must be [T, Hkv, 16]")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    splits, workspace, ws_ptr, ws_bytes = _parts(num_splits, kv_scales, B, qlen, Hq, Hkv,
                                                 workspace, dev, stream)
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), topk_idx.data_ptr(), ws_ptr,
            ws_bytes, out.data_ptr(), B, qlen, Hq, Hkv, S, NB, float(sm_scale), float(k_scale),
            float(v_scale), splits, _stream(dev, stream))
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2)
        st = _lib().msa_sparse_decode_scaled(
            q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, args[0], sc, *args[1:])
    elif _fp8(q, q_scale):
        st = _lib().msa_sparse_decode_q8(q.data_ptr(), float(q_scale), *args)
    else:
        st = _lib().msa_sparse_decode(q.data_ptr(), *args)
    _native.check(st, "msa_sparse_decode")
    return out


def dense_splits(stride: int) -> int:
    """Split count of dense_decode for a block table of `stride` columns (0:
    longer than dense_decode takes)."""
    return int(_lib().msa_dense_splits(int(stride)))


def dense_decode(q, kv, block_table, seq_lens, qlen: int, sm_scale: float, k_scale: float = 1.0,
                 v_scale: float = 1.0, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None,
                 q_scale: float = 1.0, kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Attention over every visible block, bf16 [T, Hq, 128] (msa_dense_decode;
    with more than one split the merge runs on the same stream).  kv_scales:
    page scales [NB, Hkv, 2]."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, qlen)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    splits = dense_splits(S)
    if splits == 0:
        raise ValueError("dense_decode takes block tables of at most 2048 columns")
    need = workspace_bytes(B, qlen, Hq, splits)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = _own(need, torch.uint8, dev, stream)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), ws_ptr, ws_bytes,
            out.data_ptr(), B, qlen, Hq, Hkv, S, NB, float(sm_scale), float(k_scale),
            float(v_scale), _stream(dev, stream))
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2)
        st = _lib().msa_dense_decode_scaled(
            q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, args[0], sc, *args[1:])
    elif _fp8(q, q_scale):
        st = _lib().msa_dense_decode_q8(q.data_ptr(), float(q_scale), *args)
    else:
        st = _lib().msa_dense_decode(q.data_ptr(), *args)
    _native.check(st, "msa_dense_decode")
    return out


#: Rows of at most this many candidate blocks are selected inside the attend
#: kernel (the selector keeps them in registers there); longer rows go through
#: the selector kernel, which holds up to 2048 candidates in registers.
FUSED_MAX_BLOCKS = 512


def fused_selection(stride: int) -> bool:
    """Whether decode_step selects inside the attend kernel for a block table of
    `stride` columns (the longest possible row)."""
    return stride <= FUSED_MAX_BLOCKS


def sparse_decode_select(q, kv, block_table, seq_lens, scores, qlen: int, sm_scale: float,
                         k_scale: float = 1.0, v_scale: float = 1.0,
                         topk_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         num_splits: int = 0, workspace: torch.Tensor | None = None,
                         stream=None, q_scale: float = 1.0,
                         kv_scales: torch.Tensor | None = None):
    """Selection and attention in one kernel (msa_sparse_decode_select): the
    top-16 blocks of every (token, KV head) row are selected from `scores`
    (any strides, as msa_topk) and attended.  kv_scales: page scales [NB, Hkv,
    2].  Returns (topk [T, Hkv, 16], out)."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, qlen)
    # any strided view, as for topk()
    if not (isinstance(scores, torch.Tensor) and scores.is_cuda and scores.dtype == torch.float32
            and scores.device == dev):
        raise TypeError("scores must be a float32 tensor on q's device")
    if scores.dim() != 3 or scores.shape[0] != Hkv or scores.shape[1] != B * qlen \
            or scores.shape[2] < S:
        raise ValueError("scores must be [Hkv, T, >= S]")
    if topk_out is None:
        topk_out = _empty((B * qlen, Hkv, TOPK), torch.int32, dev, stream)
    _need(topk_out, "topk_out", (torch.int32,), dev)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    splits, workspace, ws_ptr, ws_bytes = _parts(num_splits, kv_scales, B, qlen, Hq, Hkv,
                                                 workspace, dev, stream)
    sh, st, sn = scores.stride()
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), scores.data_ptr(), sh, st,
            sn, topk_out.data_ptr(), ws_ptr, ws_bytes, out.data_ptr(), B, qlen, Hq, Hkv, S, NB,
            float(sm_scale), float(k_scale), float(v_scale), splits, _stream(dev, stream))
    if kv_scales is not None:
        psc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2)
        status = _lib().msa_sparse_decode_select_scaled(
            q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, args[0], psc, *args[1:])
    elif _fp8(q, q_scale):
        status = _lib().msa_sparse_decode_select_q8(q.data_ptr(), float(q_scale), *args)
    else:
        status = _lib().msa_sparse_decode_select(q.data_ptr(), *args)
    _native.check(status, "msa_sparse_decode_select")
    return topk_out, out


def _cu_seqlens(cu_seqlens_q, batch: int, dev, q=None):
    """Checks cu_seqlens_q [B + 1]; the tokens of q."""
    _need(cu_seqlens_q, "cu_seqlens_q", (torch.int32,), dev)
    if cu_seqlens_q.shape != (batch + 1,):
        raise ValueError("cu_seqlens_q must be [B + 1]")
    return int(q.shape[0]) if q is not None else None


def _prefill_geometry(q, kv, block_table, seq_lens, cu_seqlens_q):
    """Shapes of a prefill-style batch: q holds T tokens, request b owning
    tokens cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, None)
    return dev, B, _cu_seqlens(cu_seqlens_q, B, dev, q), S, Hq, Hkv, NB


def sparse_prefill(q, kv, block_table, seq_lens, cu_seqlens_q, topk_idx, sm_scale: float,
                   k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
                   num_splits: int = 0, workspace: torch.Tensor | None = None, stream=None,
                   q_scale: float = 1.0,
                   kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Sparse attend of a prefill or chunked-prefill batch (msa_sparse_prefill):
    request b's query tokens are q[cu_seqlens_q[b] : cu_seqlens_q[b + 1]], the
    last ones of its seq_lens[b]; each token attends its own list
    topk_idx [T, Hkv, 16].  kv_scales: page scales [NB, Hkv, 2].  Returns bf16
    [T, Hq, 128]."""
    dev, B, T, S, Hq, Hkv, NB = _prefill_geometry(q, kv, block_table, seq_lens, cu_seqlens_q)
    _need(topk_idx, "topk", (torch.int32,), dev)
    if tuple(topk_idx.shape) != (T, Hkv, TOPK):
        raise ValueError("topk must be [T, Hkv, 16]")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    # one CTA per token: the single-token rule, choose_splits(T, 1, ...)
    splits, workspace, ws_ptr, ws_bytes = _parts(num_splits, kv_scales, max(T, 1), 1, Hq, Hkv,
                                                 workspace, dev, stream)
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(),
            topk_idx.data_ptr(), ws_ptr, ws_bytes, out.data_ptr(), B, T, Hq, Hkv, S, NB,
            float(sm_scale), float(k_scale), float(v_scale), splits, _stream(dev, stream))
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2)
        st = _lib().msa_sparse_prefill_scaled(
            q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, args[0], sc, *args[1:])
    elif _fp8(q, q_scale):
        st = _lib().msa_sparse_prefill_q8(q.data_ptr(), float(q_scale), *args)
    else:
        st = _lib().msa_sparse_prefill(q.data_ptr(), *args)
    _native.check(st, "msa_sparse_prefill")
    return out


def sparse_prefill_select(q, kv, block_table, seq_lens, cu_seqlens_q, scores, sm_scale: float,
                          k_scale: float = 1.0, v_scale: float = 1.0,
                          topk_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          num_splits: int = 0, workspace: torch.Tensor | None = None,
                          stream=None, q_scale: float = 1.0,
                          kv_scales: torch.Tensor | None = None):
    """Per-token causal top-16 selected from `scores` [Hkv, T, >= S] (any
    strides) and attended, for a prefill-style batch
    (msa_sparse_prefill_select).  kv_scales: page scales [NB, Hkv, 2].  Returns
    (topk [T, Hkv, 16], out)."""
    dev, B, T, S, Hq, Hkv, NB = _prefill_geometry(q, kv, block_table, seq_lens, cu_seqlens_q)
    if not (isinstance(scores, torch.Tensor) and scores.is_cuda and scores.dtype == torch.float32
            and scores.device == dev):
        raise TypeError("scores must be a float32 tensor on q's device")
    if scores.dim() != 3 or scores.shape[0] != Hkv or scores.shape[1] != T \
            or scores.shape[2] < S:
        raise ValueError("scores must be [Hkv, T, >= S]")
    if topk_out is None:
        topk_out = _empty((T, Hkv, TOPK), torch.int32, dev, stream)
    _need(topk_out, "topk_out", (torch.int32,), dev)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    # one CTA per token: the single-token rule, choose_splits(T, 1, ...)
    splits, workspace, ws_ptr, ws_bytes = _parts(num_splits, kv_scales, max(T, 1), 1, Hq, Hkv,
                                                 workspace, dev, stream)
    sh, st, sn = scores.stride()
    args = (kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(),
            scores.data_ptr(), sh, st, sn, topk_out.data_ptr(), ws_ptr, ws_bytes, out.data_ptr(),
            B, T, Hq, Hkv, S, NB, float(sm_scale), float(k_scale), float(v_scale), splits,
            _stream(dev, stream))
    if kv_scales is not None:
        psc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2)
        status = _lib().msa_sparse_prefill_select_scaled(
            q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, args[0], psc, *args[1:])
    elif _fp8(q, q_scale):
        status = _lib().msa_sparse_prefill_select_q8(q.data_ptr(), float(q_scale), *args)
    else:
        status = _lib().msa_sparse_prefill_select(q.data_ptr(), *args)
    _native.check(status, "msa_sparse_prefill_select")
    return topk_out, out


def score_prefill(q, kv, block_table, seq_lens, cu_seqlens_q, sm_scale: float,
                  k_scale: float = 1.0, scores: torch.Tensor | None = None, stream=None,
                  q_scale: float = 1.0, kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Block scores fp32 [Hkv, T, S] of a prefill or chunked-prefill batch
    (msa_score_prefill): score() with one query length per request, the tokens as in
    sparse_prefill().  `kv` may be a K-only (index-K) cache [NB, Hkv, 128, 128];
    kv_scales: page scales [NB, Hkv, 2] ([NB, Hkv, 1] of a K-only cache)."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, None, k_only_ok=True)
    T = _cu_seqlens(cu_seqlens_q, B, dev, q)
    if scores is None:
        scores = _empty((Hkv, T, S), torch.float32, dev, stream)
    _need(scores, "scores", (torch.float32,), dev)
    if scores.shape != (Hkv, T, S):
        raise ValueError("scores must be [Hkv, T, S]")
    k_only = kv.shape[3] == HEAD_DIM
    sc = None
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 1 if k_only else 2)
    if T == 0 and B == 0:
        return scores        # empty tensors have no address to check
    st = _lib().msa_score_prefill(
        q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, kv.data_ptr(), sc, int(k_only),
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(), scores.data_ptr(), B,
        T, Hq, Hkv, S, NB, float(sm_scale), float(k_scale), _stream(dev, stream))
    _native.check(st, "msa_score_prefill")
    return scores


def topk_prefill(scores: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor,
                 k: int = TOPK, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Selected blocks int32 [T, Hkv, 16] of a prefill or chunked-prefill batch
    (msa_topk_prefill): topk() with one query length per request.  `scores` is
    indexed [g, i, n] and may be any strided view."""
    if not (isinstance(scores, torch.Tensor) and scores.is_cuda and scores.dtype == torch.float32):
        raise TypeError("scores must be a CUDA float32 tensor")
    if scores.dim() != 3:
        raise ValueError("scores must be [Hkv, T, S]")
    dev = scores.device
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    Hkv, T, S = scores.shape
    B = seq_lens.shape[0]
    _cu_seqlens(cu_seqlens_q, B, dev)
    if out is None:
        out = _empty((T, Hkv, k), torch.int32, dev, stream)
    _need(out, "out", (torch.int32,), dev)
    if out.shape != (T, Hkv, k):
        raise ValueError("out must be [T, Hkv, 16]")
    if T == 0 and B == 0:
        return out
    sh, stt, sn = scores.stride()
    st = _lib().msa_topk_prefill(scores.data_ptr(), sh, stt, sn, seq_lens.data_ptr(),
                                 cu_seqlens_q.data_ptr(), out.data_ptr(), B, T, Hkv, S, k,
                                 _stream(dev, stream))
    _native.check(st, "msa_topk_prefill")
    return out


@functools.lru_cache(maxsize=None)
def _dense_prefill_bytes(index: int) -> int:
    sms = torch.cuda.get_device_properties(index).multi_processor_count
    return int(_lib().msa_dense_prefill_workspace_bytes(sms))


def dense_prefill_workspace_bytes(device=None) -> int:
    """Bytes of workspace dense_prefill uses on `device` (the current one), whatever
    the batch."""
    index = None if device is None else torch.device(device).index
    return _dense_prefill_bytes(torch.cuda.current_device() if index is None else index)


def dense_prefill(q, kv, block_table, seq_lens, cu_seqlens_q, sm_scale: float,
                  k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None, q_scale: float = 1.0,
                  kv_scales: torch.Tensor | None = None) -> torch.Tensor:
    """Attention over every visible key of a prefill or chunked-prefill batch, bf16
    [T, Hq, 128] (msa_dense_prefill): the tokens as in sparse_prefill(), their keys
    and values in the cache already.  workspace: dense_prefill_workspace_bytes();
    kv_scales: page scales [NB, Hkv, 2]."""
    dev, B, T, S, Hq, Hkv, NB = _prefill_geometry(q, kv, block_table, seq_lens, cu_seqlens_q)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    if out.shape != q.shape:
        raise ValueError("out must be [T, Hq, 128]")
    sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2) if kv_scales is not None else None
    if T == 0 and B == 0:
        return out
    need = dense_prefill_workspace_bytes(dev)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = _own(need, torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    st = _lib().msa_dense_prefill(
        q.data_ptr(), float(q_scale) if _fp8(q, q_scale) else 0.0, kv.data_ptr(), sc,
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), out.data_ptr(), B, T, Hq, Hkv, S, NB,
        float(sm_scale), float(k_scale), float(v_scale), _stream(dev, stream))
    _native.check(st, "msa_dense_prefill")
    return out


def combine(workspace: torch.Tensor, tokens: int, num_q_heads: int, num_splits: int,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Merge split-K partials (layout of msa_workspace_bytes) into bf16 [T, Hq, 128]."""
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda):
        raise TypeError("workspace must be a CUDA tensor")
    dev = workspace.device
    if out is None:
        out = _empty((tokens, num_q_heads, HEAD_DIM), torch.bfloat16, dev, stream)
    _need(out, "out", (torch.bfloat16,), dev)
    st = _lib().msa_combine(workspace.data_ptr(), out.data_ptr(), tokens, num_q_heads, num_splits,
                            _stream(dev, stream))
    _native.check(st, "msa_combine")
    return out


@dataclass
class DecodeBuffers:
    """Preallocated outputs and workspace of one decode step (reusable, and
    stable addresses for CUDA-graph capture).  chosen: num_splits is the
    caller's; else decode_step with kv_scales cuts rows as num_splits=0 does."""
    scores: torch.Tensor
    topk: torch.Tensor
    out: torch.Tensor
    workspace: torch.Tensor | None
    num_splits: int
    chosen: bool = True

    @staticmethod
    def allocate(batch: int, qlen: int, num_q_heads: int, num_kv_heads: int, stride: int,
                 device, num_splits: int = 0, stream=None) -> "DecodeBuffers":
        T = batch * qlen
        splits = num_splits if num_splits > 0 else choose_splits(batch, qlen, num_kv_heads)
        need = workspace_bytes(batch, qlen, num_q_heads, splits)
        ws = _own(need, torch.uint8, device, stream) if need else None
        return DecodeBuffers(
            scores=_empty((num_kv_heads, T, stride), torch.float32, device, stream),
            topk=_empty((T, num_kv_heads, TOPK), torch.int32, device, stream),
            out=_empty((T, num_q_heads, HEAD_DIM), torch.bfloat16, device, stream),
            workspace=ws, num_splits=splits, chosen=num_splits > 0)


def decode_step(q, kv, block_table, seq_lens, qlen: int, sm_scale: float, k_scale: float = 1.0,
                v_scale: float = 1.0, buffers: DecodeBuffers | None = None, stream=None,
                q_scale: float = 1.0, index_k: torch.Tensor | None = None,
                index_k_scale: float | None = None, kv_scales: torch.Tensor | None = None,
                index_scales: torch.Tensor | None = None):
    """One decode step in one library call (msa_decode_step): score, then
    selection + attention on one stream, no host sync -- in one kernel
    (msa_sparse_decode_select) while rows have at most FUSED_MAX_BLOCKS
    candidate blocks, else msa_topk then msa_sparse_decode (-> combine when
    split).  With `index_k` (a K-only cache [NB, Hkv, 128, 128] on the same
    block table, scale index_k_scale, default k_scale) the blocks are scored
    on it instead of kv's K halves.  kv_scales: page scales [NB, Hkv, 2] of kv,
    with index_scales [NB, Hkv, 1] those of index_k (msa_decode_step_scaled).
    Returns (scores, topk, out)."""
    dev, B, S, Hq, Hkv, NB = _geometry(q, kv, block_table, seq_lens, qlen)
    if buffers is None:
        buffers = DecodeBuffers.allocate(B, qlen, Hq, Hkv, S, dev, stream=stream)
    if index_k is not None:
        _need(index_k, "index_k", _KV_DTYPES, dev)
        if (index_k.dim() != 4 or index_k.shape[1] != Hkv or index_k.shape[2] != PAGE_SIZE
                or index_k.shape[3] != HEAD_DIM or index_k.shape[0] != NB):
            raise ValueError("index_k must be [num_blocks, Hkv, 128, 128]")
    bf = buffers
    _need(bf.scores, "scores", (torch.float32,), dev)
    _need(bf.topk, "topk", (torch.int32,), dev)
    _need(bf.out, "out", (torch.bfloat16,), dev)
    if (tuple(bf.scores.shape) != (Hkv, B * qlen, S) or tuple(bf.topk.shape) != (B * qlen, Hkv, TOPK)
            or tuple(bf.out.shape) != tuple(q.shape)):
        raise ValueError("buffers do not match the step's shapes")
    ws = bf.workspace
    ws_ptr = ws.data_ptr() if ws is not None else None
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    fp8 = _fp8(q, q_scale)
    ik_scale = (k_scale if index_k_scale is None else index_k_scale) if index_k is not None else 0.0
    if index_scales is not None and (index_k is None or kv_scales is None):
        raise ValueError("index_scales go with index_k and kv_scales")
    head = (q.data_ptr(), float(q_scale) if fp8 else 0.0, kv.data_ptr())
    index = (index_k.data_ptr() if index_k is not None else None, float(ik_scale))
    if kv_scales is not None:
        f = _lib().msa_decode_step_scaled
        head += (_page_scales(kv_scales, "kv_scales", dev, NB, Hkv, 2),)
        index += (None if index_scales is None else
                  _page_scales(index_scales, "index_scales", dev, NB, Hkv, 1),)
    else:
        f = _lib().msa_decode_step
    st = f(
        *head, *index,
        block_table.data_ptr(), seq_lens.data_ptr(), bf.scores.data_ptr(), bf.topk.data_ptr(),
        ws_ptr, ws_bytes, bf.out.data_ptr(), B, qlen, Hq, Hkv, S, NB, float(sm_scale),
        float(k_scale), float(v_scale), bf.num_splits if kv_scales is None or bf.chosen else 0,
        _stream(dev, stream))
    _native.check(st, "msa_decode_step")
    return bf.scores, bf.topk, bf.out


def _rows(t, name: str, heads: int, tokens: int, dev):
    """Checks bf16 rows [T, heads, 128] whose heads lie one behind the other and
    returns the tokens' distance in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if t.shape != (tokens, heads, HEAD_DIM):
        raise ValueError(f"{name} must be [{tokens}, {heads}, 128]")
    st, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != HEAD_DIM):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if tokens <= 1:
        return heads * HEAD_DIM
    if st % 8 or st < heads * HEAD_DIM:
        raise ValueError(f"{name}: tokens must be a multiple of 8 elements apart and not overlap")
    return st


def _append(fn, k, v, kv, block_table, seq_lens, tokens, cu, qlen, k_scale, v_scale, kv_scales,
            cos_sin, interleaved, q, q_out, q_scale, stream):
    _need(kv, "kv", _KV_DTYPES)
    dev = kv.device
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    sides = 1 if v is None else 2
    shape, table = kv.shape, block_table.shape
    if len(shape) != 4 or shape[2] != PAGE_SIZE or shape[3] != sides * HEAD_DIM:
        raise ValueError("kv must be [num_blocks, Hkv, 128, 256], or without v a K-only "
                         "[num_blocks, Hkv, 128, 128]")
    if len(table) != 2 or seq_lens.shape != table[:1]:
        raise ValueError("block_table must be [B, S] and seq_lens [B]")
    B, S = table
    NB, Hkv = shape[0], shape[1]
    Hq = GROUP * Hkv
    if tokens is None:
        tokens = B * qlen
    ks = _rows(k, "k", Hkv, tokens, dev)
    vs = _rows(v, "v", Hkv, tokens, dev) if v is not None else 0
    qs = qp = qo = None
    q8 = 0.0
    if q is not None:
        qs, qp = _rows(q, "q", Hq, tokens, dev), q.data_ptr()
        if q_out is None:
            q_out = _empty((tokens, Hq, HEAD_DIM), torch.bfloat16, dev, stream)
        _need(q_out, "q_out", (torch.bfloat16,) + ((_FP8_Q,) if _FP8_Q is not None else ()), dev)
        if q_out.shape != (tokens, Hq, HEAD_DIM):
            raise ValueError("q_out must be [T, Hq, 128]")
        qo = q_out.data_ptr()
        if _fp8(q_out, q_scale):
            q8 = float(q_scale)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    sc = None
    if kv_scales is not None:
        sc = _page_scales(kv_scales, "kv_scales", dev, NB, Hkv, sides)
    tab, max_pos, rot = None, 0, 0
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", (torch.float32,), dev)
        table = cos_sin.shape
        if len(table) != 2:
            raise ValueError("cos_sin must be [max_pos, rot_dim]")
        tab, (max_pos, rot) = cos_sin.data_ptr(), table
        if rot == 0 or rot > HEAD_DIM or rot % 16:
            raise ValueError("rot_dim must be a multiple of 16 up to 128")
    if B == 0 and tokens == 0:
        return q_out        # empty tensors have no address to check
    mid = () if cu is None else (cu.data_ptr(),)
    st = fn(
        k.data_ptr(), ks, v.data_ptr() if v is not None else None, vs, qp, qs or 0, tab, max_pos,
        rot, 1 if interleaved else 0, kv.data_ptr(), sc, qo, q8, block_table.data_ptr(),
        seq_lens.data_ptr(), *mid, B, tokens if cu is not None else qlen, Hq, Hkv, S, NB,
        k_scale, v_scale, _stream(dev, stream))
    _native.check(st, fn.__name__)
    return q_out


def append_kv(k, v, kv, block_table, seq_lens, qlen: int, k_scale: float = 1.0,
              v_scale: float = 1.0, kv_scales: torch.Tensor | None = None,
              cos_sin: torch.Tensor | None = None, interleaved: bool = False, q=None,
              q_out: torch.Tensor | None = None, q_scale: float = 1.0, stream=None):
    """Writes a decode step's keys and values into the paged cache (msa_append_kv).

    k, v bf16 [T, Hkv, 128], T = B * qlen, possibly slices of one projection's
    output (a token's heads contiguous); v None for a K-only cache.  Token j of
    request b goes to position seq_lens[b] - qlen + j (seq_lens counts the new
    tokens).  cos_sin fp32 [max_pos, rot_dim] (cosines, then sines of each
    position) rotates the first rot_dim dims of k, and of q [T, Hq, 128] into
    q_out (bf16, or fp8 e4m3 codes of q / q_scale; q itself for in place), in
    halves or, with `interleaved`, in neighbouring pairs.  kv_scales [NB, Hkv,
    2] (or 1): page scales, updated; else codes are x / k_scale, x / v_scale.
    Returns q_out (None without q)."""
    return _append(_lib().msa_append_kv, k, v, kv, block_table, seq_lens, None, None, qlen, k_scale,
                   v_scale, kv_scales, cos_sin, interleaved, q, q_out, q_scale, stream)


def append_kv_prefill(k, v, kv, block_table, seq_lens, cu_seqlens_q, k_scale: float = 1.0,
                      v_scale: float = 1.0, kv_scales: torch.Tensor | None = None,
                      cos_sin: torch.Tensor | None = None, interleaved: bool = False, q=None,
                      q_out: torch.Tensor | None = None, q_scale: float = 1.0, stream=None):
    """append_kv of a prefill or chunked-prefill batch (msa_append_kv_prefill):
    request b's tokens are rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 of k,
    v and q, the last ones of its seq_lens[b]."""
    _need(seq_lens, "seq_lens", (torch.int32,))
    _need(cu_seqlens_q, "cu_seqlens_q", (torch.int32,), seq_lens.device)
    tokens = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
    if tuple(cu_seqlens_q.shape) != (seq_lens.shape[0] + 1,):
        raise ValueError("cu_seqlens_q must be [B + 1]")
    return _append(_lib().msa_append_kv_prefill, k, v, kv, block_table, seq_lens, tokens,
                   cu_seqlens_q, None, k_scale, v_scale, kv_scales, cos_sin, interleaved, q, q_out,
                   q_scale, stream)


_CACHE_DTYPES = _KV_DTYPES + (torch.float32,)


def _caches(caches, num_blocks, dev):
    """The bytes of an msa_cache_t for each tensor [num_blocks, ...]: rows of tokens in
    [.., 128, bytes] of 8-bit types, else whole pages."""
    out = []
    for i, c in enumerate(caches):
        if not (isinstance(c, torch.Tensor) and c.dtype in _CACHE_DTYPES and c.device == dev
                and c.is_contiguous()):
            _need(c, f"caches[{i}]", _CACHE_DTYPES, dev)
        shape = c.shape
        if len(shape) < 2 or shape[0] != num_blocks:
            raise ValueError(f"caches[{i}] must be [num_blocks, ...] of the pool's pages")
        if c.dtype is torch.float32:          # page scales [NB, Hkv, sides]
            if len(shape) != 3:
                raise ValueError(f"caches[{i}]: page scales are [num_blocks, Hkv, sides]")
            rows, row_bytes = 1, 4 * shape[2]
        else:
            if len(shape) != 4 or shape[2] != PAGE_SIZE:
                raise ValueError(f"caches[{i}] must be [num_blocks, Hkv, 128, row bytes]")
            rows, row_bytes = PAGE_SIZE, shape[3]
        out.append(_native.pack_cache(c.data_ptr(), shape[1], rows, row_bytes))
    return b"".join(out)


def _int32(t, name: str, shape, dev):
    """Checks int32 `t` of `shape` (None: any length of a vector) on `dev`, which is a CUDA
    device, and returns its address."""
    try:
        if (t.dtype is torch.int32 and t.device == dev and t.is_contiguous()
                and (t.shape == shape or (shape is None and t.dim() == 1))):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, (torch.int32,), dev)
    raise ValueError(f"{name} must be " + ("a vector" if shape is None else str(list(shape))))


def _outputs(given, dev, stream):
    """Tensors and addresses of the outputs [(tensor or None, name, shape)]."""
    out, at = [], []
    for t, name, shape in given:
        if t is None:
            t = _empty(shape, torch.int32, dev, stream)
            at.append(t.data_ptr())
        else:
            at.append(_int32(t, name, shape, dev))
        out.append(t)
    return out, at


def _table(block_table, seq_lens, refs):
    if not isinstance(block_table, torch.Tensor) or not isinstance(refs, torch.Tensor):
        raise TypeError("block_table and refs must be torch.Tensors")
    if block_table.dim() != 2 or not block_table.is_cuda:
        raise ValueError("block_table must be a CUDA tensor [B, S]")
    dev, (B, S) = block_table.device, block_table.shape
    return (dev, B, S, refs.shape[0] if refs.dim() else 0,
            _int32(block_table, "block_table", (B, S), dev), _int32(seq_lens, "seq_lens", (B,), dev),
            _int32(refs, "refs", None, dev))


def fork_pages(block_table, seq_lens, parents, refs, caches=(), grow=None, block_table_out=None,
               seq_lens_out=None, refs_out=None, copies=None, stream=None):
    """The next step's rows of a block table (msa_fork_pages): new row b continues row
    parents[b] of block_table [B, S], seq_lens [B] (-1: a new, empty row) and has room
    for grow[b] more tokens; rows without a child are freed.  Full pages are shared, a
    begun page goes to the first child (where nobody else holds it) and is copied for
    the others, in every tensor of `caches` (kv [NB, Hkv, 128, 256], K-only caches, page
    scales, of any number of layers).  refs [NB]: how many rows hold each page; free
    pages (0) are taken in ascending order.  Returns (block_table, seq_lens, refs, copies [rows, 3])."""
    dev, B, S, NB, table, lens, counts = _table(block_table, seq_lens, refs)
    follows = _int32(parents, "parents", None, dev)
    rows = parents.shape[0]
    more = None if grow is None else _int32(grow, "grow", (rows,), dev)
    handles = _caches(caches, NB, dev)
    out, at = _outputs(((block_table_out, "block_table_out", (rows, S)),
                        (seq_lens_out, "seq_lens_out", (rows,)), (refs_out, "refs_out", (NB,)),
                        (copies, "copies", (rows, 3))), dev, stream)
    st = _lib().msa_fork_pages(table, lens, follows, more, counts, *at, B, rows, S, NB, handles,
                               len(caches), _stream(dev, stream))
    _native.check(st, "msa_fork_pages")
    return tuple(out)


def compact_pages(block_table, seq_lens, refs, caches=(), block_table_out=None, refs_out=None,
                  copies=None, stream=None):
    """Pages in use moved to the lowest indices (msa_compact_pages), in every tensor of
    `caches` as fork_pages() takes them.  Returns (block_table, refs, copies [NB // 2,
    3]): copies lists the moves (from, to, 128), then (-1, -1, 0)."""
    dev, B, S, NB, table, lens, counts = _table(block_table, seq_lens, refs)
    handles = _caches(caches, NB, dev)
    out, at = _outputs(((block_table_out, "block_table_out", (B, S)), (refs_out, "refs_out", (NB,)),
                        (copies, "copies", (NB // 2, 3))), dev, stream)
    st = _lib().msa_compact_pages(table, lens, counts, *at, B, S, NB, handles, len(caches),
                                  _stream(dev, stream))
    _native.check(st, "msa_compact_pages")
    return tuple(out)


def copy_pages(copies, caches, stream=None):
    """Copies of pages (msa_copy_pages): copies int32 [n, 3] of (source page,
    destination page, token rows), as fork_pages() and compact_pages() return them, in
    every tensor of `caches` (further layers' caches, say)."""
    _need(copies, "copies", (torch.int32,))
    dev = copies.device
    if copies.dim() != 2 or copies.shape[1] != 3:
        raise ValueError("copies must be [n, 3]")
    if not caches:
        return
    NB = caches[0].shape[0] if isinstance(caches[0], torch.Tensor) and caches[0].dim() else 0
    handles = _caches(caches, NB, dev)
    st = _lib().msa_copy_pages(copies.data_ptr(), copies.shape[0], NB, handles, len(caches),
                               _stream(dev, stream))
    _native.check(st, "msa_copy_pages")


def set_union_tile(enable: bool) -> bool:
    """msa_set_union_tile: attend sparse decode steps of two or more tokens per
    request over the union of each 4-token tile's lists, loading each shared
    page once (pays off when a request's tokens list mostly the same blocks).
    Off by default; dense decode always works this way, and calls with
    kv_scales= on lists never do.  Returns the previous setting."""
    return bool(_lib().msa_set_union_tile(1 if enable else 0))


def set_input_overlap(enable: bool) -> bool:
    """msa_set_input_overlap: let the first kernel of every library call start
    before the previous kernel on its stream has finished (only safe when that
    kernel wrote none of the call's inputs, e.g. another library call).  Off
    by default.  Returns the previous setting."""
    return bool(_lib().msa_set_input_overlap(1 if enable else 0))


def get_error(clear: bool = True) -> int:
    """The device's sticky MSA_ERR_* bits (synchronises the device)."""
    flags = ctypes.c_uint(0)
    _native.check(_lib().msa_get_error(ctypes.byref(flags), 1 if clear else 0), "msa_get_error")
    return int(flags.value)
