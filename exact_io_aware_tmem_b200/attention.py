"""Python entry points over the C ABI (argument marshalling only).

Every step of the forward and backward passes runs in the CUDA kernels of
libfa_b200.so; this module checks torch tensors, allocates the outputs with
torch (device memory and streams are all PyTorch provides), and passes raw
pointers and the current stream to ``fa_fwd`` / ``fa_bwd``.

Layouts (token-major, as in include/fa.h):
  dense : q [B, N, H, D], k / v [B, N, H_kv, D]; lse [B, H, N]
  packed: q [T, H, D],    k / v [T, H_kv, D] with cu_seqlens int32 [B+1]
          on the device; lse [H, T]
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import Optional

import torch

from . import _abi

# The library the entry points call: libfa_b200.so, or, inside debug_build(),
# the same kernels built with index checks and event stamps.
_lib = _abi.lib


@contextlib.contextmanager
def debug_build():
    """Route the entry points through libfa_b200_debug.so (include/fa.h,
    "Debug build") for the duration of the block."""
    global _lib
    prev = _lib
    _lib = _abi.debug_lib
    try:
        yield _abi.debug_lib()
    finally:
        _lib = prev

_DTYPES = {torch.bfloat16: _abi.FA_BF16, torch.float32: _abi.FA_F32}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The handle alone, 0.05 us instead of 2.2 through a Stream object. Not a public name of
# torch: where a release lacks it, the public one serves.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    index = torch.cuda.current_device() if device.index is None else device.index
    if _raw_stream is None:
        return torch.cuda.current_stream(index).cuda_stream
    return _raw_stream(index)


def _shape(q: torch.Tensor, k: torch.Tensor, cu_seqlens, max_seqlen):
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}; use bfloat16 or float32")
    for t in (q, k):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    if cu_seqlens is None:
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("dense inputs are [B, N, H, D]")
        B, N, H, D = q.shape
        H_kv = k.shape[2]
        return B, N, H, H_kv, D, 0, B * N
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("packed inputs are [T, H, D]")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor")
    T, H, D = q.shape
    if max_seqlen is None:
        raise ValueError("packed inputs need max_seqlen")
    return cu_seqlens.numel() - 1, 0, H, k.shape[1], D, int(max_seqlen), T


def _call(what: str, fn, device: torch.device, *args) -> None:
    """``fn(*args)`` with the tensors' device as the current one: the library launches there."""
    if device.index is None or device.index == torch.cuda.current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st:
        _abi.check(st, what)


def _is(t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device) -> bool:
    return t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()


def _aux(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple,
         device: torch.device) -> Optional[int]:
    """Pointer of an optional side tensor after its checks."""
    if t is None:
        return None
    if not _is(t, shape, dtype, device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _score_shape(q, cu_seqlens, softcap, alibi_slopes, key_begin, key_end):
    """fa_score_shape of the arguments, or None when none is given."""
    if softcap is None and alibi_slopes is None and key_begin is None and key_end is None:
        return None
    shape, device = q.shape, q.device
    tokens = shape[:1] if cu_seqlens is not None else shape[:2]
    if cu_seqlens is not None and (cu_seqlens.device != device or not cu_seqlens.is_contiguous()):
        raise ValueError(f"cu_seqlens must be contiguous on {device}")
    return _abi.ScoreShape(
        0.0 if softcap is None else float(softcap),
        _aux(alibi_slopes, "alibi_slopes", torch.float32, shape[-2:-1], device),
        _aux(key_begin, "key_begin", torch.int32, tokens, device),
        _aux(key_end, "key_end", torch.int32, tokens, device))


def _same(what: str, like: torch.Tensor, **tensors):
    """Shape, type, layout and device of ``tensors`` are those of ``like``."""
    shape, dtype, device = like.shape, like.dtype, like.device
    for name, t in tensors.items():
        if not _is(t, shape, dtype, device):
            raise ValueError(f"{name} must match {what} in shape, dtype and device and be contiguous")


def _room(workspace: torch.Tensor, device: torch.device) -> int:
    """Bytes of a workspace after its checks."""
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace.numel() * workspace.element_size()


def _beside(q: torch.Tensor, k: torch.Tensor):
    """k differs from q in its heads only."""
    a, b = q.shape, k.shape
    if k.device != q.device or k.dtype is not q.dtype or a[-1] != b[-1] or a[:-2] != b[:-2]:
        raise ValueError("k must match q but for its heads")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
        scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
        max_seqlen: Optional[int] = None, out: Optional[torch.Tensor] = None,
        lse: Optional[torch.Tensor] = None, softcap: Optional[float] = None,
        alibi_slopes: Optional[torch.Tensor] = None, key_begin: Optional[torch.Tensor] = None,
        key_end: Optional[torch.Tensor] = None):
    """Attention forward. Returns (O, LSE).

    Shaped scores (fa_fwd_shaped): ``softcap`` caps them by softcap *
    tanh(x / softcap), ``alibi_slopes`` (float32 [H]) subtracts slope * |i - j|,
    ``key_begin`` / ``key_end`` (int32 [B, N], packed [T]) limit each query to
    keys [begin, end) of its sequence; ``key_ranges`` makes them. All elements
    of q, k and v must then be finite.
    """
    B, N, H, H_kv, D, max_sl, T = _shape(q, k, cu_seqlens, max_seqlen)
    if v.shape != k.shape or v.dtype != q.dtype or k.dtype != q.dtype:
        raise ValueError("k and v must match in shape and dtype with q's dtype")
    shape = _score_shape(q, cu_seqlens, softcap, alibi_slopes, key_begin, key_end)
    rows = (B, H, N) if cu_seqlens is None else (H, T)
    if shape is not None:
        _beside(q, k)
        _same("k", k, v=v)
        if out is not None:
            _same("q", q, out=out)
        _aux(lse, "lse", torch.float32, rows, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(rows, device=q.device, dtype=torch.float32)
    s = -1.0 if scale is None else float(scale)
    if shape is not None:
        _call("fa_fwd_shaped", _lib().fa_fwd_shaped, q.device, q.data_ptr(), k.data_ptr(),
              v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, H_kv, N, D, _DTYPES[q.dtype],
              int(bool(causal)), s, _ptr(cu_seqlens), max_sl, T, ctypes.byref(shape),
              _stream(q.device))
        return out, lse
    st = _lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, H_kv, N, D,
                           _DTYPES[q.dtype], int(bool(causal)), s, _ptr(cu_seqlens), max_sl, T,
                           _stream(q.device))
    _abi.check(st, "fa_fwd")
    return out, lse


BWD_FUSED = _abi.BWD_FUSED
BWD_SPLIT = _abi.BWD_SPLIT


def workspace_size(T: int, H: int, D: int, dtype: torch.dtype, phases: int = BWD_FUSED) -> int:
    """Bytes of backward workspace for ``phases`` (fa_bwd_phases_workspace_size)."""
    return int(_lib().fa_bwd_phases_workspace_size(int(phases), T, H, D, _DTYPES[dtype]))


def bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
        o: torch.Tensor, lse: torch.Tensor, *, causal: bool = False,
        scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
        max_seqlen: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
        dv: Optional[torch.Tensor] = None, phases: int = BWD_FUSED,
        softcap: Optional[float] = None, alibi_slopes: Optional[torch.Tensor] = None,
        key_begin: Optional[torch.Tensor] = None, key_end: Optional[torch.Tensor] = None):
    """Attention backward for the loss sum(O * dO). Returns (dQ, dK, dV).

    ``softcap``, ``alibi_slopes``, ``key_begin`` and ``key_end`` as in the
    ``fwd`` call that gave ``o`` and ``lse`` (fa_bwd_shaped; ``phases`` must
    then be ``BWD_FUSED``, and the slopes get no gradient).

    ``phases`` selects the kernels to enqueue (the FA_BWD_PHASE_* bits of
    include/fa.h): the default ``BWD_FUSED`` runs the preprocess, the fused
    kernel and the dQ conversion; ``BWD_SPLIT`` runs the preprocess, the
    dK / dV kernel and the dQ kernel (bitwise reproducible dQ, smaller
    workspace); single bits enqueue one kernel, to time it.
    """
    B, N, H, H_kv, D, max_sl, T = _shape(q, k, cu_seqlens, max_seqlen)
    for t in (dout, o, v, lse):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    shape = _score_shape(q, cu_seqlens, softcap, alibi_slopes, key_begin, key_end)
    if shape is not None:
        if phases != BWD_FUSED:
            raise ValueError("shaped scores have the BWD_FUSED backward only")
        _beside(q, k)
        _same("q", q, dout=dout, o=o, **({} if dq is None else {"dq": dq}))
        _same("k", k, v=v, **{n: x for n, x in (("dk", dk), ("dv", dv)) if x is not None})
        _aux(lse, "lse", torch.float32, (B, H, N) if cu_seqlens is None else (H, T), q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if shape is not None:
        dtype = _DTYPES[q.dtype]
        if workspace is None:
            workspace = torch.empty(_lib().fa_bwd_shaped_workspace_size(T, B, H, D, dtype),
                                    dtype=torch.uint8, device=q.device)
        _call("fa_bwd_shaped", _lib().fa_bwd_shaped, q.device, q.data_ptr(), k.data_ptr(),
              v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
              dk.data_ptr(), dv.data_ptr(), B, H, H_kv, N, D, dtype, int(bool(causal)),
              -1.0 if scale is None else float(scale), _ptr(cu_seqlens), max_sl, T,
              ctypes.byref(shape), workspace.data_ptr(), _room(workspace, q.device),
              _stream(q.device))
        return dq, dk, dv
    need = workspace_size(T, H, D, q.dtype, phases)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    s = -1.0 if scale is None else float(scale)
    st = _lib().fa_bwd_phases(int(phases), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                  _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, N, D,
                                  _DTYPES[q.dtype], int(bool(causal)), s, _ptr(cu_seqlens),
                                  max_sl, T, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream(q.device))
    _abi.check(st, "fa_bwd")
    return dq, dk, dv


def key_ranges(N: Optional[int] = None, *, B: int = 1, causal: bool = True,
               doc_ids: Optional[torch.Tensor] = None,
               prefix_lens: Optional[torch.Tensor] = None, window: Optional[int] = None,
               cu_seqlens: Optional[torch.Tensor] = None, max_seqlen: Optional[int] = None,
               device="cuda"):
    """Key ranges (begin, end) of every query token for ``fwd`` and ``bwd`` (fa_key_ranges).

    ``doc_ids`` (int32, one per token): queries see their own document, the run
    of equal ids around them. ``prefix_lens`` (int32 [B], with ``causal``): the
    first keys that every query of the sequence sees. ``window``: the last keys,
    the token itself counted. Dense: [B, N]; packed (``cu_seqlens``): [N], N the
    total number of tokens. The ranges hold the causal limit; pass
    ``causal=False`` with them to ``fwd`` when there are prefixes.
    """
    if N is None:
        if doc_ids is None:
            raise ValueError("key_ranges needs N or doc_ids")
        N = int(doc_ids.shape[-1])
        B = int(doc_ids.shape[0]) if doc_ids.dim() == 2 and cu_seqlens is None else B
    for t in (cu_seqlens, doc_ids, prefix_lens):
        if t is not None:
            device = t.device
            break
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("key_ranges runs on CUDA tensors")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if cu_seqlens is not None:
        if max_seqlen is None:
            raise ValueError("packed inputs need max_seqlen")
        B = cu_seqlens.numel() - 1
        _aux(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), device)
    tokens = (N,) if cu_seqlens is not None else (B, N)
    docs = _aux(doc_ids, "doc_ids", torch.int32, tokens, device)
    prefix = _aux(prefix_lens, "prefix_lens", torch.int32, (B,), device)
    begin, end = (torch.empty(tokens, dtype=torch.int32, device=device) for _ in range(2))
    _call("fa_key_ranges", _lib().fa_key_ranges, device, docs, prefix,
          0 if window is None else int(window), int(bool(causal)), B,
          0 if cu_seqlens is not None else N, _ptr(cu_seqlens), int(max_seqlen or 0), N,
          begin.data_ptr(), end.data_ptr(), _stream(device))
    return begin, end


def decode_num_splits(B: int, H_kv: int, max_seqlen_k: int, n_split: int = 0) -> int:
    return int(_lib().fa_decode_num_splits(B, H_kv, max_seqlen_k, n_split))


def decode_balanced(D: int, q_len: int, H: int, H_kv: int, n_split: int = 0) -> bool:
    """Whether fa_decode takes its balanced kernel for this shape: automatic
    splits, D = 128 and at most 64 query rows (q_len x H / H_kv) per kv head
    (include/fa.h, fa_decode)."""
    return n_split == 0 and D == 128 and H % H_kv == 0 and q_len * (H // H_kv) <= 64


def decode_workspace_size(B: int, q_len: int, H: int, H_kv: int, D: int, max_seqlen_k: int,
                          n_split: int = 0) -> int:
    return int(_lib().fa_decode_workspace_size(B, q_len, H, H_kv, D, max_seqlen_k, n_split))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           cache_seqlens: torch.Tensor, *, q_len: int, max_seqlen_k: int,
           block_table: Optional[torch.Tensor] = None, page_size: Optional[int] = None,
           causal: bool = True, scale: Optional[float] = None, n_split: int = 0,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, softcap: Optional[float] = None,
           alibi_slopes: Optional[torch.Tensor] = None, window: Optional[int] = None,
           key_positions: Optional[torch.Tensor] = None,
           key_weights: Optional[torch.Tensor] = None):
    """Split-KV decode (fa_decode): O [B*q_len, H, D] bf16 and LSE [B*q_len, H].

    ``q`` is [B*q_len, H, D]; the caches are [rows, H_kv, D]. Contiguous
    cache: ``page_size`` is the rows per sequence (default: rows // B).
    Paged cache: ``block_table`` [B, max_blocks] int32 and ``page_size``.

    Shaped scores (fa_decode_shaped; automatic splits, at most 64 query rows per
    kv head): ``softcap`` and ``alibi_slopes`` as in ``fwd``, ``window`` the last
    positions a query sees, ``key_positions`` (int32 [B, H_kv, slots]) the
    positions of a cache that has lost slots. ``key_weights`` (float32 [B, H_kv,
    slots]) is increased in place by the attention weight each slot receives;
    ``evict`` reads it.
    """
    B = cache_seqlens.numel()
    H, D = q.shape[1], q.shape[2]
    H_kv = k_cache.shape[1]
    rows = k_cache.shape[0]
    if block_table is None and page_size is None:
        page_size = rows // max(B, 1)
    max_blocks = block_table.shape[1] if block_table is not None else 0
    if not (softcap is None and alibi_slopes is None and window is None and
            key_positions is None and key_weights is None):
        return _decode_shaped(q, k_cache, v_cache, cache_seqlens, q_len, max_seqlen_k, block_table,
                              page_size, causal, scale, n_split, out, lse, workspace, softcap,
                              alibi_slopes, window, key_positions, key_weights)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((q.shape[0], H), device=q.device, dtype=torch.float32)
    need = decode_workspace_size(B, q_len, H, H_kv, D, max_seqlen_k, n_split)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    st = _lib().fa_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(cache_seqlens),
        _ptr(block_table), B, int(q_len), H, H_kv, D, int(page_size), int(max_blocks), rows,
        int(max_seqlen_k), int(causal), -1.0 if scale is None else float(scale), int(n_split),
        _ptr(workspace) if need else None, need, _stream(q.device))
    _abi.check(st, "fa_decode")
    return out, lse


def _check_cache(k_cache, v_cache, cache_seqlens, block_table):
    """Device, type and layout of a cache as decode and evict take it."""
    dev, shape = k_cache.device, k_cache.shape
    if len(shape) != 3 or dev.type != "cuda" or not _is(k_cache, shape, torch.bfloat16, dev):
        raise ValueError("a cache is a contiguous bfloat16 CUDA tensor [rows, H_kv, D]")
    if not _is(v_cache, shape, torch.bfloat16, dev):
        raise ValueError("v_cache must match k_cache in shape, dtype and device and be contiguous")
    B = cache_seqlens.numel()
    _aux(cache_seqlens, "cache_seqlens", torch.int32, (B,), dev)
    if block_table is not None:
        _aux(block_table, "block_table", torch.int32, (B, block_table.shape[-1]), dev)


@functools.lru_cache(maxsize=256)
def _decode_shaped_need(lib, device, B, q_len, H, H_kv, D, max_seqlen_k, weights) -> int:
    """fa_decode_shaped_workspace_size on the current device (``device`` keys the cache)."""
    return lib.fa_decode_shaped_workspace_size(B, q_len, H, H_kv, D, max_seqlen_k, weights)


def _decode_shaped(q, k_cache, v_cache, cache_seqlens, q_len, max_seqlen_k, block_table, page_size,
                   causal, scale, n_split, out, lse, workspace, softcap, alibi_slopes, window,
                   key_positions, key_weights):
    if n_split != 0:
        raise ValueError("shaped scores take automatic splits only (n_split = 0)")
    B, (tokens, H, D), dev = cache_seqlens.numel(), q.shape, q.device
    rows, H_kv, D_kv = k_cache.shape
    _check_cache(k_cache, v_cache, cache_seqlens, block_table)
    if k_cache.device != dev or D_kv != D or tokens != B * q_len or \
            not _is(q, q.shape, torch.bfloat16, dev):
        raise ValueError("q must be a contiguous bfloat16 tensor [B * q_len, H, D] beside the cache")
    if out is None:
        out = torch.empty_like(q)
    else:
        _same("q", q, out=out)
    if lse is None:
        lse = torch.empty((tokens, H), device=dev, dtype=torch.float32)
    else:
        _aux(lse, "lse", torch.float32, (tokens, H), dev)
    slots = (key_weights.shape[-1] if key_weights is not None else
             key_positions.shape[-1] if key_positions is not None else 0)
    side = (B, H_kv, slots)
    shape = _abi.DecodeShape(
        0.0 if softcap is None else float(softcap),
        _aux(alibi_slopes, "alibi_slopes", torch.float32, (H,), dev),
        0 if window is None else int(window),
        _aux(key_positions, "key_positions", torch.int32, side, dev),
        _aux(key_weights, "key_weights", torch.float32, side, dev), slots)
    lib = _lib()
    span = max_seqlen_k if not window or window < 0 else min(max_seqlen_k, int(window) + q_len + 127)
    if dev.index == torch.cuda.current_device():
        need = _decode_shaped_need(lib, dev.index, B, q_len, H, H_kv, D, span,
                                   int(key_weights is not None))
    else:
        with torch.cuda.device(dev):
            need = _decode_shaped_need(lib, dev.index, B, q_len, H, H_kv, D, span,
                                       int(key_weights is not None))
    if need and (workspace is None or _room(workspace, dev) < need):
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    _call("fa_decode_shaped", lib.fa_decode_shaped, dev, q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(), cache_seqlens.data_ptr(),
          _ptr(block_table), B, int(q_len), H, H_kv, D, int(page_size),
          0 if block_table is None else block_table.shape[1], rows, int(max_seqlen_k),
          int(bool(causal)), -1.0 if scale is None else float(scale), ctypes.byref(shape),
          workspace.data_ptr() if need else None, need, _stream(dev))
    return out, lse


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, cache_seqlens: torch.Tensor,
          key_weights: torch.Tensor, *, keep: int, max_seqlen_k: int, recent: int = 0,
          block_table: Optional[torch.Tensor] = None, page_size: Optional[int] = None,
          key_positions: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
          v_out: Optional[torch.Tensor] = None, out_block_table: Optional[torch.Tensor] = None,
          out_page_size: Optional[int] = None, out_slots: Optional[int] = None,
          workspace: Optional[torch.Tensor] = None):
    """Copy the slots worth keeping of a cache into another one (fa_cache_evict).

    Each (sequence, kv head) keeps its last ``recent`` slots and the others with
    the largest ``key_weights`` (float32 [B, H_kv, slots], as ``decode`` adds
    them up), ``keep`` in all, in their order. Returns (k_out, v_out,
    seqlens int32 [B], weights float32 and positions int32 [B, H_kv,
    out_slots]); weights are 0 and positions -1 from the new length on, ready
    for new tokens. ``key_positions`` are those of a cache that has lost slots
    before. The caches are laid out as for ``decode``; without ``k_out`` and
    ``v_out`` a contiguous pair of ``out_page_size`` (default ``out_slots``)
    rows a sequence is allocated, zeroed. ``out_slots`` defaults to ``keep``.
    """
    _check_cache(k_cache, v_cache, cache_seqlens, block_table)
    dev = k_cache.device
    B, (rows, H_kv, D) = cache_seqlens.numel(), k_cache.shape
    if block_table is None and page_size is None:
        page_size = rows // max(B, 1)
    if block_table is not None and page_size is None:
        raise ValueError("a paged cache needs page_size")
    out_slots = int(keep) if out_slots is None else int(out_slots)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        if out_block_table is not None:
            raise ValueError("out_block_table needs k_out and v_out")
        out_page_size = out_slots if out_page_size is None else int(out_page_size)
        k_out, v_out = (torch.zeros((B * out_page_size, H_kv, D), dtype=k_cache.dtype, device=dev)
                        for _ in range(2))
    elif out_page_size is None:
        if out_block_table is not None:
            raise ValueError("a paged cache needs out_page_size")
        out_page_size = k_out.shape[0] // max(B, 1)
    if k_out.device != dev or k_out.shape[1:] != k_cache.shape[1:]:
        raise ValueError("k_out must have the cache's heads, head size and device")
    _check_cache(k_out, v_out, cache_seqlens, out_block_table)
    slots = key_weights.shape[-1]
    w = _aux(key_weights, "key_weights", torch.float32, (B, H_kv, slots), dev)
    pos = _aux(key_positions, "key_positions", torch.int32, (B, H_kv, slots), dev)
    seqlens = torch.empty((B,), dtype=torch.int32, device=dev)
    weights = torch.empty((B, H_kv, out_slots), dtype=torch.float32, device=dev)
    positions = torch.empty((B, H_kv, out_slots), dtype=torch.int32, device=dev)
    lib = _lib()
    need = lib.fa_cache_evict_workspace_size(B, H_kv, int(keep))
    if workspace is None or _room(workspace, dev) < need:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    _call("fa_cache_evict", lib.fa_cache_evict, dev, k_cache.data_ptr(), v_cache.data_ptr(),
          cache_seqlens.data_ptr(), _ptr(block_table), B, H_kv, D, int(page_size),
          0 if block_table is None else block_table.shape[1], rows, int(max_seqlen_k), w, pos,
          slots, int(keep), int(recent), k_out.data_ptr(), v_out.data_ptr(),
          _ptr(out_block_table), int(out_page_size),
          0 if out_block_table is None else out_block_table.shape[1], k_out.shape[0],
          seqlens.data_ptr(), weights.data_ptr(), positions.data_ptr(), out_slots,
          workspace.data_ptr(), need, _stream(dev))
    return k_out, v_out, seqlens, weights, positions


def fp8_quantize(x: torch.Tensor, B: int, N: int, *, out: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None):
    """Pass 1 of the FP8 forward: E4M3 codes (uint8, x's shape) and per-block
    steps fp32 [B, Hx, ceil(N / 128)] of a bf16 [B*N, Hx, D] (or [B, N, Hx, D]) tensor."""
    Hx, D = x.shape[-2], x.shape[-1]
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if out is None else out
    sc = torch.empty((B, Hx, (N + 127) // 128), dtype=torch.float32, device=x.device) \
        if scale is None else scale
    st = _lib().fa_fp8_quantize(_ptr(x), _ptr(x8), _ptr(sc), B, N, Hx, D, _stream(x.device))
    _abi.check(st, "fa_fp8_quantize")
    return x8, sc


def fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
            k_scale: torch.Tensor, *, B: int, N: int, causal: bool = False,
            scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None):
    """Pass 2 of the FP8 forward (fa_fwd_fp8). Returns (O bf16, LSE [B, H, N])."""
    H, D = q8.shape[-2], q8.shape[-1]
    H_kv = k8.shape[-2]
    if out is None:
        out = torch.empty(q8.shape, dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    st = _lib().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v), _ptr(q_scale), _ptr(k_scale),
                               _ptr(out), _ptr(lse), B, H, H_kv, N, D, int(bool(causal)),
                               -1.0 if scale is None else float(scale), _stream(q8.device))
    _abi.check(st, "fa_fwd_fp8")
    return out, lse


def check_device_error(device: Optional[torch.device] = None) -> tuple:
    """Synchronise the current stream; return (status, where) and clear the flag."""
    dev = torch.device("cuda") if device is None else device
    where = ctypes.c_uint(0)
    st = _lib().fa_check_device_error(_stream(dev), ctypes.byref(where))
    return st, where.value


def selftest_wait_timeout(cycles: int, device: Optional[torch.device] = None) -> None:
    dev = torch.device("cuda") if device is None else device
    _abi.check(_lib().fa_selftest_wait_timeout(int(cycles), _stream(dev)),
               "fa_selftest_wait_timeout")


def selftest_exp2(x: torch.Tensor) -> torch.Tensor:
    """2^x by the kernels' FMA-pipe exponential (fa_selftest_exp2), for a
    contiguous fp32 CUDA tensor."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("selftest_exp2 takes a contiguous float32 CUDA tensor")
    y = torch.empty_like(x)
    _abi.check(_lib().fa_selftest_exp2(_ptr(x), _ptr(y), x.numel(), _stream(x.device)),
               "fa_selftest_exp2")
    return y


def set_wait_budget(cycles: int) -> None:
    _lib().fa_set_wait_budget(int(cycles))


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)
