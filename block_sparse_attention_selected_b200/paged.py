"""Paged K/V cache: block tables and slot maps, the write of new rows, attention of new
tokens over the cache (all visible keys, or selected blocks).

The binding of the ``nsa_sel_paged_*`` calls of ``include/nsa_sel.h``; marshalling only.
One step of a server::

    cu, kv_lens, slots, positions, used = nsa_sel_paged_plan(
        new_lens, cached_lens, free_pages, block_table, page_size, total_tokens)
    for each layer:
        nsa_sel_paged_write_kv(k, v, slots, k_cache, v_cache)
        out, lse = nsa_sel_paged_attn_fwd(q, k_cache, v_cache, cu, kv_lens, block_table)
        # or, over selected blocks
        out, lse = nsa_sel_paged_sel_fwd(q, k_cache, v_cache, cu, kv_lens, block_table,
                                         block_idx, block_size)

Caches are [num_pages, page_size, hkv, d]; any strides whose columns are adjacent (heads
before tokens, K and V as two halves of one tensor) are taken as they are.
"""
from __future__ import annotations

import ctypes

import torch

from . import NSA_F16, NsaError, _check, _need, _ws_cache, get_workspace, load_library

__all__ = ["nsa_sel_paged_plan", "nsa_sel_paged_write_kv", "nsa_sel_paged_attn_workspace_size",
           "nsa_sel_paged_attn_fwd", "nsa_sel_paged_sel_fwd"]

# A decode step makes these calls once per layer on kernels of a few microseconds, so the
# host path is kept short: plain comparisons, and the stream and device queries that
# torch's own generated code uses.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_ELEM = {torch.bfloat16: 0, torch.float16: NSA_F16}


class _Cache(ctypes.Structure):   # nsa_paged_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("hkv", ctypes.c_int),
                ("head_dim", ctypes.c_int)]


def _call(fn: str, dev: torch.device, *args):
    """Calls the library with the tensors' device current."""
    f = getattr(load_library(), fn)
    if dev.index == _current_device():
        code = f(*args)
    else:
        with torch.cuda.device(dev):
            code = f(*args)
    if code:
        _check(fn, code)


def _need_strided(t, name, dtype, ndim, dev):
    """A CUDA tensor whose last dimension is adjacent; other strides are free."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"{name} must have adjacent columns (stride 1 in its last dimension)")


def _strides(t):
    # an empty tensor may have any strides; nothing is read through them
    return t.stride()[:2] if t.numel() else (0, 0)


def _cache_arg(k_cache, v_cache, et, dev):
    _need_strided(k_cache, "k_cache", et, 4, dev)
    _need_strided(v_cache, "v_cache", et, 4, dev)
    shape, strides = k_cache.shape, k_cache.stride()
    if shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if strides != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same strides")
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), *strides[:3], *shape)


def _elem(t, name):
    et = t.dtype
    if et not in _ELEM:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {et}")
    return et, _ELEM[et]


def _table_arg(block_table, R, dev):
    """(pointer, width, row stride) of a block table of R rows."""
    _need_strided(block_table, "block_table", torch.int32, 2, dev)
    rows, width = block_table.shape
    if rows != R:
        raise ValueError("block_table needs one row per request")
    return block_table.data_ptr(), width, max(block_table.stride(0), width) if R == 1 else block_table.stride(0)


def nsa_sel_paged_plan(new_lens, cached_lens, free_pages, block_table, page_size, total_tokens):
    """Block tables, slot maps and cumulative lengths of one step; returns
    (cu_seqlens int32 [R + 1], kv_lens int32 [R], slots int64 [total_tokens],
    positions int32 [total_tokens], pages_used int32 [1]).

    new_lens, cached_lens: int32 [R], tokens that each request brings and already holds.
    free_pages: int32 page numbers, taken from the front, requests in order.
    block_table: int32 [R, width], updated in place (the entries of fresh pages only).
    total_tokens: host int, at least the sum of new_lens; rows behind it get slot -1.
    pages_used[0] is what the step needs of free_pages; missing pages are -1 in the table,
    and slots on them -1."""
    dev = new_lens.device
    _need(new_lens, "new_lens", torch.int32, 1, dev)
    _need(cached_lens, "cached_lens", torch.int32, 1, dev)
    _need(free_pages, "free_pages", torch.int32, 1, dev)
    R, T = new_lens.shape[0], int(total_tokens)
    if cached_lens.shape[0] != R:
        raise ValueError("new_lens and cached_lens must have the same length")
    table = _table_arg(block_table, R, dev)
    if T < 0:
        raise ValueError("total_tokens must not be negative")
    cu, kv_lens, used = new_lens.new_empty(R + 1), new_lens.new_empty(R), new_lens.new_empty(1)
    slots, positions = new_lens.new_empty(T, dtype=torch.int64), new_lens.new_empty(T)
    _call("nsa_sel_paged_plan", dev, new_lens.data_ptr(), cached_lens.data_ptr(), R,
          free_pages.data_ptr(), free_pages.shape[0], *table, int(page_size), T, cu.data_ptr(),
          kv_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(), used.data_ptr(),
          _raw_stream(dev.index))
    return cu, kv_lens, slots, positions, used


def nsa_sel_paged_write_kv(k, v, slots, k_cache, v_cache):
    """Writes k, v [T, hkv, d] into their cache slots (int64 [T]; negative: not written).

    k and v may be slices of a wider tensor (a fused QKV projection) whose strides are
    multiples of 8 elements."""
    dev = k.device
    et, _ = _elem(k, "k")
    _need_strided(k, "k", et, 3, dev)
    _need_strided(v, "v", et, 3, dev)
    _need(slots, "slots", torch.int64, 1, dev)
    cache = _cache_arg(k_cache, v_cache, et, dev)
    shape = k.shape
    if v.shape != shape or shape[0] != slots.shape[0] or shape[1] != cache.hkv or shape[2] != cache.head_dim:
        raise ValueError("inconsistent shapes")
    _call("nsa_sel_paged_write_kv", dev, k.data_ptr(), v.data_ptr(), *_strides(k), *_strides(v),
          slots.data_ptr(), shape[0], ctypes.byref(cache), _raw_stream(dev.index))


def nsa_sel_paged_attn_workspace_size(total_tokens, num_seqs, hq, hkv, head_dim) -> int:
    n = load_library().nsa_sel_paged_attn_workspace_size(total_tokens, num_seqs, hq, hkv, head_dim)
    if n == 0:
        raise NsaError("nsa_sel_paged_attn_workspace_size", 2)
    return int(n)


_workspace_bytes: dict = {}   # head_dim -> bytes: the size depends on nothing else


def _paged_workspace(T, R, hq, hkv, d, dev, stream):
    nbytes = _workspace_bytes.get(d)
    if nbytes is None:
        nbytes = _workspace_bytes[d] = nsa_sel_paged_attn_workspace_size(T, R, hq, hkv, d)
    # A call that is being captured takes its workspace from the graph's own memory: the
    # cached one would be shared with other graphs and with eager calls, which may overlap
    # with a replay.
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws = _ws_cache.get((dev, stream))
    return ws if ws is not None and ws.numel() >= nbytes else get_workspace(nbytes, dev)


def _attend(fn, q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, selection, scale, window_size,
            out, lse, with_lse, workspace):
    dev = q.device
    et, flag = _elem(q, "q")
    _need_strided(q, "q", et, 3, dev)
    cache = _cache_arg(k_cache, v_cache, et, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1, dev)
    _need(kv_lens, "kv_lens", torch.int32, 1, dev)
    T, hq, d = shape = q.shape
    R = kv_lens.shape[0]
    table = _table_arg(block_table, R, dev)
    if d != cache.head_dim or cu_seqlens.shape[0] != R + 1:
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _need(out, "out", et, 3, dev)
        if out.shape != shape:
            raise ValueError("out must have the shape of q")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (hq, T):
            raise ValueError("lse must be [hq, T]")
    elif with_lse:
        lse = q.new_empty((hq, T), dtype=torch.float32)
    stream = _raw_stream(dev.index)
    ws = workspace
    if ws is None:
        ws = _paged_workspace(T, R, hq, cache.hkv, d, dev, stream)
    _call(fn, dev, q.data_ptr(), *_strides(q), T, hq, ctypes.byref(cache), cu_seqlens.data_ptr(),
          kv_lens.data_ptr(), R, *table, *selection, float(d ** -0.5 if scale is None else scale),
          int(window_size), out.data_ptr(), lse.data_ptr() if lse is not None else None, ws.data_ptr(),
          ws.numel(), stream, flag)
    return out, lse


def nsa_sel_paged_attn_fwd(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, scale=None,
                           window_size=0, out=None, lse=None, with_lse=True, workspace=None):
    """Causal attention of each request's new tokens over its paged cache; returns
    (out [T, hq, d], lse fp32 [hq, T]).

    q [T, hq, d] (bf16 or fp16; may be a slice of a wider tensor) holds the new tokens,
    request r's at rows cu_seqlens[r] .. cu_seqlens[r + 1]; their K/V are in the cache
    already, as the last of its kv_lens[r] tokens.  window_size > 0: each query sees the
    last window_size keys up to its own.  Rows of q behind cu_seqlens[-1] are padding:
    their outputs are not written.  with_lse=False: None is returned in its place."""
    return _attend("nsa_sel_paged_attn_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, (),
                   scale, window_size, out, lse, with_lse, workspace)


def nsa_sel_paged_sel_fwd(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx, block_size,
                          scale=None, window_size=0, out=None, lse=None, with_lse=True,
                          workspace=None):
    """Selected-block attention over the paged cache: as nsa_sel_paged_attn_fwd, over the
    keys of the blocks block_idx[t, g, :] (int32 [T, hkv, topk], block numbers local to the
    request's sequence, distinct within a row, -1 pads)."""
    _need(block_idx, "block_idx", torch.int32, 3, q.device)
    if block_idx.shape[0] != q.shape[0] or block_idx.shape[1] != k_cache.shape[2]:
        raise ValueError("inconsistent shapes")
    return _attend("nsa_sel_paged_sel_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table,
                   (block_idx.data_ptr(), block_idx.shape[2], int(block_size)), scale, window_size,
                   out, lse, with_lse, workspace)
