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
import os
import warnings

import torch

from . import NSA_F16, NsaError, _check, _ws_cache, get_workspace, load_library

__all__ = ["nsa_sel_paged_plan", "nsa_sel_paged_write_kv", "nsa_sel_paged_attn_workspace_size",
           "nsa_sel_paged_attn_fwd", "nsa_sel_paged_sel_fwd"]

# A decode step makes these calls once per layer on kernels of a few microseconds, so the
# host path is kept short: the plain case is marshalled by a small compiled module
# (csrc/paged_bind.cpp); anything it does not take comes back and is looked at here, where
# what is wrong gets its name.  The stream and device queries are those that torch's own
# generated code uses (a torch without CUDA lacks them, and has no tensors that get this far).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_ELEM = {torch.bfloat16: 0, torch.float16: NSA_F16}

_bind = None   # the compiled module; False where it was not built


def _plain(t):
    """The compiled module, for a call whose first tensor is t."""
    global _bind
    if _bind is None:
        from .build import LIB_BIND, bind_target
        try:
            from . import _paged_bind
            if _paged_bind.built_for != bind_target():
                raise ImportError(f"it was built for {_paged_bind.built_for}, this is {bind_target()}")
        except ImportError as e:
            if os.path.exists(LIB_BIND):       # there, but not for this process
                warnings.warn(f"_paged_bind.so is not used, the paged calls are marshalled in Python: {e}")
            _bind = False
            return _bind
        lib = load_library()
        _paged_bind.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.nsa_sel_paged_plan, lib.nsa_sel_paged_write_kv, lib.nsa_sel_paged_attn_fwd,
            lib.nsa_sel_paged_sel_fwd)))
        _bind = _paged_bind
    return _bind and isinstance(t, torch.Tensor) and t.is_cuda and _bind


class _Cache(ctypes.Structure):   # nsa_paged_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("hkv", ctypes.c_int),
                ("head_dim", ctypes.c_int)]


def _call(fn: str, index: int, *args):
    """Calls the library with the tensors' device current."""
    f = getattr(load_library(), fn)
    if index == _current_device():
        code = f(*args)
    else:
        with torch.cuda.device(index):
            code = f(*args)
    if code:
        _check(fn, code)


def _refuse(t, name, dtype, ndim, index):
    """Raises for a tensor that failed its test; returns where the test was too strict."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _packed(t, name, dtype, ndim, index):
    """A contiguous CUDA tensor's pointer."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == ndim
            and t.is_contiguous()):
        _refuse(t, name, dtype, ndim, index)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _strided(t, name, dtype, ndim, index):
    """The strides of a CUDA tensor whose last dimension is adjacent; the others are free."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == ndim):
        _refuse(t, name, dtype, ndim, index)
    strides = t.stride()
    if strides[-1] != 1:
        if not t.numel():       # nothing is read through an empty tensor's strides
            return (0,) * ndim
        if t.shape[-1] > 1:
            raise ValueError(f"{name} must have adjacent columns (stride 1 in its last dimension)")
    return strides


def _cache_arg(k_cache, v_cache, et, index):
    strides = _strided(k_cache, "k_cache", et, 4, index)
    other = _strided(v_cache, "v_cache", et, 4, index)
    shape = k_cache.shape
    if shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if any(a != b and n > 1 for a, b, n in zip(strides, other, shape)):
        raise ValueError("k_cache and v_cache must have the same strides")
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), *strides[:3], *shape), shape


def _elem(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    et = t.dtype
    if et not in _ELEM:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {et}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return et, _ELEM[et], t.get_device()


def _table_arg(block_table, R, index):
    """(pointer, width, row stride) of a block table of R rows."""
    strides = _strided(block_table, "block_table", torch.int32, 2, index)
    rows, width = block_table.shape
    if rows != R:
        raise ValueError("block_table needs one row per request")
    return block_table.data_ptr(), width, max(strides[0], width) if R == 1 else strides[0]


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
    bind = _plain(new_lens)
    if bind:
        device = _current_device()
        got = bind.plan(new_lens, cached_lens, free_pages, block_table, page_size, total_tokens, device,
                        _raw_stream(device))
        if got.__class__ is tuple:
            return got
        if got is not None:
            raise NsaError("nsa_sel_paged_plan", got)
    if not isinstance(new_lens, torch.Tensor) or not new_lens.is_cuda:
        raise ValueError("new_lens must be a CUDA tensor")
    index, int32 = new_lens.get_device(), torch.int32
    new = _packed(new_lens, "new_lens", int32, 1, index)
    cached = _packed(cached_lens, "cached_lens", int32, 1, index)
    free = _packed(free_pages, "free_pages", int32, 1, index)
    R, T = new_lens.shape[0], int(total_tokens)
    if cached_lens.shape[0] != R:
        raise ValueError("new_lens and cached_lens must have the same length")
    table = _table_arg(block_table, R, index)
    if T < 0:
        raise ValueError("total_tokens must not be negative")
    cu, kv_lens, used = new_lens.new_empty(R + 1), new_lens.new_empty(R), new_lens.new_empty(1)
    slots, positions = new_lens.new_empty(T, dtype=torch.int64), new_lens.new_empty(T)
    _call("nsa_sel_paged_plan", index, new, cached, R, free, free_pages.shape[0], *table, int(page_size), T,
          cu.data_ptr(), kv_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(), used.data_ptr(),
          _raw_stream(index))
    return cu, kv_lens, slots, positions, used


def nsa_sel_paged_write_kv(k, v, slots, k_cache, v_cache):
    """Writes k, v [T, hkv, d] into their cache slots (int64 [T]; negative: not written).

    k and v may be slices of a wider tensor (a fused QKV projection) whose strides are
    multiples of 8 elements."""
    bind = _plain(k)
    if bind:
        device = _current_device()
        code = bind.write(k, v, slots, k_cache, v_cache, device, _raw_stream(device))
        if code == 0:
            return
        if code is not None:
            raise NsaError("nsa_sel_paged_write_kv", code)
    et, _, index = _elem(k, "k")
    ks = _strided(k, "k", et, 3, index)
    vs = _strided(v, "v", et, 3, index)
    at = _packed(slots, "slots", torch.int64, 1, index)
    cache, cshape = _cache_arg(k_cache, v_cache, et, index)
    T, hkv, d = shape = k.shape
    if v.shape != shape or T != slots.shape[0] or hkv != cshape[2] or d != cshape[3]:
        raise ValueError("inconsistent shapes")
    _call("nsa_sel_paged_write_kv", index, k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], at, T,
          ctypes.byref(cache), _raw_stream(index))


def nsa_sel_paged_attn_workspace_size(total_tokens, num_seqs, hq, hkv, head_dim) -> int:
    n = load_library().nsa_sel_paged_attn_workspace_size(total_tokens, num_seqs, hq, hkv, head_dim)
    if n == 0:
        raise NsaError("nsa_sel_paged_attn_workspace_size", 2)
    return int(n)


_workspace_bytes: dict = {}   # head_dim -> bytes: the size depends on nothing else


def _paged_workspace(T, R, hq, hkv, d, q):
    nbytes = _workspace_bytes.get(d)
    if nbytes is None:
        nbytes = _workspace_bytes[d] = nsa_sel_paged_attn_workspace_size(T, R, hq, hkv, d)
    return get_workspace(nbytes, q.device)


def _attend_plain(fn, q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx, block_size, scale,
                  window_size, out, lse, with_lse, workspace):
    """(out, lse) by the compiled module, or None."""
    bind = _plain(q)
    if not bind:
        return None
    device = _current_device()
    stream = _raw_stream(device)
    ws = workspace
    if ws is None:
        # (being captured: not from the cache, see get_workspace)
        ws = None if _capturing() else _ws_cache.get((q.device, stream))
        if ws is None:
            return None
    got = bind.attend(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx, block_size, scale,
                      window_size, out, lse, with_lse, ws, device, stream)
    if got is None or got.__class__ is tuple:
        return got
    if got == 3 and workspace is None:      # the cached workspace is another call's, and smaller
        return None
    raise NsaError(fn, got)


def _attend(fn, q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, selection, scale, window_size,
            out, lse, with_lse, workspace):
    # selection: () or (block_idx, block_size)
    et, flag, index = _elem(q, "q")
    qs = _strided(q, "q", et, 3, index)
    cache, cshape = _cache_arg(k_cache, v_cache, et, index)
    cu = _packed(cu_seqlens, "cu_seqlens", torch.int32, 1, index)
    kv = _packed(kv_lens, "kv_lens", torch.int32, 1, index)
    T, hq, d = shape = q.shape
    R = kv_lens.shape[0]
    table = _table_arg(block_table, R, index)
    if d != cshape[3] or cu_seqlens.shape[0] != R + 1:
        raise ValueError("inconsistent shapes")
    if selection:
        block_idx, block_size = selection
        idx = _packed(block_idx, "block_idx", torch.int32, 3, index)
        if block_idx.shape[:2] != (T, cshape[2]):
            raise ValueError("inconsistent shapes")
        selection = idx, block_idx.shape[2], int(block_size)
    if out is None:
        out = q.new_empty(shape)
        to = out.data_ptr()
    else:
        to = _packed(out, "out", et, 3, index)
        if out.shape != shape:
            raise ValueError("out must have the shape of q")
    lse_to = None
    if lse is not None:
        lse_to = _packed(lse, "lse", torch.float32, 2, index)
        if lse.shape != (hq, T):
            raise ValueError("lse must be [hq, T]")
    elif with_lse:
        lse = q.new_empty((hq, T), dtype=torch.float32)
        lse_to = lse.data_ptr()
    stream = _raw_stream(index)
    if workspace is not None:
        ws = workspace
        _packed(ws, "workspace", torch.uint8, 1, index)
    else:
        ws = _paged_workspace(T, R, hq, cshape[2], d, q)
    _call(fn, index, q.data_ptr(), qs[0], qs[1], T, hq, ctypes.byref(cache), cu, kv, R, *table, *selection,
          d ** -0.5 if scale is None else float(scale), int(window_size), to, lse_to, ws.data_ptr(), ws.numel(),
          stream, flag)
    return out, lse


def nsa_sel_paged_attn_fwd(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, scale=None,
                           window_size=0, out=None, lse=None, with_lse=True, workspace=None):
    """Causal attention of each request's new tokens over its paged cache; returns
    (out [T, hq, d], lse fp32 [hq, T]).

    q [T, hq, d] (bf16 or fp16; may be a slice of a wider tensor) holds the new tokens,
    request r's at rows cu_seqlens[r] .. cu_seqlens[r + 1]; their K/V are in the cache
    already, as the last of its kv_lens[r] tokens.  window_size > 0: each query sees the
    last window_size keys up to its own.  Rows of q behind cu_seqlens[-1] are padding:
    their outputs are not written.  with_lse=False: None is returned in its place.

    The call may be captured into a CUDA graph; it then takes its workspace from the graph's
    memory (pass `workspace` to read the status of a replay with nsa_sel_check_status)."""
    got = _attend_plain("nsa_sel_paged_attn_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, None, 0,
                        scale, window_size, out, lse, with_lse, workspace)
    if got is not None:
        return got
    return _attend("nsa_sel_paged_attn_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, (),
                   scale, window_size, out, lse, with_lse, workspace)


def nsa_sel_paged_sel_fwd(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx, block_size,
                          scale=None, window_size=0, out=None, lse=None, with_lse=True,
                          workspace=None):
    """Selected-block attention over the paged cache: as nsa_sel_paged_attn_fwd, over the
    keys of the blocks block_idx[t, g, :] (int32 [T, hkv, topk], block numbers local to the
    request's sequence, distinct within a row, -1 pads)."""
    got = _attend_plain("nsa_sel_paged_sel_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx,
                        block_size, scale, window_size, out, lse, with_lse, workspace) if block_idx is not None else None
    if got is not None:
        return got
    return _attend("nsa_sel_paged_sel_fwd", q, k_cache, v_cache, cu_seqlens, kv_lens, block_table,
                   (block_idx, block_size), scale, window_size, out, lse, with_lse, workspace)
