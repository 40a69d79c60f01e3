"""The paged key/value cache of a decoding step that drafts trees: its pages
and rows, as C calls of ``include/sv_tree.h``.

A cache is two tensors ``k_cache``, ``v_cache`` ``[layers, pages, page_size,
heads, head_dim]`` (any strides with a contiguous last dimension, the same for
both) and three int32 tensors: ``page_table [slots, max_pages]`` (a slot's
pages in its leading entries, -1 behind them), ``lens [slots]`` and
``refcount [pages]`` (0 = free).  Everything stays on the GPU: no call here
synchronises, so a whole step can be captured into a CUDA graph.

    status = cache_resize(page_table, lens + nodes, refcount, page_size)   # room for a tree
    ...                                                                    # tree_attention, tree_verify
    lens = cache_commit(k_cache, v_cache, page_table, lens, path)          # keep the accepted rows
    cache_resize(page_table, lens, refcount, page_size)                    # give the rest back
"""
from __future__ import annotations

import ctypes

from . import BF16, F32, _check, _torch, library

__all__ = ["cache_resize", "cache_commit", "cache_fork", "F16", "MAX_SLOTS"]

F16 = 2             # SV_F16: caches only
MAX_SLOTS = 8192    # SV_MAX_SLOTS of the C header

_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _Cache(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("layers", _I32), ("pages", _I32), ("page_size", _I32), ("heads", _I32),
                ("head_dim", _I32), ("dtype", _I32), ("layer_stride", _I64), ("page_stride", _I64),
                ("row_stride", _I64), ("head_stride", _I64)]


_SIGNATURES = {
    "sv_cache_commit": (_I32, [ctypes.POINTER(_Cache), _VP, _I64, _I32, _I32, _VP, _VP, _I64, _I32, _VP, _VP]),
    "sv_cache_resize": (_I32, [_VP, _I64, _I32, _I32, _VP, _I32, _VP, _I32, _VP, _VP]),
    "sv_cache_fork": (_I32, [ctypes.POINTER(_Cache), _VP, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _VP]),
}
_LIB = None


def _library():
    global _LIB
    if _LIB is None:
        lib = library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _LIB = lib
    return _LIB


def _kv_code(t) -> int:
    torch = _torch()
    code = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}.get(t.dtype)
    if code is None:
        raise TypeError(f"the cache must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _ints(what, t, shape, device, rows=False):
    """Pointer of an int32 tensor of exactly this shape (contiguous, or with
    ``rows`` any stride between contiguous rows); None passes through."""
    if t is None:
        return None
    if t.dtype != _torch().int32:
        raise TypeError(f"{what} must be torch.int32, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{what} is on {t.device}, expected the CUDA device of the call ({device})")
    if rows:
        if t.numel() and (t.stride(1) != 1 and t.shape[1] > 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1):
            raise ValueError(f"{what} must have contiguous rows that do not overlap")
    elif not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _cache(k, v) -> _Cache:
    """The C description of a cache; 4-d tensors are one layer."""
    if k.dim() not in (4, 5) or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
        raise ValueError("k_cache and v_cache must be [layers, pages, page_size, heads, head_dim] tensors of one "
                         "shape, dtype and device")
    if k.stride() != v.stride() or (k.stride(-1) != 1 and k.shape[-1] > 1):
        raise ValueError("k_cache and v_cache must have the same strides and a contiguous last dimension")
    if not k.is_cuda:
        raise ValueError("k_cache and v_cache must be CUDA tensors")
    shape = k.shape if k.dim() == 5 else (1, *k.shape)
    st = k.stride() if k.dim() == 5 else (0, *k.stride())
    return _Cache(k.data_ptr(), v.data_ptr(), *shape, _kv_code(k), *(s if n > 1 else 0 for s, n in zip(st[:4], shape)))


class _on:
    """Makes the tensors' device current for a call and gives its stream."""

    def __init__(self, device, stream):
        torch = _torch()
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        self.device, self.stream = device, stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        s = _torch().cuda.current_stream(self.device) if self.stream is None else self.stream
        return s.cuda_stream

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _table(page_table):
    if page_table.dim() != 2 or page_table.shape[1] < 1:
        raise ValueError("page_table must be [slots, max_pages]")
    return page_table.shape


def cache_resize(page_table, lens, refcount, page_size, *, status=None, stream=None):
    """Every slot comes to hold ``ceil(lens / page_size)`` pages: surplus pages
    are given back first (``lens`` 0 frees a slot), then missing ones are taken,
    free pages in increasing order of their id, slots in order.  Updates
    ``page_table`` and ``refcount`` in place; returns int32 ``status [slots]``:
    0, or -1 where the slot was left unchanged (its length or entries are not
    valid, or the free pages did not reach it)."""
    slots, max_pages = _table(page_table)
    dev = page_table.device
    lib = _library()
    if status is None:
        status = _torch().empty(slots, dtype=_torch().int32, device=dev)
    if refcount.dim() != 1:
        raise ValueError("refcount must be [pages]")
    args = (_ints("page_table", page_table, (slots, max_pages), dev, rows=True), _row_stride(page_table), slots,
            max_pages, _ints("lens", lens, (slots,), dev), int(page_size),
            _ints("refcount", refcount, refcount.shape, dev), refcount.shape[0],
            _ints("status", status, (slots,), dev))
    with _on(dev, stream) as st:
        _check(lib.sv_cache_resize(*args, st), "sv_cache_resize")
    return status


def cache_commit(k_cache, v_cache, page_table, lens, path, *, out_lens=None, stream=None):
    """Compaction after verification, in all layers: with n the number of
    leading entries >= 0 of ``path[b]`` (``tree_verify`` returns it), cache row
    ``lens[b] + path[b][i]`` moves to row ``lens[b] + i`` for i < n.  Returns
    the new lengths ``lens + n`` (int32, -1 for a request that is not valid and
    was left alone); ``out_lens`` must be another tensor than ``lens``."""
    B, max_pages = _table(page_table)
    dev = page_table.device
    lib = _library()
    c = _cache(k_cache, v_cache)
    if out_lens is None:
        out_lens = _torch().empty(B, dtype=_torch().int32, device=dev)
    if path.dim() != 2:
        raise ValueError("path must be [B, width]")
    if k_cache.device != dev:
        raise ValueError(f"the cache is on {k_cache.device}, page_table on {dev}")
    args = (ctypes.byref(c), _ints("page_table", page_table, (B, max_pages), dev, rows=True), _row_stride(page_table),
            B, max_pages, _ints("lens", lens, (B,), dev), _ints("path", path, (B, path.shape[1]), dev, rows=True),
            _row_stride(path), path.shape[1], _ints("out_lens", out_lens, (B,), dev))
    with _on(dev, stream) as st:
        _check(lib.sv_cache_commit(*args, st), "sv_cache_commit")
    return out_lens


def cache_fork(k_cache, v_cache, page_table, lens, refcount, src, dst, *, status=None, stream=None):
    """Fork i makes slot ``dst[i]`` a copy of slot ``src[i]``: full pages are
    shared, the ragged last one is copied in all layers to a free page, what
    ``dst`` held is given back.  Updates ``page_table``, ``lens`` and
    ``refcount`` in place; returns int32 ``status [forks]``: 0, -1 (not valid,
    nothing changed) or -2 (no free page left: ``dst`` is left empty)."""
    slots, max_pages = _table(page_table)
    dev = page_table.device
    lib = _library()
    c = _cache(k_cache, v_cache)
    if src.dim() != 1:
        raise ValueError("src must be [forks]")
    if k_cache.device != dev:
        raise ValueError(f"the cache is on {k_cache.device}, page_table on {dev}")
    n = src.shape[0]
    if status is None:
        status = _torch().empty(n, dtype=_torch().int32, device=dev)
    args = (ctypes.byref(c), _ints("page_table", page_table, (slots, max_pages), dev, rows=True),
            _row_stride(page_table), slots, max_pages, _ints("lens", lens, (slots,), dev),
            _ints("refcount", refcount, (c.pages,), dev), _ints("src", src, (n,), dev), _ints("dst", dst, (n,), dev), n,
            _ints("status", status, (n,), dev))
    with _on(dev, stream) as st:
        _check(lib.sv_cache_fork(*args, st), "sv_cache_fork")
    return status
