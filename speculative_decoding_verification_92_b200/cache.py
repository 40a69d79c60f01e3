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

``tree.TreeStep`` is this sequence.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import BF16, F32, SpecVerifyError, library

__all__ = ["cache_resize", "cache_commit", "cache_fork", "F16", "MAX_SLOTS"]

F16 = 2             # SV_F16: caches only
MAX_SLOTS = 8192    # SV_MAX_SLOTS of the C header

_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


# sv_cache, packed: k, v, five int32 (layers, pages, page_size, heads,
# head_dim), dtype, four int64 strides.
_CACHE = struct.Struct("@2P6i4q")
_SIGNATURES = {
    "sv_cache_commit": (_I32, [ctypes.c_char_p, _VP, _I64, _I32, _I32, _VP, _VP, _I64, _I32, _VP, _VP]),
    "sv_cache_resize": (_I32, [_VP, _I64, _I32, _I32, _VP, _I32, _VP, _I32, _VP, _VP]),
    "sv_cache_fork": (_I32, [ctypes.c_char_p, _VP, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _VP]),
}
_KV_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
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


def _bad_tensor(what, t, dtype, shape, index, layout):
    """Raises what is wrong with a tensor that did not pass a quick check."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{what} is on {t.device}, expected the device of the call (cuda:{index})")
    raise ValueError(f"{what} must {layout}")


def _cuda_index(what, t) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{what} must be a CUDA tensor, got one on {t.device}")
    return index


def _dense(what, t, dtype, shape, index):
    """Pointer of a contiguous tensor of exactly this dtype, shape and CUDA
    device; None passes through.  Calls of a few microseconds are checked
    here, so the usual case is one expression."""
    if t is None:
        return None
    if t.dtype == dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _bad_tensor(what, t, dtype, shape, index, "be contiguous")


def _int_rows(what, t, shape, index):
    """Pointer and row stride of an int32 matrix with contiguous rows."""
    if t.dtype == torch.int32 and t.shape == shape and t.get_device() == index:
        s0, s1 = t.stride()
        if s1 == 1 or shape[1] <= 1:
            if shape[0] <= 1:
                return t.data_ptr(), shape[1]
            if s0 >= shape[1]:
                return t.data_ptr(), s0
    _bad_tensor(what, t, torch.int32, shape, index, "have contiguous rows that do not overlap")


def _cache(k, v, index) -> bytes:
    """The C description of a cache; 4-d tensors are one layer."""
    shape, st, dtype = k.shape, k.stride(), k.dtype
    if (len(shape) not in (4, 5) or v.shape != shape or v.dtype != dtype or v.stride() != st
            or (st[-1] != 1 and shape[-1] > 1)):
        raise ValueError("k_cache and v_cache must be [layers, pages, page_size, heads, head_dim] tensors of one "
                         "shape, dtype and layout with a contiguous last dimension")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError(f"the caches are on {k.device} and {v.device}, expected the device of the call (cuda:{index})")
    if dtype not in _KV_CODES:
        raise TypeError(f"the cache must be float32, bfloat16 or float16, got {dtype}")
    if len(shape) == 4:
        n1, n2, n3, n4 = shape
        s1, s2, s3, _ = st
        n0, s0 = 1, 0
    else:
        n0, n1, n2, n3, n4 = shape
        s0, s1, s2, s3, _ = st
    return _CACHE.pack(k.data_ptr(), v.data_ptr(), n0, n1, n2, n3, n4, _KV_CODES[dtype], s0 if n0 > 1 else 0,
                       s1 if n1 > 1 else 0, s2 if n2 > 1 else 0, s3 if n3 > 1 else 0)


def _call(fn, index, stream, *args):
    """The C call with device `index` current, on `stream` or the device's
    current stream."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status:
        raise SpecVerifyError(status, fn.__name__)


def _fresh(like, shape, stream, own=False):
    """A new tensor of the dtype and device of `like` (which the caller checks)
    for use on `stream` (None: the current one).  It is taken with that stream
    current: a block of another stream's memory may still be in use by work
    that is pending there.  What the caller gets is kept from reuse until the
    caller's stream is done with it too; `own` memory is used by the call alone."""
    if stream is None:
        return like.new_empty(shape)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape)
    if not own and stream != current:
        t.record_stream(current)
    return t


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
    dev = _cuda_index("page_table", page_table)
    if status is None:
        status = _fresh(page_table, slots, stream)
    pages = refcount.shape
    if len(pages) != 1:
        raise ValueError("refcount must be [pages]")
    table, stride = _int_rows("page_table", page_table, (slots, max_pages), dev)
    _call(_library().sv_cache_resize, dev, stream, table, stride, slots, max_pages,
          _dense("lens", lens, torch.int32, (slots,), dev), int(page_size),
          _dense("refcount", refcount, torch.int32, pages, dev), pages[0],
          _dense("status", status, torch.int32, (slots,), dev))
    return status


def cache_commit(k_cache, v_cache, page_table, lens, path, *, out_lens=None, stream=None):
    """Compaction after verification, in all layers: with n the number of
    leading entries >= 0 of ``path[b]`` (``tree_verify`` returns it), cache row
    ``lens[b] + path[b][i]`` moves to row ``lens[b] + i`` for i < n.  Returns
    the new lengths ``lens + n`` (int32, -1 for a request that is not valid and
    was left alone); ``out_lens`` must be another tensor than ``lens``."""
    B, max_pages = _table(page_table)
    dev = _cuda_index("page_table", page_table)
    c = _cache(k_cache, v_cache, dev)
    if out_lens is None:
        out_lens = _fresh(page_table, B, stream)
    if path.dim() != 2:
        raise ValueError("path must be [B, width]")
    width = path.shape[1]
    table, stride = _int_rows("page_table", page_table, (B, max_pages), dev)
    rows, path_stride = _int_rows("path", path, (B, width), dev)
    _call(_library().sv_cache_commit, dev, stream, c, table, stride, B, max_pages,
          _dense("lens", lens, torch.int32, (B,), dev), rows, path_stride, width,
          _dense("out_lens", out_lens, torch.int32, (B,), dev))
    return out_lens


def cache_fork(k_cache, v_cache, page_table, lens, refcount, src, dst, *, status=None, stream=None):
    """Fork i makes slot ``dst[i]`` a copy of slot ``src[i]``: full pages are
    shared, the ragged last one is copied in all layers to a free page, what
    ``dst`` held is given back.  Updates ``page_table``, ``lens`` and
    ``refcount`` in place; returns int32 ``status [forks]``: 0, -1 (not valid,
    nothing changed) or -2 (no free page left: ``dst`` is left empty)."""
    slots, max_pages = _table(page_table)
    dev = _cuda_index("page_table", page_table)
    c = _cache(k_cache, v_cache, dev)
    if src.dim() != 1:
        raise ValueError("src must be [forks]")
    n = src.shape[0]
    if status is None:
        status = _fresh(page_table, n, stream)
    table, stride = _int_rows("page_table", page_table, (slots, max_pages), dev)
    pages = k_cache.shape[-4]
    _call(_library().sv_cache_fork, dev, stream, c, table, stride, slots, max_pages,
          _dense("lens", lens, torch.int32, (slots,), dev), _dense("refcount", refcount, torch.int32, (pages,), dev),
          _dense("src", src, torch.int32, (n,), dev), _dense("dst", dst, torch.int32, (n,), dev), n,
          _dense("status", status, torch.int32, (n,), dev))
    return status
