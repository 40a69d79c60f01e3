"""Decoding steps that draft a tree of tokens per request: attention of the
nodes over a paged cache and lossless verification of the tree
(``include/sv_tree.h``; the cache's pages are in ``cache``).

Node 0 of a request is the root, the last token it has committed; ``parents``
int32 ``[B, N]`` gives node i's parent (below i; entry 0 is not read; None is
a chain) and ``counts`` int32 ``[B]`` the nodes in use (None: all N; 0: an
idle slot).
"""
from __future__ import annotations

import ctypes

from . import _check, _dtype_code, _torch, library
from .cache import _Cache, _cache, _ints, _on, _row_stride, _table

__all__ = ["tree_attention", "tree_attention_workspace_bytes", "tree_verify", "MAX_NODES"]

MAX_NODES = 256     # SV_MAX_NODES of the C header

_VP, _I32, _I64, _F32, _F64, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                    ctypes.c_size_t)


class _TreeShape(ctypes.Structure):
    _fields_ = [("B", _I32), ("N", _I32), ("V", _I32), ("dtype", _I32), ("row_stride", _I64)]


class _AttentionShape(ctypes.Structure):
    _fields_ = ([("B", _I32), ("N", _I32), ("q_heads", _I32), ("max_pages", _I32), ("table_stride", _I64)]
                + [(f"{t}_stride_{d}", _I64) for t in "qkvo" for d in "bnh"])


_SIGNATURES = {
    "sv_tree_attention_workspace_bytes": (_SZ, [ctypes.POINTER(_AttentionShape), ctypes.POINTER(_Cache)]),
    "sv_tree_attention": (_I32, [ctypes.POINTER(_AttentionShape), ctypes.POINTER(_Cache), _VP, _VP, _VP, _VP, _VP,
                                 _VP, _VP, _F32, _VP, _VP, _SZ, _VP]),
    "sv_tree_verify": (_I32, [ctypes.POINTER(_TreeShape), _VP, _VP, _VP, _VP, _VP, _VP, _F64, _I32, _VP, _VP, _VP,
                              _VP]),
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


def _logits(what, t, shape, device):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected the CUDA device of the call ({device})")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(what, t, shape, dtype, device):
    """Pointer of a [B, N, heads, head_dim] tensor with a contiguous last
    dimension, and its other strides (0 where there is one of a kind)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must have the cache's dtype {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected the CUDA device of the call ({device})")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{what} must have a contiguous last dimension")
    return t.data_ptr(), [s if n > 1 else 0 for s, n in zip(st[:3], shape)]


def _attention_shapes(q, k, v, out, k_cache, v_cache, page_table):
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B, N, q_heads, head_dim], the caches [pages, page_size, heads, head_dim]")
    B, N, Hq, D = q.shape
    c = _cache(k_cache, v_cache)
    dt, dev = k_cache.dtype, k_cache.device
    if tuple(page_table.shape[:1]) != (B,):
        raise ValueError(f"page_table must be [{B}, max_pages], got {tuple(page_table.shape)}")
    (qp, qs), (kp, ks), (vp, vs), (op, os) = (
        _rows("q", q, (B, N, Hq, c.head_dim), dt, dev), _rows("k", k, (B, N, c.heads, c.head_dim), dt, dev),
        _rows("v", v, (B, N, c.heads, c.head_dim), dt, dev), _rows("out", out, q.shape, dt, dev))
    _, max_pages = _table(page_table)
    return c, _AttentionShape(B, N, Hq, max_pages, _row_stride(page_table), *qs, *ks, *vs, *os), (qp, kp, vp, op)


def tree_attention_workspace_bytes(q, k, v, k_cache, v_cache, page_table) -> int:
    """Bytes of the workspace that tree_attention needs for these shapes."""
    c, shape, _ = _attention_shapes(q, k, v, q, k_cache, v_cache, page_table)
    return int(_library().sv_tree_attention_workspace_bytes(ctypes.byref(shape), ctypes.byref(c)))


def tree_attention(q, k, v, k_cache, v_cache, page_table, lens, parents=None, counts=None, *, scale=None, out=None,
                   workspace=None, stream=None):
    """One layer's attention of the drafted nodes.  ``k``, ``v [B, N, heads,
    head_dim]`` go to rows ``lens[b] + i`` of the paged cache (``k_cache``,
    ``v_cache [pages, page_size, heads, head_dim]``, one layer of the tensors
    of ``cache``); then node i of ``q [B, N, q_heads, head_dim]`` attends to
    the ``lens[b]`` cached rows before the tree, to its ancestors and to itself
    (softmax of ``scale q.k``; ``scale`` defaults to ``head_dim ** -0.5``).
    Query heads share key heads in consecutive groups.

    Returns ``out`` (like q; rows past ``counts[b]`` are left as they were,
    NaN rows mark a request that is not valid).  bfloat16 and float16,
    head_dim 64 and 128, page_size 16 to 128 (powers of two); a single new
    token per request is N = 1.  Calls that may run at the same time need
    separate workspaces."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    c, shape, (qp, kp, vp, op) = _attention_shapes(q, k, v, out, k_cache, v_cache, page_table)
    B, N, dev = shape.B, shape.N, k_cache.device
    ints = (_ints("page_table", page_table, (B, shape.max_pages), dev, rows=True), _ints("lens", lens, (B,), dev),
            _ints("parents", parents, (B, N), dev), _ints("counts", counts, (B,), dev))
    lib = _library()
    with _on(dev, stream) as st:
        if workspace is None:
            n = lib.sv_tree_attention_workspace_bytes(ctypes.byref(shape), ctypes.byref(c))
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        _check(lib.sv_tree_attention(ctypes.byref(shape), ctypes.byref(c), qp, kp, vp, *ints,
                                     c.head_dim ** -0.5 if scale is None else float(scale), op, workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), st), "sv_tree_attention")
    return out


def tree_verify(target, draft, tokens, parents, counts, uniforms, temperature=1.0, greedy=False, *, V=None, out=None,
                stream=None):
    """Verify one drafted tree per request.  ``target [B, N, row_stride]``:
    row i are the target's logits after node i; ``draft`` (same shape, or None
    when the drafter gave ids only): row i is the distribution that node i's
    children were drawn from, independently; ``tokens [B, N]``; ``uniforms
    [B, N]`` in [0, 1): node i's test, slot 0 the final draw (may be None when
    greedy).  Children are tried in index order.

    Returns int32 ``(accept_len [B], tokens [B, N], path [B, N])``: the number
    j of accepted drafts; their tokens and the last token at index j, then -1;
    node 0 and the accepted nodes, then -1 (what ``cache_commit`` takes).  A
    request that is not valid gets -1 throughout.  Only rows on the accepted
    path are read; sums are held in 64 bits."""
    torch = _torch()
    if target.dim() != 3:
        raise ValueError("target logits must be [B, N, row_stride]")
    B, N, row_stride = target.shape
    dev = target.device
    if draft is not None and draft.dtype != target.dtype:
        raise TypeError(f"draft logits must have the target's dtype {target.dtype}, got {draft.dtype}")
    if greedy:
        draft = uniforms = None
    if uniforms is not None and uniforms.dtype != torch.float32:
        raise TypeError(f"uniforms must be torch.float32, got {uniforms.dtype}")
    shape = _TreeShape(B, N, row_stride if V is None else int(V), _dtype_code(target), row_stride)
    ptrs = (_logits("target", target, (B, N, row_stride), dev),
            None if draft is None else _logits("draft", draft, (B, N, row_stride), dev),
            _ints("tokens", tokens, (B, N), dev), _ints("parents", parents, (B, N), dev),
            _ints("counts", counts, (B,), dev),
            None if uniforms is None else _logits("uniforms", uniforms, (B, N), dev))
    lib = _library()
    if out is None:
        all_out = torch.empty(2 * B * N + B, dtype=torch.int32, device=dev)
        out = all_out[2 * B * N:], all_out[:B * N].view(B, N), all_out[B * N:2 * B * N].view(B, N)
    outs = (_ints("out accept_len", out[0], (B,), dev), _ints("out tokens", out[1], (B, N), dev),
            _ints("out path", out[2], (B, N), dev))
    with _on(dev, stream) as st:
        _check(lib.sv_tree_verify(ctypes.byref(shape), *ptrs, float(temperature), int(bool(greedy)), *outs, st),
               "sv_tree_verify")
    return out
