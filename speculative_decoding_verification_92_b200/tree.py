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

__all__ = ["tree_verify", "MAX_NODES"]

MAX_NODES = 256     # SV_MAX_NODES of the C header

_VP, _I32, _I64, _F32, _F64, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                    ctypes.c_size_t)


class _TreeShape(ctypes.Structure):
    _fields_ = [("B", _I32), ("N", _I32), ("V", _I32), ("dtype", _I32), ("row_stride", _I64)]


_SIGNATURES = {
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
