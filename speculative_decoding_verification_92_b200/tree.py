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
import struct

import torch

from . import BF16, F32, library
from .cache import (_bad_tensor, _cache, _call, _cuda_index, _dense, _fresh, _int_rows, _table, cache_commit,
                    cache_resize)

__all__ = ["tree_attention", "tree_attention_workspace_bytes", "tree_verify", "TreeStep", "MAX_NODES"]

MAX_NODES = 256     # SV_MAX_NODES of the C header

_VP, _I32, _F32, _F64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_double, ctypes.c_size_t


# sv_tree_shape: B, N, V, dtype, row_stride; sv_tree_attention_shape: B, N,
# q_heads, max_pages, table_stride, strides of q, k, v and out.
_TREE_SHAPE = struct.Struct("@4iq")
_ATTENTION_SHAPE = struct.Struct("@4iq12q")
_SIGNATURES = {
    "sv_tree_attention_workspace_bytes": (_SZ, [ctypes.c_char_p, ctypes.c_char_p]),
    "sv_tree_attention": (_I32, [ctypes.c_char_p, ctypes.c_char_p, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _F32, _VP, _VP,
                                 _SZ, _VP]),
    "sv_tree_verify": (_I32, [ctypes.c_char_p, _VP, _VP, _VP, _VP, _VP, _VP, _F64, _I32, _VP, _VP, _VP, _VP]),
}
_LOGIT_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_LIB = None
_WORKSPACE = {}    # bytes by sizes


def _library():
    global _LIB
    if _LIB is None:
        lib = library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _LIB = lib
    return _LIB


def _rows(what, t, shape, dtype, index):
    """Pointer of a [B, N, heads, head_dim] tensor with a contiguous last
    dimension, and its other strides (0 where there is one of a kind)."""
    s0, s1, s2, s3 = t.stride() if t.dim() == 4 else (0, 0, 0, 0)
    if t.dtype == dtype and t.shape == shape and t.get_device() == index and s3 == 1:
        return t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0, s2 if shape[2] > 1 else 0
    _bad_tensor(what, t, dtype, shape, index, "have a contiguous last dimension")


def _attention_shapes(q, k, v, out, k_cache, v_cache, page_table):
    qshape, cshape = q.shape, k_cache.shape
    if len(qshape) != 4 or len(cshape) != 4:
        raise ValueError("q must be [B, N, q_heads, head_dim], the caches [pages, page_size, heads, head_dim]")
    B, N, Hq, D = qshape
    heads = cshape[2]
    dt, dev = k_cache.dtype, _cuda_index("k_cache", k_cache)
    c = _cache(k_cache, v_cache, dev)
    full, kv = (B, N, Hq, cshape[3]), (B, N, heads, cshape[3])
    qp, *qs = _rows("q", q, full, dt, dev)
    kp, *ks = _rows("k", k, kv, dt, dev)
    vp, *vs = _rows("v", v, kv, dt, dev)
    op, *os = _rows("out", out, full, dt, dev)
    max_pages = _table(page_table)[1]
    table, stride = _int_rows("page_table", page_table, (B, max_pages), dev)
    return (c, _ATTENTION_SHAPE.pack(B, N, Hq, max_pages, stride, *qs, *ks, *vs, *os), (qp, kp, vp, table), op,
            (B, N, Hq, heads, D, dev))


def _workspace_bytes(c, shape, sizes):
    """Asked for once per sizes: it depends on nothing else, and asking takes
    as long as a tensor's checks."""
    n = _WORKSPACE.get(sizes)
    if n is None:
        n = int(_library().sv_tree_attention_workspace_bytes(shape, c))
        if n and len(_WORKSPACE) < 4096:
            _WORKSPACE[sizes] = n
    return n


def tree_attention_workspace_bytes(q, k, v, k_cache, v_cache, page_table) -> int:
    """Bytes of the workspace that tree_attention needs for these shapes."""
    c, shape, *_ = _attention_shapes(q, k, v, q, k_cache, v_cache, page_table)
    return int(_library().sv_tree_attention_workspace_bytes(shape, c))


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
    head_dim 64 and 128, page_size 16 to 128 (powers of two).  A single new
    token per request is N = 1; a prompt fills the cache as chains of up to
    256 nodes, call by call (``parents`` None, ``lens`` growing).  Calls that may run at the same time need
    separate workspaces."""
    if out is None:
        out = _fresh(q, q.shape, stream)
    c, shape, ptrs, op, sizes = _attention_shapes(q, k, v, out, k_cache, v_cache, page_table)
    B, N, _, _, D, dev = sizes
    if workspace is None:
        n = max(_workspace_bytes(c, shape, sizes), 256)
        workspace = _fresh(q, (n + 1) // 2, stream, own=True)   # (two bytes an element)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {q.device}")
    else:
        n = workspace.numel() * workspace.element_size()
    nodes = (B, N)
    _call(_library().sv_tree_attention, dev, stream, shape, c, *ptrs, _dense("lens", lens, torch.int32, (B,), dev),
          _dense("parents", parents, torch.int32, nodes, dev), _dense("counts", counts, torch.int32, (B,), dev),
          D ** -0.5 if scale is None else float(scale), op, workspace.data_ptr(), n)
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
    path are read.  Draws and residuals come from sums in 64 bits; acceptance
    tests from sums in 32 where these settle them, else in 64."""
    if target.dim() != 3:
        raise ValueError("target logits must be [B, N, row_stride]")
    rows = target.shape
    B, N, row_stride = rows
    dev, dt = _cuda_index("target", target), target.dtype
    if dt not in _LOGIT_CODES:
        raise TypeError(f"logits must be float32 or bfloat16, got {dt}")
    if greedy:
        draft = uniforms = None
    i32, nodes = torch.int32, (B, N)
    if out is None:
        out = _fresh(tokens, B, stream), _fresh(tokens, nodes, stream), _fresh(tokens, nodes, stream)
        outs = [x.data_ptr() for x in out]
    else:
        outs = (_dense("out accept_len", out[0], i32, (B,), dev), _dense("out tokens", out[1], i32, nodes, dev),
                _dense("out path", out[2], i32, nodes, dev))
    _call(_library().sv_tree_verify, dev, stream,
          _TREE_SHAPE.pack(B, N, row_stride if V is None else int(V), _LOGIT_CODES[dt], row_stride),
          _dense("target", target, dt, rows, dev), _dense("draft", draft, dt, rows, dev),
          _dense("tokens", tokens, i32, nodes, dev), _dense("parents", parents, i32, nodes, dev),
          _dense("counts", counts, i32, (B,), dev), _dense("uniforms", uniforms, torch.float32, nodes, dev),
          float(temperature), int(bool(greedy)), *outs)
    return out


class TreeStep:
    """A decoding step over a paged cache (``cache``), for trees of up to
    ``nodes`` nodes per slot and a model with ``q_heads`` query heads:

        step = TreeStep(k_cache, v_cache, page_table, lens, refcount, nodes, q_heads)
        step.begin(parents, counts)                        # room for the trees
        for layer in range(layers):                        # the target model
            out = step.attention(layer, q, k, v)
        accept_len, tokens, path = step.finish(target, draft, drafts, uniforms)

    ``page_table``, ``lens`` and ``refcount`` are updated in place: ``begin``
    takes pages for ``lens + counts`` rows, ``finish`` verifies, moves the
    accepted rows behind the prefix, advances ``lens`` and gives surplus pages
    back.  A slot that the free pages do not reach sits the step out as an
    idle one (``status`` of the slot -1, nothing accepted, ``lens`` kept); so
    does one whose length and count do not fit its row of the table.  Pages
    that a slot holds past its rows are given back by either call.

    The step owns its workspace and the outputs of ``finish`` (the next step
    overwrites them) and never synchronises; everything runs on the current
    stream, so one step can be captured into a CUDA graph as
    ``graph.VerifyGraph`` captures a verification.  Two steps that may run at
    the same time need a TreeStep each."""

    def __init__(self, k_cache, v_cache, page_table, lens, refcount, nodes, q_heads):
        if k_cache.dim() != 5:
            raise ValueError("k_cache must be [layers, pages, page_size, heads, head_dim]")
        if not 1 <= nodes <= MAX_NODES:
            raise ValueError(f"nodes must be in [1, {MAX_NODES}], got {nodes}")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.page_table, self.lens, self.refcount, self.nodes = page_table, lens, refcount, nodes
        slots, dev = _table(page_table)[0], k_cache.device
        heads, head_dim = k_cache.shape[3:]
        index = _cuda_index("k_cache", k_cache)
        _dense("lens", lens, torch.int32, (slots,), index)
        _dense("refcount", refcount, torch.int32, k_cache.shape[1:2], index)   # (its free pages are the cache's)
        ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)
        self.status, self.counts, self.parents = ints(slots), None, None
        self._want, self._new_lens, self._full = ints(slots), ints(slots), torch.full_like(lens, nodes)
        self._counts, self._trimmed = ints(slots), ints(slots)
        self._verified = ints(slots), ints(slots, nodes), ints(slots, nodes)
        row = torch.empty(head_dim, dtype=k_cache.dtype, device=dev)   # (only shapes matter here)
        q, k = (row.expand(slots, nodes, h, head_dim) for h in (q_heads, heads))
        n = tree_attention_workspace_bytes(q, k, k, k_cache[0], v_cache[0], page_table)
        if n == 0 and slots > 0:
            raise ValueError("no tree attention for a cache of this type, page size or head count")
        self._workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)

    def begin(self, parents=None, counts=None):
        """Takes the pages of this step's trees (``parents [slots, nodes]``,
        ``counts [slots]`` as in ``tree_attention``); returns ``status``."""
        counts = self._full if counts is None else counts
        index = self.k_cache.get_device()
        # (before anything of the step's own is written: a captured graph may hold it)
        if counts.dtype != torch.int32 or counts.shape != self.lens.shape or counts.get_device() != index:
            _bad_tensor("counts", counts, torch.int32, self.lens.shape, index, "")
        _dense("parents", parents, torch.int32, (self.lens.shape[0], self.nodes), index)
        torch.clamp(counts, min=0, out=self._want)   # (a count or length that is not valid takes nothing away)
        self._want += self.lens
        torch.where(self.lens < 0, self.lens, self._want, out=self._want)
        cache_resize(self.page_table, self._want, self.refcount, self.k_cache.shape[2], status=self.status)
        # a slot without its pages is idle
        torch.mul(counts, self.status + 1, out=self._counts)
        self.parents, self.counts = parents, self._counts
        return self.status

    def attention(self, layer, q, k, v, *, scale=None, out=None):
        """``tree_attention`` of one layer of the cache."""
        return tree_attention(q, k, v, self.k_cache[layer], self.v_cache[layer], self.page_table, self.lens,
                              self.parents, self._begun(), scale=scale, out=out, workspace=self._workspace)

    def finish(self, target, draft, tokens, uniforms, temperature=1.0, greedy=False, *, V=None):
        """``tree_verify`` of the step's trees; the cache then holds the
        accepted path.  Returns ``(accept_len, tokens, path)``."""
        out = tree_verify(target, draft, tokens, self.parents, self._begun(), uniforms, temperature, greedy, V=V,
                          out=self._verified)
        cache_commit(self.k_cache, self.v_cache, self.page_table, self.lens, out[2], out_lens=self._new_lens)
        torch.where(self._new_lens < 0, self.lens, self._new_lens, out=self.lens)
        cache_resize(self.page_table, self.lens, self.refcount, self.k_cache.shape[2], status=self._trimmed)
        self.counts = None
        return out

    def _begun(self):
        if self.counts is None:
            raise RuntimeError("begin() comes first")
        return self.counts
