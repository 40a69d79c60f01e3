"""The C ABI of the tree operators on a machine without a GPU: limits, shapes
and arguments are refused on the host, before any CUDA call.  No kernel is
launched: every call here fails, or has nothing to do."""
import ctypes
import math
import re
from pathlib import Path

import pytest
import torch

import speculative_decoding_verification_92_b200 as sv
from speculative_decoding_verification_92_b200 import Status, cache, tree

FAKE = 0x10000  # 16-byte aligned, never dereferenced
HEADER = (Path(__file__).resolve().parents[1] / "include" / "sv_tree.h").read_text()


def define(name):
    return int(re.search(rf"#define {name} (\d+)", HEADER).group(1))


def test_limits_match_the_header():
    assert tree.MAX_NODES == define("SV_MAX_NODES")
    assert cache.MAX_SLOTS == define("SV_MAX_SLOTS")
    assert cache.F16 == define("SV_F16")


def struct_of(name):
    body = re.search(r"typedef struct \{([^}]*)\} " + name, HEADER).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for decl in body.split(";"):
        words = decl.split()
        if not words:
            continue
        kind = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "void": ctypes.c_void_p}[words[0]]
        fields += [(n.strip(" *"), kind) for n in decl.strip()[len(words[0]):].split(",")]
    return type(name, (ctypes.Structure,), {"_fields_": fields})


@pytest.mark.parametrize("name,packed", [("sv_cache", cache._CACHE), ("sv_tree_attention_shape", tree._ATTENTION_SHAPE),
                                         ("sv_tree_shape", tree._TREE_SHAPE)])
def test_packed_structs_have_the_header_s_layout(name, packed):
    struct = struct_of(name)
    assert ctypes.sizeof(struct) == packed.size
    values = list(range(1, len(struct._fields_) + 1))
    got = struct.from_buffer_copy(packed.pack(*values))
    assert [getattr(got, n) for n, _ in struct._fields_] == values


def kv(**kw):
    d = dict(k=FAKE, v=FAKE, layers=1, pages=8, page_size=16, heads=2, head_dim=64, dtype=sv.BF16, s_layer=0,
             s_page=16 * 2 * 64, s_row=2 * 64, s_head=64)
    d.update(kw)
    return cache._CACHE.pack(*d.values())


def shape(**kw):
    d = dict(B=2, N=3, q_heads=8, max_pages=4, table_stride=4)
    strides = {f"{t}{x}": y for t in "qkvo" for x, y in zip("bnh", (3 * 8 * 64, 8 * 64, 64))}
    d.update(strides)
    d.update(kw)
    return tree._ATTENTION_SHAPE.pack(*d.values())


def attention(s=None, c=None, q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, scale=0.1, out=FAKE, ws=FAKE,
              ws_bytes=1 << 40):
    return tree._library().sv_tree_attention(s or shape(), c or kv(), q, k, v, table, lens, None, None, scale, out,
                                             ws, ws_bytes, None)


EINVAL, EUNSUPPORTED, OK = Status.EINVAL, Status.EUNSUPPORTED, Status.OK


@pytest.mark.parametrize("want,kw", [
    (EINVAL, dict(s=dict(B=-1))), (EINVAL, dict(s=dict(N=0))), (EUNSUPPORTED, dict(s=dict(N=257))),
    (EINVAL, dict(s=dict(q_heads=7))), (EINVAL, dict(s=dict(q_heads=0))), (EUNSUPPORTED, dict(s=dict(q_heads=130))),
    (EINVAL, dict(s=dict(max_pages=0))), (EINVAL, dict(s=dict(table_stride=3))),
    (EINVAL, dict(s=dict(qn=4))), (EINVAL, dict(s=dict(ob=12))), (EINVAL, dict(s=dict(kh=-64))),
    (EUNSUPPORTED, dict(c=dict(dtype=sv.F32))), (EUNSUPPORTED, dict(c=dict(head_dim=96))),
    (EUNSUPPORTED, dict(c=dict(page_size=24))), (EUNSUPPORTED, dict(c=dict(page_size=8))),
    (EUNSUPPORTED, dict(c=dict(page_size=256))), (EINVAL, dict(c=dict(pages=0))), (EINVAL, dict(c=dict(heads=0))),
    (EINVAL, dict(c=dict(s_row=2 * 64 + 4))), (EINVAL, dict(c=dict(k=0))),
    (EINVAL, dict(q=None)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)), (EINVAL, dict(table=None)),
    (EINVAL, dict(lens=None)), (EINVAL, dict(out=None)), (EINVAL, dict(ws=None)), (EINVAL, dict(ws_bytes=64)),
    (EINVAL, dict(scale=math.nan)), (EINVAL, dict(scale=math.inf)), (EINVAL, dict(q=FAKE + 2)),
    (EINVAL, dict(ws=FAKE + 8)), (OK, dict(s=dict(B=0), q=None, k=None, v=None, table=None, lens=None, out=None))])
def test_attention_arguments(want, kw):
    kw = dict(kw)
    if "s" in kw:
        kw["s"] = shape(**kw["s"])
    if "c" in kw:
        kw["c"] = kv(**kw["c"])
    assert attention(**kw) == want


def test_attention_workspace():
    lib = tree._library()
    size = lambda s, c: lib.sv_tree_attention_workspace_bytes(s, c)
    assert size(shape(), kv()) > 0
    assert size(shape(N=257), kv()) == size(shape(), kv(head_dim=96)) == 0
    assert size(shape(B=64), kv()) >= size(shape(), kv())


def verify(B=2, N=3, V=100, dtype=sv.F32, stride=0, target=FAKE, tokens=FAKE, uniforms=FAKE, T=1.0, greedy=0,
           out=(FAKE, FAKE, FAKE)):
    return tree._library().sv_tree_verify(tree._TREE_SHAPE.pack(B, N, V, dtype, stride), target, None, tokens, None,
                                          None, uniforms, T, greedy, *out, None)


@pytest.mark.parametrize("want,kw", [
    (EINVAL, dict(B=-1)), (EINVAL, dict(N=0)), (EINVAL, dict(V=0)), (EUNSUPPORTED, dict(N=257)),
    (EUNSUPPORTED, dict(V=sv.MAX_V + 1)), (EUNSUPPORTED, dict(dtype=cache.F16)), (EINVAL, dict(stride=99)),
    (EINVAL, dict(target=None)), (EINVAL, dict(tokens=None)), (EINVAL, dict(uniforms=None)),
    (EINVAL, dict(T=0.0)), (EINVAL, dict(T=-1.0)), (EINVAL, dict(T=math.nan)), (EINVAL, dict(T=math.inf)),
    (EINVAL, dict(T=1e-45)), (EINVAL, dict(T=1e300)), (EINVAL, dict(out=(None, FAKE, FAKE))),
    (EINVAL, dict(out=(FAKE, None, FAKE))), (EINVAL, dict(out=(FAKE, FAKE, None))), (OK, dict(B=0)),
    (OK, dict(B=0, target=None, tokens=None, out=(None, None, None))), (OK, dict(B=0, uniforms=None, greedy=1, T=0.0))])
def test_verify_arguments(want, kw):
    assert verify(**kw) == want


def resize(table=FAKE, stride=4, slots=2, max_pages=4, lens=FAKE, page=16, ref=FAKE, pages=8, status=2 * FAKE):
    return cache._library().sv_cache_resize(table, stride, slots, max_pages, lens, page, ref, pages, status, None)


@pytest.mark.parametrize("want,kw", [
    (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(ref=None)), (EINVAL, dict(status=None)),
    (EINVAL, dict(slots=-1)), (EINVAL, dict(max_pages=0)), (EINVAL, dict(page=0)), (EINVAL, dict(pages=-1)),
    (EINVAL, dict(stride=3)), (EUNSUPPORTED, dict(slots=8193)), (EINVAL, dict(status=FAKE + 4)),
    (OK, dict(slots=0, table=None, lens=None, status=None))])
def test_resize_arguments(want, kw):
    assert resize(**kw) == want


def commit(c=None, table=FAKE, stride=4, B=2, max_pages=4, lens=FAKE, path=FAKE, path_stride=3, width=3, out=2 * FAKE):
    return cache._library().sv_cache_commit(c or kv(), table, stride, B, max_pages, lens, path, path_stride, width, out,
                                            None)


@pytest.mark.parametrize("want,kw", [
    (EINVAL, dict(c=dict(k=0))), (EINVAL, dict(c=dict(layers=0))), (EINVAL, dict(c=dict(head_dim=0))),
    (EUNSUPPORTED, dict(c=dict(dtype=7))), (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)),
    (EINVAL, dict(path=None)), (EINVAL, dict(out=None)), (EINVAL, dict(out=FAKE)), (EINVAL, dict(out=FAKE + 4)), (EINVAL, dict(B=-1)), (EINVAL, dict(max_pages=0)),
    (EINVAL, dict(stride=3)), (EINVAL, dict(path_stride=2)), (EINVAL, dict(width=-1)),
    (EUNSUPPORTED, dict(width=257, path_stride=257)), (OK, dict(B=0, table=None, lens=None, path=None, out=None))])
def test_commit_arguments(want, kw):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = kv(**kw["c"])
    assert commit(**kw) == want


def fork(c=None, table=FAKE, stride=4, slots=4, max_pages=4, lens=FAKE, ref=FAKE, src=2 * FAKE, dst=3 * FAKE, n=2,
         status=4 * FAKE):
    return cache._library().sv_cache_fork(c or kv(), table, stride, slots, max_pages, lens, ref, src, dst, n, status,
                                          None)


@pytest.mark.parametrize("want,kw", [
    (EINVAL, dict(c=dict(v=0))), (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(ref=None)),
    (EINVAL, dict(src=None)), (EINVAL, dict(dst=None)), (EINVAL, dict(status=None)), (EINVAL, dict(slots=-1)),
    (EINVAL, dict(n=-1)), (EINVAL, dict(stride=3)), (EUNSUPPORTED, dict(slots=8193)), (EUNSUPPORTED, dict(n=8193)),
    (EINVAL, dict(status=FAKE + 12)), (EINVAL, dict(status=2 * FAKE + 4)), (EINVAL, dict(status=3 * FAKE - 4)),
    (EINVAL, dict(src=FAKE + 8)), (EINVAL, dict(dst=FAKE)), (OK, dict(n=0, src=None, dst=None, status=None))])
def test_fork_arguments(want, kw):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = kv(**kw["c"])
    assert fork(**kw) == want


def test_tensors_on_the_cpu_are_refused():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    k = torch.zeros(1, 8, 16, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    calls = [lambda: cache.cache_resize(i(2, 4), i(2), i(8), 16),
             lambda: cache.cache_commit(k, k, i(2, 4), i(2), i(2, 3)),
             lambda: cache.cache_fork(k, k, i(2, 4), i(2), i(8), i(1), i(1)),
             lambda: tree.tree_attention(x, x, x, k[0], k[0], i(2, 4), i(2)),
             lambda: tree.tree_verify(torch.zeros(2, 3, 9), None, i(2, 3), None, None, torch.zeros(2, 3)),
             lambda: tree.TreeStep(k, k, i(2, 4), i(2), i(8), 3, 2)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
