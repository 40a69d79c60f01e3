"""cache_resize, cache_fork and cache_commit against their plain forms."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_92_b200 import SpecVerifyError, cache
from tree_reference import commit, fork, make_parents, ancestors, resize

pytestmark = pytest.mark.gpu


def t32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def pool(rng, lens, page, max_pages, extra):
    """A valid table for these lengths, in shuffled pages."""
    need = [-(-n // page) for n in lens]
    P = sum(need) + extra
    perm = rng.permutation(P).tolist()
    table, ref = np.full((len(lens), max_pages), -1, np.int32), np.zeros(P, np.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = perm.pop()
            ref[table[s, i]] += 1
    return table, ref


def check_resize(table, lens, ref, page):
    t, r = t32(table), t32(ref)
    status = cache.cache_resize(t, t32(lens), r, page)
    want = resize(table, np.asarray(lens), ref, page)
    for g, w in zip((t, r, status), want):
        assert np.array_equal(g.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("page", [1, 16, 24, 128])
@pytest.mark.parametrize("slots,most,extra", [(1, 40, 3), (7, 300, 40), (70, 900, 500), (1500, 90, 3000), (20, 9000, 20000)])
def test_resize_grows_and_shrinks(page, slots, most, extra):
    rng = np.random.default_rng(slots + page)
    old, new = rng.integers(0, most, slots), rng.integers(0, most, slots)
    new[rng.random(slots) < 0.2] = 0
    table, ref = pool(rng, old, page, most // page + 2, extra)
    table, ref, status = check_resize(table, new, ref, page)
    check_resize(table, old, ref, page)
    check_resize(table, np.zeros(slots, np.int32), ref, page)


def test_resize_short_of_pages_serves_slots_in_order():
    rng = np.random.default_rng(1)
    table, ref = pool(rng, [16, 0, 0, 0, 32, 0], 16, 6, 4)
    _, _, status = check_resize(table, [16, 32, 48, 16, 0, 16], ref, 16)
    assert list(status) == [0, 0, 0, 0, 0, -1]          # 6 free pages for 2 + 3 + 1 + 1
    _, _, status = check_resize(table, [16, 32, 64, 16, 32, 16], ref, 16)
    assert list(status) == [0, 0, -1, -1, 0, -1]


def test_resize_refuses_bad_rows_and_lengths():
    rng = np.random.default_rng(2)
    table, ref = pool(rng, [30, 30, 30, 30, 30], 16, 4, 10)
    table[1] = [table[1, 0], -1, table[1, 1], -1]
    table[2, 3] = len(ref)
    table[3, 2] = -2
    _, _, status = check_resize(table, [65, 10, 10, 10, 10], ref, 16)
    assert list(status) == [-1, -1, -1, -1, 0]
    _, _, status = check_resize(table, [-1, 0, 0, 0, 64], ref, 16)
    assert list(status) == [-1, -1, -1, -1, 0]


def test_resize_keeps_shared_pages_until_the_last_holder_lets_go():
    ref = np.array([2, 2, 0, 0], np.int32)
    table = np.array([[1, 0], [1, 0]], np.int32)
    table, ref, _ = check_resize(table, [0, 32], ref, 16)
    assert list(ref) == [1, 1, 0, 0]
    _, ref, _ = check_resize(table, [0, 0], ref, 16)
    assert list(ref) == [0, 0, 0, 0]


def caches(rng, L, P, page, H, D, dtype=torch.bfloat16, layout="nhd"):
    out = []
    for _ in range(2):
        x = torch.from_numpy(rng.integers(-1000, 1000, (L, P, page, H, D)).astype(np.float32)).to(dtype).cuda()
        out.append(x if layout == "nhd" else x.transpose(2, 3).contiguous().transpose(2, 3))
    return out


def as_np(x):
    return x.float().cpu().numpy()


@pytest.mark.parametrize("page,layout,dtype", [(16, "nhd", torch.bfloat16), (16, "hnd", torch.bfloat16),
                                               (32, "nhd", torch.float16), (5, "nhd", torch.float32),
                                               (128, "hnd", torch.float32)])
@pytest.mark.parametrize("slots,G", [(1, 1), (3, 4), (40, 3)])
def test_fork(page, layout, dtype, slots, G):
    rng = np.random.default_rng(page + slots)
    lens = np.concatenate([rng.integers(0, 3 * page + 1, slots), np.zeros(slots * G, int)]).astype(np.int32)
    lens[slots + 1::3] = page + 2                       # some destinations hold something
    table, ref = pool(rng, lens, page, 6, slots * G + 2)
    k, v = caches(rng, 3, len(ref), page, 2, 8, dtype, layout)
    src = np.repeat(np.arange(slots), G).astype(np.int32)
    dst = (slots + rng.permutation(slots * G)).astype(np.int32)
    want = fork(as_np(k), as_np(v), table, lens, ref, src, dst)
    t, n, r = t32(table), t32(lens), t32(ref)
    status = cache.cache_fork(k, v, t, n, r, t32(src), t32(dst))
    got = (as_np(k), as_np(v), t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy(), status.cpu().numpy())
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert (want[5] == 0).all()


def test_fork_refusals_and_empty_pools():
    rng = np.random.default_rng(3)
    lens = np.array([20, 33, 0, 0, 0, 0, 16, 5], np.int32)
    table, ref = pool(rng, lens, 16, 4, 1)
    table[7] = [-1, table[7, 0], -1, -1]                # not a valid row
    k, v = caches(rng, 1, len(ref), 16, 1, 8)
    src = np.array([0, 0, 1, 9, 0, 7, 6, 0, 1], np.int32)
    dst = np.array([2, 2, 0, 3, -1, 3, 4, 5, 3], np.int32)
    dst[3] = 8
    dst[5] = 4
    dst[6] = 3
    dst[8] = 5
    for s, d in ((src, dst), (np.array([0, 1, 6, 0], np.int32), np.array([5, 3, 4, 2], np.int32))):
        want = fork(as_np(k), as_np(v), table, lens, ref, s, d)
        t, n, r, kk, vv = t32(table), t32(lens), t32(ref), k.clone(), v.clone()
        status = cache.cache_fork(kk, vv, t, n, r, t32(s), t32(d))
        got = (as_np(kk), as_np(vv), t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy(), status.cpu().numpy())
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
    assert list(want[5]) == [0, -2, 0, -2]              # one free page, two ragged forks too many


def test_many_forks_over_a_large_pool():
    rng = np.random.default_rng(4)
    slots, F = 700, 600
    lens = np.zeros(slots, np.int32)
    lens[:100] = rng.integers(0, 100, 100)
    table, ref = pool(rng, lens, 16, 8, 40000)
    k, v = caches(rng, 1, len(ref), 16, 1, 8)
    src, dst = rng.integers(0, 100, F).astype(np.int32), (100 + rng.permutation(F)).astype(np.int32)
    want = fork(as_np(k), as_np(v), table, lens, ref, src, dst)
    t, n, r = t32(table), t32(lens), t32(ref)
    cache.cache_fork(k, v, t, n, r, t32(src), t32(dst))
    for g, w in zip((as_np(k), as_np(v), t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy()), want):
        assert np.array_equal(g, w)


def paths(rng, B, N, width):
    out = np.full((B, N), -1, np.int32)
    for b in range(B):
        parents = make_parents(rng, N, width)
        row = sorted(ancestors(parents, int(rng.integers(0, N))))
        out[b, :len(row)] = row
    return out


@pytest.mark.parametrize("page,layout,dtype,H,D", [(16, "nhd", torch.bfloat16, 2, 64), (16, "hnd", torch.float16, 3, 8),
                                                   (7, "nhd", torch.float32, 1, 128), (64, "hnd", torch.bfloat16, 8, 128)])
@pytest.mark.parametrize("N,width", [(1, 1), (9, 1), (20, 2), (64, None), (256, 1)])
def test_commit(page, layout, dtype, H, D, N, width):
    rng = np.random.default_rng(page + N)
    B = 7
    lens = rng.integers(0, 100, B).astype(np.int32)
    table, ref = pool(rng, lens + N, page, (100 + N) // page + 2, 3)
    k, v = caches(rng, 2, len(ref), page, H, D, dtype, layout)
    path = paths(rng, B, N, width)
    path[0] = -1                                        # nothing accepted, not even the root
    if N > 1:
        path[1, :N - 1] = np.arange(1, N)               # every row moves by one
        path[1, N - 1] = -1
    want = commit(as_np(k), as_np(v), table, lens, path)
    n = cache.cache_commit(k, v, t32(table), t32(lens), t32(path))
    for g, w in zip((as_np(k), as_np(v), n.cpu().numpy()), want):
        assert np.array_equal(g, w)


def test_commit_takes_a_view_of_the_path_and_leaves_bad_requests_alone():
    rng = np.random.default_rng(6)
    lens = np.array([10, -1, 10, 10, 10, 10], np.int32)
    table, ref = pool(rng, [26] * 6, 16, 2, 2)
    k, v = caches(rng, 2, len(ref), 16, 2, 8)
    path = np.tile(np.array([0, 2, 5, -1, 3, 9], np.int32), (6, 1))
    path[2, :3] = [0, 5, 2]
    path[3, 2] = 22                                     # past the two pages
    table[4, 0] = -1
    want = commit(as_np(k), as_np(v), table, lens, path[:, :4])
    n = cache.cache_commit(k, v, t32(table), t32(lens), t32(path)[:, :4])
    for g, w in zip((as_np(k), as_np(v), n.cpu().numpy()), want):
        assert np.array_equal(g, w)
    assert list(want[2]) == [13, -1, -1, -1, -1, 13]


def test_refusals():
    rng = np.random.default_rng(7)
    table, ref = pool(rng, [20, 20], 16, 4, 2)
    k, v = caches(rng, 1, len(ref), 16, 1, 8)
    t, n, r, p = t32(table), t32([20, 20]), t32(ref), t32([[0, 1], [0, 1]])
    for want, call in [
        (TypeError, lambda: cache.cache_resize(t.long(), n, r, 16)), (ValueError, lambda: cache.cache_resize(t, n[:1], r, 16)),
        (SpecVerifyError, lambda: cache.cache_resize(t, n, r, 0)), (ValueError, lambda: cache.cache_resize(t.cpu(), n, r, 16)),
        (SpecVerifyError, lambda: cache.cache_commit(k, v, t, n, p, out_lens=n)),
        (ValueError, lambda: cache.cache_commit(k, v[:, :1], t, n, p)),
        (SpecVerifyError, lambda: cache.cache_commit(k[..., :4].contiguous(), v[..., :4].contiguous(), t, n, p)),
        (TypeError, lambda: cache.cache_commit(k.double(), v.double(), t, n, p)),
        (ValueError, lambda: cache.cache_fork(k, v, t, n, r[:1], p[0], p[1])),
        (ValueError, lambda: cache.cache_fork(k, v, t, n, r, p[0], p[1, :1]))]:
        with pytest.raises(want):
            call()


def test_nothing_to_do():
    rng = np.random.default_rng(9)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    k, v = caches(rng, 2, 4, 16, 2, 8)
    ref = t32([1, 0, 2, 0])
    assert cache.cache_resize(e(0, 4), e(0), ref, 16).shape == (0,)
    assert cache.cache_commit(k, v, e(0, 4), e(0), e(0, 3)).shape == (0,)
    table = t32([[0, -1], [2, -1]])
    assert cache.cache_fork(k, v, table, t32([5, 6]), ref, e(0), e(0)).shape == (0,)
    assert ref.tolist() == [1, 0, 2, 0] and table.tolist() == [[0, -1], [2, -1]]


def test_overlapping_tensors_are_refused():
    lens = t32([5, 6])
    with pytest.raises(SpecVerifyError):
        cache.cache_resize(t32([[0, -1], [2, -1]]), lens, t32([1, 0, 1]), 16, status=lens)
    both = t32([1, 1, 1])
    k, v = caches(np.random.default_rng(10), 1, 3, 16, 2, 8)
    with pytest.raises(SpecVerifyError):
        cache.cache_fork(k, v, t32([[0, -1], [2, -1]]), t32([5, 6]), t32([1, 0, 1]), both[:1], both[1:2],
                         status=both[1:2])
