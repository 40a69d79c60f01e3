"""tree_attention against a 64-bit form of the same sums, at the sizes and
masks where it can go wrong."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_92_b200 import Status, SpecVerifyError, tree
from tree_reference import ancestors, attention, attention_tolerance, exact_score_tolerance, make_parents

pytestmark = pytest.mark.gpu


class Case:
    """A cache with poisoned places: rows past each request's tree, free pages
    and the padding behind strided tensors hold NaN."""

    def __init__(self, lens, counts, N, Hkv=2, g=4, D=128, page=16, dtype=torch.bfloat16, width=None, seed=0,
                 layout="nhd", gain=1.0, spare_pages=3, chain=False):
        gen = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.B, self.N, self.Hkv, self.Hq, self.D, self.page, self.dtype = B, N, Hkv, Hkv * g, D, page, dtype
        self.lens, self.counts, self.scale = list(lens), list(counts), D ** -0.5
        self.parents = [make_parents(rng, N, 1 if chain else width) for _ in range(B)]
        need = [-(-(n + m) // page) for n, m in zip(lens, counts)]
        P = sum(need) + spare_pages
        perm = rng.permutation(P).tolist()
        table = np.full((B, max(need + [1]) + 2), -1, np.int32)
        for b, n in enumerate(need):
            for i in range(n):
                table[b, i] = perm.pop()
        shape = (P, page, Hkv, D) if layout == "nhd" else (P, Hkv, page, D)
        kv = []
        for _ in range(2):
            c = torch.randn(shape, generator=gen, device="cuda").mul_(gain).to(dtype)
            kv.append(c if layout == "nhd" else c.transpose(1, 2))
        self.kc, self.vc = kv
        self.table = torch.from_numpy(table).cuda()
        for b in range(B):          # poison what no node may see
            for t in range(lens[b], need[b] * page):
                for c in kv:
                    c[table[b, t // page], t % page] = math.nan
        for x in perm:
            for c in kv:
                c[x] = math.nan
        # q, k, v as views of one fused projection
        fused = torch.randn(B, N, (self.Hq + 2 * Hkv) * D + 8, generator=gen, device="cuda").to(dtype)
        fused[..., -8:] = math.nan
        cut = lambda a, h: fused[..., a * D:(a + h) * D].unflatten(-1, (h, D))
        self.q, self.k, self.v = cut(0, self.Hq).mul_(gain), cut(self.Hq, Hkv), cut(self.Hq + Hkv, Hkv)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.lens_t, self.counts_t, self.parents_t = i32(self.lens), i32(self.counts), i32(self.parents)
        self.out = torch.full((B, N, self.Hq, D), 7.0, dtype=dtype, device="cuda")

    def rows_of(self, b, n):
        ids = self.table[b, :-(-n // self.page)].long()
        return tuple(c[ids].reshape(-1, self.Hkv, self.D)[:n] for c in (self.kc, self.vc))

    def reference(self):
        out, A = attention(self.q, self.k, self.v, self.lens, self.counts, self.parents, self.rows_of, self.scale)
        kmax = max([float(self.k.double().abs().max())] +
                   [float(self.rows_of(b, n)[0].double().abs().max()) for b, n in enumerate(self.lens) if n > 0])
        return out, attention_tolerance(self.q, kmax, torch.nan_to_num(out), torch.nan_to_num(A), self.dtype, self.scale)

    def run(self, **kw):
        args = dict(parents=self.parents_t, counts=self.counts_t, out=self.out)
        args.update(kw)
        return tree.tree_attention(self.q, self.k, self.v, self.kc, self.vc, self.table, self.lens_t, **args)

    def check(self, out=None, ref=None):
        ref, tol = ref or self.reference()
        out = self.run() if out is None else out
        torch.cuda.synchronize()
        for b in range(self.B):
            m = self.counts[b]
            got = out[b, :m].double()
            err = (got - ref[b, :m]).abs()
            worst = (err / tol[b, :m]).nan_to_num(nan=math.inf).amax().item() if m else 0.0
            assert worst <= 1.0, (b, self.lens[b], m, worst)
            assert bool((out[b, m:] == 7.0).all()), "rows past the count are left as they were"
            for i in range(m):       # the new rows are in the cache
                t = self.lens[b] + i
                at = int(self.table[b, t // self.page]), t % self.page
                assert torch.equal(self.kc[at], self.k[b, i]) and torch.equal(self.vc[at], self.v[b, i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_types_heads_and_pages(dtype, D, page):
    Case([0, 1, 127, 128, 129, 300], [5, 7, 1, 7, 6, 2], 7, D=D, page=page, dtype=dtype, seed=page + D).check()


@pytest.mark.parametrize("Hkv,g", [(1, 1), (1, 8), (2, 7), (3, 5), (8, 4), (2, 64)])
def test_head_groups(Hkv, g):
    Case([40, 0, 511], [3, 9, 9], 9, Hkv=Hkv, g=g, seed=g).check()


@pytest.mark.parametrize("g", [1, 4])
def test_single_tokens_over_many_lengths(g):
    lens = list(range(0, 40)) + [63, 64, 65, 126, 127, 128, 129, 255, 256, 257, 383, 384, 640, 1000, 1023, 1024]
    Case(lens, [1] * len(lens), 1, g=g, seed=1).check()


@pytest.mark.parametrize("N,g,width", [(32, 4, 1), (33, 4, 2), (64, 2, 3), (64, 4, 3), (65, 4, None), (100, 7, None),
                                       (128, 1, 4), (129, 2, None), (256, 1, None), (256, 8, 16)])
def test_wide_trees(N, g, width):
    Case([130, 5, 0], [N, N - 1, (N + 1) // 2], N, g=g, width=width, seed=N).check()


@pytest.mark.parametrize("page,layout", [(16, "hnd"), (128, "hnd"), (64, "nhd")])
def test_a_tree_that_crosses_pages_and_tiles_in_either_layout(page, layout):
    Case([120, 250, 383], [20, 20, 20], 20, page=page, layout=layout, seed=3).check()


def test_long_contexts_and_ragged_batches():
    Case([9000, 3, 0, 4097, 1500], [4, 9, 0, 9, 1], 9, Hkv=2, g=4, page=64, seed=4).check()


@pytest.mark.parametrize("N,g,D,page", [(9, 4, 128, 16), (1, 8, 64, 32), (64, 4, 128, 64), (40, 7, 64, 16)])
def test_runs_of_many_tiles(N, g, D, page):
    # more tiles than CTAs: every CTA runs through several heads and requests, with short and long last tiles
    lens = [600 + 37 * i for i in range(40)] + [1, 0, 128, 1790, 1920]
    Case(lens, [N - (i % 3 == 2) * (N // 2) for i in range(len(lens))], N, Hkv=8, g=g, D=D, page=page, seed=N).check()


def test_one_long_request():
    Case([20011], [2], 2, Hkv=1, g=2, page=16, seed=5).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,g,lens", [(3, 7, [12600, 9000]), (64, 4, [18000]), (1, 1, [30000, 5, 0])])
def test_few_units_cut_into_many_parts(N, g, lens, D):
    Case(lens, [N] * len(lens), N, Hkv=1, g=g, D=D, page=16, seed=20).check()


def test_many_short_requests():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 200, 300).tolist()
    counts = rng.integers(0, 6, 300).tolist()
    Case(lens, counts, 5, Hkv=2, g=2, D=64, seed=6).check()


@pytest.mark.parametrize("gain", [0.0, 6.0, 25.0])
def test_flat_and_peaked_scores(gain):
    # gain 25: scores up to some thousands; the softmax is nearly one-hot and its maximum moves all the time
    Case([700, 64], [6, 3], 6, gain=gain, seed=7).check()


def test_rising_scores_move_the_maximum_in_every_tile():
    c = Case([2000], [3], 3, Hkv=1, g=2, seed=8)
    ids = c.table[0].long()
    ramp = torch.linspace(-30, 30, 2000, device="cuda")
    for t in range(2000):
        c.kc[ids[t // c.page], t % c.page] = (c.q[0, 0, 0].float() / c.q[0, 0, 0].float().norm() * ramp[t]).to(c.dtype)
    c.check()


def test_default_chain_full_counts_and_fresh_output():
    c = Case([50, 3], [6, 6], 6, chain=True, seed=9)
    out = tree.tree_attention(c.q, c.k, c.v, c.kc, c.vc, c.table, c.lens_t)
    c.check(out)


def test_scale():
    c = Case([50, 3], [6, 6], 6, seed=10)
    c.scale = 0.3
    c.check(c.run(scale=0.3))


def test_two_calls_give_the_same_bits_and_a_later_call_sees_new_data():
    c = Case([1000, 200, 31], [8, 8, 5], 8, seed=11)
    a = c.run().clone()
    for _ in range(5):
        assert torch.equal(a.view(torch.int16), c.run().view(torch.int16))
    c.q.neg_()
    c.check()


def test_invalid_requests_are_nan_and_change_nothing():
    c = Case([40, 40, 40, 40, 40, 40], [4, 4, 4, 4, 4, 4], 4, seed=12)
    lens, counts, parents, table = c.lens_t.clone(), c.counts_t.clone(), c.parents_t.clone(), c.table.clone()
    lens[0] = -1
    counts[1] = 5                       # out of range: no row is written at all
    parents[2, 3] = 3
    table[3, 1] = c.kc.shape[0]
    lens[4] = table.shape[1] * c.page - 3
    before = c.kc.clone(), c.vc.clone()
    out = tree.tree_attention(c.q, c.k, c.v, c.kc, c.vc, table, lens, parents, counts, out=c.out)
    torch.cuda.synchronize()
    for b in (0, 2, 3, 4):
        assert out[b].isnan().all()
    assert (out[1] == 7.0).all()
    assert out[5].isfinite().all()
    for x, y, new in ((before[0], c.kc, c.k), (before[1], c.vc, c.v)):
        same = (x == y) | (x.isnan() & y.isnan())
        changed = (~same.flatten(1).all(1)).nonzero()[:, 0].tolist()
        assert set(changed) <= set(c.table[5].tolist())


def test_offsets_past_32_bits():
    # pages at the far end of a cache of more than 2^31 elements
    P, page, Hkv, D = 150000, 16, 8, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    c = Case([100, 33], [5, 5], 5, Hkv=Hkv, g=2, D=D, page=page, seed=13)
    big = []
    for x in (c.kc, c.vc):
        y = torch.empty(P, page, Hkv, D, dtype=c.dtype, device="cuda")
        y[P - x.shape[0]:] = x
        big.append(y)
    c.kc, c.vc = big
    c.table = torch.where(c.table >= 0, c.table + (P - 0) - (sum(-(-(n + 5) // page) for n in c.lens) + 3), c.table)
    c.check()


def test_on_a_side_stream_and_in_a_graph():
    c = Case([300, 20], [7, 4], 7, seed=14)
    ref = c.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = c.run()
    side.synchronize()
    c.check(out, ref)
    c.out.fill_(7.0)
    ws = torch.empty(tree.tree_attention_workspace_bytes(c.q, c.k, c.v, c.kc, c.vc, c.table), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = c.run(workspace=ws)
    for _ in range(3):
        c.out.fill_(7.0)
        g.replay()
        c.check(out, ref)
    # the replayed graph follows new lengths in its buffers
    c.lens[0] -= 9
    c.lens_t.sub_(torch.tensor([9, 0], dtype=torch.int32, device="cuda"))
    ref = c.reference()
    c.out.fill_(7.0)
    g.replay()
    c.check(out, ref)


def test_refusals():
    c = Case([5], [2], 2, seed=15)
    bad = lambda want, **kw: _refused(want, c, **kw)
    bad(TypeError, q=c.q.float())
    bad(ValueError, k=c.k[:, :, :1])
    bad(ValueError, lens=c.lens_t.cpu())
    bad(TypeError, lens=c.lens_t.long())
    bad(ValueError, parents=c.parents_t[:, :1])
    bad(ValueError, v_cache=c.vc.transpose(1, 2).contiguous().transpose(1, 2))
    bad(SpecVerifyError, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    bad(SpecVerifyError, scale=math.nan)
    bad(SpecVerifyError, q=c.q[:, :, :7], out=c.out[:, :, :7])        # 7 query heads, 2 key heads
    odd = torch.zeros(4, 24, 2, 128, dtype=c.dtype, device="cuda")    # page of 24 rows
    bad(SpecVerifyError, k_cache=odd, v_cache=odd.clone())


def _refused(want, c, **kw):
    args = dict(q=c.q, k=c.k, v=c.v, k_cache=c.kc, v_cache=c.vc, page_table=c.table, lens=c.lens_t,
                parents=c.parents_t, counts=c.counts_t, out=c.out)
    args.update(kw)
    if "q" in kw and "out" not in kw:
        args["out"] = None
    with pytest.raises(want):
        tree.tree_attention(**args)


@pytest.mark.parametrize("what", ["v", "k", "q"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_node_that_is_not_finite_harms_only_those_that_see_it(what, bad):
    """Node 2's descendants and itself (for q: itself) are unspecified; every other node is what it is without it."""
    for lens, N, g in (([120, 30], 20, 4), ([128, 1], 90, 3)):
        c = Case(lens, [N, N], N, g=g, seed=16)
        ref, tol = c.reference()
        getattr(c, what)[:, 2] = bad
        out = c.run()
        torch.cuda.synchronize()
        for b in range(2):
            for i in range(N):
                if i == 2 or (what != "q" and 2 in ancestors(c.parents[b], i)):
                    continue
                assert bool(((out[b, i].double() - ref[b, i]).abs() <= tol[b, i]).all()), (b, i)


@pytest.mark.parametrize("scale", [-0.125, 0.0, -2.0])
def test_scales_of_either_sign_in_wide_trees(scale):
    c = Case([130, 256, 0], [64, 40, 64], 64, g=4, width=3, seed=17)
    c.scale = scale
    c.check(c.run(scale=scale))


def test_no_requests():
    c = Case([5], [2], 2, seed=18)
    none = lambda x: x[:0].contiguous()
    out = tree.tree_attention(none(c.q), none(c.k), none(c.v), c.kc, c.vc, none(c.table), none(c.lens_t))
    assert out.shape == (0,) + c.q.shape[1:]


def test_a_call_s_own_tensors_on_another_stream():
    """Output and workspace made by the call, used on `stream`, are not given
    to later work of the current stream while the call may still run."""
    c = Case([4000, 3000], [9, 9], 9, page=64, seed=19)
    ref = c.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):
        outs.append(c.run(stream=side, out=None))
        torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda")   # would land in the workspace's place
    side.synchronize()
    for out in outs:
        c.check(out, ref)


def test_a_call_on_another_stream_is_not_given_memory_that_the_current_stream_still_writes():
    """Blocks of exactly the output's and the workspace's size are let go while
    long work on them is pending on the current stream; the call on the other
    stream, whose inputs are ready, runs meanwhile."""
    c = Case([900, 300], [9, 9], 9, page=64, seed=21)
    ref = c.reference()
    n = tree.tree_attention_workspace_bytes(c.q, c.k, c.v, c.kc, c.vc, c.table)
    side = torch.cuda.Stream()
    c.run(stream=side, out=None)         # all is loaded
    torch.cuda.synchronize()
    for _ in range(3):
        pending = [torch.empty(c.q.shape, dtype=c.dtype, device="cuda"),
                   torch.empty((n + 1) // 2, dtype=c.dtype, device="cuda")]
        for _ in range(300):
            for x in pending:
                x.fill_(3.0)
        del x, pending
        out = c.run(stream=side, out=None)
        torch.cuda.synchronize()
        c.check(out, ref)


class ExactCase(Case):
    """Queries and keys are whole numbers up to `most` times a power of two each,
    so that every q.k is exact in 32 bits (and some are equal); so is the scale."""

    def __init__(self, *args, most=8, scale=1.0, q_unit=1.0, k_unit=1.0, **kw):
        super().__init__(*args, **kw)
        whole = lambda x: (x.float() * most / 2).round().clamp(-most, most).to(x.dtype)
        for x, unit in ((self.q, q_unit), (self.k, k_unit), (self.kc, k_unit)):   # (NaN stays)
            x.copy_(whole(x) * unit)
        self.scale = scale

    def shift(self, at, q0, k0):
        """The first component: q0 in every query, k0 in the keys of cached rows `at` on (the new ones with them)."""
        self.q[..., 0], self.k[..., 0] = q0, k0
        for b, n in enumerate(self.lens):
            for t in range(n):
                self.kc[int(self.table[b, t // self.page]), t % self.page, :, 0] = k0 if t >= at else 0.0

    def reference(self):
        out, A = attention(self.q, self.k, self.v, self.lens, self.counts, self.parents, self.rows_of, self.scale)
        vmax = max(float(x.nan_to_num().abs().max()) for x in (self.vc, self.v))
        return out, exact_score_tolerance(out.nan_to_num(), A.nan_to_num(), self.dtype, max(self.lens) + self.N, vmax)

    def run(self, **kw):
        return super().run(scale=self.scale, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,g", [(128, 4), (64, 7)])
@pytest.mark.parametrize("scale", [2.0 ** -6, 2.0 ** -3, -2.0 ** -3, 1.0, 4.0])
def test_exact_scores_from_flat_to_one_hot(dtype, D, g, scale):
    # scores up to some thousands; with the larger scales the maximum is nearly everything, and moves all the time
    c = ExactCase([700, 64, 2900], [6, 3, 5], 6, g=g, D=D, dtype=dtype, scale=scale, page=32, seed=22)
    out, tol = c.reference()
    c.check(ref=(out, tol))
    # the tolerance tells these from the answer
    c.scale = scale * 17 / 16
    other = c.reference()[0]
    for b, m in enumerate(c.counts):
        assert bool((out[b, :m].abs() > tol[b, :m]).any())
        if abs(scale) < 1:
            assert bool(((other - out)[b, :m].abs() > tol[b, :m]).any())


@pytest.mark.parametrize("dtype,q_unit,k_unit,scale", [
    (torch.bfloat16, 2.0 ** 10, 2.0 ** 10, 0.125), (torch.bfloat16, 2.0 ** 12, 2.0 ** 12, 1.0),
    (torch.bfloat16, 2.0 ** 20, 2.0 ** 20, -1.0), (torch.bfloat16, 2.0 ** 45, 2.0 ** 45, 0.125),
    (torch.bfloat16, 2.0 ** -20, 2.0 ** 60, 2.0 ** 60), (torch.float16, 2.0 ** 11, 2.0 ** 11, 0.125),
    (torch.float16, 2.0 ** 11, 2.0 ** 11, 4.0), (torch.float16, 2.0 ** 11, 2.0 ** 11, -2.0 ** 60)])
@pytest.mark.parametrize("N,g,lens", [(6, 4, [700, 64, 2900]), (64, 4, [130, 300, 0])])
def test_scores_past_what_32_bits_hold_to_a_whole_number(dtype, q_unit, k_unit, scale, N, g, lens):
    """Finite queries and keys whose scores are so large that the step of a
    32-bit score is worth many powers of two: the largest scores take all, in
    equal shares."""
    ExactCase(lens, [N, N - 1, (N + 1) // 2], N, g=g, dtype=dtype, scale=scale, q_unit=q_unit, k_unit=k_unit, page=16,
              seed=23).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k0", [2.0 ** 11, -2.0 ** 11])
@pytest.mark.parametrize("scale,at", [(0.125, 0), (0.5, 0), (2.0, 0), (2.0, 500), (4.0, 0), (4.0, 300)])
def test_small_differences_between_large_scores(dtype, k0, scale, at):
    """Scores 2^23 and up (or down) from nothing, or from cached row `at` on,
    that differ by a few whole numbers."""
    c = ExactCase([700, 64, 1900], [6, 3, 5], 6, dtype=dtype, scale=scale, most=1, page=16, seed=24)
    c.shift(at, 2.0 ** 12, k0)
    c.check()


@pytest.mark.parametrize("g,D", [(4, 128), (1, 64)])
def test_prompts_fill_the_cache_in_chains(g, D):
    """Prompts of 600, 256 and 17 tokens, 256 a call, give what one look at all
    earlier tokens gives."""
    total, N = [600, 256, 17], 256
    whole = Case([0, 0, 0], [t if t <= N else N for t in total], N, g=g, D=D, page=16, chain=True, seed=25)
    gen = torch.Generator("cuda").manual_seed(26)
    rand = lambda h: torch.randn(3, 600, h, D, generator=gen, device="cuda").to(whole.dtype)
    q, k, v = rand(whole.Hq), rand(whole.Hkv), rand(whole.Hkv)
    pages = [-(-t // 16) for t in total]
    table = torch.full((3, max(pages)), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(sum(pages), generator=gen, device="cuda").int()
    for b in range(3):
        table[b, :pages[b]] = ids[sum(pages[:b]):sum(pages[:b + 1])]
    kc, vc = (torch.full((sum(pages), 16, whole.Hkv, D), math.nan, dtype=whole.dtype, device="cuda") for _ in range(2))
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = []
    for at in range(0, 600, N):
        counts = torch.tensor([min(max(t - at, 0), N) for t in total], dtype=torch.int32, device="cuda")
        part = lambda x: torch.nn.functional.pad(x[:, at:at + N], (0, 0, 0, 0, 0, max(0, at + N - 600))).contiguous()
        got.append(tree.tree_attention(part(q), part(k), part(v), kc, vc, table, lens, counts=counts))
        lens += counts
    got = torch.cat(got, 1)
    for b, t in enumerate(total):
        none = lambda b, n: (k[b, :0], v[b, :0])
        chain = [list(range(-1, t - 1))]
        out, A = attention(q[b:b + 1, :t], k[b:b + 1, :t], v[b:b + 1, :t], [0], [t], chain, none, D ** -0.5)
        tol = attention_tolerance(q[b:b + 1, :t], float(k[b, :t].double().abs().max()), out, A, whole.dtype, D ** -0.5)
        assert bool(((got[b:b + 1, :t].double() - out).abs() <= tol).all())
        rows = lambda c: c[table[b, :pages[b]].long()].flatten(0, 1)[:t]
        assert torch.equal(rows(kc), k[b, :t]) and torch.equal(rows(vc), v[b, :t])
