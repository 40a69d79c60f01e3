"""tree_verify against the rule written out in 64 bits: whole numbers, so
every answer has to be equal."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_92_b200 as sv
from speculative_decoding_verification_92_b200 import tree
from speculative_decoding_verification_92_b200.workload import make_workload
from helpers import device_inputs
from tree_reference import make_parents, verify

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, N, V, dtype="f32", draft=False, T=1.0, greedy=False, width=None, seed=0, counts=None,
                 boost=6.0, pad=0, noise=0.5, repeat=False):
        rng = np.random.default_rng(seed)
        self.T, self.greedy, self.V = T, greedy, V
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.parents = np.array([make_parents(rng, N, width) for _ in range(B)], np.int32)
        self.counts = np.array(counts if counts is not None else rng.integers(1, N + 1, B), np.int32)
        z = rng.standard_normal((B, N, V + pad)).astype(np.float32)
        y = z + noise * rng.standard_normal(z.shape).astype(np.float32)
        self.tokens = rng.integers(0, V, (B, N)).astype(np.int32)
        if repeat:                       # few tokens, so that siblings repeat
            self.tokens %= 3
        for b in range(B):
            for i in range(1, N):        # drafted tokens are likely under their parent
                z[b, self.parents[b, i], self.tokens[b, i]] += boost * rng.random()
        z[..., V:] = y[..., V:] = np.nan
        self.z = torch.from_numpy(z).to(dt).cuda()
        self.y = torch.from_numpy(y).to(dt).cuda() if draft else None
        self.u = rng.random((B, N), dtype=np.float32)

    def tensors(self):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return self.z, self.y, c(self.tokens), c(self.parents), c(self.counts), c(self.u)

    def run(self, **kw):
        got = tree.tree_verify(*self.tensors(), self.T, self.greedy, V=self.V, **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in got]

    def check(self, got=None):
        host = lambda x: None if x is None else x[..., :self.V].float().cpu().numpy()
        want = verify(host(self.z), host(self.y), self.tokens, self.parents, self.counts, self.u, self.T, self.greedy)
        got = self.run() if got is None else got
        for g, w in zip(got, want):
            assert np.array_equal(g, w), np.flatnonzero((g != w).reshape(len(g), -1).any(1))
        return want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["ids", "draft", "greedy"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 255, 256, 257, 1000, 4099, 20000])
def test_vocabularies(dtype, mode, V):
    Case(9, 6, V, dtype, draft=mode == "draft", greedy=mode == "greedy", seed=V).check()


@pytest.mark.parametrize("mode", ["ids", "draft", "greedy"])
@pytest.mark.parametrize("N,width", [(1, 1), (2, 1), (9, 1), (13, 3), (64, 2), (33, None), (40, 39), (256, None)])
def test_trees(mode, N, width):
    Case(8, N, 600, draft=mode == "draft", greedy=mode == "greedy", width=width, seed=N, boost=8.0).check()


@pytest.mark.parametrize("B", [1, 2, 3, 9, 19, 40, 80, 160, 400])
def test_batches_take_every_cluster_size(B):
    Case(B, 5, 30011, "bf16", seed=B, boost=12.0).check()


@pytest.mark.parametrize("B", [3, 40, 300])
@pytest.mark.parametrize("draft", [False, True])
def test_deep_walks(B, draft):
    want = Case(B, 12, 3000, "bf16", draft=draft, seed=B, boost=20.0, width=1, counts=[12] * B).check()
    assert want[0].max() >= 2            # the walks go down some levels


@pytest.mark.parametrize("B,V,dtype", [(1, 151936, "bf16"), (5, 128256, "f32")])
@pytest.mark.parametrize("draft", [False, True])
def test_full_vocabularies(B, V, dtype, draft):
    Case(B, 7, V, dtype, draft=draft, seed=B, boost=14.0, width=2, noise=0.2).check()


def test_largest_vocabulary():
    Case(1, 2, sv.MAX_V, "bf16", draft=True, seed=1, counts=[2], noise=0.1).check()


@pytest.mark.parametrize("T", [0.05, 0.6, 1.3, 50.0])
@pytest.mark.parametrize("draft", [False, True])
def test_temperatures(T, draft):
    Case(16, 7, 3001, "bf16", draft=draft, T=T, seed=2, width=3).check()


@pytest.mark.parametrize("V,pad", [(1000, 24), (1001, 7), (997, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_rows_with_nan_behind_the_vocabulary(V, pad, dtype):
    Case(6, 5, V, dtype, draft=True, pad=pad, seed=V + pad).check()


def test_unaligned_rows():
    c = Case(6, 5, 1001, "bf16", draft=True, seed=3)
    flat = torch.empty(c.z.numel() + 1, dtype=c.z.dtype, device="cuda")[1:].view(c.z.shape)
    flat.copy_(c.z)
    c.z = flat
    c.check()


@pytest.mark.parametrize("draft", [False, True])
def test_repeated_siblings(draft):
    Case(64, 24, 50, draft=draft, width=6, repeat=True, seed=4, boost=4.0).check()


@pytest.mark.parametrize("greedy", [False, True])
def test_minus_infinity_is_no_probability(greedy):
    c = Case(24, 9, 400, greedy=greedy, seed=5, width=3, boost=3.0)
    c.z[:, :, 5::2] = -float("inf")
    c.z[:, :, 0] = -1.0e38
    c.check()


def test_truncated_draft():
    c = Case(24, 9, 400, draft=True, seed=6, width=3)
    c.y[:, :, 40:] = -float("inf")       # drafted tokens there have q = 0: accepted if p > 0
    c.check()


def test_peaked_rows_leave_residuals_without_cancellation():
    # children that hold nearly all of the mass: what is left is some 1e-9 of it
    c = Case(64, 4, 3000, seed=7, width=3, counts=[4] * 64, boost=0.0)
    for b in range(64):
        c.z[b, 0, torch.from_numpy(c.tokens[b, 1:4]).long()] += 28.0
    c.u[:, 1:] = np.float32(1 - 2.0 ** -24)
    c.check()


@pytest.mark.parametrize("u", [0.0, 1 - 2.0 ** -24])
@pytest.mark.parametrize("draft", [False, True])
def test_extreme_uniforms(u, draft):
    c = Case(12, 5, 333, draft=draft, seed=8)
    c.u[:] = np.float32(u)
    c.check()


def test_equal_draft_and_target_accept_everything():
    c = Case(12, 6, 500, draft=True, seed=9, width=1, counts=[6] * 12)
    c.y = c.z.clone()
    c.u[:] = np.float32(1 - 2.0 ** -24)
    want = c.check()
    assert (want[0] == 5).all()


@pytest.mark.parametrize("ties", [2, 7])
def test_greedy_ties_go_to_the_lowest_index(ties):
    c = Case(16, 5, 4097, "bf16", greedy=True, seed=10)
    c.z = (c.z * 0.5).round().clamp(max=ties).to(torch.bfloat16)
    c.check()


def test_idle_and_invalid_requests():
    c = Case(8, 6, 100, seed=11, counts=[6, 0, 7, -1, 6, 6, 6, 3])
    c.parents[4, 2] = 2
    c.tokens[5, 3] = 100
    c.tokens[6, 1] = -1
    c.parents[7, 4] = 9                  # behind the count: not looked at
    c.tokens[7, 5] = -5
    want = c.check()
    assert list(want[0][1:7]) == [0, -1, -1, -1, -1, -1]


def test_rows_off_the_path_are_not_read():
    c = Case(20, 12, 300, draft=True, seed=12, counts=[12] * 20, boost=10.0)
    got = c.run()
    on = np.zeros((20, 12), bool)
    for b in range(20):
        on[b, got[2][b][got[2][b] >= 0]] = True
    off = torch.from_numpy(~on).cuda()
    c.z[off] = float("nan")
    c.y[off] = float("nan")
    again = c.run()
    for a, b in zip(got, again):
        assert np.array_equal(a, b)


def test_a_chain_is_spec_verify():
    # the chain form with one-hot drafts: the same rule, the uniforms one slot on
    w = make_workload(B=32, k_max=6, V=5000, dtype="f32", seed=13, boost=9.0, draft_mode="ids", fav_prob=0.9)
    d = device_inputs(w)
    n0, t0 = sv.spec_verify(d["target"], None, d["tokens"], None, d["uniforms"], 1.0)
    tokens = torch.cat([torch.zeros_like(d["tokens"][:, :1]), d["tokens"]], 1).contiguous()
    u = d["uniforms"].roll(1, 1).contiguous()
    n1, t1, path = tree.tree_verify(d["target"], None, tokens, None, None, u)
    torch.cuda.synchronize()
    # 32-bit sums there, 64-bit sums here: away from near ties they agree
    same = (n0 == n1) & (t0 == t1).all(1)
    assert same.float().mean() > 0.95
    ref = torch.arange(7, device="cuda").expand(32, 7)
    assert torch.equal(path, torch.where(ref <= n1[:, None], ref, -1).int())


@pytest.mark.parametrize("draft", [False, True])
def test_first_token_follows_the_target(draft):
    """Losslessness: over many uniforms the first emitted token has the
    target's distribution, whatever was drafted."""
    rng = np.random.default_rng(14)
    V, n = 6, 60000
    z = rng.standard_normal(V).astype(np.float32) * 1.5
    y = rng.standard_normal(V).astype(np.float32)
    q = np.exp(y) / np.exp(y).sum()
    tokens = np.zeros((n, 4), np.int32)
    tokens[:, 1:] = rng.choice(V, (n, 3), p=q) if draft else [2, 0, 4]
    parents = np.tile(np.array([-1, 0, 0, 0], np.int32), (n, 1))
    c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    zt = c(z).expand(n, 4, V).contiguous()
    yt = c(y).expand(n, 4, V).contiguous() if draft else None
    u = c(rng.random((n, 4), dtype=np.float32))
    _, out, _ = tree.tree_verify(zt, yt, c(tokens), c(parents), None, u)
    seen = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    p = np.exp(z) / np.exp(z).sum()
    chi2 = ((seen - n * p) ** 2 / (n * p)).sum()
    assert chi2 < 25.7                   # 5 degrees of freedom, 1 in 10^4


def test_on_a_side_stream_and_in_a_graph():
    c = Case(8, 9, 5000, "bf16", draft=True, seed=15, width=2)
    side = torch.cuda.Stream()
    t = c.tensors()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tree.tree_verify(*t, c.T, V=c.V)
    side.synchronize()
    c.check([x.cpu().numpy() for x in got])
    g = torch.cuda.CUDAGraph()
    out = tuple(torch.zeros_like(x) for x in got)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        tree.tree_verify(*t, c.T, V=c.V, out=out)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        c.check([x.cpu().numpy() for x in out])


def test_refusals():
    c = Case(2, 3, 50, seed=16)
    z, _, tok, par, cnt, u = c.tensors()
    for want, args in [
        (ValueError, (z[0], None, tok, par, cnt, u)), (ValueError, (z, z[:, :2], tok, par, cnt, u)),
        (TypeError, (z, z.bfloat16(), tok, par, cnt, u)), (TypeError, (z.half(), None, tok, par, cnt, u)),
        (TypeError, (z, None, tok.long(), par, cnt, u)), (ValueError, (z, None, tok, par[:1], cnt, u)),
        (ValueError, (z, None, tok, par, cnt.cpu(), u)), (TypeError, (z, None, tok, par, cnt, u.double())),
        (sv.SpecVerifyError, (z, None, tok, par, cnt, None)), (sv.SpecVerifyError, (z, None, tok, par, cnt, u, 0.0)),
        (sv.SpecVerifyError, (z, None, tok, par, cnt, u, float("nan")))]:
        with pytest.raises(want):
            tree.tree_verify(*args)


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("draft", [False, True])
def test_rows_that_are_not_finite_stay_in_bounds(fill, draft, greedy):
    """Unspecified results, but a length, tokens and nodes that exist."""
    B, N, V = 6, 7, 1000
    gen = torch.Generator("cuda").manual_seed(9)
    z = torch.randn(B, N, V, generator=gen, device="cuda")
    y = torch.randn(B, N, V, generator=gen, device="cuda") if draft else None
    z[0] = fill
    z[1, :, ::3] = fill
    z[2, :, 5] = fill
    if draft:
        y[3] = fill
        y[4, :, 7] = fill
        y[0] = fill
    tokens = torch.randint(0, V, (B, N), generator=gen, device="cuda", dtype=torch.int32)
    u = torch.rand(B, N, generator=gen, device="cuda")
    n, tok, path = (x.cpu() for x in tree.tree_verify(z, y, tokens, None, None, u, 1.0, greedy))
    for b in range(B):
        j = int(n[b])
        assert 0 <= j < N and bool(((tok[b, :j + 1] >= 0) & (tok[b, :j + 1] < V)).all())
        assert bool((tok[b, j + 1:] == -1).all()) and path[b, :j + 1].tolist() == list(range(j + 1))


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_requests_with_more_logits_than_l2_holds(dtype, draft):
    N = 70 if dtype == "f32" else 140
    Case(3, N, 160001, dtype=dtype, draft=draft, width=1, boost=14.0, pad=7, seed=21).check()
    Case(2, N + 60, 160000, dtype=dtype, draft=draft, width=2, boost=14.0, seed=22).check()


def test_no_requests():
    e = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device="cuda")
    n, tok, path = tree.tree_verify(e(0, 3, 9, dt=torch.float32), None, e(0, 3), None, None, e(0, 3, dt=torch.float32))
    assert n.shape == (0,) and tok.shape == path.shape == (0, 3)


@pytest.mark.parametrize("T", [1e-9, 2e-9, 5e-9, 2e-8, 1e-7])
@pytest.mark.parametrize("mode", ["leaf", "ids", "draft"])
@pytest.mark.parametrize("top", [20.0, 30.0, 100.0, -20.0])
def test_tiny_temperatures(T, mode, top):
    """Logits one float apart lie thousands of powers of two apart (or, at the
    largest T and the smallest logits, a few): a leaf and rejections take the
    likeliest tokens, whatever stands right below them."""
    B, N, V = 8, 3, 2000
    c = Case(B, N, V, draft=mode == "draft", T=T, seed=23, width=2, counts=[1 if mode == "leaf" else N] * B)
    top = np.float32(top)
    below = [np.nextafter(top, np.float32(-np.inf))]
    below.append(np.nextafter(below[0], np.float32(-np.inf)))
    rng = np.random.default_rng(24)
    likely = np.array([5, 40, 1300])     # the target's, the first of them where a leaf takes its reference
    z = rng.choice(np.array([below[0], below[1], top - 1, top - 7], np.float32), (B, N, V))
    z[..., likely] = top
    if mode == "draft":                  # the draft's two likely tokens have no probability under the target
        y = rng.choice(np.array([top - 1, top - 7], np.float32), (B, N, V))
        y[..., [300, 301]] = top
        z[..., [300, 301]] = top - 7
        c.y = torch.from_numpy(y).cuda()
        c.tokens[:, 1:] = rng.choice([300, 301], (B, N - 1))
    else:
        c.tokens[:, 1:] = [300, 7]       # no probability, and (at times) the reference's neighbour
        z[..., 300] = top - 7
    c.z = torch.from_numpy(z).cuda()
    c.u[:, 1:] = np.float32(0.5)
    c.u[:, 0] = np.linspace(0.02, 0.98, B, dtype=np.float32)
    want = c.check()
    assert (want[0] == 0).all()          # (1e-6 and less of the mass is theirs)
    if T <= 5e-9:
        assert np.isin(want[1][:, 0], likely).all()
