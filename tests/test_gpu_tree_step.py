"""tree.TreeStep: pages, attention, verification and compaction run together,
as a decoding loop runs them, against the plain forms on copies of the state."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_92_b200 import SpecVerifyError, cache, host, tree
from tree_reference import attention, attention_tolerance, commit, make_parents, resize, verify

pytestmark = pytest.mark.gpu

L, HKV, G, D, PAGE, V = 2, 2, 4, 64, 16, 500


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def state(lens, max_pages, spare, seed=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // PAGE) for n in lens]
    P = sum(need) + spare
    perm = rng.permutation(P).tolist()
    table, ref = np.full((len(lens), max_pages), -1, np.int32), np.zeros(P, np.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = perm.pop()
            ref[table[b, i]] = 1
    gen = torch.Generator("cuda").manual_seed(seed)
    kv = [torch.randn(L, P, PAGE, HKV, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    return kv[0], kv[1], i32(table), i32(lens), i32(ref)


def problem(rng, B, N, counts, mode):
    """One step's inputs: a tree per slot whose tokens the target often agrees with."""
    parents = np.array([make_parents(rng, N) for _ in range(B)], np.int32)
    target = rng.normal(size=(B, N, V)).astype(np.float32)
    draft = target + 0.3 * rng.normal(size=(B, N, V)).astype(np.float32) if mode == "draft" else None
    tokens = rng.integers(0, V, (B, N)).astype(np.int32)
    for b in range(B):
        for i in range(1, N):
            if rng.random() < 0.7:
                tokens[b, i] = target[b, parents[b, i]].argmax()
            target[b, parents[b, i], tokens[b, i]] += 4.0
    u = rng.random((B, N)).astype(np.float32)
    q, k, v = (torch.from_numpy(rng.normal(size=(L, B, N, h, D)).astype(np.float32)).cuda().bfloat16()
               for h in (HKV * G, HKV, HKV))
    return dict(parents=parents, counts=np.asarray(counts, np.int32), target=target, draft=draft, tokens=tokens, u=u,
                q=q, k=k, v=v)


def take(step, p, mode):
    """One step through the framework."""
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()
    status = step.begin(dev(p["parents"]), dev(p["counts"]))
    outs = [step.attention(x, p["q"][x], p["k"][x], p["v"][x]) for x in range(L)]
    return (status, outs) + tuple(step.finish(dev(p["target"]), dev(p["draft"]), dev(p["tokens"]), dev(p["u"]), 0.8,
                                              mode == "greedy"))


def as_np(x):
    return x.float().cpu().numpy()


def check_step(step, p, mode):
    k0, v0 = step.k_cache.clone(), step.v_cache.clone()
    table, lens, ref = (x.cpu().numpy() for x in (step.page_table, step.lens, step.refcount))
    got = take(step, p, mode)
    torch.cuda.synchronize()
    # pages
    table, ref, status = resize(table, lens + p["counts"], ref, PAGE)
    assert np.array_equal(got[0].cpu().numpy(), status)
    counts = np.where(status < 0, 0, p["counts"])
    # attention, layer by layer
    B, N = p["parents"].shape
    for x in range(L):
        def rows_of(b, n):
            ids = torch.from_numpy(table[b, :-(-n // PAGE)]).cuda().long()
            return tuple(c[x][ids].reshape(-1, HKV, D)[:n] for c in (k0, v0))
        want, A = attention(p["q"][x], p["k"][x], p["v"][x], lens, counts, p["parents"].tolist(), rows_of, D ** -0.5)
        kmax = max(float(k0[x].abs().max()), float(p["k"].abs().max()))
        tol = attention_tolerance(p["q"][x], kmax, torch.nan_to_num(want), torch.nan_to_num(A), torch.bfloat16, D ** -0.5)
        for b in range(B):
            m = int(counts[b])
            assert bool(((got[1][x][b, :m].double() - want[b, :m]).abs() <= tol[b, :m]).all())
            for i in range(m):
                t = int(lens[b]) + i
                k0[x, table[b, t // PAGE], t % PAGE] = p["k"][x, b, i]
                v0[x, table[b, t // PAGE], t % PAGE] = p["v"][x, b, i]
    # verification, compaction, pages given back
    n, tok, path = verify(p["target"], p["draft"], p["tokens"], p["parents"], counts, p["u"], 0.8, mode == "greedy")
    for g, w in zip(got[2:], (n, tok, path)):
        assert np.array_equal(g.cpu().numpy(), w)
    kn, vn, new = commit(as_np(k0), as_np(v0), table, lens, path)
    assert np.array_equal(new, lens + np.where(counts > 0, n + 1, 0))
    table, ref, _ = resize(table, new, ref, PAGE)
    for g, w in ((step.lens, new), (step.page_table, table), (step.refcount, ref)):
        assert np.array_equal(g.cpu().numpy(), w)
    # every row that a slot still holds
    for b in range(B):
        for t in range(int(new[b])):
            at = int(table[b, t // PAGE]), t % PAGE
            assert np.array_equal(as_np(step.k_cache[:, at[0], at[1]]), kn[:, at[0], at[1]])
            assert np.array_equal(as_np(step.v_cache[:, at[0], at[1]]), vn[:, at[0], at[1]])
    return n


@pytest.mark.parametrize("mode", ["ids", "draft", "greedy"])
def test_a_decoding_loop(mode):
    rng = np.random.default_rng(3)
    N, lens = 9, [15, 0, 128, 40]
    step = tree.TreeStep(*state(lens, 12, 20), N, HKV * G)
    accepted = 0
    for counts in ([9, 9, 9, 9], [1, 9, 0, 5], [9, 2, 9, 9]):
        accepted += check_step(step, problem(rng, 4, N, counts, mode), mode).sum()
    assert accepted > 0


def test_slots_without_pages_sit_the_step_out():
    rng = np.random.default_rng(4)
    step = tree.TreeStep(*state([16, 16, 16], 12, 2), 17, HKV * G)
    p = problem(rng, 3, 17, [17, 2, 2], "ids")      # the first takes both free pages, the others miss one each
    check_step(step, p, "ids")
    assert step.status.tolist() == [0, -1, -1]
    check_step(step, problem(rng, 3, 17, [0, 2, 2], "ids"), "ids")


def test_counts_and_lengths_that_are_not_valid_change_nothing():
    rng = np.random.default_rng(5)
    step = tree.TreeStep(*state([17, 33, 20, 20], 12, 9), 4, HKV * G)
    step.lens[3] = -1
    before = [x.clone() for x in (step.k_cache, step.v_cache, step.page_table, step.lens, step.refcount)]
    p = problem(rng, 4, 4, [-1, -20, 5, 4], "ids")
    n = take(step, p, "ids")[2]
    assert n.tolist() == [-1, -1, -1, 0]
    for x, y in zip((step.k_cache, step.v_cache, step.page_table, step.lens, step.refcount), before):
        assert torch.equal(x, y)


def test_forked_slots_go_their_own_ways():
    """A prompt forked into three completions that share its full pages."""
    rng = np.random.default_rng(6)
    k, v, table, lens, ref = state([37, 0, 0], 12, 12)
    assert cache.cache_fork(k, v, table, lens, ref, i32([0, 0]), i32([1, 2])).tolist() == [0, 0]
    assert lens.tolist() == [37] * 3 and ref.max().item() == 3
    step = tree.TreeStep(k, v, table, lens, ref, 6, HKV * G)
    for _ in range(2):
        check_step(step, problem(rng, 3, 6, [6, 6, 6], "ids"), "ids")
    assert ref.max().item() == 3                     # the prompt's pages are still shared
    shared = table[0, :2].tolist()
    assert table[1, :2].tolist() == shared and table[2, :2].tolist() == shared


def test_captured_steps_are_eager_steps():
    """Two graphs (a step object each, in turn) replayed over several steps' inputs."""
    rng = np.random.default_rng(7)
    N, lens = 5, [30, 100]
    problems = [problem(rng, 2, N, [5, 4], "draft") for _ in range(4)]
    eager = tree.TreeStep(*state(lens, 12, 12), N, HKV * G)
    take(eager, problems[0], "draft")                # everything is loaded before a capture
    eager = [tree.TreeStep(*state(lens, 12, 12, s), N, HKV * G) for s in (0, 1)]
    steps = [tree.TreeStep(*state(lens, 12, 12, s), N, HKV * G) for s in (0, 1)]
    dev = lambda x: torch.from_numpy(x).cuda()
    static = {n: (dev(x) if isinstance(x, np.ndarray) else x.clone()) for n, x in problems[0].items()}
    graphs, results = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            s.begin(static["parents"], static["counts"])
            outs = [s.attention(x, static["q"][x], static["k"][x], static["v"][x]) for x in range(L)]
            results.append((outs, s.finish(static["target"], static["draft"], static["tokens"], static["u"], 0.8)))
        graphs.append(g)
    for p in problems:
        for n, x in p.items():
            static[n].copy_(dev(x) if isinstance(x, np.ndarray) else x)
        for i in (0, 1):
            graphs[i].replay()
        for i in (0, 1):
            want = take(eager[i], p, "draft")
            torch.cuda.synchronize()
            got = results[i]
            for a, b in zip(got[0], want[1]):
                for s in (0, 1):
                    assert torch.equal(a[s, :p["counts"][s]], b[s, :p["counts"][s]])
            for a, b in zip(got[1], want[2:]):
                assert torch.equal(a, b)
            for name in ("k_cache", "v_cache", "page_table", "lens", "refcount", "status"):
                assert torch.equal(getattr(steps[i], name), getattr(eager[i], name)), name


def test_a_tree_of_a_drafters_candidates():
    """The ngram drafter's chain with its other candidates for the first token
    as siblings, verified greedily: the candidate that the target takes is found
    wherever it stands."""
    ng = host.NgramDrafter(max_n=3, window=2)
    ng.begin_step()
    for tail in ([7, 8, 9, 10], [7, 8, 9, 11], [20, 21, 22, 23], [30, 31, 32, 33]):
        ng.add(1, np.array([1, 2, 3] + tail, np.int32))
    ids, lens = ng.draft_batch([1], [np.array([5, 1, 2, 3], np.int32)], k_max=3)
    first = ng.candidates(1, np.array([5, 1, 2, 3], np.int32), 4)
    chain = ids[0][:lens[0]].tolist()
    others = [int(x) for x in first if x != chain[0]]
    tokens = [0] + chain + others
    parents = [-1] + list(range(len(chain))) + [0] * len(others)
    N = len(tokens)
    assert len(chain) >= 1 and len(others) >= 1
    for taken in [chain[0]] + others:
        step = tree.TreeStep(*state([20], 4, 3), N, HKV * G)
        target = np.full((1, N, V), -5.0, np.float32)
        target[0, :, 499] = 0.0                      # what follows everything else
        target[0, 0, taken] = 5.0
        p = problem(np.random.default_rng(8), 1, N, [N], "greedy")
        p.update(parents=np.array([parents], np.int32), tokens=np.array([tokens], np.int32), target=target)
        assert check_step(step, p, "greedy").tolist() == [1]
        assert step.lens.tolist() == [22]


def test_refusals():
    k, v, table, lens, ref = state([20, 30], 4, 3)
    for want, args in ((ValueError, (k[0], v[0], table, lens, ref, 4, 8)), (ValueError, (k, v, table, lens, ref, 0, 8)),
                       (ValueError, (k, v, table, lens, ref, 257, 8)), (ValueError, (k, v, table, lens, ref, 4, 7)),
                       (TypeError, (k, v, table, lens.long(), ref, 4, 8)),
                       (ValueError, (k, v[:, :, :8], table, lens, ref, 4, 8)),
                       (ValueError, (k.float(), v.float(), table, lens, ref, 4, 8))):
        with pytest.raises(want):
            tree.TreeStep(*args)
    step = tree.TreeStep(k, v, table, lens, ref, 4, 8)
    x = torch.zeros(2, 4, 8, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        step.attention(0, x, x[:, :, :2], x[:, :, :2])
    with pytest.raises(RuntimeError):
        step.finish(torch.zeros(2, 4, V, device="cuda"), None, i32(np.zeros((2, 4))), None, greedy=True)
    with pytest.raises(TypeError):
        step.begin(counts=lens.long())
    step.begin()
    with pytest.raises(ValueError):
        step.attention(0, x[:1], x[:1, :, :2], x[:1, :, :2])
    with pytest.raises(IndexError):
        step.attention(2, x, x[:, :, :2], x[:, :, :2])


def test_a_step_takes_no_more_memory_than_it_keeps():
    k, v, table, lens, ref = state([0] * 64, 4, 8)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    step = tree.TreeStep(k, v, table, lens, ref, 256, 64 * HKV)
    kept = torch.cuda.memory_allocated() - before
    assert torch.cuda.max_memory_allocated() - before <= kept + (1 << 20)   # (as many queries alone are 268 MB)
    assert step.begin().tolist() == [-1] * 64


def test_a_pool_of_another_size_than_the_cache_is_refused():
    k, v, table, lens, ref = state([20, 30], 4, 3)
    for other in (torch.cat([ref, ref]), ref[:-1], ref[None]):
        with pytest.raises(ValueError):
            tree.TreeStep(k, v, table, lens, other, 4, 8)
    with pytest.raises(TypeError):
        tree.TreeStep(k, v, table, lens, ref.long(), 4, 8)
