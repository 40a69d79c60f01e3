"""What is measured of the tree operators: attention of a drafted token tree
over a paged cache, verification of the tree from given uniforms, compaction
of the cache to the accepted path, and forking of cached sequences.

``own`` selects the framework's kernels; otherwise the operators run in their
plain form, in elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # One request, one new token: plain decoding, where latency is all.
        dict(name="attend-one-token", op="attend", B=1, N=1, w=1, ctx=500, Hkv=8, g=4, D=128, page=16, dtype="bf16"),
        # A rollout batch verifying chains of 8 drafts (9 nodes with the root).
        dict(name="attend-chain-batch", op="attend", B=64, N=9, w=1, ctx=2000, Hkv=8, g=4, D=128, page=16, dtype="bf16"),
        # Long rollouts (8k to 16k tokens, batch 16) with a wide tree.
        dict(name="attend-tree-long", op="attend", B=16, N=64, w=3, ctx=16384, Hkv=8, g=4, D=128, page=64, dtype="bf16"),
        # Odd sizes: group of 7 heads, small head, ragged short contexts.
        dict(name="attend-tree-odd", op="attend", B=7, N=25, w=2, ctx=1501, Hkv=4, g=7, D=64, page=32, dtype="f16"),
        # Tiny sanity size of the verification workloads, with draft logits.
        dict(name="verify-tiny", op="verify", B=4, N=5, w=2, V=1000, dtype="f32", draft=True, T=1.0, greedy=False),
        # Model-free drafter (ids only), full vocabulary, candidate trees.
        dict(name="verify-ids-batch", op="verify", B=128, N=40, w=3, V=151936, dtype="bf16", draft=False, T=1.0, greedy=False),
        # Draft model with logits in 32 bits: siblings drawn from one row.
        dict(name="verify-draft-batch", op="verify", B=64, N=13, w=3, V=128256, dtype="f32", draft=True, T=1.0, greedy=False),
        # Few straggling requests, greedy decoding.
        dict(name="verify-greedy-few", op="verify", B=8, N=25, w=2, V=151936, dtype="bf16", draft=False, T=1.0, greedy=True),
        # Compaction after a step: two requests, few layers.
        dict(name="commit-small", op="commit", B=2, N=8, w=2, ctx=100, L=4, Hkv=2, D=64, page=16, dtype="bf16"),
        # Compaction after a step of a whole batch through 32 layers.
        dict(name="commit-batch", op="commit", B=64, N=40, w=3, ctx=200, L=32, Hkv=8, D=128, page=16, dtype="bf16"),
        # One prompt forked into four completions.
        dict(name="fork-small", op="fork", S=1, G=4, ctx=100, L=4, Hkv=2, D=64, page=16, dtype="bf16"),
        # Eight prompts forked into eight completions each.
        dict(name="fork-batch", op="fork", S=8, G=8, ctx=300, L=32, Hkv=8, D=128, page=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "verify", "commit", "fork"])
    if op == "attend":
        c = dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 64), w=rng.choice([1, 2, 3, 4]), ctx=_log(rng, 1, 16384),
                 Hkv=rng.choice([1, 2, 4, 5, 8]), g=rng.choice([1, 2, 4, 5, 7, 8]), D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "f16"]))
        while c["B"] > 1 and c["B"] * c["ctx"] * c["Hkv"] * max(1, c["N"] * c["g"] / 256) > 16 * 16384 * 8:
            c["B"] = (c["B"] + 1) // 2
    elif op == "verify":
        c = dict(op=op, B=_log(rng, 1, 200), N=_log(rng, 1, 64), w=rng.choice([1, 2, 3, 4]), V=_log(rng, 500, 151936),
                 dtype=rng.choice(["f32", "bf16"]), draft=rng.random() < 0.4, T=rng.choice([0.6, 1.0, 1.3]),
                 greedy=rng.random() < 0.2)
        c["draft"] = c["draft"] and not c["greedy"]
        es = 4 if c["dtype"] == "f32" else 2
        while c["B"] > 1 and c["B"] * c["N"] * c["V"] * (es + 4 * c["draft"]) > 10 ** 9:
            c["B"] = (c["B"] + 1) // 2
    elif op == "commit":
        c = dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 2, 40), w=rng.choice([1, 2, 3]), ctx=_log(rng, 1, 300),
                 L=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32]),
                 dtype=rng.choice(["bf16", "f16"]))
    else:
        c = dict(op=op, S=_log(rng, 1, 8), G=_log(rng, 1, 8), ctx=_log(rng, 1, 400), L=_log(rng, 1, 32),
                 Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32]),
                 dtype=rng.choice(["bf16", "f16"]))
    return c


# ---------------------------------------------------------------------------
# Shapes.  Node i's parent is (i - 1) // w: a chain for w = 1, else a w-ary
# tree in breadth-first order, so that any prefix of the nodes is a tree.


def _depth(n, w):
    d, i = 0, n - 1
    while i > 0:
        i, d = (i - 1) // w, d + 1
    return d


def _lens(c):
    """Cached lengths of the requests, known from the case alone: ragged, from
    a third of ctx to ctx (the first request has ctx)."""
    n = c.get("B") or c["S"]
    return [c["ctx"] - (i * 7919 * (c["ctx"] // 3 * 2 + 1) // 10007) % (c["ctx"] // 3 * 2 + 1) for i in range(n)]


def _counts(c):
    """Nodes of each request: mostly all N, every fourth request fewer."""
    return [c["N"] if b % 4 != 3 else max(1, c["N"] - 1 - (5 * b) % c["N"]) for b in range(c["B"])]


def _paths(c):
    """Accepted nodes of each request for the compaction: a walk from the root
    that stops after a while, as verification leaves it."""
    width = _depth(c["N"], c["w"]) + 1
    rows = []
    for b, n in enumerate(_counts(c)):
        row, i = [0], 0
        while len(row) < width and (b * 31 + len(row) * 17) % 5:
            i = i * c["w"] + 1 + (b + len(row)) % c["w"]
            if i >= n:
                break
            row.append(i)
        rows.append(row + [-1] * (width - len(row)))
    return rows


# Shares of the target's mass on the drafted candidates, by rank (log of the
# odds against the rest of the vocabulary), and how often a candidate is right.
ODDS = (0.9, -0.9, -1.9, -2.5)
HIT = 0.9


def _accept(c):
    """Expected chance that some child of an inner node is accepted."""
    if c["greedy"]:
        return HIT
    if c["draft"]:
        return 0.9 if c["w"] == 1 else 0.97
    mass = [math.exp(o) for o in ODDS]
    return HIT * sum(mass[:c["w"]]) / (1 + sum(mass))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    dev, dt = "cuda", DTYPES[c["dtype"]]
    i32 = dict(dtype=torch.int32, device=dev)

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    s = dict(c)
    if c["op"] == "verify":
        B, N, V, w = c["B"], c["N"], c["V"], c["w"]
        s["parents"] = torch.tensor([[-1] + [(i - 1) // w for i in range(1, N)]] * B, **i32)
        s["counts"] = torch.tensor(_counts(c), **i32)
        s["uniforms"] = torch.rand(B, N, generator=gen, device=dev)
        s["depth"], s["draft_logits"] = _depth(N, w), None
        # the target's candidates: a few likely tokens in every row
        spread = torch.arange(len(ODDS), device=dev) * (V // (len(ODDS) + 1) + 1)
        fav = (torch.randint(0, V, (B, N, 1), generator=gen, device=dev) + spread) % V
        boost = (torch.tensor(ODDS, device=dev) + math.log(V) + 0.5 / c["T"] ** 2) * c["T"]
        target = normal(B, N, V).scatter_(2, fav, boost.to(dt).expand(B, N, -1))
        tokens = torch.randint(0, V, (B, N), generator=gen, device=dev)
        if not c["draft"]:
            # a drafter that gives ids: the candidates, some of them wrong
            child = torch.arange(1, N, device=dev)
            right = torch.rand(B, N, generator=gen, device=dev)[:, 1:] < HIT
            tokens[:, 1:] = torch.where(right, fav[:, (child - 1) // w, (child - 1) % w], tokens[:, 1:])
        else:
            # a draft model near the target; a node's children are drawn from its row
            s["draft_logits"] = target + 0.2 * normal(B, N, V)
            inner = (N - 1 + w - 1) // w
            if inner:
                q = torch.softmax(s["draft_logits"][:, :inner].float() / c["T"], 2)
                x = torch.multinomial(q.reshape(-1, V), w, replacement=True, generator=gen).reshape(B, -1)
                tokens[:, 1:] = x[:, :N - 1]
        s["target"], s["tokens"] = target, tokens.to(torch.int32)
        return s

    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    lens = _lens(c)
    if c["op"] == "attend":
        B, N, w = c["B"], c["N"], c["w"]
        pages = [-(-(n + N) // page) for n in lens]
        s["counts"] = torch.tensor(_counts(c), **i32)
        s["parents"] = torch.tensor([[-1] + [(i - 1) // w for i in range(1, N)]] * B, **i32)
        s["q"] = normal(B, N, Hkv * c["g"], D)
        s["k"], s["v"] = normal(B, N, Hkv, D), normal(B, N, Hkv, D)
        s["out"] = torch.zeros_like(s["q"])
        P = sum(pages) + 3
        s["k_cache"], s["v_cache"] = normal(P, page, Hkv, D), normal(P, page, Hkv, D)
    elif c["op"] == "commit":
        pages = [-(-n // page) for n in lens]
        s["nodes"] = c["N"]
        P = sum(-(-(n + c["N"]) // page) for n in lens) + 5
        s["path"] = torch.tensor(_paths(c), **i32)
    else:
        S, G = c["S"], c["G"]
        pages = [-(-n // page) for n in lens] + [0] * (S * G)
        P = sum(pages) + S * G + 7
        s["src"] = torch.tensor([i for i in range(S) for _ in range(G)], **i32)
        s["dst"] = torch.tensor([S + i for i in range(S * G)], **i32)
        lens = lens + [0] * (S * G)
    if c["op"] != "attend":
        s["k_cache"], s["v_cache"] = (normal(c["L"], P, page, Hkv, D) for _ in range(2))
    most = max(pages) if c["op"] != "commit" else max(-(-(n + c["N"]) // page) for n in lens)
    ids = torch.randperm(P, generator=gen, device=dev).tolist()
    rows, ref = [], [0] * P
    for n in pages:
        row = [ids.pop() for _ in range(n)]
        for i in row:
            ref[i] = 1
        rows.append(row + [-1] * (most - n))
    s["table"], s["lens"], s["refcount"] = torch.tensor(rows, **i32), torch.tensor(lens, **i32), torch.tensor(ref, **i32)
    return s


def run(state):
    return {"attend": _attend, "verify": _verify, "commit": _commit, "fork": _fork}[state["op"]](state)


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "attend":
        kv = sum(n + m for n, m in zip(_lens(c), _counts(c)))
        rows = sum(_counts(c))
        row = c["Hkv"] * c["D"] * es
        pairs = sum(m * n + sum(_depth(i + 1, c["w"]) + 1 for i in range(m)) for n, m in zip(_lens(c), _counts(c)))
        return {"bytes": 2 * kv * row + 2 * rows * row + 2 * rows * row * c["g"],
                "flops": 4 * pairs * c["Hkv"] * c["g"] * c["D"]}
    if c["op"] == "verify":
        # the rows on the accepted path, as far as it goes on average
        a = _accept(c)
        rows = sum(sum(a ** d for d in range(_depth(n, c["w"]) + 1)) for n in _counts(c))
        both = 2 * rows - sum(a ** _depth(n, c["w"]) for n in _counts(c)) if c["draft"] else rows
        return {"bytes": both * c["V"] * es, "flops": 4 * both * c["V"]}
    row = 2 * c["L"] * c["Hkv"] * c["D"] * es
    if c["op"] == "commit":
        moved = sum(1 for r in _paths(c) for i, n in enumerate(r) if n > i)
        return {"bytes": 2 * moved * row + 4 * 4 * c["B"] * (c["N"] // c["page"] + 2), "flops": 0}
    ragged = sum(n % c["page"] for n in _lens(c))
    return {"bytes": ragged * row * (1 + c["G"]) + 4 * c["S"] * c["G"] * (c["ctx"] // c["page"] + 2), "flops": 0}


def exact(case, seed):
    if case["op"] != "attend":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    B, N, Hkv, g, D = s["B"], s["N"], s["Hkv"], s["g"], s["D"]
    out = torch.zeros(B, N, Hkv, g, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, m = int(s["lens"][b]), int(s["counts"][b])
        pages = s["table"][b, :-(-n // s["page"])].long()
        k, v = (torch.cat([x[pages].reshape(-1, Hkv, D)[:n], y[b, :m]]).double().transpose(0, 1)
                for x, y in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])))
        see = torch.zeros(m, n + m, dtype=torch.bool)
        see[:, :n] = True
        for i in range(m):
            j = i
            while j >= 0:
                see[i, n + j] = True
                j = (j - 1) // s["w"] if j else -1
        see = see.cuda()
        q = s["q"][b, :m].double().reshape(m, Hkv, g, D).permute(1, 2, 0, 3)
        x = torch.matmul(q, k.transpose(1, 2)[:, None]) / math.sqrt(D)
        p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
        out[b, :m] = torch.matmul(p, v[:, None]).permute(2, 0, 1, 3)
    return [out.reshape(B, N, Hkv * g, D), None, None]


# ---------------------------------------------------------------------------
# Attention: the nodes' keys and values go to the cache, then every node
# attends to the cached prefix and to its ancestors.


def _attend(s):
    if own:
        from speculative_decoding_verification_92_b200 import tree
        out = tree.tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                  s["parents"], s["counts"], out=s["out"])
        return [out, s["k_cache"], s["v_cache"]]
    B, N, Hkv, g, D, page = (s[x] for x in ("B", "N", "Hkv", "g", "D", "page"))
    dev = s["q"].device
    table, lens = s["table"].long(), s["lens"].long()
    node = torch.arange(N, device=dev)
    valid = node < s["counts"][:, None]
    pos = lens[:, None] + node
    at = table.gather(1, pos // page), pos % page
    for cached, new in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        cached[at] = torch.where(valid[..., None, None], new, cached[at])
    k, v = (x[table.clamp(min=0)].reshape(B, -1, Hkv, D).float().transpose(1, 2) for x in (s["k_cache"], s["v_cache"]))
    # ancestors: (1 - P)^-1 = 1 + P + P^2 + ..., P the parent matrix (0/1, exact)
    up = (s["parents"][..., None] == node).float()
    eye = torch.eye(N, device=dev).expand(B, N, N)
    anc = torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True) > 0.5
    t = torch.arange(k.shape[2], device=dev)
    rel = t - lens[:, None]
    in_tree = anc.gather(2, rel.clamp(0, N - 1)[:, None].expand(B, N, -1)) & ((rel >= 0) & (rel < N))[:, None]
    see = (rel < 0)[:, None] | in_tree
    q = s["q"].float().reshape(B, N, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * N, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).reshape(B, Hkv, g, N, -1)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(e.reshape(B, Hkv, g * N, -1), v).reshape(B, Hkv, g, N, D) / e.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hkv * g, D).to(s["q"].dtype)
    return [torch.where(valid[..., None, None], o, s["out"]), s["k_cache"], s["v_cache"]]


# ---------------------------------------------------------------------------
# Verification: all requests walk down their trees level by level.  In 64
# bits: the answers are whole numbers, next to borders of running sums.


def _verify(s):
    if own:
        from speculative_decoding_verification_92_b200 import tree
        return tree.tree_verify(s["target"], s["draft_logits"], s["tokens"], s["parents"], s["counts"], s["uniforms"],
                                s["T"], s["greedy"])
    B, N, V = s["B"], s["N"], s["V"]
    dev = s["target"].device
    every, node = torch.arange(B, device=dev), torch.arange(N, device=dev)
    tokens, valid = s["tokens"].long(), node < s["counts"][:, None]
    u = s["uniforms"].double()
    at = torch.zeros(B, dtype=torch.long, device=dev)
    path = torch.full((B, N), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0
    out = torch.full((B, N), -1, dtype=torch.long, device=dev)
    n = torch.zeros(B, dtype=torch.long, device=dev)
    live = torch.ones(B, dtype=torch.bool, device=dev)
    for level in range(s["depth"] + 1):
        child = (s["parents"] == at[:, None]) & valid
        z = s["target"][every, at]
        if s["greedy"]:
            last = z.argmax(1)
            ok = child & (tokens == last[:, None])
        else:
            p = torch.softmax(z.double() / s["T"], 1)
            px = p.gather(1, tokens)
            if s["draft_logits"] is None:
                # an earlier sibling with the same token has taken its mass
                same = (tokens[:, :, None] == tokens[:, None]) & child[:, None] & (node < node[:, None])
                px = px.masked_fill(same.any(2) | ~child, 0)
                ok = child & (u * (1 - (px.cumsum(1) - px)) < px)
                keep = torch.zeros(B, V, dtype=torch.int32, device=dev).scatter_add_(1, tokens, child.int()) == 0
                w = p * keep
            else:
                q = torch.softmax(s["draft_logits"][every, at].double() / s["T"], 1)
                qx, rank = q.gather(1, tokens), child.long().cumsum(1)
                lam, norm, ok, w = px.new_zeros(B, 1), px.new_ones(B, 1), torch.zeros_like(child), p
                for r in range(1, s["w"] + 1):
                    mine = child & (rank == r)
                    ok = ok | (mine & (u * norm * qx < (px - lam * qx).clamp(min=0)))
                    has = mine.any(1, keepdim=True)
                    lam = torch.where(has, lam + norm, lam)
                    w = torch.where(has, (p - lam * q).clamp(min=0), w)
                    norm = torch.where(has, w.sum(1, keepdim=True), norm)
            w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
            cdf = w.cumsum(1)
            last = (cdf <= u[:, :1] * cdf[:, -1:]).sum(1)
        first = torch.where(ok, node, N).amin(1)
        went = live & (first < N)
        stop = live & (first == N)
        to = first.clamp(max=N - 1)
        out[every, n] = torch.where(went, tokens[every, to], torch.where(stop, last, out[every, n]))
        n = n + went
        path[every, n] = torch.where(went, to, path[every, n])
        at = torch.where(went, to, at)
        live = went
    return tuple(x.to(torch.int32) for x in (n, out, path))


# ---------------------------------------------------------------------------
# The cache's pages.  table [slots, pages] of page ids (-1: none), refcount
# [pages].  New pages are the free ones with the lowest ids, in slot order.


def _resize(table, lens, ref, page):
    need = (lens + page - 1) // page
    idx = torch.arange(table.shape[1], device=table.device)
    drop = (idx >= need[:, None]) & (table >= 0)
    ref.index_add_(0, table.clamp(min=0).flatten(), -drop.int().flatten())
    table.masked_fill_(drop, -1)
    miss = (idx < need[:, None]) & (table < 0)
    fits = (miss.sum(1).cumsum(0) <= (ref == 0).sum()) | ~miss.any(1)
    take = miss & fits[:, None]
    free = torch.sort((ref != 0).int(), stable=True).indices
    ids = free[(take.flatten().cumsum(0) - 1).clamp(0, len(free) - 1)].reshape(table.shape).int()
    table.copy_(torch.where(take, ids, table))
    ref.index_add_(0, table.clamp(min=0).flatten(), take.int().flatten())
    return fits.int() - 1


def _commit(s):
    table, lens, ref, page, path = s["table"], s["lens"], s["refcount"], s["page"], s["path"]
    if own:
        from speculative_decoding_verification_92_b200 import cache
        first = cache.cache_resize(table, lens + s["nodes"], ref, page)
        new = cache.cache_commit(s["k_cache"], s["v_cache"], table, lens, path)
        second = cache.cache_resize(table, new, ref, page)
    else:
        first = _resize(table, lens + s["nodes"], ref, page)
        valid = path >= 0
        to = (lens[:, None] + torch.arange(path.shape[1], device=path.device)).long()
        come = torch.where(valid, lens[:, None] + path, to).long()
        ids = table.long()
        for x in (s["k_cache"], s["v_cache"]):
            x[:, ids.gather(1, to // page), to % page] = x[:, ids.gather(1, come // page), come % page]
        new = (lens + valid.sum(1)).int()
        second = _resize(table, new, ref, page)
    return [new, first, second, table, ref, s["k_cache"], s["v_cache"]]


def _fork(s):
    table, lens, ref, page = s["table"], s["lens"], s["refcount"], s["page"]
    if own:
        from speculative_decoding_verification_92_b200 import cache
        status = cache.cache_fork(s["k_cache"], s["v_cache"], table, lens, ref, s["src"], s["dst"])
    else:
        src, dst = s["src"].long(), s["dst"].long()
        old = table[dst]
        ref.index_add_(0, old.clamp(min=0).flatten(), -(old >= 0).int().flatten())
        full, rag = lens[src] // page, lens[src] % page
        idx = torch.arange(table.shape[1], device=table.device)
        share = idx < full[:, None]
        row = torch.where(share, table[src], -1)
        ref.index_add_(0, row.clamp(min=0).flatten(), share.int().flatten())
        # each ragged copy a free page of its own (the others, past them, stay as they are)
        free = torch.sort((ref != 0).int(), stable=True).indices
        rank = torch.sort((rag == 0).int(), stable=True).indices.argsort()
        ids = free[rank]
        row = torch.where((idx == full[:, None]) & (rag > 0)[:, None], ids[:, None].int(), row)
        come = table[src].long().gather(1, full.long()[:, None].clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0)
        keep = (torch.arange(page, device=table.device) < rag[:, None])[None, :, :, None, None]
        for x in (s["k_cache"], s["v_cache"]):
            x[:, ids] = torch.where(keep, x[:, come], x[:, ids])
        ref.index_add_(0, ids, (rag > 0).int())
        table[dst] = row
        lens[dst] = lens[src]
        status = torch.zeros_like(s["src"])
    return [status, table, lens, ref, s["k_cache"], s["v_cache"]]
