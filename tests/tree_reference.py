"""Plain 64-bit forms of the tree operators, written request by request from
their definitions, and generators of small trees."""
from __future__ import annotations

import math
from collections import deque

import numpy as np
import torch


def make_parents(rng, n, width=None):
    """Parents of n nodes: a chain (width 1), a complete tree, or any tree."""
    if width is None:
        return [-1] + [int(rng.integers(0, i)) for i in range(1, n)]
    return [-1] + [(i - 1) // width for i in range(1, n)]


def ancestors(parents, i):
    while i > 0:
        yield i
        i = parents[i]
    yield 0


# ---------------------------------------------------------------------------
# attention


def attention(q, k, v, lens, counts, parents, rows_of, scale):
    """(out, A) in float64: out [B, N, Hq, D] (NaN rows past the counts) and
    A = sum_t p_t |v_t|, which scales the rounding of p.  ``rows_of(b, n)``
    gives the first n cached keys and values of request b."""
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    out = torch.full((B, N, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    A = out.clone()
    for b in range(B):
        n, m = lens[b], counts[b]
        if m <= 0 or n < 0:
            continue
        kc, vc = rows_of(b, n)
        kk = torch.cat([kc, k[b, :m]]).double().repeat_interleave(Hq // Hkv, 1)
        vv = torch.cat([vc, v[b, :m]]).double().repeat_interleave(Hq // Hkv, 1)
        see = torch.zeros(m, n + m, dtype=torch.bool)
        see[:, :n] = True
        for i in range(m):
            see[i, [n + a for a in ancestors(parents[b], i)]] = True
        see = see.to(q.device)
        for i in range(m):
            t = see[i].nonzero()[:, 0]
            s = torch.einsum("hd,thd->ht", q[b, i].double(), kk[t]) * scale
            p = torch.softmax(s, 1)
            out[b, i] = torch.einsum("ht,thd->hd", p, vv[t])
            A[b, i] = torch.einsum("ht,thd->hd", p, vv[t].abs())
    return out, A


def attention_tolerance(q, kmax, out, A, dtype, scale):
    """Per element: half a step for rounding the result; the weights p are
    rounded to the cache's type before they meet v, and so is their sum
    (at most eps/2 each of A); scores are sums of D products in 32 bits, whose
    error e changes a weight by the factor exp(e) (twice: weight and sum), and
    2^-20 covers exp2, the running sums and their joining."""
    eps = torch.finfo(dtype).eps
    D = q.shape[-1]
    score = D * 2.0 ** -24 * q.double().abs().amax() * kmax * D * abs(scale)
    return eps / 2 * out.abs() + (eps + 2 * (float(score) + 2.0 ** -20)) * A


# ---------------------------------------------------------------------------
# verification, straight from the rule: the residual is renormalised after
# every rejection


def softmax(z, T):
    z = z.astype(np.float64) / T
    z = np.exp(z - z.max())
    return z / z.sum()


def draw(w, u):
    c = np.cumsum(w)
    return int(np.argmax(c > u * c[-1]))


def verify_one(target, draft, tokens, parents, count, uniforms, T, greedy):
    N, V = target.shape
    out, path = np.full(N, -1, np.int32), np.full(N, -1, np.int32)
    if count == 0:
        return 0, out, path
    if not 0 <= count <= N or any(not 0 <= parents[i] < i or not 0 <= tokens[i] < V for i in range(1, count)):
        return -1, out, path
    at, j = 0, 0
    path[0] = 0
    while True:
        kids = [i for i in range(1, count) if parents[i] == at]
        went = None
        if greedy:
            last = int(np.argmax(target[at]))
            went = next((i for i in kids if tokens[i] == last), None)
        else:
            full = p = softmax(target[at], T)
            for i in kids:
                if draft is None:
                    q = np.zeros(V)
                    q[tokens[i]] = 1.0
                else:
                    q = softmax(draft[at], T)
                x = tokens[i]
                if float(uniforms[i]) * q[x] < p[x]:
                    went = i
                    break
                r = np.maximum(0.0, p - q)
                if draft is None:      # a point mass takes all that the token had
                    r = p.copy()
                    r[x] = 0.0
                if r.sum() <= 0:
                    r = full
                p = r / r.sum()
            if went is None:
                last = draw(p, float(uniforms[0]))
        if went is None:
            out[j] = last
            return j, out, path
        out[j] = tokens[went]
        j += 1
        path[j] = went
        at = went


def verify(target, draft, tokens, parents, counts, uniforms, T=1.0, greedy=False):
    got = [verify_one(target[b], None if draft is None else draft[b], tokens[b], parents[b], int(counts[b]),
                      uniforms[b], T, greedy) for b in range(len(target))]
    return (np.array([g[0] for g in got], np.int32), np.stack([g[1] for g in got]), np.stack([g[2] for g in got]))


# ---------------------------------------------------------------------------
# pages


def row_state(row, pages):
    """Held pages of a table row, None when it is not valid."""
    held = [x for x in row if x >= 0]
    if any(x < -1 or x >= pages for x in row) or list(row[:len(held)]) != held:
        return None
    return held


def resize(table, lens, ref, page):
    table, ref = table.copy(), ref.copy()
    status = np.zeros(len(table), np.int32)
    want = {}
    for s, row in enumerate(table):
        held, need = row_state(row, len(ref)), -(-int(lens[s]) // page)
        if lens[s] < 0 or need > table.shape[1] or held is None:
            status[s] = -1
            continue
        for i in range(need, len(held)):
            ref[row[i]] -= 1
            row[i] = -1
        if len(held) < need:
            want[s] = (len(held), need)
    free = deque(int(p) for p in np.flatnonzero(ref == 0))
    left = len(free)
    for s, (a, z) in want.items():
        left -= z - a
        if left < 0:
            status[s] = -1
            continue
        for i in range(a, z):
            table[s, i] = free.popleft()
            ref[table[s, i]] = 1
    return table, ref, status


def fork(k, v, table, lens, ref, src, dst):
    """numpy copies of everything after the forks; k, v [L, P, page, H, D]."""
    k, v, table, lens, ref = (x.copy() for x in (k, v, table, lens, ref))
    page, slots = k.shape[2], len(table)
    status, todo = np.zeros(len(src), np.int32), []
    for i, (s, d) in enumerate(zip(src, dst)):
        ok = 0 <= s < slots and 0 <= d < slots and list(dst).count(d) == 1 and d not in src
        if ok:
            held = row_state(table[s], len(ref))
            ok = held is not None and row_state(table[d], len(ref)) is not None and lens[s] >= 0 \
                and -(-int(lens[s]) // page) <= len(held)
        if ok:
            todo.append(i)
        else:
            status[i] = -1
    for i in todo:
        for x in table[dst[i]]:
            if x >= 0:
                ref[x] -= 1
        table[dst[i]] = -1
    free = deque(int(p) for p in np.flatnonzero(ref == 0))
    for i in todo:
        s, d = src[i], dst[i]
        full, rag = int(lens[s]) // page, int(lens[s]) % page
        if rag and not free:
            status[i], lens[d] = -2, 0
            continue
        table[d, :full] = table[s, :full]
        for x in table[s, :full]:
            ref[x] += 1
        if rag:
            new = free.popleft()
            table[d, full] = new
            ref[new] = 1
            for c in (k, v):
                c[:, new, :rag] = c[:, table[s, full], :rag]
        lens[d] = lens[s]
    return k, v, table, lens, ref, status


def commit(k, v, table, lens, path):
    k, v = k.copy(), v.copy()
    page, pages = k.shape[2], k.shape[1]
    out = np.full(len(lens), -1, np.int32)
    for b, row in enumerate(path):
        n = next((i for i, x in enumerate(row) if x < 0), len(row))
        ids, base = [int(x) for x in row[:n]], int(lens[b])
        if base < 0 or any(y <= x for x, y in zip(ids, ids[1:])) or (n and base + ids[-1] >= table.shape[1] * page):
            continue
        moves = [(base + x, base + i) for i, x in enumerate(ids) if x != i]
        if any(not 0 <= table[b, t // page] < pages for m in moves for t in m):
            continue
        for s, d in moves:
            for c in (k, v):
                c[:, table[b, d // page], d % page] = c[:, table[b, s // page], s % page]
        out[b] = base + n
    return k, v, out


def exact_score_tolerance(out, A, dtype, rows, vmax):
    """Per element, where products and sums of q.k are exact in 32 bits: half a
    step for rounding the result and half a step of A for the weights p.  The
    exponent x = (s - reference) c has an error of at most 3 2^-24 (|x| + 16)
    (c is rounded twice, the fused operation once; the reference is within 2^16
    of the largest weight), below 2^-16 for every weight above 2^-100; 2^x one of 1.0e-4
    (bf16) or 2.8e-6 (fp16); 2^-20 is for running sums and their joining: all
    of them twice, for the weight and for the sum.  Smaller weights may be lost,
    2^-100 of v each, and fp16 weights, which are kept 2^6 up, lose 2^-25 each
    below 2^-14 (next to a sum of at least 2^6)."""
    half = torch.finfo(dtype).eps / 2
    exp2 = 1.0e-4 if dtype == torch.bfloat16 else 2.8e-6
    lost = rows * vmax * (2.0 ** -31 if dtype == torch.float16 else 2.0 ** -100)
    return (half * out.abs() + (half + 2 * (2.0 ** -16 + exp2 + 2.0 ** -20)) * A + lost) * (1 + 2 * half)
