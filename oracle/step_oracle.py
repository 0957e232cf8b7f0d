"""CPU oracle of the operators of a step over the paged cache. Written from the
definitions in include/lmhead.h, element by element, in fp64 (where a definition
rounds to fp32, so does this)."""
from __future__ import annotations

import math

import numpy as np


def rotary(x, positions, turns, interleaved=False, backward=False, magnitude=1.0):
    """x: T x heads x dim (fp64), in a copy. Negative positions leave their rows."""
    y = np.array(x, dtype=np.float64)
    half = len(turns)
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        for i, f in enumerate(turns):
            part = (int(pos) * int(f)) % (1 << 64)  # exactly
            if part >= 1 << 63:
                part -= 1 << 64
            a = 2 * math.pi * (part / 2.0 ** 64) * (-1 if backward else 1)
            c, s = magnitude * math.cos(a), magnitude * math.sin(a)
            j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, v = x[t, :, j].astype(np.float64), x[t, :, k].astype(np.float64)
            y[t, :, j], y[t, :, k] = u * c - v * s, v * c + u * s
    return y


def _draw(w, u):
    run = np.cumsum(w.astype(np.float64))
    at = int(np.searchsorted(run, float(u) * run[-1], side="right"))
    return min(at, int(np.nonzero(w > 0)[0][-1]))


def verify_tree(p, tokens, parent, r, u, cand_ids=None, cand_q=None):
    """One request: p N x n fp32. Returns (tokens, path) or None for a tree that is
    not one."""
    f32 = np.float32
    clean = lambda x: np.where(np.asarray(x) > 0, x, 0).astype(f32)
    n = p.shape[1]
    cur, path, said = 0, [0], []

    def arrive(c):
        w = clean(p[c])
        g = np.zeros(n, dtype=f32)
        known = np.zeros(n, dtype=bool)
        if cand_ids is not None:
            for j, q in zip(cand_ids[c], cand_q[c]):
                if 0 <= j < n and not known[j]:
                    g[j], known[j] = clean(q), True
        return w, g, known
    w, g, known = arrive(0)
    Z = Q = 1.0
    for x in range(1, len(tokens)):
        if parent[x] != cur:
            continue
        t = int(tokens[x])
        if not 0 <= t < n:
            return None
        if cand_ids is None:
            yes = float(r[x]) * Z < float(w[t])
            if not yes:
                Z = max(Z - float(w[t]), 0.0)
                w[t] = 0
        else:
            if not known[t]:
                return None
            yes = float(r[x]) * Z * float(g[t]) < float(w[t]) * Q
            if not yes:
                took = np.minimum(w, f32(Z / Q if Q > 0 else 0.0) * g)
                w = w - took
                Z = max(Z - float(took.astype(np.float64).sum()), 0.0)
                Q -= float(g[t])
                g[t] = 0
        if yes:
            said.append(t)
            path.append(x)
            cur = x
            w, g, known = arrive(x)
            Z = Q = 1.0
    if not (w > 0).any():
        w = clean(p[cur])
    said.append(_draw(w, u) if (w > 0).any() else n - 1)
    return said, path


def cache_keep(cache, table, kept, first, page):
    """cache: pages x page x heads (x dim), changed in place; kept: S x (heads x) n."""
    heads = cache.shape[2]
    lens = []
    for s in range(len(table)):
        f = int(first[s]) if first is not None else 0
        per = np.asarray(kept[s])
        per = np.broadcast_to(per, (heads, per.shape[-1]))
        place = lambda pos: (table[s][pos // page], pos % page)
        for a in range(heads):
            for i, x in enumerate(per[a]):  # upwards: what is read has not been written
                if x >= 0:
                    cache[place(f + i)][a] = cache[place(f + int(x))][a]
        some = np.nonzero(per[0] >= 0)[0]
        lens.append(f + (int(some[-1]) + 1 if len(some) else 0))
    return np.array(lens)


def page_release(held, new_lens, table, free, count, page):
    free = list(free[:count])
    for s, (h, m) in enumerate(zip(held, new_lens)):
        free += [int(x) for x in table[s][-(-int(m) // page):-(-int(h) // page)]]
    return free


def cache_weights(q, k_cache, table, lens, cu, lse, weights, scale, window=0, tree=None, decay=1.0):
    """All fp64; weights pages x page x kv_heads, in a copy. Returns (weights, rows):
    the number of terms of each entry (0: not a cached token's)."""
    weights = np.array(weights, dtype=np.float64)
    rows = np.zeros(weights.shape)
    H = q.shape[1]
    P, Hk = k_cache.shape[1], k_cache.shape[2]
    G = H // Hk
    for s in range(len(lens)):
        l, m = int(lens[s]), int(cu[s + 1] - cu[s])
        for j in range(l + m):
            at = (int(table[s][j // P]), j % P)
            for a in range(Hk):
                total, n = 0.0, 0
                for i in range(m):
                    t = int(cu[s]) + i
                    if tree is not None:
                        see = j < l or (j - l < 64 and (int(tree[t]) >> (j - l)) & 1)
                    else:
                        see = j <= l + i and (not window or j > l + i - window)
                    if not see:
                        continue
                    x = scale * (q[t, a * G:(a + 1) * G] @ k_cache[at][a]) - lse[t, a * G:(a + 1) * G]
                    total += float(np.exp(x).sum())
                    n += G
                old = decay * weights[at][a] if j < l and decay else 0.0
                weights[at][a] = old + total
                rows[at][a] = n + 1
    return weights, rows


def cache_select(weights, table, lens, page, budget, sinks, recent):
    """weights pages x page x kv_heads. Returns S x kv_heads x budget."""
    Hk = weights.shape[2]
    out = np.full((len(lens), Hk, budget), -1, dtype=np.int64)
    for s, l in enumerate(lens):
        l = int(l)
        j = np.arange(l)
        for a in range(Hk):
            if l <= budget:
                out[s, a, :l] = j
                continue
            w = weights[np.asarray(table[s])[j // page], j % page, a].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            nan = np.isnan(weights[np.asarray(table[s])[j // page], j % page, a])
            lo, hi = min(sinks, l), max(min(sinks, l), l - recent)
            mid = sorted(range(lo, hi), key=lambda x: (nan[x], -w[x], x))[:budget - lo - (l - hi)]
            out[s, a] = sorted(list(range(lo)) + mid + list(range(hi, l)))
    return out
