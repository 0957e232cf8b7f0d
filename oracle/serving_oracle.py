"""fp64 CPU oracle of the serving operators around the head. Written from the
definitions in include/lmhead.h, element by element."""
from __future__ import annotations

import numpy as np


def page_plan(lens, new, table, free_pages, free_count, page, max_tokens):
    """Returns (slots, positions, cu, granted, free_left, table)."""
    table = np.array(table)
    width = table.shape[1]
    F = max(0, min(int(free_count), len(free_pages)))
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int64)
    cu, granted, before, left = [0], [], 0, F
    for s, (l, m) in enumerate(zip(lens, new)):
        l, m = int(l), int(m)
        fits = l >= 0 and m >= 0 and l + m <= width * page
        need = -(-(l + m) // page) - -(-l // page) if fits else 0
        ok = fits and (need == 0 or before + need <= F)
        if ok:
            held = -(-l // page)
            for j in range(need):
                table[s, held + j] = free_pages[F - 1 - before - j]
            left -= need
            for i in range(m):
                t = cu[-1] + i
                if t < max_tokens:
                    positions[t] = l + i
                    slots[t] = int(table[s, (l + i) // page]) * page + (l + i) % page
        before += need
        granted.append(int(ok))
        cu.append(cu[-1] + max(m, 0))
    return slots, positions, np.array(cu), np.array(granted), left, table


def beam_step(logits, scores, beams, k, finished=None):
    """Per sequence: [(score, flat index)] of its k best, best first, ties to the
    lower index, entries that score -inf or NaN left out."""
    rows, n = logits.shape
    res = []
    for s in range(rows // beams):
        val, idx = [], []
        for b in range(beams):
            r = s * beams + b
            if finished is not None and finished[r]:
                val.append(np.array([scores[r]], dtype=np.float64))
                idx.append(np.array([b * n]))
                continue
            with np.errstate(all="ignore"):
                x = logits[r].astype(np.float64)
                top = x.max()
                val.append(float(scores[r]) + ((x - top) - np.log(np.exp(x - top).sum())))
            idx.append(b * n + np.arange(n))
        val, idx = np.concatenate(val), np.concatenate(idx)
        keep = val > -np.inf  # false for NaN too
        val, idx = val[keep], idx[keep]
        order = np.lexsort((idx, -val))[:k]
        res.append([(val[o], int(idx[o])) for o in order])
    return res


def q4_rows(codes, scales, mins, group):
    """The weights of 4-bit rows in fp64."""
    c = np.empty((codes.shape[0], codes.shape[1] * 2))
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    c = c.reshape(codes.shape[0], -1, group)
    w = (c - 8) * scales[..., None] if mins is None else c * scales[..., None] + mins[..., None]
    return w.reshape(codes.shape[0], -1)


def chunk_attention(q, k_cache, v_cache, table, lens, cu, scale, window=0, tree=None, granted=None):
    """q T x H x D, caches pages x P x Hk x D (the chunk's own K and V already in
    them), all fp64. Returns (out, lse, magnitude, reach): magnitude is sum_j
    p_j |v_j| and reach max_j scale sum_d |q_d k_jd| over the visible keys. Requests
    with granted 0 see none."""
    T, H, D = q.shape
    P, Hk = k_cache.shape[1], k_cache.shape[2]
    G = H // Hk
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, reach = np.full((T, H), -np.inf), np.zeros((T, H))
    for s in range(len(lens)):
        l, m = int(lens[s]), int(cu[s + 1] - cu[s])
        if granted is not None and not granted[s]:
            continue
        j = np.arange(l + m)
        slot = np.asarray(table[s])[j // P].astype(np.int64) * P + j % P
        K = k_cache.reshape(-1, Hk, D)[slot]
        V = v_cache.reshape(-1, Hk, D)[slot]
        for i in range(m):
            t = int(cu[s]) + i
            if tree is None:
                lo = max(0, l + i + 1 - window) if window else 0
                keys = np.arange(lo, l + i + 1)
            else:
                bits = int(tree[t]) & ((1 << 64) - 1)
                keys = np.array(list(range(l)) + [l + x for x in range(min(m, 64)) if bits >> x & 1], dtype=int)
            if not len(keys):
                continue
            for b in range(Hk):
                Ka, Va, qa = K[keys, b], V[keys, b], q[t, b * G:(b + 1) * G]
                x = scale * (qa @ Ka.T)
                top = x.max(axis=1, keepdims=True)
                e = np.exp(x - top)
                z = e.sum(axis=1, keepdims=True)
                heads = slice(b * G, (b + 1) * G)
                out[t, heads], mag[t, heads] = (e / z) @ Va, (e / z) @ np.abs(Va)
                lse[t, heads] = (top + np.log(z))[:, 0]
                reach[t, heads] = scale * (np.abs(qa) @ np.abs(Ka).T).max(axis=1)
    return out, lse, mag, reach
