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
