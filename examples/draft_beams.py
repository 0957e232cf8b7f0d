"""Beam drafting over a paged cache with a 4-bit head: every serving operator of
the library in one loop, on the GPU throughout.

    python examples/draft_beams.py

A drafter of one attention layer with random weights reads prompts of different
lengths (page_plan, chunk_attention), then extends each of them by a few tokens
with a beam search: candidates by the low-rank head (lowrank_score_topk), their
logits from the 4-bit rows (q4_gather_logits), the best continuations over all
beams (beam_select), and the beams' states moved to their parents' places
(beam_reorder) before the next token's attention.

The beams of a prompt share its full pages. What follows them - the prompt's
last, partial page and the drafted tokens - is a beam's own: its tail pages. They
exist twice, and a reordering copies them from one set to the other, so that two
children of one beam never write to the same page.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import draft_lm_head_gb300 as L  # noqa: E402
from draft_lm_head_gb300 import prep  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class Drafter:
    """Random weights of one attention layer and of the head in both forms."""

    def __init__(self, n=4096, d=256, heads=8, kv_heads=2, dim=64, r=32, group=64, seed=0, device="cuda"):
        self.n, self.d, self.heads, self.kv_heads, self.dim, self.group = n, d, heads, kv_heads, dim, group
        rng = np.random.default_rng(seed)
        W = prep.bf16_bits(rng.standard_normal((n, d)) / np.sqrt(d))
        fac = prep.freq_aware_factors(W, rng.integers(0, 50, n), r, rng.permutation(n))
        q4 = prep.quantise_rows(W, group)

        def bits(x):
            return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).to(device).view(BF16)

        def rand(*shape):
            return torch.from_numpy(rng.standard_normal(shape) / np.sqrt(shape[0])).to(device, BF16)

        self.A, self.B = bits(fac["A"]), bits(fac["B"])
        self.token_ids = torch.from_numpy(fac["token_ids"]).to(device)
        self.codes, self.scales = torch.from_numpy(q4["codes"]).to(device), bits(q4["scales"])
        self.embed = rand(n, d) * 8
        self.qkv = rand(d, (heads + 2 * kv_heads) * dim)
        self.out = rand(heads * dim, d)
        self.ws = L.Workspace()

    def attend(self, x, cache, table, lens, cu, slots, granted=None):
        """x (tokens x d) through the layer, its K and V into the cache."""
        H, Hk, D = self.heads, self.kv_heads, self.dim
        qkv = (x @ self.qkv).view(-1, H + 2 * Hk, D)
        o = L.chunk_attention(qkv[:, :H], cache[0], cache[1], table, lens, cu, k=qkv[:, H:H + Hk],
                              v=qkv[:, H + Hk:], slots=slots, workspace=self.ws, granted=granted)
        return x + o.view(-1, H * D) @ self.out

    def candidates(self, h):
        """Candidate ids of each row of h and their logits from the 4-bit rows."""
        ids = L.lowrank_score_topk(L.LOCAL, self.A, self.B, h, self.token_ids, 256, 2)
        return ids, L.q4_gather_logits(self.codes, self.scales, h, ids, self.group)


def draft(model, prompts, beams, steps, page=16):
    """The `beams` best continuations of `steps` tokens of each prompt (a list of
    token lists): tokens S x beams x steps and scores S x beams."""
    dev = model.embed.device
    S, lens = len(prompts), [len(p) for p in prompts]
    full = [n // page for n in lens]                       # pages shared by the beams
    tail = max(-(-(n % page + steps) // page) for n in lens)  # pages of a beam's own
    own = S * beams * tail
    pool = sum(-(-n // page) for n in lens)
    Hk, D = model.kv_heads, model.dim
    # the pool: the prompts' pages, then two sets of tail pages
    cache = [torch.zeros(pool + 2 * own, page, Hk, D, dtype=BF16, device=dev) for _ in range(2)]

    def i32(x):
        return torch.tensor(x, dtype=I32, device=dev)

    # ---- the prompts
    table = torch.zeros(S, max(-(-n // page) for n in lens), dtype=I32, device=dev)
    free = torch.arange(pool, dtype=I32, device=dev)
    plan = L.page_plan(i32([0] * S), i32(lens), table, free, i32([pool]), page, sum(lens))
    x = model.embed[torch.tensor(sum(prompts, []), device=dev)]
    h = model.attend(x, cache, table, i32([0] * S), plan.cu, plan.slots, plan.granted)
    h = h[(plan.cu[1:] - 1).long()]                        # of each prompt's last token

    # ---- tables of the beams, for either set of tail pages
    rows = S * beams
    width = max(full) + tail
    tables = []
    for half in range(2):
        t = torch.zeros(S, beams, width, dtype=I32, device=dev)
        first = pool + half * own
        for s in range(S):
            t[s, :, :full[s]] = table[s, :full[s]]
            t[s, :, full[s]:full[s] + tail] = (first + s * beams * tail + torch.arange(
                beams * tail, device=dev)).view(beams, tail).to(I32)
            if half == 0 and lens[s] % page:               # the partial page, once per beam
                for c in cache:
                    c[t[s, :, full[s]].long()] = c[table[s, full[s]].long()].clone()
        tables.append(t.view(rows, width))
    tails = [[c[pool + half * own: pool + (half + 1) * own].view(rows, -1) for c in cache] for half in range(2)]

    # ---- the beams: at first one is alive, at the prompt's last state
    h = h.repeat_interleave(beams, 0).contiguous()
    scores = torch.full((S, beams), -float("inf"), device=dev)
    scores[:, 0] = 0
    tokens = torch.zeros(rows, steps, dtype=I32, device=dev)
    cu = torch.arange(rows + 1, dtype=I32, device=dev)
    length = i32([n for n in lens for _ in range(beams)])
    for step in range(steps):
        ids, logits = model.candidates(h)
        parent, token, scores = L.beam_select(logits, scores.view(-1), beams, beams, ids=ids, workspace=model.ws)
        a, b = step & 1, 1 - (step & 1)
        tokens, _, _ = L.beam_reorder(parent, [tokens, *tails[a]], beams,
                                      out=[torch.empty_like(tokens), *tails[b]])
        tokens[:, step] = token.view(-1)
        if step + 1 == steps:
            break
        x = model.embed[token.view(-1).long()]
        page_of = torch.gather(tables[b], 1, (length // page).long()[:, None])[:, 0]
        h = model.attend(x, cache, tables[b], length, cu, page_of * page + length % page)
        length = length + 1
    return tokens.view(S, beams, steps), scores


def main():
    rng = np.random.default_rng(1)
    model = Drafter()
    prompts = [rng.integers(0, model.n, n).tolist() for n in (5, 40, 64, 33)]
    tokens, scores = draft(model, prompts, beams=4, steps=6)
    assert L.last_device_error() == 0
    for s, p in enumerate(prompts):
        print(f"prompt of {len(p)} tokens")
        for b in range(tokens.shape[1]):
            print(f"  {scores[s, b].item():9.4f}  {tokens[s, b].tolist()}")


if __name__ == "__main__":
    main()
