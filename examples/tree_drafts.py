"""Speculative steps with draft trees over a paged cache that is cut down when it has
grown: every operator of a step in one loop, on the GPU throughout.

    python examples/tree_drafts.py

A target of one attention layer with random weights reads prompts of different
lengths (page_plan, rotary, chunk_attention). Then each step drafts a tree behind every
sequence's last token (dense_head and draft_select over the drafts' embeddings), runs
all trees through the target in one pass, takes the path that the target accepts and one
token more (verify_tree), keeps that path's rows in the cache (cache_keep) and gives
the other pages back (page_release). How much attention each cached token draws from the
tokens that stay is summed up on the way (cache_weights, behind the verdict); a sequence
with more than `budget` tokens is cut down to those that draw most (cache_select,
cache_keep, page_release).
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
# the draft tree: node 0 is the last token, three drafts behind it, three behind those
PARENT = [-1, 0, 0, 0, 1, 1, 2]
DEPTH = [0, 1, 1, 1, 2, 2, 2]
RANK = [0, 0, 1, 2, 0, 1, 0]  # which of its parent's most likely tokens a node is


class Target:
    """Random weights of one attention layer and a head."""

    def __init__(self, n=2048, d=256, heads=8, kv_heads=2, dim=64, seed=0, device="cuda"):
        self.n, self.d, self.heads, self.kv_heads, self.dim = n, d, heads, kv_heads, dim
        rng = np.random.default_rng(seed)

        def rand(*shape):
            return torch.from_numpy(rng.standard_normal(shape) / np.sqrt(shape[-1])).to(device, BF16)

        self.embed = rand(n, d) * 8
        self.qkv = rand((heads + 2 * kv_heads) * dim, d)
        self.out = rand(d, heads * dim)
        # the head likes what it saw: drafts by embeddings are worth trying
        self.W = ((self.embed.float() * 0.3).roll(1, 0) + rand(n, d).float()).to(BF16).contiguous()
        self.ids = torch.arange(n, dtype=I32, device=device)
        self.turns = torch.from_numpy(prep.rotary_turns(dim, 10000.0, "wavelength", 4.0, 1024)).to(device)
        self.ws = L.Workspace()

    def attend(self, tokens, positions, cache, table, lens, plan, tree=None):
        """States behind the tokens, whose keys and values go to the cache, and what
        cache_weights takes of them: queries and lse."""
        H, Hk, D = self.heads, self.kv_heads, self.dim
        x = self.embed[tokens.long()]
        qkv = (x @ self.qkv.T).view(-1, H + 2 * Hk, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        L.rotary(q, k, positions, self.turns)
        o, lse = L.chunk_attention(q, cache[0], cache[1], table, lens, plan.cu, k=k, v=v, slots=plan.slots, tree=tree,
                                   with_lse=True, workspace=self.ws, granted=plan.granted)
        return x + o.view(-1, H * D) @ self.out.T, q, lse

    def weigh(self, q, lse, cache, weights, table, lens, plan, tree=None):
        """What the tokens' queries drew on goes to the weights."""
        L.cache_weights(q, cache[0], table, lens, plan.cu, lse, weights, tree=tree, decay=0.9, granted=plan.granted,
                        workspace=self.ws)

    def forward(self, tokens, positions, cache, weights, table, lens, plan, tree=None):
        """Both, for tokens that all count."""
        h, q, lse = self.attend(tokens, positions, cache, table, lens, plan, tree)
        self.weigh(q, lse, cache, weights, table, lens, plan, tree)
        return h

    def probabilities(self, h, temperature):
        logits, p = L.dense_head(self.W, h.contiguous(), temperature)
        return p

    def draft(self, tokens):
        """The most likely tokens behind each token, by its embedding alone."""
        _, q = L.dense_head(self.W, self.embed[tokens.long()].contiguous())
        return L.draft_select(q, self.ids.expand(q.shape[0], -1).contiguous(), 3)[0]


def generate(model, prompts, steps, page=16, budget=None, seed=1, temperature=1.0):
    """`steps` speculative steps behind each prompt. Returns (tokens: a list of lists, the
    caches, table, lens, free pages and their count, positions) for those who look."""
    dev = model.embed.device
    S, N, depth = len(prompts), len(PARENT), max(DEPTH)
    Hk, D = model.kv_heads, model.dim
    i32 = lambda x: torch.tensor(x, dtype=I32, device=dev)  # noqa: E731
    width = -(-(max(len(p) for p in prompts) + steps * (depth + 1) + N) // page)
    pages = S * width
    cache = [torch.zeros(pages, page, Hk, D, dtype=BF16, device=dev) for _ in range(2)]
    # of each head the tokens of a page side by side
    weights = torch.zeros(pages, Hk, page, device=dev).transpose(1, 2)
    g = torch.Generator(device=dev).manual_seed(seed)
    free = torch.randperm(pages, generator=g, device=dev).to(I32)
    table = torch.zeros(S, width, dtype=I32, device=dev)
    lens, free_count = i32([0] * S), i32([pages])

    # ---- the prompts: all but their last token, which is the first tree's root
    new = [len(p) - 1 for p in prompts]
    plan = L.page_plan(lens, i32(new), table, free, free_count, page, max(1, sum(new)))
    if sum(new):
        model.forward(i32(sum((p[:-1] for p in prompts), [])), plan.positions, cache, weights, table, lens, plan)
    lens, free_count = i32(new), plan.free_left
    at = lens.clone()                             # positions go on where rows are evicted
    last = i32([p[-1] for p in prompts])
    said = []

    # ---- the trees, the same for all sequences
    bits = []
    for c, p in enumerate(PARENT):
        bits.append((bits[p] if c else 0) | 1 << c)
    tree = torch.tensor(bits * S, dtype=torch.int64, device=dev)
    parent, level, count = i32(PARENT * S), i32(DEPTH), i32([N] * S)
    for _ in range(steps):
        # drafts, level by level
        tokens = torch.zeros(S, N, dtype=I32, device=dev)
        tokens[:, 0] = last
        for up in sorted({p for p in PARENT if p >= 0}):
            kids = [c for c in range(N) if PARENT[c] == up]
            tokens[:, kids] = model.draft(tokens[:, up])[:, [RANK[c] for c in kids]]
        tokens = tokens.view(-1)
        # the target's pass over them: a node's position is its depth's
        plan = L.page_plan(lens, count, table, free, free_count, page, S * N)
        h, q, lse = model.attend(tokens, (at[:, None] + level[None, :]).view(-1), cache, table, lens, plan, tree)
        p = model.probabilities(h, temperature)
        r, u = torch.rand(S * N, generator=g, device=dev), torch.rand(S, generator=g, device=dev)
        out, path, accepted = L.verify_tree(p, tokens, parent, plan.cu, r, u, depth, granted=plan.granted)
        # rejected drafts draw nothing: a row of -inf; the others while their keys are in the chunk's places
        on = torch.zeros(S, N + 1, dtype=torch.bool, device=dev).scatter_(1, path.long() % (N + 1), True)[:, :N]
        model.weigh(q, lse.masked_fill_(~on.reshape(-1, 1), float("-inf")), cache, weights, table, lens, plan, tree)
        new_lens = L.cache_keep([*cache, weights], table, path, first=lens)
        free_count = L.page_release(lens, new_lens, table, free, plan.free_left, page, cu=plan.cu, granted=plan.granted)
        at = at + (new_lens - lens)
        lens = new_lens
        last = out.gather(1, accepted.clamp(min=0).long()[:, None])[:, 0].contiguous()
        said.append(out)
        if budget is not None:
            kept = L.cache_select(weights, table, lens, budget, sinks=2, recent=budget // 2)
            new_lens = L.cache_keep([*cache, weights], table, kept)
            free_count = L.page_release(lens, new_lens, table, free, free_count, page)
            lens = new_lens
    said = torch.cat(said, 1).cpu().tolist()
    tokens = [p + [t for t in row if t >= 0] for p, row in zip(prompts, said)]
    return tokens, cache, table, lens, free, free_count, at


def main():
    rng = np.random.default_rng(1)
    model = Target()
    prompts = [rng.integers(0, model.n, n).tolist() for n in (5, 40, 64, 1)]
    for budget in (None, 24):
        tokens, _, _, lens, _, left, _ = generate(model, prompts, 8, budget=budget)
        assert L.last_device_error() == 0
        print(f"budget {budget}: cached {lens.tolist()}, free pages {left.item()}")
        for p, t in zip(prompts, tokens):
            print(f"  prompt of {len(p)} tokens, {len(t) - len(p)} more in 8 steps: {t[len(p):]}")


if __name__ == "__main__":
    main()
