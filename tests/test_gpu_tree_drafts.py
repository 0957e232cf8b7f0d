"""The operators of a step together, through the example that uses all of them: what the
cache holds in the end is what each sequence's tokens, read from the start, would have
put there, and every page is either free or one sequence's."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _pages_are_whole(table, lens, free, left, page, pages):
    held = [int(x) for s, n in enumerate(lens.tolist()) for x in table[s, :-(-n // page)].tolist()]
    spare = free[:int(left)].tolist()
    assert sorted(held + spare) == list(range(pages))


def _rows(model, tokens):
    """Keys and values of a sequence's tokens, rotated, as the model rounds them."""
    import torch
    from oracle import step_oracle as O
    H, Hk, D = model.heads, model.kv_heads, model.dim
    x = model.embed[torch.tensor(tokens, device="cuda")]
    qkv = (x @ model.qkv.T).view(-1, H + 2 * Hk, D)
    k = O.rotary(qkv[:, H:H + Hk].double().cpu().numpy(), np.arange(len(tokens)), model.turns.cpu().numpy())
    return k, qkv[:, H + Hk:].double().cpu().numpy()


def _close(got, want):
    """bf16 products of other batches may round the other way, once before the rotation
    and once behind it, which mixes a pair: 2^-7 of the pair's size and a little more."""
    size = np.abs(want).max(axis=-1, keepdims=True)
    return np.all(np.abs(got - want) <= 2.0 ** -6 * size)


@pytest.mark.parametrize("page,steps", [(16, 1), (16, 9), (32, 6)])
def test_cache_holds_the_accepted_tokens(page, steps):
    import torch
    from gpu_util import lib
    L = lib()
    import tree_drafts as E
    model = E.Target()
    rng = np.random.default_rng(page + steps)
    prompts = [rng.integers(0, model.n, n).tolist() for n in (1, 5, 16, 37, 64)]
    tokens, cache, table, lens, free, left, at = E.generate(model, prompts, steps, page)
    assert L.last_device_error() == 0
    _pages_are_whole(table, lens, free, left, page, cache[0].shape[0])
    more = 0
    for s, (p, t) in enumerate(zip(prompts, tokens)):
        n = int(lens[s])
        # everything but the last token, which no pass has read yet
        assert t[:len(p)] == p and n == len(t) - 1 == int(at[s]) and len(p) + steps <= len(t) <= len(p) + 3 * steps
        more += len(t) - len(p) - steps
        k, v = _rows(model, t[:n])
        j = torch.arange(n, device="cuda")
        pg = table[s].long()[j // page]
        assert _close(cache[0][pg, j % page].double().cpu().numpy(), k)
        assert _close(cache[1][pg, j % page].double().cpu().numpy(), v)
    assert steps == 1 or more > 0  # some drafts were accepted


def test_eviction_in_the_loop():
    import torch
    from gpu_util import lib
    L = lib()
    import tree_drafts as E
    model = E.Target()
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, model.n, n).tolist() for n in (2, 30, 100, 64)]
    tokens, cache, table, lens, free, left, at = E.generate(model, prompts, 7, 16, budget=24)
    assert L.last_device_error() == 0
    _pages_are_whole(table, lens, free, left, 16, cache[0].shape[0])
    for s, (p, t) in enumerate(zip(prompts, tokens)):
        assert int(at[s]) == len(t) - 1 and int(lens[s]) == min(24, len(t) - 1)
        # the first two and the last twelve are always among them, in their order
        k, v = _rows(model, t[:-1])
        n = int(lens[s])
        j = torch.arange(n, device="cuda")
        pg = table[s].long()[j // 16]
        for got, want in ((cache[0][pg, j % 16].double().cpu().numpy(), k), (cache[1][pg, j % 16].double().cpu().numpy(), v)):
            assert _close(got[:2], want[:2][:n]) and _close(got[-min(12, n):], want[-min(12, n):])


def test_rejected_drafts_draw_nothing(monkeypatch):
    """What the weights are summed up from: of a tree's rows those of the accepted path."""
    import torch
    from gpu_util import lib
    L = lib()
    import tree_drafts as E
    model = E.Target()
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, model.n, n).tolist() for n in (3, 20, 33)]
    calls, paths = [], []
    weigh, verify = L.cache_weights, L.verify_tree

    def weights(q, kc, table, lens, cu, lse, w, **kw):
        if kw.get("tree") is not None:
            calls.append(lse.clone())
        return weigh(q, kc, table, lens, cu, lse, w, **kw)

    def verdict(*args, **kw):
        paths.append(verify(*args, **kw))
        return paths[-1]
    monkeypatch.setattr(E.L, "cache_weights", weights)
    monkeypatch.setattr(E.L, "verify_tree", verdict)
    E.generate(model, prompts, 4)
    assert L.last_device_error() == 0 and len(calls) == len(paths) == 4
    for lse, (_, path, _) in zip(calls, paths):
        lse = lse.view(3, len(E.PARENT), -1)
        for s in range(3):
            on = {x for x in path[s].tolist() if x >= 0}
            for c in range(len(E.PARENT)):
                assert bool(torch.isfinite(lse[s, c]).all() if c in on else (lse[s, c] == -float("inf")).all()), (s, c)


def test_a_step_captured_and_replayed():
    """Plan, rotary, attention, weights, verification, kept rows and pages given back in one
    graph, replayed on two states, against the same calls made one by one."""
    import torch
    from gpu_util import lib
    L = lib()
    import tree_drafts as E
    model = E.Target()
    S, N, P, dev = 3, len(E.PARENT), 16, "cuda"
    g = torch.Generator(device=dev).manual_seed(5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    bits = []
    for c, p in enumerate(E.PARENT):
        bits.append((bits[p] if c else 0) | 1 << c)
    tree, parent, level = torch.tensor(bits * S, dtype=torch.int64, device=dev), i32(E.PARENT * S), i32(E.DEPTH)

    def state(seed):
        g.manual_seed(seed)
        return dict(tokens=torch.randint(0, model.n, (S * N,), generator=g, device=dev, dtype=torch.int32),
                    lens=torch.randint(1, 90, (S,), generator=g, device=dev, dtype=torch.int32),
                    table=torch.randperm(S * 8, generator=g, device=dev).to(torch.int32).view(S, 8),
                    k=torch.randn(S * 8, P, 2, 64, generator=g, device=dev).to(torch.bfloat16),
                    v=torch.randn(S * 8, P, 2, 64, generator=g, device=dev).to(torch.bfloat16),
                    w=torch.rand(S * 8, P, 2, generator=g, device=dev), free=torch.randperm(40, generator=g, device=dev).to(torch.int32) % 24,
                    r=torch.rand(S * N, generator=g, device=dev) * 0.02, u=torch.rand(S, generator=g, device=dev))

    count, free_count = i32([N] * S), i32([24])

    def step(st):
        # (the tables' pages stand in for new ones: the plan takes none where a page has room)
        plan = L.page_plan(st["lens"], count, st["table"], st["free"], free_count, P, S * N)
        h = model.forward(st["tokens"], (st["lens"][:, None] + level[None, :]).view(-1), [st["k"], st["v"]], st["w"], st["table"],
                          st["lens"], plan, tree)
        p = model.probabilities(h, 1.0)
        out, path, acc = L.verify_tree(p, st["tokens"], parent, plan.cu, st["r"], st["u"], 2, granted=plan.granted)
        new = L.cache_keep([st["k"], st["v"], st["w"]], st["table"], path, first=st["lens"])
        left = L.page_release(st["lens"], new, st["table"], st["free"], plan.free_left, P, cu=plan.cu, granted=plan.granted)
        return [out, path, acc, new, left, st["k"], st["v"], st["w"], st["free"]]

    # pages that the plan hands out are distinct from the tables': 24 tables' pages, so the pool has 24 more
    def fresh(seed):
        st = state(seed)
        st["k"], st["v"] = (torch.cat([x, x.flip(0)]) for x in (st["k"], st["v"]))
        st["w"] = torch.cat([st["w"], st["w"].flip(0)])
        st["free"] = (torch.randperm(24, generator=g, device=dev) + 24).to(torch.int32)
        return st

    want = [[x.clone() for x in step(fresh(s))] for s in (1, 2)]
    held = fresh(1)
    step(fresh(3))  # workspaces are as large as they get
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for s in (1, 2):
        for name, x in fresh(s).items():
            held[name].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[s - 1]):
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert L.last_device_error() == 0
