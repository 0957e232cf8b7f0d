"""The operators of a step over the paged cache, as timed cases.

Four groups: rotary (rotary positions of a step's queries and keys, and their gradient), verify (a draft
tree against the target's probabilities, the accepted rows kept in the cache, the other pages given back),
weights (how much attention each cached token has drawn, summed up) and evict (which tokens stay by those
weights, the rows moved together, the pages given back). `own` picks between the plain torch form of each
and the framework's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
INF = math.inf


def listed():
    return [
        # a decoding step of 8 sequences, in place in the projection's output: the smallest call
        dict(name="rotary decode 8", op="rotary", tokens=8, heads=32, kv_heads=8, dim=128, rot=128, pairs=False, far=4000,
             scaled=False, back=False, inplace=True, dtype="bf16"),
        # prompts far into a long context, frequencies stretched for it, refused tokens at the end
        dict(name="rotary prompts 16384", op="rotary", tokens=16384, heads=32, kv_heads=8, dim=128, rot=128, pairs=False,
             far=900000, scaled=True, back=False, inplace=False, dtype="bf16"),
        # the gradient of a chunk in full precision, neighbours paired, half of each head
        dict(name="rotary backward 5001", op="rotary", tokens=5001, heads=64, kv_heads=8, dim=64, rot=32, pairs=True, far=130000,
             scaled=False, back=True, inplace=False, dtype="fp32"),
        # one sequence's tree of 10 nodes, children the most likely tokens
        dict(name="verify 1x10", op="verify", requests=1, nodes=10, ragged=False, depth=5, vocab=128256, cands=64, drawn=False,
             ctx=2000, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # 8 concurrent sequences, children drawn from the head's candidates
        dict(name="verify 8x10 drawn", op="verify", requests=8, nodes=10, ragged=False, depth=5, vocab=201088, cands=1572, drawn=True,
             ctx=4100, kv_heads=8, dim=64, page=64, dtype="bf16"),
        # a batch of wide trees of different sizes
        dict(name="verify 64x60 drawn", op="verify", requests=64, nodes=60, ragged=True, depth=8, vocab=128256, cands=1002, drawn=True,
             ctx=2000, kv_heads=8, dim=128, page=32, dtype="fp16"),
        # one new token of one sequence
        dict(name="weights token", op="weights", requests=1, new=1, ctx=2000, ragged=False, heads=32, kv_heads=8, dim=128, page=16,
             mask="causal", window=0, decay=1.0, dtype="bf16"),
        # decoding of a ragged batch: all of the cached keys are read
        dict(name="weights decode 32", op="weights", requests=32, new=1, ctx=8000, ragged=True, heads=32, kv_heads=8, dim=128, page=32,
             mask="causal", window=0, decay=0.97, dtype="fp16"),
        # chunks of two long prompts over what was cached before
        dict(name="weights prompt 2x2048", op="weights", requests=2, new=2048, ctx=6144, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, mask="causal", window=0, decay=1.0, dtype="bf16"),
        # one sequence halved
        dict(name="evict 4096 to 2048", op="evict", requests=1, ctx=4096, ragged=False, budget=2048, sinks=4, recent=256, kv_heads=8,
             dim=128, page=16, dtype="bf16"),
        # a ragged batch that has outgrown its budget by a little
        dict(name="evict 64 decoding", op="evict", requests=64, ctx=2176, ragged=True, budget=2000, sinks=4, recent=500, kv_heads=8,
             dim=64, page=64, dtype="bf16"),
        # long prompts cut down to what is read most
        dict(name="evict 16 prompts", op="evict", requests=16, ctx=32768, ragged=True, budget=4097, sinks=1, recent=1024, kv_heads=8,
             dim=128, page=32, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "verify", "weights", "weights", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        dim = rng.choice([64, 80, 96, 128])
        rot = 16 * rng.randint(1, dim // 16)
        most = 16384 * 40 * 128 // ((heads + kv_heads) * dim * 2)
        return dict(op=op, tokens=_log(rng, 1, most), heads=heads, kv_heads=kv_heads, dim=dim, rot=rot, pairs=rng.random() < 0.4,
                    far=_log(rng, 100, 2000000), scaled=rng.random() < 0.5, back=rng.random() < 0.3, inplace=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "verify":
        nodes = rng.randint(1, 64)
        vocab = _log(rng, 500, 200000)
        return dict(op=op, requests=_log(rng, 1, max(1, min(64, 480_000_000 // (nodes * vocab)))), nodes=nodes, ragged=rng.random() < 0.5,
                    depth=rng.randint(1, 10), vocab=vocab, cands=max(64, _log(rng, 64, min(2376, vocab))), drawn=rng.random() < 0.5,
                    ctx=_log(rng, 1, 4000), kv_heads=kv_heads, dim=dim, page=page, dtype=rng.choice(["bf16", "fp16"]))
    if op == "weights":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        mask = rng.choice(["causal", "causal", "tree", "window"])
        new = rng.randint(1, 64) if mask == "tree" else rng.choice([1, _log(rng, 1, 2048)])
        ctx = rng.choice([rng.randint(0, 200), _log(rng, 1, 16000)])
        most = min(0.2e12 / (2.0 * new * (ctx + new) * heads * dim), 3e8 / (2.0 * kv_heads * dim * (ctx + new)), 64)
        return dict(op=op, requests=_log(rng, 1, max(1, int(most))), new=new, ctx=ctx, ragged=rng.random() < 0.6, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page, mask=mask, window=rng.choice([1, 100, 128, 1000]) if mask == "window" else 0,
                    decay=rng.choice([1.0, 1.0, 0.9, 0.0]), dtype=rng.choice(["bf16", "fp16"]))
    ctx = _log(rng, 10, 32768)
    budget = rng.randint(1, min(ctx + 10, 8192))
    sinks = rng.randint(0, min(4, budget))
    most = 16 * 32768 * 8 * 128 // (ctx * kv_heads * dim)
    return dict(op=op, requests=_log(rng, 1, max(1, min(64, most))), ctx=ctx, ragged=rng.random() < 0.6, budget=budget, sinks=sinks,
                recent=rng.randint(0, (budget - sinks) // 2), kv_heads=kv_heads, dim=dim, page=page, dtype=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------- inputs

def _lengths(case, seed):
    """Cached tokens and new ones of each request, on the host: what a scheduler knows. The seed deals
    the same lengths out in another order, so that a case's sizes are its own."""
    r = random.Random(13)
    new = case.get("nodes", case.get("new", 0))
    if case["ragged"]:
        pairs = [(r.randint(case["ctx"] // 2, case["ctx"]), r.randint(max(1, new // 2), new) if new else 0) for _ in range(case["requests"])]
    else:
        pairs = [(case["ctx"], new)] * case["requests"]
    random.Random(seed).shuffle(pairs)
    return [p[0] for p in pairs], [p[1] for p in pairs]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _starts(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _pages(case, lens, new, g):
    """A pool whose pages lie in no order, and the requests' tables of them. Its last pages are no
    request's."""
    P = case["page"]
    pages = [-(-(l + m) // P) for l, m in zip(lens, new)]
    total, width = sum(pages) + 3, max(max(pages), 1)
    perm = torch.randperm(total - 1, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < _i32(pages)[:, None]] = perm[: sum(pages)]
    free = torch.zeros(total, dtype=torch.int32, device=DEV)
    free[:2] = perm[sum(pages):]
    return total, table, free


def _turns(case):
    """Turns a position, in units of 2^-64: base 10000, or 500000 with the slow frequencies divided by 8
    and those between two wavelengths blended."""
    half = case["rot"] // 2
    f = []
    for i in range(half):
        w = (500000.0 if case["scaled"] else 10000.0) ** (-i / half)
        if case["scaled"]:
            keep = min(1.0, max(0.0, (8192 * w / (2 * math.pi) - 1) / 3))
            w = w * keep + w / 8 * (1 - keep)
        f.append(round(w / (2 * math.pi) * 2.0 ** 64))
    return torch.tensor(f, dtype=torch.int64, device=DEV)


def _tree_bits(new, r):
    """Ancestor bits (own bit included) of each node of a random draft tree."""
    bits = []
    for i in range(new):
        bits.append((bits[r.randint(max(0, i - 4), i - 1)] if i else 0) | (1 << i))
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def _tree(m, depth, r):
    """Parents of a draft tree's nodes (node 0 is its root) and each node's rank among its siblings."""
    parent, level, rank, kids = [-1], [0], [0], [0]
    for c in range(1, m):
        p = r.choice([x for x in range(max(0, c - 12), c) if level[x] < depth] or [0])
        parent.append(p)
        level.append(level[p] + 1)
        rank.append(kids[p])
        kids[p] += 1
        kids.append(0)
    return parent, rank


def _paged(total, case, g):
    return torch.randn(total, case["page"], case["kv_heads"], case["dim"], generator=g, device=DEV, dtype=TYPES[case["dtype"]])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "rotary":
        T, H, Hk, D, t = case["tokens"], case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
        # the projection's output: q, k and v side by side (a gradient comes as two tensors)
        qkv = torch.randn(T, H + 2 * Hk, D, generator=g, device=DEV, dtype=torch.float32).to(t)
        q, k = qkv[:, :H], qkv[:, H: H + Hk]
        if case["back"]:
            q, k = q.contiguous(), k.contiguous()
        pos = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        pos[T - T // 50:] = -1
        out = None if case["inplace"] else (torch.zeros(T, H, D, dtype=t, device=DEV), torch.zeros(T, Hk, D, dtype=t, device=DEV))
        st.update(q=q, k=k, pos=pos, turns=_turns(case), out=out, magnitude=1.0 + 0.1 * math.log(8) if case["scaled"] else 1.0)
        return st
    lens, new = _lengths(case, seed)
    S = len(lens)
    total, table, free = _pages(case, lens, new, g)
    cu = _starts(new)
    kc = _paged(total, case, g)
    st.update(lens=_i32(lens), cu=_i32(cu), table=table, kc=kc, host_lens=lens, host_new=new, free=free, free_count=_i32([2]))
    if op == "verify":
        T, n, K = cu[-1], case["vocab"], case["cands"]
        r = random.Random(seed * 31 + 7)
        trees = [_tree(m, case["depth"], r) for m in new]
        parent, rank = _i32(sum((x[0] for x in trees), [])), _i32(sum((x[1] for x in trees), [])).long()
        root = torch.repeat_interleave(_i32(cu[:-1]).long(), _i32(new).long())
        # the candidates carry most of the target's mass; the drafter's view of them is a little off
        start = torch.randint(0, n, (T, 1), generator=g, device=DEV)
        ids = (start + torch.arange(K, device=DEV) * 1000003) % n
        x = torch.randn(T, n, generator=g, device=DEV)
        mine = 2.5 * torch.randn(T, K, generator=g, device=DEV) + 8
        x.scatter_(1, ids, mine)
        p = torch.softmax(x, 1)
        del x
        q = torch.softmax(mine + 0.5 * torch.randn(T, K, generator=g, device=DEV), 1)
        # children: the most likely candidates of their parent, or drawn from it without replacement
        order = torch.log(q)
        if case["drawn"]:
            order = order - torch.log(-torch.log(torch.rand(T, K, generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
        order = torch.topk(order, min(64, K), 1).indices
        up = root + parent.long().clamp(min=0)
        tokens = ids[up, order[up, rank.clamp(max=order.shape[1] - 1)]].to(torch.int32)
        st.update(p=p, tokens=tokens, parent=parent, r=torch.rand(T, generator=g, device=DEV), u=torch.rand(S, generator=g, device=DEV),
                  vc=_paged(total, case, g), ids=ids.to(torch.int32) if case["drawn"] else None, q=q if case["drawn"] else None)
    elif op == "weights":
        T, H, Hk, D = cu[-1], case["heads"], case["kv_heads"], case["dim"]
        st.update(q=torch.randn(T, H + 2 * Hk, D, generator=g, device=DEV).to(TYPES[case["dtype"]])[:, :H], scale=D ** -0.5,
                  # of each K/V head the tokens of a page side by side
                  w=torch.rand(total, Hk, case["page"], generator=g, device=DEV).transpose(1, 2), tree=None)
        if case["mask"] == "tree":
            r = random.Random(seed * 31 + 5)
            st["tree"] = torch.tensor([b for m in new for b in _tree_bits(m, r)], dtype=torch.int64, device=DEV)
        st["lse"] = _log_sums(st)
    else:
        # few tokens draw most of the attention, some none at all
        w = torch.exp(2 * torch.randn(total, case["kv_heads"], case["page"], generator=g, device=DEV))
        w[torch.rand(w.shape, generator=g, device=DEV) < 0.1] = 0
        st.update(vc=_paged(total, case, g), w=w.transpose(1, 2))
        # what is chosen by stays as it is, so that each pass finds the same to do; its copy moves with the rows
        st["moved"] = w.clone().transpose(1, 2)
    return st


# ---------------------------------------------------------------- plain forms and calls

def _rotary_plain(st):
    c = st["case"]
    half = c["rot"] // 2
    turn = (st["pos"].long()[:, None] * st["turns"][None, :]).double() * 2.0 ** -64  # whole turns drop out
    co = (torch.cos(2 * math.pi * turn) * st["magnitude"]).float()[:, None]
    si = (torch.sin(2 * math.pi * turn) * st["magnitude"]).float()[:, None]
    if c["back"]:
        si = -si
    there = (st["pos"] >= 0)[:, None, None]

    def turned(x, out):
        f = x[..., : c["rot"]].float()
        a, b = (f[..., 0::2], f[..., 1::2]) if c["pairs"] else (f[..., :half], f[..., half:])
        y = (a * co - b * si, b * co + a * si)
        y = torch.stack(y, -1).flatten(-2) if c["pairs"] else torch.cat(y, -1)
        y = torch.cat([y.to(x.dtype), x[..., c["rot"]:]], -1)
        return out.copy_(torch.where(there, y, out))

    out = st["out"] or (st["q"], st["k"])
    return dict(q=turned(st["q"], out[0]), k=turned(st["k"], out[1]))


def _padded(st):
    """The requests' tokens side by side, in rows of one length: (row of each in the chunk, which of them
    there are)."""
    lens, cu = st["lens"].long(), st["cu"].long()
    i = torch.arange(max(max(st["host_new"]), 1), device=DEV)[None, :]
    there = i < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + i, torch.zeros_like(i)), there


def _slots(st, pos, there):
    """Slots of positions of each request (S x ...); those that are not there are the pool's last."""
    P = st["case"]["page"]
    page = torch.gather(st["table"].long(), 1, (pos.clamp(min=0) // P).clamp(max=st["table"].shape[1] - 1).flatten(1)).view(pos.shape)
    return torch.where(there, page * P + pos % P, torch.full_like(pos, st["kc"].shape[0] * P - 1))


def _scores(st):
    """Scores of every new token's heads against every key of its request, -inf where it sees none:
    S x kv_heads x (tokens, heads) x keys, with the rows' places."""
    c = st["case"]
    Hk, D = c["kv_heads"], c["dim"]
    G = c["heads"] // Hk
    rows, there = _padded(st)
    S, M = rows.shape
    lens = st["lens"].long()
    n = lens + there.sum(1)
    j = torch.arange(max(l + m for l, m in zip(st["host_lens"], st["host_new"])), device=DEV)[None, :].expand(S, -1)
    K = st["kc"].view(-1, Hk, D)[_slots(st, j, j < n[:, None])].permute(0, 2, 3, 1).float()
    q = st["q"][rows].view(S, M, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hk, M * G, D).float()
    x = torch.matmul(q, K) * st["scale"]
    i, at = torch.arange(M, device=DEV)[None, :, None], (j - lens[:, None])[:, None, :]
    if c["mask"] == "tree":
        bit = (st["tree"][rows][:, :, None] >> at.clamp(0, 63)) & 1
        see = (at < 0) | ((bit == 1) & (at < 64))
    else:
        see = at <= i
        if c["window"]:
            see = see & (at > i - c["window"])
    see = see & there[:, :, None] & (j < n[:, None])[:, None, :]
    x = x.view(S, Hk, M, G, -1).masked_fill_(~see[:, None, :, None, :], -INF).view(S, Hk, M * G, -1)
    return x, rows, there, j, n


def _log_sums(st):
    """log sum exp of each token's and head's scores, as attention leaves it."""
    c = st["case"]
    x, rows, there, _, _ = _scores(st)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    lse = (top + torch.log(torch.exp(x.sub_(top)).sum(-1, keepdim=True)))[..., 0]
    S, Hk, M = lse.shape[0], c["kv_heads"], rows.shape[1]
    lse = lse.view(S, Hk, M, -1).transpose(1, 2).reshape(S, M, c["heads"])
    return lse[there].contiguous()


def _weights_plain(st):
    c = st["case"]
    Hk, P = c["kv_heads"], c["page"]
    x, rows, there, j, n = _scores(st)
    S, M = rows.shape
    lse = st["lse"][rows].view(S, M, Hk, -1).transpose(1, 2).reshape(S, Hk, -1, 1)
    drawn = torch.exp(x.sub_(lse)).sum(2).transpose(1, 2)  # S x keys x kv_heads
    slot = _slots(st, j, j < n[:, None])
    old = st["w"][slot // P, slot % P]
    kept = old * c["decay"] if c["decay"] else torch.zeros_like(old)
    fresh = torch.where((j < st["lens"].long()[:, None])[..., None], kept, torch.zeros_like(old)) + drawn
    st["w"][slot // P, slot % P] = torch.where((j < n[:, None])[..., None], fresh, old)
    return dict(weights=st["w"])


def _moved(st, caches, kept, first):
    """Row first + i of each request (and K/V head) becomes what row first + kept[i] was."""
    P, Hk = st["case"]["page"], st["case"]["kv_heads"]
    S, k = kept.shape[0], kept.shape[-1]
    kept = kept.long().view(S, -1, k).expand(S, Hk, k)
    there = kept >= 0
    base = first.long()[:, None, None]
    head = torch.arange(Hk, device=DEV)[None, :, None].expand(S, Hk, k)
    last = torch.full_like(kept, st["kc"].shape[0] * P - 1)
    src = _slots(st, base + kept, there)
    to = torch.where(there, _slots(st, base + torch.arange(k, device=DEV), there), last)
    for cache in caches:
        cache[to // P, to % P, head] = cache[src // P, src % P, head]
    return (first + there[:, 0].sum(1)).to(torch.int32)


def _released(st, held, new_lens):
    """The pages between new_lens and held tokens, behind the free ones."""
    P, free = st["case"]["page"], st["free"]
    at = torch.arange(st["table"].shape[1], device=DEV)[None, :]
    gone = (at >= ((new_lens + P - 1) // P)[:, None]) & (at < ((held + P - 1) // P)[:, None])
    place = st["free_count"].long() - 1 + torch.cumsum(gone.view(-1).long(), 0)
    last = free.numel() - 1
    place = torch.where(gone.view(-1), place, torch.full_like(place, last))
    free[place] = torch.where(gone.view(-1), st["table"].view(-1), free[last])
    return (st["free_count"] + gone.sum()).to(torch.int32)


def _verify_plain(st):
    c = st["case"]
    p, drawn = st["p"], c["drawn"]
    rows, there = _padded(st)
    S, N = rows.shape
    at = torch.arange(S, device=DEV)
    root = st["cu"].long()[:-1]
    tokens = st["tokens"].long()[rows]
    parent = torch.where(there, st["parent"].long()[rows], torch.full_like(rows, -2))
    r = st["r"][rows].double()
    one = torch.ones(S, dtype=torch.float64, device=DEV)
    if drawn:
        ids = st["ids"].long()
        mine, w, g = ids[root], torch.gather(p[root], 1, ids[root]), st["q"][root]
    else:
        # the target's probability of each node where its parent stands, nothing for one tried before
        px = p[root[:, None] + parent.clamp(min=0), tokens].double()
        again = (parent[:, :, None] == parent[:, None, :]) & (tokens[:, :, None] == tokens[:, None, :])
        px = torch.where((again & torch.ones(N, N, dtype=torch.bool, device=DEV).tril(-1)).any(2), torch.zeros_like(px), px)
    cur, count, Z, Q = torch.zeros_like(root), torch.zeros_like(root), one, one
    path = torch.full((S, c["depth"] + 1), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    said = torch.full((S, c["depth"] + 1), -1, dtype=torch.int64, device=DEV)
    place = torch.arange(c["depth"] + 1, device=DEV)[None, :]
    for x in range(1, N):
        tried = parent[:, x] == cur
        if drawn:
            hit = mine == tokens[:, x, None]
            gx, wx = (g * hit).sum(1).double(), (w * hit).sum(1).double()
            yes = tried & (r[:, x] * Z * gx < wx * Q)
            no = tried & ~yes
            share = torch.where(Q > 0, Z / Q, torch.zeros_like(Q)).float()
            took = torch.where(no[:, None], torch.minimum(w, share[:, None] * g), torch.zeros_like(w))
            Z = (Z - took.double().sum(1)).clamp(min=0)
            Q = torch.where(no, Q - gx, Q)
            w, g = w - took, torch.where(no[:, None] & hit, torch.zeros_like(g), g)
            row = root + x * there[:, x]
            moved = yes[:, None]
            mine, g = torch.where(moved, ids[row], mine), torch.where(moved, st["q"][row], g)
            w = torch.where(moved, p[row[:, None], mine], w)
            Q = torch.where(yes, one, Q)
        else:
            yes = tried & (r[:, x] * Z < px[:, x])
            Z = torch.where(tried & ~yes, (Z - px[:, x]).clamp(min=0), Z)
        Z = torch.where(yes, one, Z)
        said = torch.where(yes[:, None] & (place == count[:, None]), tokens[:, x, None], said)
        count = count + yes
        path = torch.where(yes[:, None] & (place == count[:, None]), x, path)
        cur = torch.where(yes, torch.full_like(cur, x), cur)
    left = p[root + cur]
    if drawn:
        left = left.scatter(1, mine, w)
    else:
        gone = torch.where(parent == cur[:, None], torch.zeros_like(r, dtype=torch.float32), torch.gather(left, 1, tokens))
        left = left.scatter_reduce(1, tokens, gone, "amin")
    left = torch.where((left > 0).any(1, keepdim=True), left, p[root + cur]).double()
    run_ = torch.cumsum(left, 1)
    pick = torch.searchsorted(run_, (st["u"].double() * run_[:, -1])[:, None], right=True)[:, 0]
    last = torch.where(left > 0, torch.arange(left.shape[1], device=DEV), -1).amax(1)
    said = torch.where(place == count[:, None], torch.minimum(pick, last)[:, None], said)
    new_lens = _moved(st, [st["kc"], st["vc"]], path, st["lens"])
    left = _released(st, st["lens"] + (st["cu"][1:] - st["cu"][:-1]), new_lens)
    i = torch.int32
    return dict(tokens=said.to(i), path=path.to(i), accepted=count.to(i), lens=new_lens, k_cache=st["kc"], v_cache=st["vc"],
                free=st["free"], left=left)


def _evict_plain(st):
    c = st["case"]
    lens = st["lens"].long()[:, None]
    j = torch.arange(max(st["host_lens"]), device=DEV)[None, :].expand(lens.shape[0], -1)
    slot = _slots(st, j, j < lens)
    w = st["w"][slot // c["page"], slot % c["page"]]  # S x positions x kv_heads
    stay = (j < c["sinks"]) | (j >= lens - c["recent"])
    w = torch.where(stay[..., None], torch.full_like(w, INF), w)
    w = torch.where((j < lens)[..., None], w, torch.full_like(w, -INF)).transpose(1, 2)
    kept = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., : c["budget"]]
    past = j.shape[1]
    kept = torch.sort(torch.where(kept < lens[..., None], kept, torch.full_like(kept, past)), dim=-1).values
    kept = torch.where(kept == past, torch.full_like(kept, -1), kept)
    if kept.shape[-1] < c["budget"]:
        kept = torch.cat([kept, kept.new_full((*kept.shape[:2], c["budget"] - kept.shape[-1]), -1)], -1)
    new_lens = _moved(st, [st["kc"], st["vc"], st["moved"]], kept, torch.zeros_like(st["lens"]))
    left = _released(st, st["lens"], new_lens)
    return dict(kept=kept.to(torch.int32), lens=new_lens, k_cache=st["kc"], v_cache=st["vc"], weights=st["moved"], free=st["free"], left=left)


def run(st):
    c = st["case"]
    if not own:
        return dict(rotary=_rotary_plain, verify=_verify_plain, weights=_weights_plain, evict=_evict_plain)[c["op"]](st)
    import draft_lm_head_gb300 as L
    if c["op"] == "rotary":
        q, k = L.rotary(st["q"], st["k"], st["pos"], st["turns"], interleaved=c["pairs"], backward=c["back"], magnitude=st["magnitude"],
                        out=st["out"])
        return dict(q=q, k=k)
    if c["op"] == "weights":
        if "ws" not in st:
            st["ws"] = L.Workspace()
        w = L.cache_weights(st["q"], st["kc"], st["table"], st["lens"], st["cu"], st["lse"], st["w"], tree=st["tree"], window=c["window"],
                            scale=st["scale"], decay=c["decay"], workspace=st["ws"])
        return dict(weights=w)
    if c["op"] == "verify":
        tokens, path, accepted = L.verify_tree(st["p"], st["tokens"], st["parent"], st["cu"], st["r"], st["u"], c["depth"],
                                               cand_ids=st["ids"], cand_q=st["q"])
        lens = L.cache_keep([st["kc"], st["vc"]], st["table"], path, first=st["lens"])
        left = L.page_release(st["lens"], lens, st["table"], st["free"], st["free_count"], c["page"], cu=st["cu"])
        return dict(tokens=tokens, path=path, accepted=accepted, lens=lens, k_cache=st["kc"], v_cache=st["vc"], free=st["free"], left=left)
    kept = L.cache_select(st["w"], st["table"], st["lens"], c["budget"], sinks=c["sinks"], recent=c["recent"])
    lens = L.cache_keep([st["kc"], st["vc"], st["moved"]], st["table"], kept)
    left = L.page_release(st["lens"], lens, st["table"], st["free"], st["free_count"], c["page"])
    return dict(kept=kept, lens=lens, k_cache=st["kc"], v_cache=st["vc"], weights=st["moved"], free=st["free"], left=left)


# ---------------------------------------------------------------- work and 64-bit values

def work(case):
    op = case["op"]
    if op == "rotary":
        x = case["tokens"] * (case["heads"] + case["kv_heads"])
        return dict(bytes=2 * x * case["dim"] * SIZE[case["dtype"]], flops=3 * x * case["rot"])
    lens, new = _lengths(case, 1)
    Hk, D = case["kv_heads"], case["dim"]
    if op == "verify":
        # one row of the target's probabilities a request, the root's candidates, two rows moved
        S = case["requests"]
        return dict(bytes=S * (4 * case["vocab"] + (12 * case["cands"] if case["drawn"] else 0) + 4 * 2 * 2 * Hk * D),
                    flops=2 * S * case["vocab"])
    if op == "weights":
        pairs = keys = 0
        for l, m in zip(lens, new):
            w = case["window"]
            pairs += sum(min(w, l + i + 1) for i in range(m)) if w else m * l + m * (m + 1) // 2
            keys += min(l + m, w + m - 1) if w else l + m
        T = sum(new)
        return dict(bytes=2 * keys * Hk * D + 8 * keys * Hk + 2 * T * case["heads"] * D + 4 * T * case["heads"],
                    flops=2 * pairs * case["heads"] * D)
    stay = [min(l, case["budget"]) for l in lens]
    # a row that moves is read and written: all but the leading ones that stay where they are
    moved = sum(max(0, b - case["sinks"]) for b, l in zip(stay, lens) if l > case["budget"])
    return dict(bytes=4 * Hk * sum(lens) + 4 * Hk * sum(stay) + 2 * moved * Hk * (2 * D * 2 + 4), flops=Hk * sum(lens))


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None
    st = prepare(case, seed)
    if op == "rotary":
        rot, half = case["rot"], case["rot"] // 2
        out = {}
        for name, x in (("q", st["q"]), ("k", st["k"])):
            y = x.double().clone()
            back = torch.zeros_like(y) if st["out"] else x.double()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
                whole = st["pos"].long() * int(st["turns"][i])
                th = whole.double() * (math.pi * 2.0 ** -63)
                z = torch.polar(torch.full_like(th, st["magnitude"]), -th if case["back"] else th)[:, None]
                z = z * torch.complex(x[..., a].double(), x[..., b].double())
                y[..., a], y[..., b] = z.real, z.imag
            y[st["pos"] < 0] = back[st["pos"] < 0]
            out[name] = y
        return out
    P, Hk = case["page"], case["kv_heads"]
    if op == "weights":
        G = case["heads"] // Hk
        res = st["w"].double().clone()
        t = 0
        for s, (l, m) in enumerate(zip(st["host_lens"], st["host_new"])):
            where = torch.arange(l + m, device=DEV)
            page, off = st["table"][s].long()[where // P], where % P
            age = (l + torch.arange(m, device=DEV))[:, None] - where[None, :]
            hidden = age < 0
            if case["mask"] == "tree":
                hidden = torch.zeros(m, l + m, dtype=torch.bool, device=DEV)
                for node in range(m):
                    hidden[:, l + node] = ((st["tree"][t: t + m] >> node) & 1) == 0
            elif case["window"]:
                hidden = hidden | (age >= case["window"])
            for a in range(Hk):
                K = st["kc"][page, off, a].double()
                got = torch.zeros(l + m, dtype=torch.float64, device=DEV)
                for h in range(a * G, a * G + G):
                    y = (st["q"][t: t + m, h].double() @ K.T) * st["scale"] - st["lse"][t: t + m, h].double()[:, None]
                    got += torch.exp(y).masked_fill_(hidden, 0).sum(0)
                if case["decay"]:
                    got[:l] += case["decay"] * res[page[:l], off[:l], a]
                res[page, off, a] = got
            t += m
        return dict(weights=res)
    caches = {"k_cache": st["kc"], "v_cache": st["vc"], "weights": st["moved"]}
    for s, l in enumerate(st["host_lens"]):
        if l <= case["budget"]:
            continue
        where = torch.arange(l, device=DEV)
        page, off = st["table"][s].long()[where // P], where % P
        for a in range(Hk):
            w = st["w"][page, off, a].double()
            must = (where < case["sinks"]) | (where >= l - case["recent"])
            some = where[~must]
            more = case["budget"] - int(must.sum())
            top = torch.sort(w[some], descending=True, stable=True).indices[:more]
            keep = torch.sort(torch.cat([where[must], some[top]])).values
            n = keep.numel()
            for x in caches.values():
                x[page[:n], off[:n], a] = x[page[keep], off[keep], a]
    return dict(kept=None, lens=None, free=None, left=None, **caches)
