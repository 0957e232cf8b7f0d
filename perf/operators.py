"""The serving operators around the draft head, as timed cases.

Four operators: page_plan (block tables and slot maps from request lengths), chunk_attention (a chunk
of new tokens over a paged cache, their K and V written first), q4 (4-bit head with group scales, over
every row or over candidate rows) and beams (selection over beams and vocabulary, then the states'
reordering). `own` picks between the plain torch form of each and the framework's call.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one decoding step of 64 requests: a token each, a page now and then
        dict(name="pages decode 64", op="pages", requests=64, new_lo=1, new_hi=1, ctx=4096, page=16, scarce=False),
        # admission of prompts next to decoding requests, the pool running out on the way
        dict(name="pages prompts 1500", op="pages", requests=1500, new_lo=0, new_hi=700, ctx=3000, page=32, scarce=True),
        # the smallest call: one request, one token
        dict(name="attn token", op="attn", requests=1, new=1, ctx=2000, ragged=False, heads=32, kv_heads=8, dim=128,
             page=16, mask="causal", window=0, dtype="bf16"),
        # 8 concurrent sequences, a 10-node draft tree each
        dict(name="attn tree 8x10", op="attn", requests=8, new=10, ctx=4100, ragged=True, heads=64, kv_heads=8, dim=64,
             page=64, mask="tree", window=0, dtype="bf16"),
        # decoding of a ragged batch: all of the cache is read
        dict(name="attn decode 32", op="attn", requests=32, new=1, ctx=8000, ragged=True, heads=32, kv_heads=8, dim=128,
             page=32, mask="causal", window=0, dtype="fp16"),
        # chunks of two long prompts over what was cached before
        dict(name="attn prompt 2x2048", op="attn", requests=2, new=2048, ctx=6144, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, mask="causal", window=0, dtype="bf16"),
        # one hidden vector through the whole vocabulary
        dict(name="q4 head 1", op="q4", rows=128256, d=4096, group=128, vectors=1, cands=0, mins=False, dtype="bf16"),
        # the candidates of 64 hidden vectors
        dict(name="q4 candidates 64", op="q4", rows=128256, d=4096, group=128, vectors=64, cands=1002, mins=False, dtype="bf16"),
        # a wide head, small groups with offsets, several hidden vectors
        dict(name="q4 wide head 16", op="q4", rows=151936, d=5120, group=64, vectors=16, cands=0, mins=True, dtype="fp16"),
        # one drafted sequence: 4 beams over the head's candidates
        dict(name="beam candidates 4", op="beam", seqs=1, beams=4, k=4, entries=1002, ids=True, d=4096, dtype="fp32", done=False),
        # 16 sequences over the whole vocabulary
        dict(name="beam vocabulary 16x4", op="beam", seqs=16, beams=4, k=4, entries=128256, ids=False, d=4096, dtype="bf16", done=True),
        # the largest: 64 sequences of 8 beams
        dict(name="beam vocabulary 64x8", op="beam", seqs=64, beams=8, k=8, entries=151936, ids=False, d=5120, dtype="fp32", done=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "attn", "attn", "q4", "q4", "beam"])
    if op == "pages":
        lo = rng.choice([0, 1])
        requests = _log(rng, 1, 1500)
        return dict(op=op, requests=requests, new_lo=lo, new_hi=max(lo, _log(rng, 1, 700)), ctx=_log(rng, 1, 20000),
                    page=rng.choice([16, 32, 64, 128]), scarce=rng.random() < 0.4)
    if op == "attn":
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        dim = rng.choice([64, 128])
        mask = rng.choice(["causal", "causal", "tree", "window"])
        new = rng.randint(1, 64) if mask == "tree" else rng.choice([1, _log(rng, 1, 2048)])
        ctx = rng.choice([rng.randint(0, 200), _log(rng, 1, 16000)])
        most = min(0.4e12 / (4.0 * new * (ctx + new) * heads * dim), 6e8 / (4.0 * kv_heads * dim * (ctx + new)), 64)
        return dict(op=op, requests=_log(rng, 1, max(1, int(most))), new=new, ctx=ctx, ragged=rng.random() < 0.6, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]), mask=mask,
                    window=rng.choice([1, 100, 128, 1000]) if mask == "window" else 0, dtype=rng.choice(["bf16", "fp16"]))
    if op == "q4":
        group = rng.choice([32, 64, 128])
        d = group * rng.randint(max(1, 256 // group), 5120 // group)
        rows = _log(rng, 1000, 150000)
        cands = rng.choice([0, _log(rng, 1, 2376)])
        return dict(op=op, rows=rows, d=d, group=group, vectors=_log(rng, 1, 64 if cands else 16), cands=cands,
                    mins=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
    entries = _log(rng, 50, 150000)
    beams = rng.randint(1, 16)
    seqs = _log(rng, 1, max(1, min(64, 70_000_000 // (entries * beams))))
    return dict(op=op, seqs=seqs, beams=beams, k=rng.randint(1, 16), entries=entries, ids=rng.random() < 0.5,
                d=8 * rng.randint(8, 640), dtype=rng.choice(["fp32", "bf16", "fp16"]), done=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lengths(case, seed):
    """Context and new lengths of each request, on the host: what a scheduler knows. The seed deals
    the same lengths out in another order, so that a case's sizes are its own."""
    r = random.Random(13)
    n = case["requests"]
    if case["op"] == "pages":
        pairs = [(r.randint(0, case["ctx"]), r.randint(case["new_lo"], case["new_hi"])) for _ in range(n)]
    elif not case["ragged"]:
        pairs = [(case["ctx"], case["new"])] * n
    else:
        pairs = [(r.randint(case["ctx"] // 2, case["ctx"]), r.randint(max(1, case["new"] // 2), case["new"])) for _ in range(n)]
    random.Random(seed).shuffle(pairs)
    return [p[0] for p in pairs], [p[1] for p in pairs]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tree_bits(new, r):
    """Ancestor bits (own bit included) of each node of a random draft tree."""
    bits = []
    for i in range(new):
        bits.append((bits[r.randint(max(0, i - 4), i - 1)] if i else 0) | (1 << i))
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "pages":
        lens, new = _lengths(case, seed)
        P = case["page"]
        held = [-(-l // P) for l in lens]
        need = [-(-(l + m) // P) - h for l, m, h in zip(lens, new, held)]
        width = max(h + n for h, n in zip(held, need)) or 1
        pool = sum(held) + (sum(need) * 2 // 3 if case["scarce"] else sum(need) + 64)
        perm = torch.randperm(max(pool, 1), generator=g, device=DEV).to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(width, device=DEV)
        mask = col[None, :] < _i32(held)[:, None]
        table[mask] = perm[: sum(held)]
        free = perm[sum(held):].contiguous()
        if free.numel() == 0:
            free = torch.zeros(1, dtype=torch.int32, device=DEV)
        st.update(lens=_i32(lens), new=_i32(new), table=table, free=free, free_count=_i32([pool - sum(held)]),
                  tokens=max(1, sum(new)))
    elif op == "attn":
        lens, new = _lengths(case, seed)
        t, P, D = TYPES[case["dtype"]], case["page"], case["dim"]
        Hq, Hk = case["heads"], case["kv_heads"]
        pages = [-(-(l + m) // P) for l, m in zip(lens, new)]
        total = sum(pages) + 3
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(max(pages), device=DEV)[None, :] < _i32(pages)[:, None]] = perm[: sum(pages)]
        T = sum(new)
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        # the projection's output: q, k and v side by side
        qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device=DEV).to(t)
        kc, vc = (torch.randn(total, P, Hk, D, generator=g, device=DEV, dtype=t) for _ in range(2))
        lens_t, cu_t = _i32(lens), _i32(cu)
        req = torch.repeat_interleave(torch.arange(len(new), device=DEV), _i32(new).long())
        pos = torch.arange(T, device=DEV) - cu_t[req] + lens_t[req]
        slots = (table[req, pos // P] * P + pos % P).to(torch.int32)
        tree = None
        if case["mask"] == "tree":
            r = random.Random(seed * 31 + 5)
            tree = torch.tensor([b for m in new for b in _tree_bits(m, r)], dtype=torch.int64, device=DEV)
        st.update(lens=lens_t, cu=cu_t, table=table, q=qkv[:, :Hq], k=qkv[:, Hq: Hq + Hk], v=qkv[:, Hq + Hk:], kc=kc, vc=vc,
                  slots=slots, tree=tree, host_lens=lens, host_new=new, scale=D ** -0.5,
                  out=torch.empty(T, Hq, D, dtype=t, device=DEV), lse=torch.empty(T, Hq, device=DEV))
    elif op == "q4":
        t, n, d, grp, M = TYPES[case["dtype"]], case["rows"], case["d"], case["group"], case["vectors"]
        codes = torch.randint(0, 256, (n, d // 2), generator=g, device=DEV, dtype=torch.uint8)
        scales = ((torch.rand(n, d // grp, generator=g, device=DEV) + 0.5) / (4 * math.sqrt(d))).to(t)
        mins = (-scales.float() * (6 + 3 * torch.rand(n, d // grp, generator=g, device=DEV))).to(t) if case["mins"] else None
        h = torch.randn(M, d, generator=g, device=DEV).to(t)
        ids = None
        if case["cands"]:
            ids = torch.randint(0, n, (M, case["cands"]), generator=g, device=DEV, dtype=torch.int32)
        out = torch.empty(M, case["cands"] or n, device=DEV)
        st.update(codes=codes, scales=scales, mins=mins, h=h, ids=ids, out=out)
    else:
        t, S, B, n, k = TYPES[case["dtype"]], case["seqs"], case["beams"], case["entries"], case["k"]
        logits = torch.empty(S * B, n, device=DEV, dtype=torch.float32).normal_(0, 3, generator=g).to(t)
        scores = -5 * torch.rand(S * B, generator=g, device=DEV)
        ids = None
        if case["ids"]:
            ids = torch.randint(0, 150000, (S * B, n), generator=g, device=DEV, dtype=torch.int32)
        done = None
        if case["done"]:
            done = torch.rand(S * B, generator=g, device=DEV) < 0.1
        hidden = torch.randn(S * B, case["d"], generator=g, device=DEV).to(torch.bfloat16)
        tables = torch.randint(0, 100000, (S * B, 128), generator=g, device=DEV, dtype=torch.int32)
        st.update(logits=logits, scores=scores, ids=ids, done=done, hidden=hidden, tables=tables)
    if own:
        import draft_lm_head_gb300 as L
        st["L"] = L
        st["ws"] = L.Workspace()
    return st


# ---------------------------------------------------------------- plain forms and calls

def _pages_plain(st):
    P = st["case"]["page"]
    lens, new, table, free = st["lens"].long(), st["new"].long(), st["table"], st["free"]
    F = st["free_count"].long()
    T = st["tokens"]
    held = (lens + P - 1) // P
    need = (lens + new + P - 1) // P - held
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    fits = lens + new <= table.shape[1] * P
    need = torch.where(fits, need, torch.zeros_like(need))
    incl = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (incl <= F))
    excl = incl - need
    j = torch.arange(table.shape[1], device=DEV)[None, :] - held[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & granted[:, None]
    at = (F - 1 - excl[:, None] - j).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    tok = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=lens.numel() - 1)
    live = (tok < cu[-1]) & granted[req]
    pos = torch.where(live, lens[req] + tok - cu[req], torch.full_like(tok, -1))
    page = table[req, (pos.clamp(min=0) // P).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live, page * P + pos % P, torch.full_like(tok, -1))
    left = F - torch.where(granted, need, torch.zeros_like(need)).sum()
    i = torch.int32
    return dict(slots=slots.to(i), positions=pos.to(i), cu=cu.to(i), granted=granted.to(i), left=left.to(i), table=table)


def _attn_plain(st):
    c = st["case"]
    P, Hk, D = c["page"], c["kv_heads"], c["dim"]
    G = c["heads"] // Hk
    flat_k, flat_v = st["kc"].view(-1, Hk, D), st["vc"].view(-1, Hk, D)
    flat_k[st["slots"].long()] = st["k"]
    flat_v[st["slots"].long()] = st["v"]
    t0 = 0
    for s, (l, m) in enumerate(zip(st["host_lens"], st["host_new"])):
        n = l + m
        pages = st["table"][s, : -(-n // P)].long()
        K = st["kc"][pages].view(-1, Hk, D)[:n].float()
        V = st["vc"][pages].view(-1, Hk, D)[:n].float()
        i = torch.arange(m, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        if c["mask"] == "tree":
            bit = (st["tree"][t0: t0 + m, None] >> (j - l).clamp(min=0)) & 1
            see = (j < l) | (bit == 1)
        else:
            see = j <= l + i
            if c["window"]:
                see = see & (j > l + i - c["window"])
        for a in range(Hk):
            q = st["q"][t0: t0 + m, a * G: (a + 1) * G].float().transpose(0, 1)
            x = torch.matmul(q, K[:, a].T) * st["scale"]
            x = x.masked_fill(~see, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            o = torch.matmul(p, V[:, a]) / z
            st["out"][t0: t0 + m, a * G: (a + 1) * G] = o.transpose(0, 1).to(st["out"].dtype)
            st["lse"][t0: t0 + m, a * G: (a + 1) * G] = (top + torch.log(z))[..., 0].T
        t0 += m
    return dict(out=st["out"], lse=st["lse"], k_cache=st["kc"], v_cache=st["vc"])


def _q4_weight(st, rows, t):
    """The rows' weights in type t: low nibble first."""
    c = st["codes"][rows]
    q = torch.stack([c & 15, c >> 4], -1).view(*c.shape[:-1], -1, st["case"]["group"]).to(t)
    s = st["scales"][rows].to(t)[..., None]
    w = (q - 8) * s if st["mins"] is None else q * s + st["mins"][rows].to(t)[..., None]
    return w.view(*c.shape[:-1], -1)


def _q4_plain(st):
    h = st["h"].float()
    if st["ids"] is None:
        step = 32768
        for r in range(0, st["codes"].shape[0], step):
            w = _q4_weight(st, slice(r, r + step), torch.float32)
            st["out"][:, r: r + step] = torch.matmul(h, w.T)
    else:
        for m in range(h.shape[0]):
            st["out"][m] = torch.matmul(_q4_weight(st, st["ids"][m].long(), torch.float32), h[m])
    return dict(logits=st["out"])


def _beam_plain(st):
    c = st["case"]
    S, B, n, k = c["seqs"], c["beams"], c["entries"], c["k"]
    # 64 bits: scores of different beams come close to one another at the border of the k
    x = st["logits"].double()
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    x = st["scores"].double()[:, None] + (x - lse)
    eos = 2
    if st["done"] is not None:
        x = torch.where(st["done"][:, None], torch.full_like(x, -math.inf), x)
        x[:, 0] = torch.where(st["done"], st["scores"].double(), x[:, 0])
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x).view(S, B * n)
    index = torch.arange(B * n, device=DEV)[None, :]
    score, flat = [], []
    for _ in range(k):
        v = x.amax(1, keepdim=True)
        at = torch.where(x == v, index, B * n).amin(1, keepdim=True)
        score.append(v)
        flat.append(torch.where(v == -math.inf, -1, at))
        x.scatter_(1, at, -math.inf)
    score, flat = torch.cat(score, 1), torch.cat(flat, 1)
    live = flat >= 0
    beam = torch.where(live, flat // n, -1)
    row = torch.arange(S, device=DEV)[:, None] * B + beam.clamp(min=0)
    entry = flat.clamp(min=0) % n
    token = entry if st["ids"] is None else st["ids"][row, entry].long()
    if st["done"] is not None:
        token = torch.where(st["done"][row], eos, token)
    token = torch.where(live, token, -1)
    moved = [torch.where(live.view(-1, 1), t[row.view(-1)], torch.zeros_like(t[:1])) for t in (st["hidden"], st["tables"])]
    return dict(parent=beam.to(torch.int32), token=token.to(torch.int32), score=score.float(), hidden=moved[0], tables=moved[1])


def run(st):
    c = st["case"]
    if not own:
        return dict(pages=_pages_plain, attn=_attn_plain, q4=_q4_plain, beam=_beam_plain)[c["op"]](st)
    L, ws = st["L"], st["ws"]
    if c["op"] == "pages":
        p = L.page_plan(st["lens"], st["new"], st["table"], st["free"], st["free_count"], c["page"], st["tokens"])
        return dict(slots=p.slots, positions=p.positions, cu=p.cu, granted=p.granted, left=p.free_left, table=st["table"])
    if c["op"] == "attn":
        L.chunk_attention(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["cu"], k=st["k"], v=st["v"], slots=st["slots"],
                          tree=st["tree"], window=c["window"], scale=st["scale"], workspace=ws, out=(st["out"], st["lse"]))
        return dict(out=st["out"], lse=st["lse"], k_cache=st["kc"], v_cache=st["vc"])
    if c["op"] == "q4":
        if st["ids"] is None:
            L.q4_head(st["codes"], st["scales"], st["h"], c["group"], mins=st["mins"], workspace=ws, out=st["out"])
        else:
            L.q4_gather_logits(st["codes"], st["scales"], st["h"], st["ids"], c["group"], mins=st["mins"], workspace=ws, out=st["out"])
        return dict(logits=st["out"])
    parent, token, score = L.beam_select(st["logits"], st["scores"], c["beams"], c["k"], ids=st["ids"], finished=st["done"], eos=2,
                                         workspace=ws)
    hidden, tables = L.beam_reorder(parent, [st["hidden"], st["tables"]], c["beams"])
    return dict(parent=parent, token=token, score=score, hidden=hidden, tables=tables)


# ---------------------------------------------------------------- work and 64-bit values

def work(case):
    op = case["op"]
    if op == "pages":
        S, new = case["requests"], (case["new_lo"] + case["new_hi"]) / 2
        return dict(bytes=int(16 * S + S * new * 8 + S * (new / case["page"]) * 8), flops=int(S * new * 4))
    if op == "attn":
        lens, new = _lengths(case, 1)
        Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        pairs = keys = 0
        for l, m in zip(lens, new):
            w = case["window"]
            if w:
                pairs += sum(min(w, l + i + 1) for i in range(m))
                keys += min(l + m, w + m - 1)
            else:
                pairs += m * l + m * (m + 1) // 2
                keys += l + m
        T = sum(new)
        # what is cached is read once; the chunk's own K and V are read and written; q and out once
        bytes_ = 2 * (2 * keys * Hk * D + 4 * T * Hk * D + 2 * T * Hq * D) + 4 * T * Hq
        return dict(bytes=bytes_, flops=4 * pairs * Hq * D)
    if op == "q4":
        M, d, n = case["vectors"], case["d"], case["rows"]
        rows = min(n, M * case["cands"]) if case["cands"] else n
        outs = M * (case["cands"] or n)
        per = d // 2 + 2 * (d // case["group"]) * (2 if case["mins"] else 1)
        return dict(bytes=rows * per + 2 * M * d + 4 * outs * (2 if case["cands"] else 1), flops=2 * outs * d)
    S, B, n = case["seqs"], case["beams"], case["entries"]
    moved = S * case["k"] * (2 * case["d"] + 512)
    return dict(bytes=S * B * n * SIZE[case["dtype"]] + 2 * moved, flops=4 * S * B * n)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        return None
    if op == "attn":
        Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
        G = Hq // Hk
        st["kc"].view(-1, Hk, D)[st["slots"].long()] = st["k"]
        st["vc"].view(-1, Hk, D)[st["slots"].long()] = st["v"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
        t = 0
        for s, (l, m) in enumerate(zip(st["host_lens"], st["host_new"])):
            where = torch.arange(l + m, device=DEV)
            slot = st["table"][s].long()[where // P] * P + where % P
            hidden = torch.zeros(m, l + m, dtype=torch.bool, device=DEV)
            if case["mask"] == "tree":
                for node in range(m):
                    hidden[:, l + node] = ((st["tree"][t: t + m] >> node) & 1) == 0
            else:
                age = (l + torch.arange(m, device=DEV))[:, None] - where[None, :]
                hidden = age < 0
                if case["window"]:
                    hidden |= age >= case["window"]
            for a in range(Hq):
                K = st["kc"].view(-1, Hk, D)[slot, a // G].double()
                V = st["vc"].view(-1, Hk, D)[slot, a // G].double()
                x = (st["q"][t: t + m, a].double() @ K.T) * st["scale"]
                x[hidden] = -math.inf
                lse[t: t + m, a] = torch.logsumexp(x, 1)
                out[t: t + m, a] = torch.softmax(x, 1) @ V
            t += m
        return dict(out=out, lse=lse, k_cache=st["kc"].double(), v_cache=st["vc"].double())
    if op == "q4":
        h, grp = st["h"].double(), case["group"]
        n = case["rows"]
        out = torch.empty(st["out"].shape, dtype=torch.float64, device=DEV)
        for r in range(0, h.shape[0] if case["cands"] else n, 1 if case["cands"] else 16384):
            rows = st["ids"][r].long() if case["cands"] else torch.arange(r, min(n, r + 16384), device=DEV)
            code = st["codes"][rows].to(torch.int16)
            hs = h[r: r + 1] if case["cands"] else h
            y = torch.zeros(hs.shape[0], rows.numel(), dtype=torch.float64, device=DEV)
            for b in range(case["d"] // grp):
                part = code[:, b * grp // 2: (b + 1) * grp // 2]
                hb = hs[:, b * grp: (b + 1) * grp]
                dot = hb[:, 0::2] @ (part % 16).double().T + hb[:, 1::2] @ (part // 16).double().T
                s = st["scales"][rows, b].double()
                low = -8 * s if st["mins"] is None else st["mins"][rows, b].double()
                y += dot * s + hb.sum(1, keepdim=True) * low
            if case["cands"]:
                out[r] = y[0]
            else:
                out[:, r: r + rows.numel()] = y
        return dict(logits=out)
    S, B, n, k = case["seqs"], case["beams"], case["entries"], case["k"]
    best = torch.empty(S, k, dtype=torch.float64, device=DEV)
    for s in range(S):
        rows = slice(s * B, (s + 1) * B)
        v = torch.log_softmax(st["logits"][rows].double(), 1) + st["scores"][rows].double()[:, None]
        if st["done"] is not None:
            v = torch.cat([v[~st["done"][rows]].reshape(-1), st["scores"][rows][st["done"][rows]].double()])
        v = v.reshape(-1)
        take = min(k, v.numel())
        best[s, :take] = torch.topk(v, take).values
        best[s, take:] = -math.inf
    return dict(parent=None, token=None, score=best, hidden=None, tables=None)
