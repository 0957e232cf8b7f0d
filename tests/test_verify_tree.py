"""Verification of draft trees: the oracle by hand and by what its tokens are
distributed as, refusals on the host, and the kernel against it. Tokens, paths and
counts have to be equal: both take the same decisions on the same fp32 weights, with
masses and running sums of 48 bits or more on either side, so a decision could
differ only where a uniform lies within 1e-13 of its border."""
import numpy as np
import pytest

from oracle import speculative_oracle as SP
from oracle import step_oracle as O

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


def test_oracle_by_hand():
    p = np.array([[0.5, 0.3, 0.2, 0.0], [0.1, 0.1, 0.1, 0.7], [0.25, 0.25, 0.25, 0.25]], dtype=np.float32)
    tok, par = [9, 1, 0], [-1, 0, 0]
    # 1 accepted: the last token from p behind it
    assert O.verify_tree(p, tok, par, [0, 0.2, 0], 0.5) == ([1, 3], [0, 1])
    # 1 rejected (0.3 = p), then 0 accepted: 0.7 * 0.71 < 0.5
    assert O.verify_tree(p, tok, par, [0, 0.31, 0.71], 0.3) == ([0, 1], [0, 2])
    # both rejected: 2 is all that is left
    assert O.verify_tree(p, tok, par, [0, 0.31, 0.72], 0.99) == ([2], [0])
    # the same token twice: nothing is left of it
    assert O.verify_tree(p, [9, 1, 1], par, [0, 0.31, 0.0], 0.0) == ([0], [0])
    # drawn from q: 1 has q = 0.6, accepted below 0.3 / 0.6; then w = (0.5 - 0.4, 0, 0.2), Z = 0.3 and q = (1, 0)
    ids, q = [[0, 1]] * 3, [[0.4, 0.6]] * 3
    assert O.verify_tree(p, tok, par, [0, 0.49, 0], 0.0, ids, q)[1] == [0, 1]
    assert O.verify_tree(p, tok, par, [0, 0.51, 0.33], 0.0, ids, q)[1] == [0, 2]
    assert O.verify_tree(p, tok, par, [0, 0.51, 0.34], 0.0, ids, q) == ([2], [0])
    assert O.verify_tree(p, [9, 3, 0], par, [0, 0.5, 0.5], 0.0, ids, q) is None


@pytest.mark.parametrize("drawn", [False, True])
def test_tokens_come_out_as_the_targets(drawn):
    """Two children of the root, one child of the first: over many draws the first
    token is distributed as p at the root, and the second, behind each first, as p
    there. 40000 draws: a share's standard deviation is at most 0.0025."""
    rng = np.random.default_rng(5)
    n, N = 6, 40000
    p = rng.dirichlet(np.ones(n) * 0.7, 4).astype(np.float32)
    q = rng.dirichlet(np.ones(4), 4).astype(np.float32)
    ids = np.array([[0, 1, 3, 5]] * 4)
    first = np.zeros(n)
    for _ in range(N):
        if drawn:
            kids = ids[0][rng.choice(4, 2, replace=False, p=q[0] / q[0].astype(float).sum())]
            grand = ids[1][rng.choice(4, p=q[1] / q[1].astype(float).sum())]
        else:
            kids, grand = [1, 3], 0
        said, path = O.verify_tree(p, [0, kids[0], kids[1], grand], [-1, 0, 0, 1], rng.random(4), rng.random(),
                                   ids if drawn else None, q if drawn else None)
        first[said[0]] += 1
    assert np.abs(first / N - p[0]).max() < 0.0125  # five standard deviations


@pytest.mark.parametrize("drawn", [False, True])
def test_second_tokens_come_out_as_the_targets(drawn):
    """Behind each accepted first token the second is distributed as the target behind that
    token, whose row depends on it: over m such draws every share p within five standard
    deviations, 5 sqrt(p (1 - p) / m), and eight draws more for rare ones."""
    rng = np.random.default_rng(15)
    n, N = 6, 40000
    root = np.array([0.25, 0.3, 0.05, 0.2, 0.1, 0.1], dtype=np.float32)  # (each child is met often)
    behind = rng.dirichlet(np.ones(n) * 0.7, n).astype(np.float32)  # by the token before
    q = rng.dirichlet(np.ones(4), 2).astype(np.float32)
    ids = np.array([0, 1, 3, 5])
    pick = lambda row, k: ids[rng.choice(4, k, replace=False, p=row / row.astype(float).sum())]
    second = np.zeros((n, n))
    for _ in range(N):
        kids = pick(q[0], 2) if drawn else [1, 3]
        grand = [pick(q[1], 2) if drawn else np.argsort(-behind[k])[:2] for k in kids]  # (given: the likely ones)
        tokens = [0, kids[0], kids[1], grand[0][0], grand[1][0], grand[0][1], grand[1][1]]
        p = np.stack([root, behind[kids[0]], behind[kids[1]]] + [behind[0]] * 4)
        said, path = O.verify_tree(p, tokens, [-1, 0, 0, 1, 2, 1, 2], rng.random(7), rng.random(), [ids] * 7 if drawn else None,
                                   [q[0], q[1], q[1]] + [q[0]] * 4 if drawn else None)
        if len(path) > 1:
            second[said[0], said[1]] += 1
    met = second.sum(1)
    assert (met > 4000).sum() >= 2
    for t in np.nonzero(met > 1000)[0]:
        b = behind[t].astype(float)
        assert np.all(np.abs(second[t] / met[t] - b) < 5 * np.sqrt(b * (1 - b) / met[t]) + 8 / met[t]), t


def test_a_chain_is_the_chain_rule():
    rng = np.random.default_rng(6)
    n, K, Kd = 50, 12, 4
    for _ in range(300):
        p = rng.dirichlet(np.ones(n), Kd + 1).astype(np.float32)
        ids = np.stack([rng.permutation(n)[:K] for _ in range(Kd + 1)])
        q = rng.dirichlet(np.ones(K), Kd + 1).astype(np.float32)
        x = [ids[t][rng.integers(K)] for t in range(Kd)]
        r, u = rng.random(Kd).astype(np.float32), np.float32(rng.random())
        count, out = SP.verify_chain(p, x, ids[:Kd], q[:Kd], r, np.full(Kd + 1, u))
        said, path = O.verify_tree(p, [0] + x, list(range(-1, Kd)), np.concatenate([[0], r]), u, ids, q)
        assert said == out and path == list(range(count + 1))


@pytest.fixture(scope="module")
def clib():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    return _lib.load()


@pytest.mark.parametrize("want,kw", [
    (-1, dict(p=None)), (-1, dict(tokens=None)), (-1, dict(ids=OK)), (-1, dict(path=None)), (-1, dict(u=None)),
    (-2, dict(n=0)), (-2, dict(n=1 << 31)), (-2, dict(S=0)), (-2, dict(T=0)), (-2, dict(depth=-1)), (-2, dict(depth=64)), (-2, dict(path=2 * OK + 28)), (-2, dict(path=3 * OK - 4)),
    (-2, dict(ids=OK, q=OK, K=0)), (-5, dict(ids=OK, q=OK, K=4097)), (-2, dict(S=70000)),
])
def test_refusals(clib, want, kw):
    a = dict(p=OK, n=100, tokens=OK, u=OK, ids=None, q=None, K=8, S=2, T=4, depth=3, path=4 * OK)
    a.update(kw)
    assert clib.lmhead_verify_tree(a["p"], a["n"], a["tokens"], OK, OK, None, OK, a["u"], a["ids"], a["q"], a["K"], a["S"], a["T"],
                                   a["depth"], 2 * OK, a["path"], 3 * OK, None) == want


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        L.verify_tree(torch.zeros(2, 4), i, i, i, torch.zeros(2), torch.zeros(1), 2)


def _tree(rng, m, spread):
    return [-1 if c == 0 else int(rng.integers(max(0, c - spread), c)) for c in range(m)]


def _depths(parent):
    d = []
    for c, p in enumerate(parent):
        d.append(0 if c == 0 or not 0 <= p < c else d[p] + 1)
    return d


def _case(rng, counts, n, K, drawn, spread, flat=False):
    """Trees whose children are candidates of their parent, likely ones first or
    drawn without replacement, and a target not far from the drafter."""
    T = sum(counts)
    logits = rng.standard_normal((T, n)) * (0.1 if flat else 1.0)
    ids = np.stack([rng.permutation(n)[:K] for _ in range(T)])
    mine = rng.standard_normal((T, K)) * 2 + np.log(n)
    np.put_along_axis(logits, ids, mine, 1)
    soft = lambda x: (lambda e: (e / e.sum(1, keepdims=True)).astype(np.float32))(np.exp(x - x.max(1, keepdims=True)))
    p, q = soft(logits), soft(mine + 0.7 * rng.standard_normal((T, K)))
    parent, tokens, base = [], np.zeros(T, dtype=np.int64), 0
    for m in counts:
        par = _tree(rng, m, spread)
        for c in range(m):
            kids = [x for x in range(c + 1, m) if par[x] == c]
            if kids:
                key = np.log(np.maximum(q[base + c], 1e-30))
                if drawn:
                    key = key + rng.gumbel(size=K)
                order = np.argsort(-key, kind="stable")
                for i, x in enumerate(kids):
                    tokens[base + x] = ids[base + c][order[i % K]]
        parent += par
        base += m
    return dict(p=p, q=q, ids=ids, tokens=tokens, parent=np.array(parent, dtype=np.int64), r=rng.random(T).astype(np.float32),
                u=rng.random(len(counts)).astype(np.float32), cu=np.concatenate([[0], np.cumsum(counts)]))


def _run(L, c, drawn, depth, granted=None, stream=None):
    import torch
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    f32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")
    return L.verify_tree(f32(c["p"]), i32(c["tokens"]), i32(c["parent"]), i32(c["cu"]), f32(c["r"]), f32(c["u"]), depth,
                         cand_ids=i32(c["ids"]) if drawn else None, cand_q=f32(c["q"]) if drawn else None,
                         granted=None if granted is None else i32(granted), stream=stream)


def _want(c, s, drawn):
    a, b = int(c["cu"][s]), int(c["cu"][s + 1])
    return O.verify_tree(c["p"][a:b], c["tokens"][a:b], c["parent"][a:b], c["r"][a:b], c["u"][s], c["ids"][a:b] if drawn else None,
                         c["q"][a:b] if drawn else None)


def _compare(c, got, drawn, depth, gone=()):
    said, path, acc = (x.cpu().numpy() for x in got)
    total = 0
    for s in range(len(c["cu"]) - 1):
        want = None if s in gone or c["cu"][s] == c["cu"][s + 1] else _want(c, s, drawn)
        if want is None:
            assert acc[s] == -1 and (said[s] == -1).all() and (path[s] == -1).all(), s
            continue
        pad = lambda x: list(x) + [-1] * (depth + 1 - len(x))
        assert acc[s] == len(want[1]) - 1 and path[s].tolist() == pad(want[1]) and said[s].tolist() == pad(want[0]), (s, want, said[s])
        total += acc[s]
    return total


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("counts,n,K,spread", [
    ([1], 1, 1, 1), ([2], 7, 3, 1), ([64], 1000, 40, 6), ([10] * 8, 5000, 64, 4), ([1, 5, 64, 3, 0, 17], 999, 100, 12),
    ([12] * 40, 33, 20, 3), ([6, 6], 300007, 4096, 6), ([9] * 3, 128256, 1002, 9), ([30] * 5, 40, 33, 30)])
def test_against_oracle(drawn, counts, n, K, spread):
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(n + K)
    for flat in (False, True):
        c = _case(rng, counts, n, K, drawn, spread, flat)
        depth = min(63, max(max(_depths(c["parent"][a:b])) if b > a else 0 for a, b in zip(c["cu"], c["cu"][1:])))
        got = _run(L, c, drawn, depth)
        assert L.last_device_error() == 0
        _compare(c, got, drawn, depth)


@pytest.mark.gpu
def test_repeated_runs_accept_and_reject():
    """Over many uniforms every kind of end is met: none, some and all accepted."""
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(2)
    for drawn in (False, True):
        seen = set()
        for _ in range(6):
            c = _case(rng, [8] * 60, 500, 30, drawn, 2)
            got = _run(L, c, drawn, 7)
            _compare(c, got, drawn, 7)
            seen |= set(got[2].cpu().tolist())
        assert {0, 1, 2, 3} <= seen


@pytest.mark.gpu
def test_edges():
    """Uniforms at their ends, weights of nothing, the same token and the same
    candidate twice, nodes that are no one's children, NaN and negative entries."""
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(3)
    for drawn in (False, True):
        c = _case(rng, [10] * 12, 3000, 50, drawn, 4)
        c["u"][:3] = 0.0
        c["u"][3:6] = 1.0
        c["u"][6] = np.float32(1 - 2 ** -24)
        c["r"][:30] = 0.0
        c["r"][30:60] = 1.0
        for t in range(60, 80):  # one entry has it all
            c["p"][t] = 0
            c["p"][t, rng.integers(3000)] = 1
        c["p"][80:90, 100:] = 0
        c["p"][85] = 0          # a row of nothing
        c["p"][90:100, ::7] = np.nan
        c["p"][100:110, ::5] = -0.25
        c["parent"][rng.random(120) < 0.1] = -1
        c["parent"][5], c["parent"][17] = 9, 7  # no earlier node
        c["tokens"][44:48] = c["tokens"][41]
        if drawn:
            c["ids"][:40, 1] = c["ids"][:40, 0]  # listed twice
            c["ids"][40:50, 30:] = -1
            c["ids"][50:60, 40:] = 3000
            c["q"][60:70] = 0
        got = _run(L, c, drawn, 9)
        bad = [s for s in range(12) if _want(c, s, drawn) is None]
        assert (L.last_device_error() == -7) == bool(bad)
        _compare(c, got, drawn, 9)


@pytest.mark.gpu
def test_what_is_no_tree():
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(4)
    c = _case(rng, [6, 6, 6, 6], 200, 20, False, 1)
    c["r"][:] = 0  # all accepted: five drafts
    assert _run(L, c, False, 5)[2].tolist() == [5] * 4 and L.last_device_error() == 0
    assert _run(L, c, False, 4)[2].tolist() == [-1] * 4 and L.last_device_error() == -7  # deeper than depth
    got = _run(L, c, False, 5, granted=[1, 0, 1, 5])
    assert L.last_device_error() == 0
    _compare(c, got, False, 5, gone=(1,))
    d = dict(c, tokens=c["tokens"].copy())
    d["tokens"][7] = 200
    d["tokens"][13] = -1
    assert _run(L, d, False, 5)[2].tolist() == [5, -1, -1, 5] and L.last_device_error() == -7
    for cu in ([0, 6, 3, 9, 24], [-1, 6, 12, 18, 24], [0, 6, 12, 18, 25]):
        acc = _run(L, dict(c, cu=np.array(cu)), False, 5)[2].tolist()
        assert -1 in acc and L.last_device_error() == -7
    big = _case(rng, [65, 3], 200, 20, False, 4)
    assert _run(L, big, False, 63)[2].tolist()[0] == -1 and L.last_device_error() == -7


@pytest.mark.gpu
def test_chain_agrees_with_verify_chain():
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(8)
    B, Kd, n, K = 16, 5, 2000, 40
    c = _case(rng, [Kd + 1] * B, n, K, True, 1)
    said, path, acc = _run(L, c, True, Kd)
    dev = lambda x, t: torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")
    at = np.arange(B * (Kd + 1)).reshape(B, Kd + 1)
    tok, count = L.verify_chain(dev(c["p"].reshape(B, Kd + 1, n), torch.float32), dev(c["tokens"][at[:, 1:]], torch.int32),
                                dev(c["ids"][at[:, :-1]], torch.int32), dev(c["q"][at[:, :-1]], torch.float32),
                                dev(c["r"][at[:, 1:]], torch.float32), dev(np.repeat(c["u"][:, None], Kd + 1, 1), torch.float32))
    assert torch.equal(acc, count) and torch.equal(said, tok)


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
def test_rows_behind_the_first_billions(drawn):
    """The last rows of a p with more than 2^31 entries."""
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(10)
    n, T, m = 200001, 10800, 12
    assert T * n > 2 ** 31
    c = _case(rng, [m], n, 40, drawn, 3)
    p = torch.full((T, n), 0.5, device="cuda")
    p[T - m:] = torch.tensor(c["p"], device="cuda")
    i32 = lambda x: torch.tensor(np.concatenate([np.zeros((T - m,) + x.shape[1:], dtype=x.dtype), x]), dtype=torch.int32, device="cuda")
    f32 = lambda x: torch.tensor(np.concatenate([np.zeros((T - m,) + x.shape[1:], dtype=x.dtype), x]), dtype=torch.float32, device="cuda")
    cu = torch.tensor([T - m, T], dtype=torch.int32, device="cuda")
    got = L.verify_tree(p, i32(c["tokens"]), i32(c["parent"]), cu, f32(c["r"]), torch.tensor(c["u"], device="cuda"), m,
                        cand_ids=i32(c["ids"]) if drawn else None, cand_q=f32(c["q"]) if drawn else None)
    _compare(c, got, drawn, m)


@pytest.mark.gpu
def test_streams_graphs_and_binding():
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(9)
    c = _case(rng, [10] * 4, 3000, 50, True, 3)
    want = _run(L, c, True, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(L, c, True, 9, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    f32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")
    args = [f32(c["p"]), i32(c["tokens"]), i32(c["parent"]), i32(c["cu"]), f32(c["r"]), f32(c["u"]), 9]
    cands = dict(cand_ids=i32(c["ids"]), cand_q=f32(c["q"]))
    out = tuple(torch.zeros_like(x) for x in want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.verify_tree(*args, **cands, out=out)
    for _ in range(2):
        for x in out:
            x.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    for bad in (dict(cand_ids=cands["cand_ids"]), dict(cands, cand_q=cands["cand_q"][:, :3]), dict(cands, granted=i32([1])),
                dict(cands, out=(out[0], out[1][:, :4], out[2]))):
        with pytest.raises((TypeError, ValueError)):
            L.verify_tree(*args, **bad)
    with pytest.raises(ValueError):
        L.verify_tree(*args[:6], 64, **cands)
    with pytest.raises((TypeError, ValueError)):
        L.verify_tree(args[0].t().contiguous().t(), *args[1:], **cands)


# ---- targets between two sums. The kernel adds up a row of p in levels (8 CTAs, 16 warps, 32
# lanes) in pairs of fp32 numbers; sums of the same entries taken in two orders differ in their
# last bit. A target that lies between the two belongs to the entry before or behind.

f32 = np.float32


def _add(a, b):
    s, (h, l) = f32(a[0] + b[0]), (a[0], b[0])
    t = f32(s - h)
    e = f32(f32(f32(h - f32(s - t)) + f32(l - t)) + f32(a[1] + b[1]))
    r = f32(s + e)
    return r, f32(e - f32(r - s))


def _scan(x):
    x = list(x) + [(f32(0), f32(0))] * (32 - len(x))
    o = 1
    while o < 32:
        x = [_add(x[i - o], x[i]) if i >= o else x[i] for i in range(32)]
        o *= 2
    return x


def _butterfly(x):
    o = len(x) // 2
    while o:
        x = [_add(x[i], x[i ^ o]) for i in range(len(x))]
        o //= 2
    return x[0]


def _exactly(pair):
    from fractions import Fraction
    return Fraction(float(pair[0])) + Fraction(float(pair[1]))


def _filled(row, at, total):
    """row with the entries at `at` (two places) such that it sums to `total`, exactly or less."""
    from fractions import Fraction
    need = total - sum(Fraction(float(x)) for x in row)
    if need <= 0:
        return False
    for i in at:
        x = f32(float(need))
        x = np.nextafter(x, f32(0)) if Fraction(float(x)) > need else x
        row[i] = x
        need -= Fraction(float(x))
    return True


def _between(rng, step):
    """A row of 4096 of which half the sum lies between the sum of its first four parts of
    `step` entries, one by one, and the same four in a tree; or, with step 1, between the
    first 32 in a tree and in another. Returns it and the two entries at that border."""
    while True:
        row = np.zeros(4096, dtype=f32)
        if step > 1:
            at = lambda c: [c * step + 3, c * step + 20]
            for c in range(7):
                big = (rng.random() * 0.1 + 0.02) * (0.6 if c > 3 else 1.0)
                row[at(c)] = big, big * 2.0 ** -25 * (1 + rng.random())
            part = [_add((row[at(c)[0]], f32(0)), (row[at(c)[1]], f32(0))) for c in range(7)]
            to = _scan(part)
            low, high = _add(to[2], part[3]), to[3]
            fill, border = at(7), (at(3)[1], at(4)[0])
        else:
            row[:32] = (rng.random(32) + 0.5) * 2.0 ** -rng.integers(4, 40, 32)
            each = [(x, f32(0)) for x in row[:32]]
            low, high = _scan(each)[31], _butterfly(each)
            fill, border = [40, 300], (31, 40)
        if low < high and _filled(row, fill, 2 * _exactly(low)):
            return row, border


@pytest.mark.gpu
@pytest.mark.parametrize("step", [512, 32, 1])
def test_targets_between_two_sums(step):
    """(512 entries a CTA, 32 a warp, one a lane.) Every request gets an entry at the border,
    whatever the results held before."""
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(step)
    S = 32
    rows, borders = zip(*(_between(rng, step) for _ in range(S)))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    for spread in (0, 1):  # with nothing behind, and with entries that do not reach the sum's last bit
        p = np.stack(rows)
        if spread:
            p[:, 2000::500] = np.where(p[:, 2000::500] > 0, p[:, 2000::500], 1e-30)
        out = tuple(torch.full(s, -5, dtype=torch.int32, device="cuda") for s in ((S, 1), (S, 1), (S,)))
        L.verify_tree(torch.tensor(p, device="cuda"), i32([0] * S), i32([-1] * S), i32(range(S + 1)), torch.zeros(S, device="cuda"),
                      torch.full((S,), 0.5, device="cuda"), 0, out=out)
        assert L.last_device_error() == 0 and out[2].tolist() == [0] * S
        got = out[0][:, 0].tolist()
        # (an entry of 1e-30 between the two lies at the border itself: any sum of pairs, 2^-48 of
        # some 0.4 at its finest, is the same with it and without)
        right = [b[0] <= g <= b[1] and row[g] > 0 for g, b, row in zip(got, borders, p)]
        assert all(right), [(g, b) for g, b, r in zip(got, borders, right) if not r][:5]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [5, 4096, 300007])
def test_uniforms_outside_their_range(n):
    """Below 0: the first entry with a weight; 1, above it and NaN: the last."""
    import torch
    from gpu_util import lib
    L = lib()
    u = [-0.25, -1e-30, -np.inf, -3e38, 1.0, 1.5, np.inf, np.nan]
    S = len(u)
    p = torch.zeros(S, n, device="cuda")
    p[:, 1:n - 1] = torch.rand(S, n - 2, device="cuda") + 0.1
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    out = tuple(torch.full(s, -5, dtype=torch.int32, device="cuda") for s in ((S, 1), (S, 1), (S,)))
    L.verify_tree(p, i32([0] * S), i32([-1] * S), i32(range(S + 1)), torch.zeros(S, device="cuda"),
                  torch.tensor(u, dtype=torch.float32, device="cuda"), 0, out=out)
    assert L.last_device_error() == 0
    assert out[0][:, 0].tolist() == [1] * 4 + [n - 2] * 4
