"""Attention weights summed up, the choice of tokens by them, rows moved together and
pages given back: oracles by hand, refusals on the host, the kernels against fp64.

What a summed weight may be off by, with R = max scale sum_d |q_d k_jd| and l = max
|lse| over the rows that see the key, n its terms: a logit's D products and its
scaling, each within one fp32 step: delta = (D + 4) 2^-23 R, a weight by 2 delta of
itself; the exponential and its argument (a difference of sizes R and l, both scaled
to base 2): 2^-20 + 2^-22 (R + l); the sum of n positive terms by n 2^-23; the
decayed old value by 2^-22 of itself. Choices and moved rows have to be equal."""
import numpy as np
import pytest

from oracle import step_oracle as O

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


# ------------------------------------------------------------------ no GPU

def test_oracles_by_hand():
    w = np.array([[5.0, 1.0], [3.0, 3.0], [np.nan, 9.0]])[:, :, None]  # three pages of two
    table = [[2, 0, 1]]
    pick = lambda L, b, s, r: O.cache_select(w, table, [L], 2, b, s, r)[0, 0].tolist()
    # positions hold NaN, 9, 5, 1, 3, 3
    assert pick(6, 3, 0, 0) == [1, 2, 4] and pick(6, 4, 0, 0) == [1, 2, 4, 5]
    assert pick(6, 3, 1, 1) == [0, 1, 5] and pick(6, 2, 2, 0) == [0, 1] and pick(6, 2, 0, 2) == [4, 5]
    assert pick(3, 5, 0, 0) == [0, 1, 2, -1, -1] and pick(0, 2, 1, 1) == [-1, -1] and pick(6, 1, 0, 0) == [1]
    c = np.arange(6.0).reshape(3, 2, 1)
    assert O.cache_keep(c, table, [[1, 2, 5, -1]], None, 2).tolist() == [3]
    assert c[2].ravel().tolist() == [5, 0] and c[0].ravel().tolist() == [3, 1]
    assert O.page_release([5, 2], [2, 2], [[7, 8, 9], [4, 5, 6]], [1, 2], 1, 2) == [1, 8, 9]
    # one head of one dimension, two cached keys and two new ones
    k = np.log(np.array([1., 2., 1., 4.])).reshape(2, 2, 1, 1)
    q = np.ones((2, 1, 1))
    lse = np.log([[4.0], [8.0]])
    old = np.array([[[10.0], [20.0]], [[30.0], [np.nan]]])
    got, _ = O.cache_weights(q, k, [[0, 1]], [2], [0, 2], lse, old, 1.0, decay=0.5)
    assert np.allclose(got.ravel(), [5 + 1 / 4 + 1 / 8, 10 + 2 / 4 + 2 / 8, 1 / 4 + 1 / 8, 4 / 8])
    got, _ = O.cache_weights(q, k, [[0, 1]], [2], [0, 2], lse, old, 1.0, window=2, decay=0.0)
    assert np.allclose(got.ravel(), [0, 2 / 4, 1 / 4 + 1 / 8, 4 / 8])
    got, _ = O.cache_weights(q, k, [[0, 1]], [2], [0, 2], lse, old, 1.0, tree=[0b01, 0b10])
    assert np.allclose(got.ravel(), [10 + 3 / 8, 20 + 6 / 8, 1 / 4, 4 / 8])


@pytest.fixture(scope="module")
def clib():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    return _lib.load()


@pytest.mark.parametrize("want,kw", [
    (-1, dict(q=None)), (-1, dict(kc=None)), (-1, dict(lse=None)), (-1, dict(w=None)),
    (-5, dict(dtype=2)), (-5, dict(D=96)), (-5, dict(P=24)), (-5, dict(P=512)), (-5, dict(tree=OK, window=4)),
    (-2, dict(S=0)), (-2, dict(T=0)), (-2, dict(Hk=3)), (-2, dict(H=516, Hk=4)), (-2, dict(scale=0.0)), (-2, dict(decay=-0.5)),
    (-2, dict(decay=float("nan"))), (-2, dict(scale=float("inf"))), (-2, dict(window=-1)), (-2, dict(pages=0)), (-2, dict(q_tok=1023)),
    (-2, dict(q_tok=0)), (-2, dict(kc_tok=64)), (-2, dict(w_tok=0)), (-2, dict(width=1 << 28)), (-2, dict(S=70000)),
    (-3, dict(q=OK + 8)), (-3, dict(kc=OK + 2)), (-3, dict(w=OK + 2)),
    (-4, dict(ws=None)), (-4, dict(ws=OK + 16)), (-4, dict(wsb=16)),
])
def test_weights_refusals(clib, want, kw):
    a = dict(dtype=0, q=OK, q_tok=1024, kc=OK, kc_tok=256, pages=10, P=16, width=8, lse=OK, S=2, T=4, H=8, Hk=2, D=128, window=0,
             tree=None, scale=0.1, decay=1.0, w=OK, w_tok=2, ws=OK, wsb=1 << 40)
    a.update(kw)
    assert clib.lmhead_cache_weights(a["dtype"], a["q"], a["q_tok"], 128, a["kc"], 4096, a["kc_tok"], 128, a["pages"], a["P"], OK,
                                     a["width"], OK, OK, None, a["tree"], a["lse"], a["S"], a["T"], a["H"], a["Hk"], a["D"], a["window"],
                                     a["scale"], a["decay"], a["w"], 32, a["w_tok"], 1, a["ws"], a["wsb"], None) == want


@pytest.mark.parametrize("want,kw", [
    (-1, dict(w=None)), (-1, dict(out=None)), (-2, dict(P=0)), (-2, dict(S=0)), (-2, dict(budget=0)), (-2, dict(sinks=-1)),
    (-2, dict(recent=-1)), (-2, dict(sinks=20, recent=81)), (-2, dict(recent=101)), (-2, dict(budget=1 << 30)), (-2, dict(Hk=0)),
    (-2, dict(w_tok=-1)), (-3, dict(w=OK + 2)),
])
def test_select_refusals(clib, want, kw):
    a = dict(w=OK, w_tok=2, pages=10, P=16, Hk=2, S=2, budget=100, sinks=4, recent=10, out=OK)
    a.update(kw)
    assert clib.lmhead_cache_select(a["w"], 32, a["w_tok"], 1, a["pages"], a["P"], a["Hk"], OK, 8, OK, a["S"], a["budget"], a["sinks"],
                                    a["recent"], a["out"], None) == want


@pytest.mark.parametrize("want,kw", [
    (-1, dict(base=[None])), (-1, dict(kept=None)), (-5, dict(base=[])), (-5, dict(base=[OK + (i << 30) for i in range(9)])),
    (-2, dict(row=0)), (-2, dict(tok=128)), (-2, dict(tok=-256)), (-2, dict(base=[OK, OK])), (-2, dict(P=0)), (-2, dict(P=1 << 17)),
    (-2, dict(Hk=0)), (-2, dict(n=0)), (-2, dict(S=0)), (-2, dict(first=OK, out=OK + 4)),
])
def test_keep_refusals(clib, want, kw):
    import ctypes
    a = dict(base=[OK], row=256, tok=512, P=16, Hk=2, kept=OK, n=5, S=2, first=None, out=2 * OK)
    a.update(kw)
    m = max(1, len(a["base"]))
    arr = lambda x: ctypes.addressof(keep.setdefault(len(keep), (ctypes.c_int64 * m)(*x)))
    keep = {}
    assert clib.lmhead_cache_keep(len(a["base"]), arr([b or 0 for b in a["base"]] or [0]), arr([8192] * m), arr([a["tok"]] * m),
                                  arr([256] * m), arr([a["row"]] * m), 10, a["P"], a["Hk"], OK, 8, a["kept"], a["n"], 0, a["first"],
                                  a["S"], a["out"], None) == want


@pytest.mark.parametrize("heads", [2, 1])
@pytest.mark.parametrize("by", [4, 128, 255, -16])
def test_keep_refuses_parts_of_a_row_that_meet(clib, by, heads):
    import ctypes
    arr = lambda *x: (ctypes.c_int64 * len(x))(*x)
    a = [arr(OK, OK + (1 << 30), OK + by), arr(*[8192] * 3), arr(*[512] * 3), arr(*[256] * 3), arr(256, 256, 64)]
    a[3][2] = 256 if heads > 1 else 64  # (the stride of a dimension of one means nothing)
    a[4][2] = 256 if by < 0 else 64  # (one in front of it reaches into it)
    assert clib.lmhead_cache_keep(3, *(ctypes.addressof(x) for x in a), 10, 16, heads, OK, 8, OK, 5, 0, None, 2, 2 * OK, None) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [2, 1])
def test_keep_parts_of_one_row(heads):
    """K and V side by side in one tensor's rows are two caches; the row and a part of it are not."""
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(4)
    table, pages = _paged(rng, [40, 70], 16)
    kv = torch.randint(0, 1000, (pages, 16, heads, 24), device="cuda", dtype=torch.int32)
    kept = np.stack([np.sort(rng.choice(40, 20, replace=False)) for _ in range(2)])
    want = kv.cpu().numpy().copy()
    O.cache_keep(want, table, kept, None, 16)
    L.cache_keep([kv[..., :16], kv[..., 16:]], _i32(table), _i32(kept))
    assert L.last_device_error() == 0 and np.array_equal(kv.cpu().numpy(), want)
    for two in ([kv, kv[..., 16:]], [kv[..., 8:], kv[..., :9]]):
        with pytest.raises(L.LmheadError):
            L.cache_keep(two, _i32(table), _i32(kept))
    assert np.array_equal(kv.cpu().numpy(), want)


@pytest.mark.parametrize("want,kw", [
    (-1, dict(lens=None)), (-1, dict(free=None)), (-2, dict(S=0)), (-2, dict(cap=-1)), (-2, dict(P=0)), (-2, dict(left=OK)),
    (-2, dict(S=1 << 20, width=1 << 20)), (-2, dict(free=OK + 8)),
])
def test_release_refusals(clib, want, kw):
    a = dict(lens=OK, S=4, width=8, free=2 * OK, cap=16, P=16, left=3 * OK)
    a.update(kw)
    assert clib.lmhead_page_release(a["lens"], OK, None, None, a["S"], OK, a["width"], a["free"], a["cap"], OK, a["P"], a["left"],
                                    None) == want


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    i, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 16, 1)
    for call in (lambda: L.cache_weights(torch.zeros(1, 1, 64), torch.zeros(1, 16, 1, 64), i.view(1, 1), i, i, w, w),
                 lambda: L.cache_select(w, i.view(1, 1), i, 4), lambda: L.cache_keep([w], i.view(1, 1), i.view(1, 1)),
                 lambda: L.page_release(i, i, i.view(1, 1), i, i, 16)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


# ----------------------------------------------------------------- weights

def _paged(rng, lens, P, extra=2):
    need = [-(-int(x) // P) for x in lens]
    ids = rng.permutation(sum(need) + extra)
    table = np.full((len(lens), max(max(need), 1) + 1), -7, dtype=np.int64)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = ids[at:at + k]
        at += k
    return table, sum(need) + extra


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _n64(x):
    return x.detach().double().cpu().numpy()


def _weights_case(lens, new, H, Hk, D, P, dtype, seed, mask="causal", heads_first=True):
    """Random q and keys, NaN in every slot that is no token's; lse from fp64."""
    import torch
    t = getattr(torch, dtype)
    rng = np.random.default_rng(seed)
    table, pages = _paged(rng, [a + b for a, b in zip(lens, new)], P)
    T = int(sum(new))
    cu = np.concatenate([[0], np.cumsum(new)])
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * Hk, D, generator=g, device="cuda") * 1.5).to(t)
    kc = torch.full((pages, P, Hk, D), float("nan"), dtype=t, device="cuda")
    w = torch.full((pages, Hk, P) if heads_first else (pages, P, Hk), float("nan"), device="cuda")
    w = w.transpose(1, 2) if heads_first else w
    for s in range(len(lens)):
        j = np.arange(lens[s] + new[s])
        pg, off = torch.tensor(table[s][j // P], device="cuda"), torch.tensor(j % P, device="cuda")
        kc[pg, off] = torch.randn(len(j), Hk, D, generator=g, device="cuda").to(t)
        w[pg[:lens[s]], off[:lens[s]]] = torch.rand(lens[s], Hk, generator=g, device="cuda") * 3
    tree = None
    if mask == "tree":
        bits = rng.integers(0, 1 << 63, T, dtype=np.uint64) | (rng.integers(0, 2, T, dtype=np.uint64) << np.uint64(63))
        bits[rng.random(T) < 0.2] = 0
        tree = torch.tensor(bits.view(np.int64), device="cuda")
    return dict(q=qkv[:, :H], kc=kc, table=_i32(table), lens=_i32(lens), cu=_i32(cu), w=w, tree=tree)


def _lse(c, window):
    """lse of every row by attention's definition, as fp32."""
    import torch
    from oracle import serving_oracle as SO
    q, kc = _n64(c["q"]), np.nan_to_num(_n64(c["kc"]))
    tree = None if c["tree"] is None else c["tree"].cpu().numpy()
    _, lse, _, reach = SO.chunk_attention(q, kc, kc, c["table"].cpu().numpy(), c["lens"].cpu().numpy(), c["cu"].cpu().numpy(),
                                          q.shape[2] ** -0.5, window, tree)
    return torch.tensor(lse, dtype=torch.float32, device="cuda"), reach


def _check_weights(L, c, window=0, decay=1.0, **kw):
    lse, reach = _lse(c, window)
    D = c["q"].shape[2]
    scale = D ** -0.5
    old = _n64(c["w"])
    tree = None if c["tree"] is None else c["tree"].cpu().numpy()
    l64 = _n64(lse)
    want, rows = O.cache_weights(_n64(c["q"]), _n64(c["kc"]), c["table"].cpu().numpy(), c["lens"].cpu().numpy(), c["cu"].cpu().numpy(),
                                 l64, old, scale, window, tree, decay)
    got = _n64(L.cache_weights(c["q"], c["kc"], c["table"], c["lens"], c["cu"], lse, c["w"], tree=c["tree"], window=window, decay=decay,
                               **kw))
    assert L.last_device_error() == 0
    touched = rows > 0
    assert np.array_equal(got[~touched], old[~touched], equal_nan=True)  # no token's: left as it was
    R, l = reach.max(initial=0), np.abs(l64[np.isfinite(l64)]).max(initial=0)
    rel = 2 * (D + 4) * 2.0 ** -23 * R + 2.0 ** -20 + 2.0 ** -22 * (R + l) + (rows + 2) * 2.0 ** -23
    err = np.abs(got - want)[touched]
    tol = (rel * want)[touched] + 1e-30
    assert np.isfinite(want[touched]).all() and np.all(err <= tol), (err / tol).max()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lens,new,H,Hk,D,P", [
    ([0], [1], 1, 1, 64, 16), ([5], [1], 4, 1, 128, 16), ([200, 3, 129, 0], [1, 1, 1, 1], 8, 2, 128, 32),
    ([300, 127], [9, 40], 6, 2, 64, 64), ([0, 128, 255], [130, 1, 33], 3, 3, 128, 128), ([17], [70], 32, 2, 64, 256),
    ([40, 0, 0, 500], [0, 3, 0, 5], 10, 2, 64, 16), ([1000], [3], 40, 8, 128, 64), ([70], [2], 256, 2, 64, 16)])
@pytest.mark.parametrize("mask,window,decay", [("causal", 0, 1.0), ("causal", 0, 0.0), ("causal", 50, 0.75), ("tree", 0, 0.9)])
def test_weights_against_oracle(dtype, lens, new, H, Hk, D, P, mask, window, decay):
    from gpu_util import lib
    c = _weights_case(lens, new, H, Hk, D, P, dtype, sum(lens) + H, mask, heads_first=bool(P & 0x50))
    _check_weights(lib(), c, window, decay)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,H,Hk,D,P,dtype,mask,window", [
    ([700, 30], [300, 513], 8, 2, 128, 64, "bfloat16", "causal", 0), ([2049], [1], 4, 1, 64, 32, "float16", "causal", 0),
    ([0], [600], 12, 1, 128, 16, "float16", "causal", 0), ([1500], [200], 4, 4, 64, 128, "bfloat16", "causal", 700),
    ([900] * 3, [64] * 3, 16, 2, 128, 64, "bfloat16", "tree", 0), ([3000, 1], [2, 400], 5, 1, 64, 16, "bfloat16", "causal", 1),
    # a CTA goes through many tiles of queries
    ([2100, 900], [2048, 1500], 32, 8, 128, 64, "bfloat16", "causal", 0), ([500], [2500], 16, 2, 64, 128, "float16", "causal", 900),
    ([37], [1900], 24, 1, 128, 32, "float16", "causal", 0),
    # more requests than a CTA has threads
    ([i * 37 % 300 for i in range(700)], [1] * 700, 8, 2, 128, 16, "bfloat16", "causal", 0),
    ([i * 53 % 600 for i in range(1300)], [1 + i % 3 for i in range(1300)], 4, 1, 64, 32, "float16", "tree", 0),
    ([i * 41 % 200 for i in range(700)], [33] * 700, 8, 1, 64, 16, "bfloat16", "causal", 90)],
    ids=lambda x: f"x{len(x)}" if isinstance(x, list) and len(x) > 9 else None)
def test_longer_weights(lens, new, H, Hk, D, P, dtype, mask, window):
    """Many tiles of keys and of queries, against fp64 on the GPU's own lse."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case(lens, new, H, Hk, D, P, dtype, 7, mask)
    q, G, scale = c["q"].double(), H // Hk, D ** -0.5
    old = c["w"].clone()
    T = q.shape[0]
    lse = torch.full((T, H), -float("inf"), device="cuda", dtype=torch.float64)
    scores, reach = [], 0.0
    for s in range(len(lens)):
        n, m, t0 = lens[s] + new[s], new[s], int(c["cu"][s])
        j = torch.arange(n, device="cuda")
        pg = c["table"][s].long()[j // P]
        K = c["kc"][pg, j % P].double().repeat_interleave(G, 1)
        x = torch.einsum("ihd,jhd->hij", q[t0:t0 + m], K) * scale
        reach = max(reach, (torch.einsum("ihd,jhd->hij", q[t0:t0 + m].abs(), K.abs()) * scale).max().item())
        age = lens[s] + torch.arange(m, device="cuda")[:, None] - j[None]
        see = age >= 0
        if mask == "tree":
            bit = (c["tree"][t0:t0 + m, None] >> (j - lens[s]).clamp(0, 63)[None]) & 1
            see = (j < lens[s])[None] | ((bit == 1) & (j - lens[s] < 64)[None])
        elif window:
            see = see & (age < window)
        x = x.masked_fill(~see[None], -float("inf"))
        lse[t0:t0 + m] = torch.logsumexp(x, 2).T
        scores.append((x, pg, j % P, see.sum(0) * G))
    l32 = lse.float()
    got = L.cache_weights(c["q"], c["kc"], c["table"], c["lens"], c["cu"], l32, c["w"], tree=c["tree"], window=window, decay=0.5)
    assert L.last_device_error() == 0
    left = torch.ones_like(old, dtype=torch.bool)
    top = l32[l32.isfinite()].abs().max().item()
    for s, (x, pg, off, terms) in enumerate(scores):
        t0, m = int(c["cu"][s]), new[s]
        e = torch.exp(x - l32[t0:t0 + m].double().T[:, :, None].clamp(min=-1e30)).sum(1).view(Hk, G, -1).sum(1).T
        base = old[pg, off].double() * 0.5
        base[lens[s]:] = 0
        want, have = base + e, got[pg, off].double()
        rel = 2 * (D + 4) * 2.0 ** -23 * reach + 2.0 ** -20 + 2.0 ** -22 * (reach + top) + (terms[:, None] + 3) * 2.0 ** -23
        assert bool(((have - want).abs() <= rel * want + 1e-30).all()), ((have - want).abs() / (rel * want + 1e-30)).max()
        left[pg, off] = False
    assert np.array_equal(_n64(got)[_n64(left) > 0], _n64(old)[_n64(left) > 0], equal_nan=True)


@pytest.mark.gpu
def test_weights_of_one_pass_sum_to_its_rows():
    """With attention's own lse, a chunk's weights over all keys sum to its tokens x
    heads; chunk after chunk they add up. lse and each weight are within 2^-12 of theirs."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case([300, 50], [40, 129], 8, 2, 64, 32, "bfloat16", 3)
    c["kc"] = torch.nan_to_num(c["kc"])
    _, lse = L.chunk_attention(c["q"], c["kc"], c["kc"].clone(), c["table"], c["lens"], c["cu"], with_lse=True)
    w = torch.zeros_like(c["w"])
    for k in range(1, 4):
        L.cache_weights(c["q"], c["kc"], c["table"], c["lens"], c["cu"], lse, w)
        have = w.double().sum((0, 1))
        # old values of new tokens are dropped each time: what is left of them is one pass
        new = sum(w[int(c["table"][s, j // 32]), j % 32].double() for s, (a, b) in enumerate([(300, 340), (50, 179)]) for j in range(a, b))
        want = k * (169 * 4 - new) + new
        assert ((have - want).abs() <= 2.0 ** -12 * want).all()


@pytest.mark.gpu
def test_weights_refused_and_bad_requests():
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case([40, 30, 20, 64], [2, 3, 1, 4], 4, 2, 64, 16, "float16", 5)
    lse, _ = _lse(c, 0)
    call = lambda w, **kw: L.cache_weights(c["q"], c["kc"], kw.pop("table", c["table"]), kw.pop("lens", c["lens"]),
                                           kw.pop("cu", c["cu"]), kw.pop("lse", lse), w, **kw)
    base, want = c["w"].clone(), call(c["w"].clone())
    pages = [c["table"][s][c["table"][s] >= 0].long() for s in range(4)]
    eq = lambda a, b: np.array_equal(_n64(a), _n64(b), equal_nan=True)
    got = call(base.clone(), granted=_i32([1, 0, 3, 1]))  # refused: left alone
    assert L.last_device_error() == 0
    assert eq(got[pages[1]], base[pages[1]]) and all(eq(got[pages[s]], want[pages[s]]) for s in (0, 2, 3))
    for lens in ([40, -1, 20, 64], [40, 1 << 30, 20, 64], [40, 2 ** 31 - 2, 20, 64]):
        got = call(base.clone(), lens=_i32(lens))
        assert L.last_device_error() == -7
        assert eq(got[pages[1]], base[pages[1]]) and all(eq(got[pages[s]], want[pages[s]]) for s in (0, 2, 3))
    t = c["table"].clone()
    t[0, 1], t[3, 0] = -1, 1 << 20
    got = call(base.clone(), table=t)
    assert L.last_device_error() == -7
    for s, gone in ((0, 1), (1, None), (2, None), (3, 0)):
        for i, pg in enumerate(pages[s].tolist()):
            assert eq(got[pg], base[pg] if i == gone else want[pg]), (s, i)
    for cu in ([0, 5, 2, 6, 10], [-3, 2, 5, 6, 10], [0, 2, 5, 6, 11]):
        got = call(base.clone(), cu=_i32(cu))
        assert L.last_device_error() == -7 and eq(got, base)
    l2 = lse.clone()
    l2[0] = -float("inf")  # a row that sees nothing draws nothing
    got, first = call(base.clone(), lse=l2), call(base.clone(), lse=torch.where(torch.arange(10, device="cuda")[:, None] == 0, 1e30, lse))
    assert eq(got, first)


@pytest.mark.gpu
def test_weights_streams_graphs_and_determinism():
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case([1500, 800], [64, 300], 8, 2, 128, 64, "bfloat16", 11)
    lse = torch.randn(364, 8, device="cuda") * 0.1 + 8
    args = (c["q"], c["kc"], c["table"], c["lens"], c["cu"], lse)
    eq = lambda a, b: np.array_equal(_n64(a), _n64(b), equal_nan=True)
    want = L.cache_weights(*args, c["w"].clone())
    for _ in range(3):
        assert eq(L.cache_weights(*args, c["w"].clone()), want)
    s = torch.cuda.Stream()
    w = c["w"].clone()
    s.wait_stream(torch.cuda.current_stream())
    L.cache_weights(*args, w, stream=s)
    s.synchronize()
    assert eq(w, want)
    # two graphs that share a workspace, replayed in turn
    ws = L.Workspace()
    a, b = c["w"].clone(), c["w"].clone()
    L.cache_weights(*args, a.clone(), workspace=ws)
    graphs = []
    torch.cuda.synchronize()
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.cache_weights(*args, x, workspace=ws)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert eq(a, want) and eq(b, want)
    # two calls at once, of different sizes
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    d = _weights_case([5000], [1], 8, 2, 128, 64, "bfloat16", 12)
    other = (d["q"], d["kc"], d["table"], d["lens"], d["cu"], torch.full((1, 8), 9.0, device="cuda"))
    wanted = L.cache_weights(*other, d["w"].clone())
    x, y = [c["w"].clone() for _ in range(4)], [d["w"].clone() for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        L.cache_weights(*args, x[i], stream=one)
        L.cache_weights(*other, y[i], stream=two)
    torch.cuda.synchronize()
    assert all(eq(i, want) for i in x) and all(eq(i, wanted) for i in y)
    for bad in (dict(lse=lse[:5]), dict(lse=lse.double()), dict(w=c["w"][:-1]), dict(w=c["w"].half()), dict(q=c["q"].float())):
        k = dict(q=c["q"], lse=lse, w=c["w"])
        k.update(bad)
        with pytest.raises((TypeError, ValueError)):
            L.cache_weights(k["q"], c["kc"], c["table"], c["lens"], c["cu"], k["lse"], k["w"])


@pytest.mark.gpu
def test_weights_of_lengths_near_2_31():
    """Within the table, but with places of blocks behind them that 32 bits do not hold: left
    alone with the error recorded, the other requests served."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case([300, 40], [2, 1], 4, 2, 64, 256, "bfloat16", 31)
    lse, _ = _lse(c, 0)
    width = (2 ** 31 - 1) // 256
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"]
    call = lambda lens: L.cache_weights(c["q"], c["kc"], table, _i32(lens), c["cu"], lse, c["w"].clone(), decay=0.5)
    want = call([300, 40])
    assert L.last_device_error() == 0
    mine, other = c["table"][0, :2].long(), c["table"][1, :1].long()
    for n in (width * 256 - 2, width * 256 - 3, 2 ** 31 - 513, 2 ** 31 - 65537, 2 ** 31 - 1):
        got = call([n, 40])
        assert L.last_device_error() == -7
        assert np.array_equal(_n64(got[other]), _n64(want[other]), equal_nan=True)
        assert np.array_equal(_n64(got[mine]), _n64(c["w"][mine]), equal_nan=True)


# ------------------------------------------------------------------ select

def _select_case(rng, lens, P, Hk, ties):
    import torch
    table, pages = _paged(rng, lens, P)
    w = np.exp(2 * rng.standard_normal((pages, P, Hk)))
    if ties:
        w = np.round(w * 2) / 2
    w[rng.random(w.shape) < 0.1] = 0
    if ties > 1:
        w[rng.random(w.shape) < 0.05] = np.nan
        w[rng.random(w.shape) < 0.05] = np.inf
        w[rng.random(w.shape) < 0.1] = -1
    w = w.astype(np.float32)
    return w, table, torch.tensor(w, device="cuda"), _i32(table)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,P,Hk,budget,sinks,recent", [
    ([1], 16, 1, 1, 0, 0), ([2, 0, 5], 1, 3, 2, 1, 1), ([100, 33, 64, 65], 16, 2, 64, 4, 16), ([1000], 48, 8, 7, 0, 0),
    ([5000, 4999, 17], 128, 2, 2000, 3, 700), ([3000], 16, 1, 500, 500, 0), ([3000], 32, 2, 500, 0, 500), ([3001], 64, 1, 3000, 1, 5),
    ([60000, 70001], 256, 1, 5000, 4, 100), ([200] * 70, 32, 4, 100, 2, 10)])
@pytest.mark.parametrize("ties", [0, 1, 2])
def test_select_against_oracle(lens, P, Hk, budget, sinks, recent, ties):
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(sum(lens) + budget + ties)
    w, table, wd, td = _select_case(rng, lens, P, Hk, ties)
    want = O.cache_select(w, table, lens, P, budget, sinks, recent)
    got = L.cache_select(wd, td, _i32(lens), budget, sinks, recent)
    assert L.last_device_error() == 0
    assert np.array_equal(got.cpu().numpy(), want)
    first = wd.transpose(1, 2).contiguous().transpose(1, 2)  # a head's tokens side by side
    assert np.array_equal(L.cache_select(first, td, _i32(lens), budget, sinks, recent).cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,P,Hk,budget,sinks,recent", [
    ([60001, 45003, 7], 256, 2, 5001, 5, 101), ([41500, 50002], 64, 3, 41000, 3, 2), ([52001], 16, 2, 600, 0, 0),
    ([70002, 41111], 20, 2, 30001, 4093, 7)])
@pytest.mark.parametrize("ties", [0, 1, 2])
def test_select_of_long_lists_by_fours(lens, P, Hk, budget, sinks, recent, ties):
    """More tokens than have room in shared memory, a head's side by side (read four at a time from
    a multiple of four on, the sinks' end or not), the heads' side by side too."""
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(sum(lens) + budget + ties)
    w, table, wd, td = _select_case(rng, lens, P, Hk, ties)
    want = O.cache_select(w, table, lens, P, budget, sinks, recent)
    first = wd.transpose(1, 2).contiguous().transpose(1, 2)
    assert first.stride(1) == 1
    for x in (first, wd):
        assert np.array_equal(L.cache_select(x, td, _i32(lens), budget, sinks, recent).cpu().numpy(), want)
    assert L.last_device_error() == 0


@pytest.mark.gpu
def test_select_bad_requests_and_equal_weights():
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(1)
    w, table, wd, td = _select_case(rng, [100, 100, 100], 16, 2, 0)
    room = table.shape[1] * 16
    got = L.cache_select(wd, td, _i32([100, -1, room + 1]), 10).cpu().numpy()
    assert L.last_device_error() == -7
    assert (got[1:] == -1).all() and np.array_equal(got[0], O.cache_select(w, table, [100], 16, 10, 0, 0)[0])
    t = td.clone()
    t[0, 0], t[1, 2] = -1, 10 ** 6
    got = L.cache_select(wd, t, _i32([100, 100, 100]), 60).cpu().numpy()
    assert L.last_device_error() == -7
    assert (got[0] >= 16).all() and not ((got[1] >= 32) & (got[1] < 48)).any()
    z = torch.zeros_like(wd)
    assert np.array_equal(L.cache_select(z, td, _i32([100] * 3), 10, 2, 3).cpu().numpy()[2, 1], [0, 1, 2, 3, 4, 5, 6, 97, 98, 99])


@pytest.mark.gpu
def test_select_of_lengths_near_2_31():
    """Within the table, but so that a loop's next place would pass 2^31: -1 throughout."""
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(3)
    w, table, wd, _ = _select_case(rng, [100], 256, 2, 0)
    width = (2 ** 31 - 1) // 256
    td = _i32(np.zeros((2, width)))
    for n in (2 ** 31 - 65535, 2 ** 31 - 8192, width * 256):
        got = L.cache_select(wd, td, _i32([n, 100]), 10, 2, 3).cpu().numpy()
        assert L.last_device_error() == -7 and (got[0] == -1).all()
        assert np.array_equal(got[1], O.cache_select(w, [[0]], [100], 256, 10, 2, 3)[0])


# -------------------------------------------------------------------- keep

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [("bfloat16", 128), ("float16", 64), ("float32", 0), ("uint8", 3), ("int16", 5), ("float32", 12),
                                     ("bfloat16", 1000)])
@pytest.mark.parametrize("lens,P,Hk,n,per_head", [
    ([1], 16, 1, 1, False), ([50, 3, 0, 17], 16, 2, 20, True), ([400, 300], 32, 3, 200, False), ([5000], 48, 2, 2500, True),
    ([90] * 6, 1, 1, 5, False)])
def test_keep_against_oracle(dtype, D, lens, P, Hk, n, per_head):
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(n + D + P)
    S = len(lens)
    first = rng.integers(0, 12, S) if n < 100 else None
    table, pages = _paged(rng, [x + 16 for x in lens], P)
    kept = np.full((S, Hk if per_head else 1, n), -1)
    for s, l in enumerate(lens):
        for a in range(kept.shape[1]):
            k = min(n, l)
            some = np.sort(rng.choice(l, k, replace=False)) if k else np.zeros(0)
            kept[s, a, :k] = some
    if n == 20:
        kept[0, :, 5] = -1       # a hole
        kept[0, :, 7] = kept[0, :, 6]  # a row twice (it is behind its place, or at it)
        kept[0, :, 7] = np.maximum(kept[0, :, 7], 7)
    t = getattr(torch, dtype)
    shape = (pages, Hk, P, D) if D else (pages, Hk, P)
    raw = torch.randint(0, 100, shape, device="cuda").to(t)
    plain = torch.randint(0, 100, (pages, P, Hk), device="cuda", dtype=torch.int32)
    caches = [raw.transpose(1, 2), plain]
    want = [c.cpu().float().numpy().copy() for c in caches]
    lens_want = [O.cache_keep(c, table, kept, first, P) for c in want][0]
    got = L.cache_keep(caches, _i32(table), _i32(kept if per_head else kept[:, 0]), first=None if first is None else _i32(first))
    assert L.last_device_error() == 0
    assert np.array_equal(got.cpu().numpy(), lens_want)
    for c, w in zip(caches, want):
        assert np.array_equal(c.cpu().float().numpy(), w)


@pytest.mark.gpu
def test_pages_far_apart():
    """Caches of pages with offsets past 2^31 elements and 2^32 bytes: the same bits as of pages
    side by side, from the weights to the rows moved."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _weights_case([700, 90], [3, 1], 8, 2, 128, 64, "bfloat16", 21)
    lse = torch.full((4, 8), 20.0, device="cuda")
    pages, P, Hk, D = c["kc"].shape
    far = lambda t, step: torch.empty(pages * step, dtype=t.dtype, device="cuda").as_strided(t.shape, (step, *t.stride()[1:])).copy_(t)
    step = (1 << 32) // pages + 4096 & -4096
    assert (pages - 1) * step > 2 ** 31
    out = []
    for kc, w in ((c["kc"].clone(), c["w"].clone()), (far(c["kc"], step), far(c["w"], step // 2))):
        L.cache_weights(c["q"], kc, c["table"], c["lens"], c["cu"], lse, w, decay=0.5)
        lens = c["lens"] + c["cu"].diff()
        kept = L.cache_select(w, c["table"], lens, 64, 2, 16)
        out.append([L.cache_keep([kc, w], c["table"], kept), kept, kc, w])
    assert L.last_device_error() == 0
    for a, b in zip(*out):
        assert np.array_equal(_n64(a), _n64(b), equal_nan=True)


@pytest.mark.gpu
def test_keep_bad_lists():
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(2)
    table, pages = _paged(rng, [40, 40, 40], 16)
    c = torch.randint(0, 1000, (pages, 16, 1, 8), device="cuda", dtype=torch.int32)
    was = c.cpu().numpy().copy()
    place = lambda s, j: (table[s][j // 16], j % 16)
    kept = np.array([[2, 0, 5], [3, 1000, 7], [1, 2, 3]])  # one below its place, one past the table
    got = L.cache_keep([c], _i32(table), _i32(kept), first=_i32([0, 1, -4]))
    assert L.last_device_error() == -7 and got.tolist() == [3, 4, -4]
    now = c.cpu().numpy()
    want = was.copy()
    want[place(0, 0)], want[place(0, 2)] = was[place(0, 2)], was[place(0, 5)]
    want[place(1, 1)], want[place(1, 3)] = was[place(1, 4)], was[place(1, 8)]
    assert np.array_equal(now, want)
    bad = table.copy()
    bad[0, 0], bad[1, 2] = pages, -1
    L.cache_keep([c], _i32(bad), _i32([[20, -1], [-1, 35], [-1, -1]]))
    assert L.last_device_error() == -7 and np.array_equal(c.cpu().numpy(), want)
    for x in ([], [c] * 2, [c, c[:, :8]], [c[..., ::2]], [c.cpu()]):
        with pytest.raises((TypeError, ValueError, L.LmheadError)):
            L.cache_keep(x, _i32(table), _i32(kept))


@pytest.mark.gpu
@pytest.mark.parametrize("per_head", [False, True])
def test_keep_entries_at_their_place_past_the_table(per_head):
    """They move nothing, but there is no such row: the error is recorded. New lengths stay
    within 32 bits."""
    import torch
    from gpu_util import lib
    L = lib()
    table, pages = _i32([[0, 1], [2, 3]]), 4
    c = torch.randint(0, 1000, (pages, 16, 2, 8), device="cuda", dtype=torch.int32)
    was = c.clone()

    def run(kept, first):
        k = np.asarray(kept)
        k = np.stack([np.full_like(k, -1), k], 1) if per_head else k  # the second head's own list
        new = L.cache_keep([c], table, _i32(k), first=_i32(first))
        assert torch.equal(c, was)
        return new.tolist(), L.last_device_error()
    at = [0, 1, 2, 3]
    own = lambda first, n: first if per_head else min(first + n, 2 ** 31 - 1)
    assert run([at, at], [28, 0]) == ([own(28, 4), own(0, 4)], 0)
    assert run([at, at], [29, 0]) == ([own(29, 4), own(0, 4)], -7)
    assert run([at, [0, 1, 2, -1]], [0, 30]) == ([own(0, 4), own(30, 3)], -7)
    assert run([at, [-1] * 4], [2 ** 31 - 2, 50]) == ([own(2 ** 31 - 2, 4), 50], -7)
    assert run([[-1] * 4] * 2, [33, 2 ** 31 - 1]) == ([33, 2 ** 31 - 1], 0)  # (no row at all)


# ----------------------------------------------------------------- release

@pytest.mark.gpu
@pytest.mark.parametrize("S", [1, 7, 8, 9, 300, 1025])
@pytest.mark.parametrize("page", [1, 16, 48, 128])
def test_release_against_oracle(S, page):
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(S + page)
    lens, new = rng.integers(0, 5 * page + 3, S), np.where(rng.random(S) < 0.3, 0, rng.integers(0, 3 * page, S))
    granted = (rng.random(S) < 0.8).astype(int)
    table = rng.integers(0, 10 ** 6, (S, 9))
    F = 5
    for with_new in (False, True):
        held = lens + (new * granted if with_new else 0)
        now = (held * rng.random(S)).astype(int) + (rng.random(S) < 0.2)
        now = np.minimum(now, held)
        total = int((-(-held // page) - -(-now // page)).sum())
        free = rng.integers(0, 10 ** 6, F + total + 3)
        want = O.page_release(held, now, table, free.tolist(), F, page)
        fd = _i32(free)
        kw = dict(cu=_i32(np.concatenate([[0], np.cumsum(new)])), granted=_i32(granted)) if with_new else {}
        left = L.page_release(_i32(lens), _i32(now), _i32(table), fd, _i32([F]), page, **kw)
        assert L.last_device_error() == 0
        assert int(left[0]) == len(want) and fd.cpu().tolist() == want + free.tolist()[len(want):]
        # a list without room for all of them
        if total > 1:
            fd = _i32(free[:F + total - 1])
            left = L.page_release(_i32(lens), _i32(now), _i32(table), fd, _i32([F]), page, **kw)
            assert L.last_device_error() == -7 and int(left[0]) == F + total - 1 and fd.cpu().tolist() == want[:-1]


@pytest.mark.gpu
def test_release_bad_lengths():
    import torch
    from gpu_util import lib
    L = lib()
    table = _i32(np.arange(18).reshape(6, 3))
    free = _i32([90, 91, -1, -1, -1, -1])
    left = L.page_release(_i32([40, -1, 20, 49, 33, 40]), _i32([16, 0, 21, 0, -2, 40]), table, free, _i32([2]), 16)
    assert L.last_device_error() == -7
    assert left.tolist() == [4] and free.tolist() == [90, 91, 1, 2, -1, -1]
    left = L.page_release(_i32([40]), _i32([16]), table[:1], free, _i32([99]), 16)  # a count above the list's length
    assert L.last_device_error() == -7 and left.tolist() == [6]
    left = L.page_release(_i32([16]), _i32([16]), table[:1], torch.zeros(0, dtype=torch.int32, device="cuda"), _i32([0]), 16)
    assert L.last_device_error() == 0 and left.tolist() == [0]


@pytest.mark.gpu
@pytest.mark.parametrize("S,width", [(1, 3), (8, 9), (9, 40), (300, 9), (17, 1500), (2, 9001), (1030, 30)])
def test_release_entries_that_are_no_pages(S, width):
    """A request with an entry below 0 among the pages that it would give back gives none
    back, and the error is recorded; entries before and behind those are not looked at."""
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(S + width)
    held = rng.integers(0, width * 16 + 1, S)
    now = np.where(rng.random(S) < 0.5, (held * rng.random(S)).astype(int), np.maximum(held - 40, 0))
    held[-1], now[-1] = width * 16, 0
    lo, hi = -(-now // 16), -(-held // 16)
    table = rng.integers(0, 10 ** 6, (S, width))
    for s in range(S):  # around them anything
        table[s, :lo[s]] = -1
        table[s, hi[s]:] = -(1 << 31)
    F = 3
    room = int((hi - lo).sum())
    args = _i32(held), _i32(now)

    def run(table, then, status):
        free = _i32([5, 6, 7] + [-9] * room)
        left = L.page_release(*args, _i32(table), free, _i32([F]), 16)
        assert L.last_device_error() == status
        want = O.page_release(held, then, table, [5, 6, 7], F, 16)
        assert left.tolist() == [len(want)] and free.cpu().tolist() == want + [-9] * (F + room - len(want))

    run(table, now, 0)
    for turn in range(6):
        bad = table.copy()
        some = [s for s in range(S) if hi[s] > lo[s] and (rng.random() < 0.4 or s == S - 1)]
        for s in some:  # one entry each: the first, the last or one between
            bad[s, [lo[s], hi[s] - 1, rng.integers(lo[s], hi[s])][turn % 3]] = -1 if turn < 3 else -(1 << 31)
        run(bad, np.where(np.isin(np.arange(S), some), held, now), -7)


@pytest.mark.gpu
def test_weights_waits_that_run_out():
    """With no time to wait a call gives up, says so, and the next one is right."""
    from gpu_util import lib
    L = lib()
    c = _weights_case([600, 70], [300, 3], 8, 2, 128, 64, "bfloat16", 13)
    lse, _ = _lse(c, 0)
    args = (c["q"], c["kc"], c["table"], c["lens"], c["cu"], lse)
    want = L.cache_weights(*args, c["w"].clone())
    assert L.last_device_error() == 0
    L.debug_set_wait_cycles(0)
    try:
        L.cache_weights(*args, c["w"].clone())
        status = L.last_device_error()
    finally:
        L.debug_set_wait_cycles(-1)
    assert status == -8
    assert np.array_equal(_n64(L.cache_weights(*args, c["w"].clone())), _n64(want), equal_nan=True)
    assert L.last_device_error() == 0
