"""Chunk attention over a paged cache: refusals on the host (no GPU: every call
fails validation first), the oracle by hand, and the kernels against fp64.

What an output may be off by, with u the half step of its 16-bit type, A = sum_j
p_j |v_j| and R = max_j scale sum_d |q_d k_jd| over a row's keys:
  - each weight rounded to 16 bits before it meets its value: u A;
  - the output rounded once: u (|o| + what came before);
  - a logit's D products and its scaling, each addition within one fp32 step:
    delta = (D + 4) 2^-23 R, which changes a weight by 2 delta of itself;
  - the exponential and its argument: 2^-21 and 2^-23 of the distance from the
    maximum, at most 2 R: within 2^-20 + 2^-22 R;
  - sums over n keys in fp32: n 2^-23 A, and as much for the weights' own sum.
lse is off by delta and by the relative error of that sum, plus 2^-23 |lse|."""
import numpy as np
import pytest

from oracle import serving_oracle as SO

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def clib():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    return _lib.load()


def _call(lib, **kw):
    a = dict(dtype=0, q=OK, q_tok=1024, q_head=128, k=OK, k_tok=256, k_head=128, v=OK, kc=OK, kc_page=4096,
             kc_tok=256, kc_head=128, pages=10, P=16, slots=OK, tree=None, S=2, T=4, H=8, Hk=2, D=128, window=0,
             scale=0.1, out=OK, ws=OK, wsb=1 << 40)
    a.update(kw)
    return lib.lmhead_chunk_attention(
        a["dtype"], a["q"], a["q_tok"], a["q_head"], a["k"], a["k_tok"], a["k_head"], a["v"], a["k_tok"],
        a["k_head"], a["kc"], a["kc_page"], a["kc_tok"], a["kc_head"], OK, a["kc_page"], a["kc_tok"],
        a["kc_head"], a["pages"], a["P"], OK, 8, OK, OK, a["slots"], a["tree"], a["S"], a["T"], a["H"], a["Hk"],
        a["D"], a["window"], a["scale"], a["out"], None, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("want,kw", [
    (-1, dict(q=None)), (-1, dict(kc=None)), (-1, dict(out=None)), (-1, dict(v=None)),
    (-1, dict(slots=None)),                       # new K and V need their slots
    (-5, dict(dtype=2)), (-5, dict(D=96)), (-5, dict(P=24)), (-5, dict(P=8)), (-5, dict(P=512)),
    (-5, dict(tree=OK, window=4)),
    (-2, dict(S=0)), (-2, dict(T=0)), (-2, dict(Hk=3)), (-2, dict(H=0)), (-2, dict(H=516, Hk=4)),
    (-2, dict(scale=0.0)), (-2, dict(scale=float("nan"))), (-2, dict(window=-1)), (-2, dict(pages=0)),
    (-2, dict(q_tok=1023)), (-2, dict(kc_tok=64)), (-2, dict(kc_head=-128)), (-2, dict(pages=1 << 40)),
    (-3, dict(q=OK + 8)), (-3, dict(kc=OK + 2)), (-3, dict(out=OK + 4)),
    (-4, dict(ws=None)), (-4, dict(ws=OK + 16)), (-4, dict(wsb=16)),
])
def test_refusals(clib, want, kw):
    assert _call(clib, **kw) == want


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        L.chunk_attention(torch.zeros(1, 1, 64), torch.zeros(1, 16, 1, 64), torch.zeros(1, 16, 1, 64),
                          i.view(1, 2), i[:1], i)


def test_oracle_by_hand():
    """Two cached tokens and two new ones, one head of one dimension: the first
    new token sees three keys, with a window of two its own and one more."""
    k = np.log(np.array([1., 2., 1., 4.])).reshape(2, 2, 1, 1)[::-1]
    v = np.array([1., 2., 3., 4.]).reshape(2, 2, 1, 1)[::-1]
    q = np.ones((2, 1, 1))
    out, lse, _, _ = SO.chunk_attention(q, k, v, [[1, 0]], [2], [0, 2], 1.0)
    assert np.allclose(out[:, 0, 0], [(1 + 4 + 3) / 4, (1 + 4 + 3 + 16) / 8]) and np.allclose(lse[:, 0], np.log([4, 8]))
    out, lse, _, _ = SO.chunk_attention(q, k, v, [[1, 0]], [2], [0, 2], 1.0, window=2)
    assert np.allclose(out[:, 0, 0], [7 / 3, 19 / 5])
    out, lse, _, _ = SO.chunk_attention(q, k, v, [[1, 0]], [2], [0, 2], 1.0, tree=[0b10, 0])
    assert np.allclose(out[:, 0, 0], [(1 + 4 + 16) / 7, 5 / 3])


def _case(lens, new, H, Hk, D, P, dtype, seed, mask="causal", extra=2, fill=None):
    """Inputs on the GPU: a shuffled table, garbage (NaN by default) in every slot
    that is no token's, q, k and v side by side in one buffer."""
    import torch
    t = getattr(torch, dtype)
    rng = np.random.default_rng(seed)
    dev = "cuda"
    S, T = len(lens), int(sum(new))
    need = [-(-(l + m) // P) for l, m in zip(lens, new)]
    pages = sum(need) + extra
    ids = rng.permutation(pages)
    width = max(max(need), 1) + 1
    table = np.full((S, width), -7, dtype=np.int32)
    at = 0
    for s in range(S):
        table[s, :need[s]] = ids[at:at + need[s]]
        at += need[s]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = torch.Generator(device=dev).manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * Hk, D, generator=g, device=dev) * 1.5).to(t)
    kc = torch.full((pages, P, Hk, D), float("nan") if fill is None else fill, dtype=t, device=dev)
    vc = kc.clone()
    for s in range(S):
        j = np.arange(lens[s])
        if len(j):
            sl = torch.tensor(table[s][j // P] * P + j % P, device=dev).long()
            kc.view(-1, Hk, D)[sl] = torch.randn(len(j), Hk, D, generator=g, device=dev).to(t)
            vc.view(-1, Hk, D)[sl] = torch.randn(len(j), Hk, D, generator=g, device=dev).to(t)
    slots = np.concatenate([table[s][(lens[s] + np.arange(new[s])) // P] * P + (lens[s] + np.arange(new[s])) % P
                            for s in range(S)]) if T else np.zeros(0)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)
    tree = None
    if mask == "tree":
        # random ancestor sets, the own bit not always in them; high bits on too
        bits = rng.integers(0, 1 << 63, T, dtype=np.uint64) | (rng.integers(0, 2, T, dtype=np.uint64) << np.uint64(63))
        bits[rng.random(T) < 0.2] = 0
        tree = torch.tensor(bits.view(np.int64), device=dev)
    return dict(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], kc=kc, vc=vc, table=i32(table), lens=i32(lens),
                cu=i32(cu), slots=i32(slots), tree=tree)


def _check(L, c, dtype, scale=None, window=0, stream=None):
    import torch
    q = c["q"]
    T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, lse = L.chunk_attention(q, c["kc"], c["vc"], c["table"], c["lens"], c["cu"], k=c["k"], v=c["v"], slots=c["slots"],
                                 tree=c["tree"], window=window, scale=scale, with_lse=True, stream=stream)
    torch.cuda.synchronize()
    n64 = lambda x: x.double().cpu().numpy()
    tree = None if c["tree"] is None else c["tree"].cpu().numpy()
    want, wl, A, R = SO.chunk_attention(n64(q), n64(c["kc"]), n64(c["vc"]), c["table"].cpu().numpy(), c["lens"].cpu().numpy(),
                                        c["cu"].cpu().numpy(), scale, window, tree)
    u = torch.finfo(getattr(torch, dtype)).eps / 2
    n = int(c["lens"].max()) + T
    delta = (D + 4) * 2.0 ** -23 * R
    rel = 2 * delta + 2.0 ** -20 + 2.0 ** -22 * R + 2 * n * 2.0 ** -23
    tol = (u + rel[..., None] * (1 + u)) * A
    tol = tol + u * (np.abs(want) + tol) + 2.0 ** -24  # fp16 also rounds below its normal range
    got = n64(out)
    assert np.all(np.abs(got - want) <= tol), np.nanmax(np.abs(got - want) / tol)
    gl = n64(lse)
    dead = ~np.isfinite(wl)
    assert np.array_equal(dead, gl == -np.inf) and np.all(got[dead] == 0)
    live = ~dead
    assert np.all(np.abs(gl - wl)[live] <= (delta + 2.0 ** -20 + 2.0 ** -22 * R + n * 2.0 ** -23 + 2.0 ** -23 * np.abs(np.where(dead, 0, wl)))[live])
    assert L.last_device_error() == 0
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("H,Hk,D,P", [(1, 1, 64, 16), (8, 2, 128, 16), (6, 2, 64, 32), (5, 1, 128, 64), (16, 1, 64, 128),
                                      (4, 4, 128, 256), (64, 8, 64, 64)])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([37], [1]), ([128, 0, 127, 300], [1, 1, 1, 1]), ([0, 5], [130, 17]),
                                      ([1000, 3, 0], [3, 40, 0]), ([255, 256, 257], [2, 1, 9])])
def test_causal(lens, new, H, Hk, D, P, dtype):
    from gpu_util import lib
    _check(lib(), _case(lens, new, H, Hk, D, P, dtype, sum(lens) + H), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 1000])
def test_window(window, H, Hk, D):
    from gpu_util import lib
    _check(lib(), _case([0, 511, 130, 77], [5, 1, 300, 64], H, Hk, D, 32, "bfloat16", window), "bfloat16", window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("H,Hk,D", [(8, 1, 64), (12, 4, 128)])
def test_tree(H, Hk, D, dtype):
    """Trees of up to 64 nodes, words with no bit at all: over an empty context
    such a row sees nothing; a chunk longer than its words can name."""
    from gpu_util import lib
    _check(lib(), _case([0, 100, 0, 640, 64], [10, 64, 3, 33, 1], H, Hk, D, 16, dtype, H, mask="tree"), dtype)
    _check(lib(), _case([20, 0], [100, 70], H, Hk, D, 16, dtype, H, mask="tree"), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_long(D):
    """Long contexts shared out over the GPU, and a long chunk."""
    from gpu_util import lib
    _check(lib(), _case([20000, 7], [2, 2], 4, 1, D, 64, "bfloat16", 1), "bfloat16")
    _check(lib(), _case([300, 1500], [700, 260], 4, 2, D, 128, "float16", 2), "float16")


@pytest.mark.gpu
def test_many_requests():
    from gpu_util import lib
    rng = np.random.default_rng(0)
    lens, new = rng.integers(0, 400, 400), rng.integers(0, 4, 400)
    _check(lib(), _case(list(lens), list(new), 8, 2, 64, 16, "bfloat16", 5), "bfloat16")


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-4, 0.088, 3.0])
def test_scales(scale):
    """Flat and nearly one-hot weights."""
    from gpu_util import lib
    _check(lib(), _case([500, 40], [4, 150], 8, 2, 128, 32, "bfloat16", 9), "bfloat16", scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["rising", "falling", "late", "spikes"])
def test_scores_that_outgrow_the_reference(shape, D, dtype):
    """Scores along one direction that climb by far more than the softmax's
    reference allows, between blocks and within them, for one tile and for two."""
    import torch
    from gpu_util import lib
    c = _case([700, 0, 90], [1, 300, 40], 4, 1, D, 32, dtype, 3)
    T, t = c["q"].shape[0], c["q"].dtype
    u = torch.ones(D, device="cuda") / 4
    qkv = torch.cat([(u * 2).expand(T, 4, D).to(t), c["k"], c["v"]], 1)
    a = torch.arange(1024, device="cuda", dtype=torch.float32)
    a = {"rising": a / 8, "falling": 80 - a / 8, "late": 60.0 * (a % 128 >= 100) + a / 16,
         "spikes": 90.0 * (a % 150 == 77) * (1 + a / 400)}[shape]
    # position j of every request has the key a_j u (and some of the direction's noise)
    key = (a[:, None] * u + 0.05 * torch.randn(1024, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1))).to(t)
    lens, cu = c["lens"].tolist(), c["cu"].tolist()
    for s, l in enumerate(lens):
        m = cu[s + 1] - cu[s]
        j = torch.arange(l, device="cuda")
        slot = (c["table"][s].long()[j // 32] * 32 + j % 32)
        c["kc"].view(-1, 1, D)[slot, 0] = key[:l]
        qkv[cu[s]:cu[s + 1], 4] = key[l:l + m]
    c.update(q=qkv[:, :4], k=qkv[:, 4:5], v=qkv[:, 5:])
    _check(lib(), c, dtype)


@pytest.mark.gpu
def test_waits_that_run_out():
    """With no time to wait the kernel gives up, says so and leaves the GPU as it
    was: the next call is right."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _case([300, 1000], [3, 200], 8, 2, 128, 32, "bfloat16", 5)
    want, _ = _check(L, c, "bfloat16")
    before = L.debug_set_wait_cycles(0)
    try:
        L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"])
        assert L.last_device_error() == -8
    finally:
        L.debug_set_wait_cycles(-1)
    assert before > 0
    assert torch.equal(L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"]), want)
    assert L.last_device_error() == 0


@pytest.mark.gpu
def test_other_cache_orders_and_streams():
    """Heads before tokens in a page, a cache that is part of a larger one, no
    new K and V (already cached), another stream."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _case([200, 31], [3, 20], 8, 4, 128, 32, "bfloat16", 4)
    a, al = _check(L, c, "bfloat16")
    kv = torch.stack([c["kc"], c["vc"]], 1).transpose(2, 3).contiguous()  # pages x 2 x heads x tokens x dim
    d = dict(c, kc=kv[:, 0].transpose(1, 2), vc=kv[:, 1].transpose(1, 2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, bl = _check(L, d, "bfloat16", stream=s)
    assert torch.equal(a, b) and torch.equal(al, bl)
    e = L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"])
    assert torch.equal(a, e)
    with pytest.raises(ValueError, match="k, v, slots"):
        L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], k=c["k"])
    with pytest.raises(ValueError, match="v_cache"):
        L.chunk_attention(c["q"], c["kc"], c["vc"][1:], c["table"], c["lens"], c["cu"])
    with pytest.raises(TypeError, match="k_cache"):
        L.chunk_attention(c["q"], c["kc"].half(), c["vc"], c["table"], c["lens"], c["cu"])
    with pytest.raises(ValueError, match="cu"):
        L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"][1:])


@pytest.mark.gpu
def test_bad_pages_and_missing_slots():
    """A page id out of range: its request's rows are NaN, the others' are not;
    a token without a slot is not written."""
    import torch
    from gpu_util import lib
    L = lib()
    for bad in (-1, 1 << 20):
        c = _case([100, 50, 300], [2, 3, 4], 4, 2, 64, 16, "bfloat16", 6)
        good, _ = L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], k=c["k"], v=c["v"],
                                    slots=c["slots"], with_lse=True)
        c["table"][1, 1] = bad
        out, lse = L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], with_lse=True)
        assert L.last_device_error() == -7
        assert torch.isnan(out[2:5]).all() and torch.isnan(lse[2:5]).all()
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
    c = _case([16], [4], 2, 2, 64, 16, "bfloat16", 6, fill=0.0)
    slots = c["slots"].clone()
    slots[1] = -1
    slots[2] = 1 << 24
    L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], k=c["k"], v=c["v"], slots=slots)
    assert L.last_device_error() == -7
    flat = c["kc"].view(-1, 2, 64)[c["slots"].long()]
    assert torch.equal(flat[0], c["k"][0]) and torch.equal(flat[3], c["k"][3])
    assert not flat[1].any() and not flat[2].any()


@pytest.mark.gpu
def test_graph_capture():
    """A captured step replayed on other lengths and pages of the same buffers."""
    import torch
    from gpu_util import lib
    L = lib()
    a = _case([700, 90], [1, 1], 8, 2, 128, 16, "bfloat16", 8, extra=3)
    b = _case([90, 700], [1, 1], 8, 2, 128, 16, "bfloat16", 9, extra=3)
    ws = L.Workspace()
    run = lambda c, out: L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], k=c["k"], v=c["v"],
                                           slots=c["slots"], workspace=ws, out=out)
    want = [run(c, None).clone() for c in (a, b)]
    live = {k: (v.clone() if v is not None else None) for k, v in a.items()}
    out = torch.empty_like(want[0])
    run(live, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(live, out)
    for c, w in zip((b, a), (want[1], want[0])):
        for k, v in live.items():
            if v is not None:
                v.copy_(c[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def _call_guarded(L, c, cu, lens):
    """A call on other ranges and lengths with bytes behind its workspace that it
    must leave alone: (out, lse, error)."""
    import torch
    S, (T, H, D) = c["lens"].shape[0], c["q"].shape
    need = L.load().lmhead_chunk_attention_workspace_size(S, T, H, c["kc"].shape[2], D)
    ws = torch.full((need + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    out = (torch.zeros(T, H, D, dtype=c["q"].dtype, device="cuda"), torch.zeros(T, H, device="cuda"))
    L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], lens, cu, workspace=ws[:need], out=out)
    err = L.last_device_error()
    assert torch.all(ws[need:] == 0x5a)
    return out[0], out[1], err


@pytest.mark.gpu
@pytest.mark.parametrize("S", [2, 40, 700])
def test_token_ranges_that_decrease(S):
    """Ranges that overlap would be more work than the workspace has places for:
    nothing is computed, every row is NaN and the error is recorded."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _case([40] * S, [2] * S, 4, 2, 64, 16, "bfloat16", 1)
    good, _ = _check(L, c, "bfloat16")
    T = 2 * S
    back = c["cu"].clone()
    back[1::2], back[0::2] = T, 0
    one = c["cu"].clone()
    one[S // 2] = T + 1
    low = c["cu"].clone()
    low[0] = -3
    for cu in (back, one, low):
        out, lse, err = _call_guarded(L, c, cu, c["lens"])
        assert err == -7 and torch.isnan(out).all() and torch.isnan(lse).all()
    # a plan's ranges may pass its tokens: the rest has no rows
    past = c["cu"].clone()
    past[-1] = T + 1000
    out, _, err = _call_guarded(L, c, past, c["lens"])
    assert err == 0 and torch.equal(out, good)


@pytest.mark.gpu
@pytest.mark.parametrize("len_of", [-1, -2 ** 31, 2 ** 31 - 1, "past"])
@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_lengths_that_no_table_holds(mask, len_of):
    """Such a request's rows are NaN and the error is recorded, whatever the
    length; the others' are right."""
    import torch
    from gpu_util import lib
    L = lib()
    c = _case([100, 50, 300], [2, 70, 4], 4, 2, 64, 16, "float16", 2, mask=mask)
    call = lambda lens: L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], lens, c["cu"], tree=c["tree"], with_lse=True)
    _check(L, c, "float16")
    good, gl = call(c["lens"])
    lens = c["lens"].clone()
    lens[1] = c["table"].shape[1] * 16 - (64 if mask == "tree" else 70) + 1 if len_of == "past" else len_of
    out, lse = call(lens)
    assert L.last_device_error() == -7
    assert torch.isnan(out[2:72]).all() and torch.isnan(lse[2:72]).all()
    for got, want in ((out, good), (lse, gl)):
        assert torch.equal(got[:2], want[:2]) and torch.equal(got[72:], want[72:])
    assert L.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("stale", [True, False])
@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_refused_requests_of_a_plan(mask, stale):
    """A plan whose pool runs out, into attention: the granted requests' rows are
    right, the refused ones' are zero and -inf, nothing is recorded, whether the
    table names other requests' pages in their places or none."""
    import torch
    from gpu_util import lib
    L = lib()
    P, H, Hk, D = 16, 8, 2, 64
    rng = np.random.default_rng(3)
    lens, new = [30, 5, 0, 64, 17, 200], [2, 300, 40, 1, 60, 8]
    held = [-(-l // P) for l in lens]
    ids = rng.permutation(120)
    table = np.full((6, 24), -1)
    if stale:
        table[:] = ids[:24]
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = ids[at:at + n]
        at += n
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    tab, T = i32(table), sum(new)
    # 19 pages are wanted by the second request and 18 are there
    plan = L.page_plan(i32(lens), i32(new), tab, i32(ids[at:]), i32([18]), P, T)
    ok = plan.granted.cpu().numpy()
    assert 0 < ok.sum() < 6
    g = torch.Generator("cuda").manual_seed(0)
    kc, vc = (torch.randn(120, P, Hk, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    qkv = torch.randn(T, H + 2 * Hk, D, generator=g, device="cuda").to(torch.bfloat16)
    tree = None
    if mask == "tree":
        tree = torch.tensor(rng.integers(0, 1 << 62, T), dtype=torch.int64, device="cuda")
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    out = (torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda"))
    L.chunk_attention(q, kc, vc, tab, i32(lens), plan.cu, k=k, v=v, slots=plan.slots, tree=tree, out=out,
                      granted=plan.granted)
    assert L.last_device_error() == 0
    n64 = lambda x: x.double().cpu().numpy()
    tr = None if tree is None else tree.cpu().numpy()
    cu = plan.cu.cpu().numpy()
    want, wl, A, R = SO.chunk_attention(n64(q), n64(kc), n64(vc), tab.cpu().numpy(), lens, cu, D ** -0.5, 0, tr, ok)
    got, gl = n64(out[0]), n64(out[1])
    u = 2.0 ** -8
    delta = (D + 4) * 2.0 ** -23 * R
    rel = 2 * delta + 2.0 ** -20 + 2.0 ** -22 * R + 2 * 520 * 2.0 ** -23
    tol = (u + rel[..., None] * (1 + u)) * A
    assert np.all(np.abs(got - want) <= tol + u * (np.abs(want) + tol))
    live = np.isfinite(wl)
    assert np.array_equal(live, np.isfinite(gl))
    assert np.all(np.abs(gl - np.where(live, wl, 0))[live] <= (
        delta + 2.0 ** -20 + 2.0 ** -22 * R + 520 * 2.0 ** -23 + 2.0 ** -23 * np.abs(np.where(live, wl, 0)))[live])
    for s in range(6):
        if not ok[s]:
            rows = slice(cu[s], cu[s + 1])
            assert not out[0][rows].any() and torch.all(out[1][rows] == -float("inf"))
    # none granted
    L.chunk_attention(q, kc, vc, tab, i32(lens), plan.cu, out=out, granted=torch.zeros_like(plan.granted))
    assert not out[0].any() and torch.all(out[1] == -float("inf")) and L.last_device_error() == 0
    with pytest.raises(ValueError, match="granted"):
        L.chunk_attention(q, kc, vc, tab, i32(lens), plan.cu, granted=plan.granted[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("H,Hk,D,P", [(5, 1, 64, 16), (8, 2, 128, 16), (12, 4, 64, 64), (2, 2, 128, 128), (6, 2, 64, 256)])
@pytest.mark.parametrize("window", [1, 63, 128, 300])
def test_windows_of_either_type_over_any_pages(window, H, Hk, D, P, dtype):
    """The pages that lie wholly before every window have been given away: their
    table entries are no page's."""
    import torch
    from gpu_util import lib
    c = _case([0, 511, 1300, 77], [5, 1, 140, 64], H, Hk, D, P, dtype, window)
    want, wl = _check(lib(), c, dtype, window=window)
    for s, l in enumerate([0, 511, 1300, 77]):
        c["table"][s, :max(0, l + 1 - window) // P] = -1
    L = lib()
    got, gl = L.chunk_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], window=window, with_lse=True)
    assert torch.equal(got, want) and torch.equal(gl, wl) and L.last_device_error() == 0
