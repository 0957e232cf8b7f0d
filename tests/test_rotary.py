"""Rotary positions: the frequencies, refusals on the host (no GPU: every call
fails validation first), and the kernel against fp64.

What a result may be off by, with u the half step of its type (2^-24 for fp32): the
fraction of a turn is rounded to 2^-33 and then, as a float of half turns, to 2^-25
of a half turn at most: the angle is off by 2 pi (2^-33 + 2^-26) < 1.0e-7; sine and
cosine by two steps of fp32 below 1 (2^-23) more, the magnitude, the product and the
sum by 2^-24 of theirs each: e = 1e-7 + 2^-23 + 3 2^-24 < 4.2e-7 of m (|a| + |b|),
then the result by u of its value once."""
import numpy as np
import pytest

from oracle import step_oracle as O

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


def test_frequencies():
    from draft_lm_head_gb300 import prep
    full = lambda t: t.view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    w = full(prep.rotary_turns(128, 10000.0))
    assert np.allclose(w, 10000.0 ** (-np.arange(64) / 64), rtol=1e-15, atol=1e-18)
    assert np.allclose(full(prep.rotary_turns(128, 10000.0, "linear", 4.0)), w / 4, rtol=1e-15, atol=1e-18)
    b = full(prep.rotary_turns(128, 10000.0, "base", 4.0))
    assert np.isclose(b[0], w[0]) and np.isclose(b[-1], w[-1] / 4)
    for kind in ("wavelength", "ramp"):
        x = full(prep.rotary_turns(128, 500000.0, kind, 8.0, 8192, 1.0, 4.0))
        y = full(prep.rotary_turns(128, 500000.0))
        n = 8192 * y / (2 * np.pi)
        ratio = y / x
        assert np.allclose(ratio[n >= 5], 1) and np.allclose(ratio[n <= 0.5], 8)
        assert np.all(np.diff(ratio) >= -1e-9) and 1.01 < ratio[np.argmin(abs(n - 2))] < 7.99
    # in turns the blend is that of the definition
    x = full(prep.rotary_turns(64, 500000.0, "wavelength", 8.0, 8192, 1.0, 4.0))
    y = full(prep.rotary_turns(64, 500000.0))
    k = np.clip((8192 * y / (2 * np.pi) - 1) / 3, 0, 1)
    assert np.allclose(x, y * k + y / 8 * (1 - k), rtol=1e-14)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, scaling="other"), dict(rot=2, scaling="base"),
                dict(rot=8, scaling="ramp", low=4.0, high=4.0), dict(rot=8, factor=0.0)):
        with pytest.raises(ValueError):
            prep.rotary_turns(**bad)


@pytest.mark.parametrize("rot,base,factor,original,low,high", [
    (128, 10000.0, 4.0, 131072, 1.0, 32.0),  # the slowest pair turns 2.4 times
    (128, 10000.0, 8.0, 65536, 1.0, 4.0), (64, 10000.0, 16.0, 10 ** 6, 1.0, 32.0),
    (128, 10000.0, 8.0, 100, 1.0, 32.0),     # and the fastest 15.9 times
    (128, 500000.0, 8.0, 8192, 1.0, 4.0), (2, 10000.0, 2.0, 100, 1.0, 32.0)])
def test_ramps_past_the_pairs(rot, base, factor, original, low, high):
    """Pair by pair against the definition: the ramp runs between the whole indices that turn
    `high` times or more and `low` times or fewer, found by counting, wherever they lie."""
    from draft_lm_head_gb300 import prep
    w = lambda i: base ** (-2 * i / rot)
    turns = lambda i: original * w(i) / (2 * np.pi)
    first = max(i for i in range(-3 * rot, 3 * rot) if turns(i) >= high)
    last = min(i for i in range(-3 * rot, 3 * rot) if turns(i) <= low)
    assert first >= 0 or last >= 0
    got = prep.rotary_turns(rot, base, "ramp", factor, original, low, high).view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    for i in range(rot // 2):
        k = min(max((last - i) / (last - first), 0.0), 1.0)
        assert np.isclose(got[i], w(i) * k + w(i) / factor * (1 - k), rtol=1e-12), i


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_ramp_needs_falling_frequencies(base):
    from draft_lm_head_gb300 import prep
    with pytest.raises(ValueError, match="base"):
        prep.rotary_turns(8, base, "ramp", 4.0)
    prep.rotary_turns(8, base, "linear", 4.0)


@pytest.mark.parametrize("scaling", ["wavelength", "ramp"])
@pytest.mark.parametrize("original", [0, -8192.0, float("nan")])
def test_original_length_is_positive(scaling, original):
    from draft_lm_head_gb300 import prep
    with pytest.raises(ValueError, match="original"):
        prep.rotary_turns(8, 10000.0, scaling, 4.0, original)


def test_oracle_by_hand():
    """A quarter turn a position: (1, 2) -> (-2, 1) -> (-1, -2); its transpose the
    other way; in the far, whole turns drop out."""
    q = np.int64(1 << 62)
    x = np.array([[[1.0, 2.0, 5.0]]])
    assert np.allclose(O.rotary(x, [1], [q]), [[[-2, 1, 5]]])
    assert np.allclose(O.rotary(x, [2], [q], magnitude=3.0), [[[-3, -6, 5]]])
    assert np.allclose(O.rotary(x, [1], [q], backward=True), [[[2, -1, 5]]])
    assert np.allclose(O.rotary(x, [2 ** 31 - 1], [q]), [[[2, -1, 5]]])
    assert np.allclose(O.rotary(x, [-1], [q]), x)
    y = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    assert np.allclose(O.rotary(y, [1], [q, 0]), [[[-3, 2, 1, 4]]])
    assert np.allclose(O.rotary(y, [1], [q, 0], interleaved=True), [[[-2, 1, 3, 4]]])


@pytest.fixture(scope="module")
def clib():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    return _lib.load()


@pytest.mark.parametrize("want,kw", [
    (-1, dict(q=None)), (-1, dict(pos=None)), (-1, dict(turns=None)), (-1, dict(oq=None)), (-1, dict(k=None)), (-1, dict(ok=None)),
    (-5, dict(dtype=3)), (-2, dict(T=0)), (-2, dict(H=0)), (-2, dict(Hk=0)), (-2, dict(rot=5)), (-2, dict(rot=0)), (-2, dict(rot=66)),
    (-2, dict(m=float("inf"))), (-2, dict(q_tok=-64)), (-2, dict(T=1 << 30)),
    (-2, dict(q_tok=1 << 37, T=1 << 27)),          # offsets near 2^63
    (-2, dict(oq_tok=32)), (-2, dict(oq_head=32)),  # results that meet
    (-2, dict(oq_tok=64, oq_head=64)),
    (-2, dict(oq=OK, oq_tok=1024)),                # in place with other strides
    (-2, dict(oq=OK + 64)),                        # over part of the input
    (-2, dict(oq=OK + (1 << 32))),                 # q and k to one place
    (-2, dict(oq=OK + (1 << 32) - 1024 * 3)),      # a result that begins in the other one
    (-2, dict(oq=OK + (1 << 30) - 1024)),          # a result over the other's input
    (-3, dict(q=OK + 1)), (-3, dict(turns=OK + 4)),
])
def test_refusals(clib, want, kw):
    a = dict(dtype=0, q=OK, q_tok=512, q_head=64, k=OK + (1 << 30), pos=OK, turns=OK, T=4, H=8, Hk=2, dim=64, rot=64, m=1.0,
             oq=OK + (1 << 31), oq_tok=512, oq_head=64, ok=OK + (1 << 32))
    a.update(kw)
    assert clib.lmhead_rotary(a["dtype"], a["q"], a["q_tok"], a["q_head"], a["k"], 128, 64, a["pos"], a["turns"], a["T"], a["H"],
                              a["Hk"], a["dim"], a["rot"], 0, 0, a["m"], a["oq"], a["oq_tok"], a["oq_head"], a["ok"], 128, 64,
                              None) == want


@pytest.mark.parametrize("k,heads,clear", [
    (512 * 2, 2, True), (512 * 2, 4, True), (512 * 2, 5, False), (511 * 2, 2, False), (512 * 2 + 1, 2, False), (-256 * 2, 4, True),
    (-256 * 2, 5, False), (768 * 3 * 2 + 512 * 2, 4, True), (768 * 3 * 2 + 448 * 2, 4, False), (0, 1, False)])
def test_parts_of_one_tensor(clib, k, heads, clear):
    """8 query heads and k's, of one row of 768 elements a token, both in place: a call whose
    tensors are clear of one another gets as far as the check of alignment, which it fails."""
    assert clib.lmhead_rotary(0, OK, 768, 64, OK + k, 768, 64, OK, OK + 4, 4, 8, heads, 64, 64, 0, 0, 1.0, OK, 768, 64, OK + k, 768, 64,
                              None) == (-3 if clear else -2)


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    with pytest.raises(TypeError, match="CUDA"):
        L.rotary(torch.zeros(1, 1, 4), None, torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64))


def _n64(x):
    return x.detach().double().cpu().numpy()


def _check(got, x, want, dtype, m, interleaved, half):
    import torch
    u = torch.finfo(getattr(torch, dtype)).eps / 2
    pairs = np.abs(x[..., :2 * half])
    both = pairs[..., 0::2] + pairs[..., 1::2] if interleaved else pairs[..., :half] + pairs[..., half:]
    both = np.repeat(both, 2, -1) if interleaved else np.concatenate([both, both], -1)
    tol = np.zeros_like(want)
    tol[..., :2 * half] = 4.2e-7 * m * both
    tol = tol + u * (np.abs(want) + tol) + 2.0 ** -25  # fp16 rounds absolutely below its normal range
    if dtype != "float16":
        tol -= 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / np.maximum(tol, 1e-300)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("T,H,Hk,dim,rot", [
    (1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (3, 5, 1, 64, 32), (257, 3, 3, 80, 80), (33, 8, 2, 96, 48), (7, 4, 2, 72, 10),
    (600, 20, 4, 64, 64), (2, 9, 0, 130, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_against_oracle(dtype, T, H, Hk, dim, rot, interleaved):
    """Every type, layout and part of a head, in place in a projection's output and
    into others, forward and back, positions from none to the last one."""
    import torch
    from draft_lm_head_gb300 import prep
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(T * 1000 + dim)
    t = getattr(torch, dtype)
    turns = torch.from_numpy(prep.rotary_turns(rot, 500000.0, "wavelength", 4.0)).cuda()
    pos = rng.integers(0, 200000, T)
    pos[rng.random(T) < 0.2] = -1
    pos[0] = 2 ** 31 - 1
    pos[-1] = -5 if T > 2 else 0
    p32 = torch.tensor(np.concatenate([pos, [7, 7]]), dtype=torch.int32, device="cuda")  # longer, as a plan's may be
    for backward, m, inplace in ((False, 1.0, True), (True, 1.25, False)):
        qkv = torch.randn(T, H + 2 * Hk, dim, device="cuda").to(t)
        q, k = qkv[:, :H], qkv[:, H:H + Hk] if Hk else None
        xs = [_n64(x) for x in (q, k) if x is not None]
        rest = qkv[:, H + Hk:].clone()
        out = None if inplace else (torch.full((T, H, dim), 9.0, dtype=t, device="cuda"),
                                    torch.full((T, Hk, dim), 9.0, dtype=t, device="cuda") if Hk else None)
        got = L.rotary(q, k, p32, turns, interleaved=interleaved, backward=backward, magnitude=m, out=out)
        assert L.last_device_error() == 0
        for g, x in zip(got, xs):
            want = O.rotary(x, pos, turns.cpu().numpy(), interleaved, backward, m)
            if not inplace:
                want[pos < 0] = 9.0
            _check(_n64(g), x, want, dtype, m, interleaved, rot // 2)
            assert np.array_equal(_n64(g)[..., rot:], want[..., rot:])
        assert torch.equal(qkv[:, H + Hk:], rest)


@pytest.mark.gpu
def test_backward_is_the_gradient():
    """Against differences of the forward pass, which is linear: <dy, R x> = <R' dy, x>
    for every pair of unit vectors is R' = R^T; with fp32 to its precision."""
    import torch
    from draft_lm_head_gb300 import prep
    from gpu_util import lib
    L = lib()
    turns = torch.from_numpy(prep.rotary_turns(16)).cuda()
    eye = torch.eye(20, device="cuda").view(1, 20, 20)  # heads x dim: the unit vectors
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    for inter in (False, True):
        f = [L.rotary(eye.clone(), None, pos, turns, interleaved=inter, magnitude=1.5, backward=b)[0][0] for b in (False, True)]
        assert (f[0] - f[1].t()).abs().max() <= 1e-6
        x = torch.randn(1, 1, 20, device="cuda", dtype=torch.float64)
        y = [L.rotary((x + d).float(), None, pos, turns, interleaved=inter, magnitude=1.5)[0].double() for d in (0.5, -0.5)]
        dy = torch.ones(1, 1, 20, device="cuda")
        g = L.rotary(dy, None, pos, turns, interleaved=inter, magnitude=1.5, backward=True)[0]
        # a step along all elements at once changes sum(y) by the sum of its gradient
        assert abs((y[0] - y[1]).sum().item() - g.double().sum().item()) <= 1e-4


@pytest.mark.gpu
def test_tokens_far_apart():
    """Offsets past 2^31 elements and 2^32 bytes."""
    import torch
    from draft_lm_head_gb300 import prep
    from gpu_util import lib
    L = lib()
    turns = torch.from_numpy(prep.rotary_turns(64)).cuda()
    pos = torch.tensor([5, 70, 9], dtype=torch.int32, device="cuda")
    step = (1 << 30) + 8
    base = torch.empty(2 * step + 512, dtype=torch.bfloat16, device="cuda")
    q, k = base.as_strided((3, 4, 64), (step, 64, 1)), base[256:].as_strided((3, 2, 64), (step, 128, 1))
    q.copy_(torch.randn(3, 4, 64, device="cuda"))
    k.copy_(torch.randn(3, 2, 64, device="cuda"))
    want = L.rotary(q.contiguous(), k.contiguous(), pos, turns)
    L.rotary(q, k, pos, turns)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.gpu
def test_layouts_streams_and_refusals():
    import torch
    from draft_lm_head_gb300 import prep
    from gpu_util import lib
    L = lib()
    turns = torch.from_numpy(prep.rotary_turns(64)).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    x = torch.randn(50, 4, 64, device="cuda")
    want, _ = L.rotary(x.clone(), None, pos, turns)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(L.rotary(heads_first, None, pos, turns)[0], want)
    odd = torch.empty(50 * 4 * 65 + 1, device="cuda")[1:].view(50, 4, 65)[..., :64]  # no 16-byte rows
    odd.copy_(x)
    assert torch.equal(L.rotary(odd, None, pos, turns)[0], want)
    s = torch.cuda.Stream()
    y = x.clone()
    s.wait_stream(torch.cuda.current_stream())
    L.rotary(y, None, pos, turns, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    z, out = x.clone(), torch.zeros_like(x)
    with torch.cuda.graph(g):
        L.rotary(z, None, pos, turns, out=(out, None))
    g.replay()
    assert torch.equal(out, want)
    for bad in (lambda: L.rotary(x, None, pos[:3], turns), lambda: L.rotary(x, None, pos.long(), turns),
                lambda: L.rotary(x, x[:, :, :32], pos, turns), lambda: L.rotary(x, None, pos, turns.int()),
                lambda: L.rotary(x, None, pos, turns, out=(out.half(), None)), lambda: L.rotary(x, None, pos, turns, out=(out, out)),
                lambda: L.rotary(x[..., ::2], None, pos, turns[:8]), lambda: L.rotary(x.double(), None, pos, turns),
                lambda: L.rotary(x, None, pos, turns, out=(x[:1].expand(50, 4, 64), None)),
                lambda: L.rotary(x[:49], None, pos[:49], turns, out=(x[1:], None))):
        with pytest.raises((TypeError, ValueError, L.LmheadError)):
            bad()
