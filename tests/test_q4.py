"""The 4-bit head: refusals on the host (no GPU: every call fails validation
first), the offline codes, and the kernels against fp64.

Codes minus 8 times 16-bit values are exact, so a logit is off by its fp32
additions alone: along a group's chain of matrix instructions (16 products each,
d/16 of them over the row, each addition within one step, 2^-23 of the running
sum) and then a multiplication and an addition a group (half a step each). With
an offset the group's constant min + 8 s and the sum of h are rounded too. Every
running sum is at most A = sum_G (|s| sum |c - 8||h| + |o| sum |h|)."""
import numpy as np
import pytest

from oracle import serving_oracle as SO

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


def test_refusals():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    lib = _lib.load()

    def head(dtype=0, codes=OK, scales=OK, mins=None, h=OK, n=100, d=256, group=64, M=2):
        return lib.lmhead_q4_head(dtype, codes, scales, mins, h, n, d, group, M, OK, None)
    assert head(codes=None) == -1
    assert head(h=None) == -1
    assert head(dtype=2) == -5
    assert head(group=48) == -5
    assert head(d=200) == -2
    assert head(d=0) == -2
    assert head(n=0) == -2
    assert head(M=0) == -2
    assert head(d=65536 + 128) == -2
    assert head(codes=OK + 8) == -3
    assert head(h=OK + 2) == -3
    assert head(scales=OK + 1) == -3
    assert head(mins=OK + 1) == -3
    gather = lib.lmhead_q4_gather_logits
    assert gather(0, OK, OK, None, OK, None, 100, 256, 64, 2, 8, OK, None) == -1
    assert gather(0, OK, OK, None, OK, OK, 100, 256, 64, 2, 0, OK, None) == -2
    assert gather(1, OK, OK, None, OK, OK, 100, 256, 64, 60000, 60000, OK, None) == -2


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    with pytest.raises(TypeError, match="CUDA"):
        L.q4_head(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1), torch.zeros(1, 32), 32)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("fp16", [False, True])
def test_quantise_rows(group, offsets, fp16):
    """Every weight is within half a code of what is stored, plus what rounding
    the scale and the offset costs (half a step each, the scale's times the code)."""
    from draft_lm_head_gb300 import prep
    rng = np.random.default_rng(group + offsets)
    W = rng.standard_normal((37, 2 * group))
    W[3] = 0.0
    W[5, :group] = 0.25
    q = prep.quantise_rows(W, group, offsets, fp16, block=16)
    as64 = (lambda x: x.astype(np.float64)) if fp16 else prep._bits_to_f64
    s = as64(q["scales"])
    mins = as64(q["mins"]) if offsets else None
    back = SO.q4_rows(q["codes"], s, mins, group)
    u = 2.0 ** -11 if fp16 else 2.0 ** -8
    per = np.repeat(s, group, axis=1)
    span = 15 * per + np.repeat(np.abs(mins), group, axis=1) if offsets else 8 * per
    assert np.all(np.abs(back - W) <= 0.5 * per + u * span * (1 + u) + 1e-12)
    with pytest.raises(ValueError):
        prep.quantise_rows(W, 48)


def _inputs(n, d, group, M, dtype, mins, seed):
    import torch
    t = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, d // group, generator=g, device="cuda") * 0.02 - 0.004).to(t)
    off = (torch.randn(n, d // group, generator=g, device="cuda") * 0.05).to(t) if mins else None
    h = torch.randn(M, d, generator=g, device="cuda").to(t)
    return codes, scales, off, h


def _exact(codes, scales, off, h, group):
    """Logits M x n in fp64 and what they may be off by."""
    s = scales.double().cpu().numpy()
    o = None if off is None else off.double().cpu().numpy()
    x = h.double().cpu().numpy()
    c = codes.cpu().numpy()
    w = SO.q4_rows(c, s, o, group)
    A = np.abs(x) @ np.abs(SO.q4_rows(c, s, None, group)).T
    const = np.zeros_like(s) if o is None else o + 8 * s
    A += np.abs(x).reshape(len(x), -1, group).sum(2) @ np.abs(const).T
    d = x.shape[1]
    steps = d / 16 + d / group + (0 if o is None else group + 2 * d / group)
    return x @ w.T, A * steps * 2.0 ** -23 + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group,d", [(32, 32), (32, 224), (64, 64), (64, 2880), (128, 128), (128, 4096), (32, 2880),
                                     (64, 5120)])
@pytest.mark.parametrize("n,M", [(1, 1), (33, 3), (1000, 8), (517, 9), (301, 17), (200, 37)])
def test_head(n, M, group, d, mins, dtype):
    import torch
    from gpu_util import lib
    L = lib()
    codes, scales, off, h = _inputs(n, d, group, M, dtype, mins, n + d)
    got = L.q4_head(codes, scales, h, group, mins=off)
    want, tol = _exact(codes, scales, off, h, group)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    assert torch.equal(got, L.q4_head(codes, scales, h, group, mins=off))  # the same sums each time
    K = max(1, n // 3)
    ids = torch.randint(0, n, (M, K), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(4))
    got = L.q4_gather_logits(codes, scales, h, ids, group, mins=off)
    at = ids.long().cpu().numpy()
    assert np.all(np.abs(got.double().cpu().numpy() - np.take_along_axis(want, at, 1)) <= np.take_along_axis(tol, at, 1))
    assert L.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 16])
def test_many_rows(M):
    """More row tiles than the GPU holds at once."""
    from gpu_util import lib
    codes, scales, off, h = _inputs(100003, 256, 64, M, "bfloat16", True, 1)
    got = lib().q4_head(codes, scales, h, 64, mins=off)
    want, tol = _exact(codes, scales, off, h, 64)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d", [(1, 65536), (8, 20480), (16, 9600)])
def test_wide_rows(M, d):
    """h past the shared memory: the row is summed in pieces."""
    from gpu_util import lib
    codes, scales, off, h = _inputs(65, d, 64, M, "float16", True, 2)
    got = lib().q4_head(codes, scales, h, 64, mins=off)
    want, tol = _exact(codes, scales, off, h, 64)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    import torch
    ids = torch.arange(64, -1, -1, device="cuda", dtype=torch.int32).repeat(M, 1)
    got = lib().q4_gather_logits(codes, scales, h, ids, 64, mins=off)
    assert np.all(np.abs(got.double().cpu().numpy()[:, ::-1] - want) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,scale", [("bfloat16", 1e-30), ("bfloat16", 1e30), ("float16", 1e-4), ("float16", 1e4),
                                         ("bfloat16", 0.0)])
@pytest.mark.parametrize("mins", [False, True])
def test_hidden_vectors_of_any_size(dtype, scale, mins):
    """Large, small and zero vectors, and elements far apart within one: they are
    held relative to a vector's largest, to 2^-36 of it at least."""
    import torch
    from gpu_util import lib
    L = lib()
    codes, scales, off, h = _inputs(300, 512, 64, 5, dtype, mins, 4)
    g = torch.Generator(device="cuda").manual_seed(2)
    e = torch.randint(-25, 1, h.shape, generator=g, device="cuda").float()
    h = (h.float() * torch.exp2(e) * scale).to(h.dtype)
    got = L.q4_head(codes, scales, h, 64, mins=off).double().cpu().numpy()
    want, tol = _exact(codes, scales, off, h, 64)
    rest = np.abs(SO.q4_rows(codes.cpu().numpy(), scales.double().cpu().numpy(),
                             None if off is None else off.double().cpu().numpy(), 64)).sum(1)
    tol = tol + 2.0 ** -36 * h.double().abs().amax(1).cpu().numpy()[:, None] * rest
    assert np.all(np.abs(got - want) <= tol)
    ids = torch.arange(300, device="cuda", dtype=torch.int32).repeat(5, 1)
    got = L.q4_gather_logits(codes, scales, h, ids, 64, mins=off).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(7, 1), (3, 33), (40, 65), (1, 3000)])
def test_gather_of_few_and_many(M, K):
    """Runs of tiles over several hidden vectors, one tile, and many."""
    import torch
    from gpu_util import lib
    codes, scales, off, h = _inputs(1000, 1024, 128, M, "bfloat16", False, M)
    ids = torch.randint(0, 1000, (M, K), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(K))
    got = lib().q4_gather_logits(codes, scales, h, ids, 128).double().cpu().numpy()
    want, tol = _exact(codes, scales, off, h, 128)
    at = ids.long().cpu().numpy()
    assert np.all(np.abs(got - np.take_along_axis(want, at, 1)) <= np.take_along_axis(tol, at, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group,d", [(32, 256), (64, 512), (128, 1024), (64, 4096), (128, 3968)])
@pytest.mark.parametrize("n,M", [(20011, 1), (9973, 7)])
def test_shared_tiles_and_scales_anywhere(n, M, group, d, mins):
    """Tiles divided between warps at every stage; scales at an address that allows
    wide copies and at one that allows none."""
    import torch
    from gpu_util import lib
    L = lib()
    codes, scales, off, h = _inputs(n, d, group, M, "bfloat16", mins, n + d)

    def moved(x):
        if x is None:
            return None
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return y.copy_(x)

    want, tol = _exact(codes, scales, off, h, group)
    ids = torch.randint(0, n, (M, 333), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(d))
    at = ids.long().cpu().numpy()
    for sc, mi in ((scales, off), (moved(scales), moved(off))):
        got = L.q4_head(codes, sc, h, group, mins=mi).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol)
        got = L.q4_gather_logits(codes, sc, h, ids, group, mins=mi).double().cpu().numpy()
        assert np.all(np.abs(got - np.take_along_axis(want, at, 1)) <= np.take_along_axis(tol, at, 1))


@pytest.mark.gpu
def test_bad_ids_streams_and_refusals():
    import torch
    from gpu_util import lib
    L = lib()
    codes, scales, off, h = _inputs(50, 256, 64, 2, "bfloat16", False, 3)
    ids = torch.tensor([[0, 50, 3], [-1, 49, 1]], device="cuda", dtype=torch.int32)
    got = L.q4_gather_logits(codes, scales, h, ids, 64)
    assert torch.isnan(got).cpu().tolist() == [[False, True, False], [True, False, False]]
    assert L.last_device_error() == -7 and L.last_device_error() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = L.q4_head(codes, scales, h, 64, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, L.q4_head(codes, scales, h, 64))
    with pytest.raises(ValueError, match="group"):
        L.q4_head(codes, scales, h, 96)
    with pytest.raises(ValueError, match="scales"):
        L.q4_head(codes, scales[:, :1].contiguous(), h, 64)
    with pytest.raises(TypeError, match="scales"):
        L.q4_head(codes, scales.half(), h, 64)
    with pytest.raises(ValueError, match="ids"):
        L.q4_gather_logits(codes, scales, h, ids[:1], 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group,d", [(32, 128), (64, 512), (128, 1024)])
@pytest.mark.parametrize("M", [5, 12])
def test_infinite_and_nan_elements(M, group, d, mins, dtype):
    """A vector with one gives no finite logit; the others' are what they were."""
    import torch
    from gpu_util import lib
    L = lib()
    codes, scales, off, h = _inputs(300, d, group, M, dtype, mins, M)
    ids = torch.randint(0, 300, (M, 77), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(1))
    ids[:, -1] = ids[:, 0]
    calls = (lambda x: L.q4_head(codes, scales, x, group, mins=off),
             lambda x: L.q4_gather_logits(codes, scales, x, ids, group, mins=off))
    want = [f(h) for f in calls]
    bad = h.clone()
    bad[1, 3], bad[2, d - 1], bad[3, d // 2] = float("inf"), float("nan"), -float("inf")
    rest = [0] + list(range(4, M))
    for f, w in zip(calls, want):
        got = f(bad)
        assert not torch.isfinite(got[1:4]).any()
        assert torch.equal(got[rest], w[rest])
    assert L.last_device_error() == 0
