"""Beam selection and the reordering of states: refusals on the host (no GPU:
every call fails validation first), and the kernels against the oracle.

A score is parent + (x - lse), rounded to fp32 once (half a step, 2^-24 of its
value). lse = top + log(sum): each exp is within 2 steps (2^-22) of its value,
its argument x - top is rounded once (2^-24 |x - top|; terms beyond 32 below the
top weigh less than e^-32), and a thread adds at most 32 terms a tile in fp32 (2^-24
each time, at most 64 of them here). Places may be exchanged, if at all, only
between entries whose exact scores lie closer together than that."""
import ctypes

import numpy as np
import pytest

from oracle import serving_oracle as SO

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced
LSE_TOL = 2.0 ** -22 + 2.0 ** -24 * (32 + 64)


def test_refusals():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    lib = _lib.load()

    def call(dtype=2, logits=OK, stride=100, S=2, beams=4, n=100, k=4, ws=OK, wsb=1 << 40):
        return lib.lmhead_beam_select(dtype, logits, stride, OK, None, None, S, beams, n, k, -1, OK, OK, OK, ws,
                                      wsb, None)
    assert call(logits=None) == -1
    assert call(dtype=3) == -5
    assert call(k=33) == -5
    assert call(beams=257) == -5
    assert call(k=0) == -2
    assert call(n=0) == -2
    assert call(S=0) == -2
    assert call(S=20000) == -2
    assert call(n=1 << 30, beams=2, stride=1 << 30) == -2
    assert call(stride=99) == -2
    assert call(logits=OK + 2) == -3
    assert call(ws=None) == -4
    assert call(ws=OK + 16) == -4
    assert call(wsb=8) == -4
    assert lib.lmhead_beam_workspace_size(2, 4, 100, 33) == 0
    one, none = (ctypes.c_void_p * 1)(OK), (ctypes.c_void_p * 1)(None)
    size, zero = (ctypes.c_int64 * 1)(64), (ctypes.c_int64 * 1)(0)
    re = lib.lmhead_beam_reorder
    assert re(None, 2, 4, 4, 1, one, one, size, None) == -1
    assert re(OK, 2, 4, 4, 1, none, one, size, None) == -1
    assert re(OK, 2, 4, 4, 0, one, one, size, None) == -5
    assert re(OK, 2, 4, 4, 9, one, one, size, None) == -5
    assert re(OK, 2, 4, 4, 1, one, one, zero, None) == -2
    assert re(OK, 0, 4, 4, 1, one, one, size, None) == -2


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    with pytest.raises(TypeError, match="CUDA"):
        L.beam_select(torch.zeros(2, 8), torch.zeros(2), 2, 1)
    with pytest.raises(TypeError, match="CUDA"):
        L.beam_reorder(torch.zeros(1, 2, dtype=torch.int32), [torch.zeros(2)], 2)


def test_oracle_by_hand():
    x = np.log(np.array([[.5, .25, .25], [.1, .8, .1]]))
    got = SO.beam_step(x, np.log([.5, .25]), 2, 4)[0]
    assert [i for _, i in got] == [0, 4, 1, 2]  # .25, .2, .125, .125
    assert np.allclose(np.exp([v for v, _ in got]), [.25, .2, .125, .125])
    got = SO.beam_step(x, np.log([.5, .25]), 2, 2, finished=[True, False])[0]
    assert [i for _, i in got] == [0, 4]


def _check(L, x, scores, beams, k, ids=None, finished=None, eos=7, stream=None):
    import torch
    n = x.shape[1]
    t = lambda v, d: None if v is None else torch.tensor(np.asarray(v), dtype=d, device="cuda")
    parent, token, score = L.beam_select(x, t(scores, torch.float32), beams, k, ids=t(ids, torch.int32),
                                         finished=t(finished, torch.bool), eos=eos, stream=stream)
    torch.cuda.synchronize()
    parent, token, score = (v.cpu().numpy() for v in (parent, token, score))
    x64 = x.double().cpu().numpy()
    want = SO.beam_step(x64, np.asarray(scores, dtype=np.float32), beams, k + 8, finished)
    for s, w in enumerate(want):
        live = min(len(w), k)
        assert np.all(parent[s, live:] == -1) and np.all(token[s, live:] == -1) and np.all(score[s, live:] == -np.inf)
        seen = set()
        for j in range(live):
            b = int(parent[s, j])
            row = s * beams + b
            tol = LSE_TOL + 2.0 ** -24 * abs(w[j][0])
            assert score[s, j] == pytest.approx(w[j][0], abs=tol, rel=0), (s, j)
            if finished is not None and finished[row]:
                assert token[s, j] == eos
                flat = b * n
            else:
                near = [i for v, i in w if abs(v - w[j][0]) <= 2 * tol and i // n == b
                        and (ids[row][i % n] if ids is not None else i % n) == token[s, j]]
                assert near, (s, j, b, token[s, j], w[j])
                flat = near[0]
                gaps = [abs(w[o][0] - w[j][0]) for o in (j - 1, j + 1) if 0 <= o < len(w)]
                # alone, or equal within one row: the place is the oracle's
                if all(g > 2 * tol for g in gaps):
                    assert flat == w[j][1]
            if ids is None:
                assert flat not in seen
                seen.add(flat)
    return parent, token, score


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("S,beams,n,k", [(1, 1, 1, 1), (1, 1, 1, 4), (2, 3, 2, 32), (1, 4, 1002, 4), (3, 2, 8191, 5),
                                         (1, 1, 8193, 32), (2, 5, 20011, 17), (1, 2, 128256, 8), (40, 8, 999, 8),
                                         (300, 4, 300, 2), (1, 256, 50, 9)])
def test_against_oracle(S, beams, n, k, dtype):
    import torch
    from gpu_util import lib
    rng = np.random.default_rng(n + k)
    x = torch.tensor(rng.standard_normal((S * beams, n)) * 3, device="cuda").to(getattr(torch, dtype))
    _check(lib(), x, -rng.random(S * beams) * 5, beams, k)


@pytest.mark.gpu
def test_many_tiles_a_slice():
    """More rows than the GPU holds CTAs: every CTA walks over several tiles and
    keeps its best between them, in ascending and descending order too."""
    import torch
    from gpu_util import lib
    rng = np.random.default_rng(3)
    for kind in ("random", "up", "down"):
        x = rng.standard_normal((1300, 20001)).astype(np.float32)
        if kind != "random":
            x = np.sort(x, axis=1)
            x = x[:, ::-1].copy() if kind == "down" else x
        _check(lib(), torch.tensor(x, device="cuda"), -rng.random(1300), 2, 7)


@pytest.mark.gpu
def test_ids_finished_and_dead_beams():
    import torch
    from gpu_util import lib
    rng = np.random.default_rng(11)
    S, B, n, k = 6, 4, 700, 9
    x = torch.tensor(rng.standard_normal((S * B, n)), dtype=torch.float32, device="cuda")
    ids = np.stack([rng.permutation(5000)[:n] for _ in range(S * B)])
    scores = (-rng.random(S * B)).astype(np.float32)
    done = rng.random(S * B) < 0.4
    done[:B] = True          # a whole sequence has ended: B entries, the rest empty
    scores[B:2 * B - 1] = -np.inf   # a first step: one beam alive
    scores[2 * B] = np.nan
    _check(lib(), x, scores, B, k, ids, done)
    _check(lib(), x, scores, B, k, ids, np.zeros(S * B, dtype=bool))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [37, 5000, 30000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_ties_and_masked_entries(n, dtype):
    """Equal logits in one row go by index (far more of them than the buffer
    holds at the larger sizes), equal beams by beam; masked entries (-inf) are
    never taken, the type's lowest value is; rows of nothing, NaN or +inf give
    nothing."""
    import torch
    from gpu_util import lib
    t = getattr(torch, dtype)
    x = torch.zeros(8, n, dtype=t, device="cuda")
    x[1] = x[0]
    x[2, : n // 2] = -np.inf
    x[3] = -np.inf
    x[4] = torch.finfo(t).min
    x[5] = torch.finfo(t).min
    x[5, 3] = 2.0
    x[6, n // 3] = float("nan")
    x[7, n // 2] = float("inf")
    scores = np.zeros(8, dtype=np.float32)
    parent, token, score = _check(lib(), x, scores, 2, 6)
    assert parent[0].tolist() == [0] * 6 and token[0].tolist() == list(range(6))
    assert parent[1].tolist() == [0] * 6 and token[1].tolist() == list(range(n // 2, n // 2 + 6))
    assert parent[2].tolist() == [1] + [0] * 5 and token[2].tolist() == [3] + list(range(5))
    assert np.all(parent[3] == -1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strides_alignment_and_streams(dtype):
    import torch
    from gpu_util import lib
    L = lib()
    rng = np.random.default_rng(5)
    t = getattr(torch, dtype)
    wide = torch.tensor(rng.standard_normal((4, 20011)), device="cuda").to(t)
    scores = -rng.random(4)
    for a, b in ((1, 9000), (3, 16390), (7, 20010), (8, 8200)):
        _check(L, wide[:, a:b], scores, 2, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _check(L, wide[:, 5:9999], scores, 4, 8, stream=s)
    with pytest.raises(TypeError, match="rows"):
        L.beam_select(wide.t().contiguous().t(), torch.zeros(4, device="cuda"), 2, 2)
    with pytest.raises(ValueError, match="k"):
        L.beam_select(wide, torch.zeros(4, device="cuda"), 2, 33)
    with pytest.raises(ValueError, match="scores"):
        L.beam_select(wide, torch.zeros(3, device="cuda"), 2, 2)
    assert L.last_device_error() == 0


@pytest.mark.gpu
def test_reorder():
    import torch
    from gpu_util import lib
    L = lib()
    g = torch.Generator(device="cuda").manual_seed(1)
    S, B, k = 5, 4, 7
    parent = torch.randint(-1, B, (S, k), generator=g, device="cuda", dtype=torch.int32)
    parent[0, 0] = -1
    states = [torch.randn(S * B, 4096, generator=g, device="cuda").to(torch.bfloat16),
              torch.randint(0, 99, (S * B, 3, 5), generator=g, device="cuda", dtype=torch.int32),
              torch.randint(0, 99, (S * B, 13), generator=g, device="cuda", dtype=torch.uint8),
              torch.randn(S * B, 9000, generator=g, device="cuda"),
              torch.randn(S * B * 40 + 1, generator=g, device="cuda")[1:].view(S * B, 40)]
    got = L.beam_reorder(parent, states, B)
    row = (torch.arange(S, device="cuda")[:, None] * B + parent.clamp(min=0)).view(-1)
    for t, o in zip(states, got):
        want = torch.where((parent >= 0).view(-1, *[1] * (t.dim() - 1)), t[row.long()], torch.zeros_like(t[:1]))
        assert torch.equal(o, want)
    assert L.last_device_error() == 0
    parent[1, 2] = B
    bad = L.beam_reorder(parent, states[:1], B)[0]
    assert not bad[k + 2].any() and L.last_device_error() == -7
    with pytest.raises(ValueError, match="states"):
        L.beam_reorder(parent, [], B)
    with pytest.raises(ValueError, match="states"):
        L.beam_reorder(parent, [states[0][1:]], B)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("climb", [1.5, 3, 10, 20, 30, 45, 59.5, 200])
def test_rows_that_climb(climb, dtype):
    """Few values at 0 to 1 in a row's first tile, and two far above them in a late
    one that decide the sum, in a row of one slice.

    A value may lie 1 above the reference that its exponential is taken from (and no
    value matters that lies far below the top: z e^-z < 1). An exponential is within
    2^-22, its argument is rounded three times (difference, product, the factor
    itself: 2^-24 of its size each), and the same goes for the scaling of a lane's
    sum to its warp's and of a slice's to its row's, and for two moves of the
    reference. With at most four values a lane every sum is rounded four times in it."""
    import torch
    from gpu_util import lib
    L = lib()
    g = torch.Generator("cuda").manual_seed(int(climb * 10))
    R, n = 4000, 6000
    x = torch.full((R, n), -np.inf, device="cuda")
    first = torch.arange(0, 512, 4, device="cuda")
    x[:, first] = torch.rand(R, 128, generator=g, device="cuda")
    x[:, 3200] = climb + torch.rand(R, generator=g, device="cuda")
    x[:, 3205] = climb + torch.rand(R, generator=g, device="cuda")
    x = x.to(getattr(torch, dtype))
    scores = -torch.rand(R, generator=g, device="cuda")
    parent, token, score = L.beam_select(x, scores, 2, 3)
    x64 = x.double()
    want = scores.double()[:, None] + (x64 - torch.logsumexp(x64, 1, keepdim=True))
    want, flat = want.view(R // 2, 2 * n).topk(4, dim=1)
    tol = 5 * (2.0 ** -22 + 3 * 2.0 ** -24) + 4 * 2.0 ** -24
    off = (score.double() - want[:, :3]).abs() - 2.0 ** -24 * want[:, :3].abs()
    assert off.max().item() <= tol, (off.max().item(), tol)
    # where the scores are that far apart, so is their order
    got = parent.long() * n + token.long()
    alone = torch.ones_like(got, dtype=torch.bool)
    gap = want[:, :3] - want[:, 1:]
    wide = 2 * (tol + 2.0 ** -24 * want[:, 1:].abs())
    alone &= gap > wide
    alone[:, 1:] &= (gap > wide)[:, :2]
    assert torch.equal(got[alone], flat[:, :3][alone])


def test_reorder_within_a_buffer_is_refused():
    """S = 2, 4 beams, k = 3: 8 source rows and 6 destination rows of 64 bytes."""
    from draft_lm_head_gb300 import build, _lib
    build.build()
    re = _lib.load().lmhead_beam_reorder
    at = lambda *x: (ctypes.c_void_p * len(x))(*x)
    size = (ctypes.c_int64 * 2)(64, 64)
    A, B, PARENT = 1 << 20, 1 << 21, 1 << 22
    for dst in (A, A + 511, A - 383, PARENT + 23, PARENT - 383):
        assert re(PARENT, 2, 4, 3, 1, at(A), at(dst), size, None) == -2
    assert re(PARENT, 2, 4, 3, 2, at(A, B), at(3 * A, B - 383), size, None) == -2    # the other's source
    assert re(PARENT, 2, 4, 3, 2, at(A, B), at(3 * A, 3 * A + 383), size, None) == -2  # the other's destination


@pytest.mark.gpu
def test_reorder_next_to_its_source():
    """Destinations that begin where a source ends."""
    import torch
    from gpu_util import lib
    L = lib()
    buf = torch.arange(8 * 16 + 6 * 16, device="cuda", dtype=torch.int32)
    parent = torch.tensor([[3, 0, -1], [1, 1, 2]], device="cuda", dtype=torch.int32)
    src, dst = buf[:128].view(8, 16), buf[128:].view(6, 16)
    want = torch.cat([src[3:4], src[:1], torch.zeros_like(src[:1]), src[5:6], src[5:6], src[6:7]])
    got, = L.beam_reorder(parent, [src], 4, out=[dst])
    assert torch.equal(got, want)
    with pytest.raises(L.LmheadError):
        L.beam_reorder(parent, [src], 4, out=[src[2:]])
