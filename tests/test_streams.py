"""Memory of calls that run on a stream other than the current one: the
allocator may not hand it out again before that stream is done with it. Shown by
addresses alone, while a stream is kept busy for a while."""
import pytest
import torch

import draft_lm_head_gb300 as L
from draft_lm_head_gb300 import _memory


class Named(torch.Tensor):
    """A tensor that lists the streams it is told about."""

    def record_stream(self, s):
        self.seen = getattr(self, "seen", []) + [s]


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_scratch_is_named_to_the_allocator():
    cpu = torch.device("cpu")
    a, b = FakeStream(1), FakeStream(2)
    t = torch.empty(512, dtype=torch.uint8).as_subclass(Named)
    assert _memory.scratch(t, 256, cpu, a) is t and t.seen == [a]
    ws = L.Workspace()
    ws.buf = torch.empty(512, dtype=torch.uint8).as_subclass(Named)
    for s in (a, b, a, b):  # once a stream
        assert _memory.scratch(ws, 512, cpu, s) is ws.buf
    assert ws.buf.seen == [a, b]


def test_workspace_tensors_are_checked():
    cpu, meta = torch.device("cpu"), torch.device("meta")
    t = torch.zeros(1024, dtype=torch.uint8)
    assert _memory.scratch(t, 512, cpu, None) is t
    assert _memory.scratch(torch.zeros(256), 512, cpu, None).numel() == 1024
    for bad, dev in ((t, meta), (t[::2], cpu), (torch.zeros(32, 32).t(), cpu)):
        with pytest.raises(ValueError, match="workspace"):
            _memory.scratch(bad, 512, dev, None)


class Elsewhere(torch.Tensor):
    """A host tensor that says to be on the second GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def test_tensors_of_another_device_are_refused(monkeypatch):
    from draft_lm_head_gb300 import serving
    monkeypatch.setattr(serving, "_current_device", lambda: 0)
    x = torch.zeros(4, 4).as_subclass(Elsewhere)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: L.page_plan(x, i, i, i, i, 16, 4), lambda: L.chunk_attention(x, x, x, i, i, i),
                 lambda: L.q4_head(i, x, x, 32), lambda: L.q4_gather_logits(i, x, x, i, 32),
                 lambda: L.beam_select(x, x, 2, 2), lambda: L.beam_reorder(x, [x], 2)):
        with pytest.raises(ValueError, match="current device"):
            call()


def _overlap(a: torch.Tensor, ptr: int, nbytes: int) -> bool:
    return a.data_ptr() < ptr + nbytes and ptr < a.data_ptr() + a.numel() * a.element_size()


def _busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(1_000_000_000)  # about half a second


def _beams(n):
    g = torch.Generator("cuda").manual_seed(n)
    return torch.randn(64, n, device="cuda", generator=g), torch.zeros(64, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("explicit", [True, False])
def test_workspace_that_grows_while_its_stream_is_busy(explicit):
    from gpu_util import lib
    lib()
    small, large = _beams(4000), _beams(200000)
    want = [L.beam_select(x, sc, 4, 8) for x, sc in (small, large)]
    s = torch.cuda.Stream()
    ws = L.Workspace()
    L.beam_select(*small, 4, 8, workspace=ws)  # allocated on the current stream
    torch.cuda.synchronize()
    _busy(s)
    if explicit:
        got = [L.beam_select(*small, 4, 8, workspace=ws, stream=s)]
    else:
        with torch.cuda.stream(s):
            got = [L.beam_select(*small, 4, 8, workspace=ws)]
    old = ws.buf.data_ptr(), ws.buf.numel()
    got.append(L.beam_select(*large, 4, 8, workspace=ws))
    assert ws.buf.numel() > old[1]
    blocks = [torch.empty(old[1], dtype=torch.uint8, device="cuda") for _ in range(4)]
    idle = s.query()
    assert idle or not any(_overlap(b, *old) for b in blocks)
    assert not idle  # the wait was long enough for the test to mean something
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_scratch_of_a_call_on_a_busy_stream():
    """No workspace given: the one of the call is gone when it returns."""
    from gpu_util import lib
    lib()
    x, sc = _beams(4000)
    need = L.load().lmhead_beam_workspace_size(16, 4, 4000, 8)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    taken = []
    real = _memory._allocate
    try:
        _memory._allocate = lambda *a: taken.append(real(*a)) or taken[-1]
        _busy(s)
        L.beam_select(x, sc, 4, 8, stream=s)
    finally:
        _memory._allocate = real
    old = taken[0].data_ptr(), taken[0].numel()
    assert old[1] >= need
    taken.clear()
    blocks = [torch.empty(old[1], dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not s.query()
    assert not any(_overlap(b, *old) for b in blocks)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_results_of_a_call_on_another_stream():
    """Memory that the current stream is not done with is not taken for the
    result of a call on another stream; nor is such a result's own memory while
    the current stream still reads it."""
    from gpu_util import lib
    lib()
    g = torch.Generator("cuda").manual_seed(0)
    codes = torch.randint(0, 256, (60000, 128), device="cuda", dtype=torch.uint8, generator=g)
    scales = torch.rand(60000, 4, device="cuda", generator=g).to(torch.bfloat16)
    h = torch.randn(8, 256, device="cuda", generator=g).to(torch.bfloat16)
    want = L.q4_head(codes, scales, h, 64)
    cur, s = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks in both pools, so that no call below has to ask the driver (which waits)
    for at in (cur, s):
        with torch.cuda.stream(at):
            blocks = [torch.empty_like(want) for _ in range(4)]
            del blocks
    # a tensor that the current stream writes late, freed before the call
    kept, y = torch.empty_like(want), torch.empty_like(want)
    _busy(cur)
    y.zero_()
    old = y.data_ptr(), y.numel() * 4
    del y
    out = L.q4_head(codes, scales, h, 64, stream=s)
    assert not cur.query() and not _overlap(out, *old)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the result, read late by the current stream and freed before the next call
    h2 = h * 2
    torch.cuda.synchronize()
    _busy(cur)
    kept.copy_(out)
    old = out.data_ptr(), out.numel() * 4
    del out
    again = L.q4_head(codes, scales, h2, 64, stream=s)
    assert not cur.query() and not _overlap(again, *old)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


@pytest.mark.gpu
def test_calls_on_a_stream_of_a_capture():
    """A stream that joins the capture and takes a call with its results and
    workspace; a device without an index is the current one."""
    from gpu_util import lib
    lib()
    x, sc = _beams(4000)
    want = L.beam_select(x, sc, 4, 8)
    ws, s = L.Workspace(), torch.cuda.Stream()
    assert ws.get(1000, torch.device("cuda")).numel() >= 1000
    L.beam_select(x, sc, 4, 8, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        a = L.beam_select(x, sc, 4, 8, workspace=ws, stream=s)
        b = L.beam_select(x, sc, 4, 8, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for y in (*a, *b):
        y.zero_()
    g.replay()
    torch.cuda.synchronize()
    for y, z, w in zip(a, b, want):
        assert torch.equal(y, w) and torch.equal(z, w)
