"""Page plan: the oracle by hand, refusals on the host (no GPU: every call fails
validation first), and the kernel against the oracle."""
import numpy as np
import pytest

from oracle import serving_oracle as SO

OK = 1 << 20  # 16-byte aligned fake address; never dereferenced


def test_oracle_by_hand():
    """Four pages free: the first request takes one, the second needs three and
    three are left, the third stays in the page it holds."""
    table = np.array([[7, 8, -1, -1], [5, -1, -1, -1], [9, -1, -1, -1]])
    slots, pos, cu, ok, left, tab = SO.page_plan([4, 1, 1], [1, 7, 1], table, [1, 2, 3, 4], 4, 2, 12)
    assert ok.tolist() == [1, 1, 1] and left == 0 and cu.tolist() == [0, 1, 8, 9]
    assert tab.tolist() == [[7, 8, 4, -1], [5, 3, 2, 1], [9, -1, -1, -1]]
    assert slots.tolist() == [8, 11, 6, 7, 4, 5, 2, 3, 19, -1, -1, -1]
    assert pos.tolist() == [4, 1, 2, 3, 4, 5, 6, 7, 1, -1, -1, -1]


def test_refusals():
    from draft_lm_head_gb300 import build, _lib
    build.build()
    lib = _lib.load()

    def call(lens=OK, S=4, width=8, free=OK, cap=16, page=16, T=32, left=2 * OK):
        return lib.lmhead_page_plan(lens, OK, S, OK, width, free, cap, OK, page, T, OK, OK, OK, OK, left, None)
    assert call(lens=None) == -1
    assert call(free=None) == -1
    assert call(S=0) == -2
    assert call(width=0) == -2
    assert call(cap=-1) == -2
    assert call(page=0) == -2
    assert call(T=0) == -2
    assert call(S=1 << 20, width=1 << 20) == -2
    assert call(left=OK) == -2  # the result must not alias the count it is made from


def test_binding_takes_cuda_tensors_only():
    import torch
    import draft_lm_head_gb300 as L
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        L.page_plan(i, i, i.view(2, 1), i, i[:1], 16, 4)


def _run(lens, new, table, free, count, page, T):
    import torch
    from gpu_util import lib
    L = lib()
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    tab = dev(table)
    p = L.page_plan(dev(lens), dev(new), tab, dev(free), dev([count]), page, T)
    want = SO.page_plan(lens, new, table, free, count, page, T)
    got = [x.cpu().numpy() for x in (p.slots, p.positions, p.cu, p.granted)] + [int(p.free_left[0]), tab.cpu().numpy()]
    for g, w, name in zip(got, want, ("slots", "positions", "cu", "granted", "left", "table")):
        assert np.array_equal(g, w), name
    return L


@pytest.mark.gpu
@pytest.mark.parametrize("S", [1, 7, 8, 9, 300, 1025])
@pytest.mark.parametrize("page", [1, 16, 48, 128])
def test_against_oracle(S, page):
    """Lengths from nothing to many pages, requests without new tokens, a pool
    that runs out on the way, room past the last token."""
    rng = np.random.default_rng(S * 1000 + page)
    lens = rng.integers(0, 5 * page + 3, S)
    new = np.where(rng.random(S) < 0.3, 0, rng.integers(0, 3 * page + 2, S))
    need = -(-(lens + new) // page) - -(-lens // page)
    width = int((-(-(lens + new) // page)).max()) or 1
    ids = rng.permutation(S * width + 40)
    table = np.full((S, width), -1)
    at = 0
    for s in range(S):
        h = -(-int(lens[s]) // page)
        table[s, :h] = ids[at:at + h]
        at += h
    for frac in (1.0, 0.5, 0.0):
        count = int(need.sum() * frac)
        free = np.concatenate([ids[at:], [0]])[:max(count, 1)]
        L = _run(lens, new, table, free, count, page, int(new.sum()) + 5)
        assert L.last_device_error() == 0


@pytest.mark.gpu
def test_bad_lengths_and_small_buffers():
    table = np.arange(12).reshape(4, 3)
    # negative lengths, and one past the table's width, are not granted and take nothing
    L = _run([-1, 3, 40, 5], [2, -4, 10, 20], table, [20, 21, 22, 23], 4, 16, 40)
    assert L.last_device_error() == 0
    _run([0, 16], [8, 8], table[:2], [20, 21, 22], 3, 16, 10)  # six tokens without a place
    assert L.last_device_error() == -7
    # a free count above the list's length is the length
    _run([0, 0], [40, 40], table[:2], [20, 21, 22], 99, 16, 80)
    assert L.last_device_error() == 0


@pytest.mark.gpu
def test_other_stream_and_reused_buffers():
    import torch
    from gpu_util import lib
    L = lib()
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    lens, new, free, count = dev([5, 30]), dev([20, 4]), dev([9, 8, 7, 6]), dev([4])
    a, b = dev([[1, -1, -1], [2, 3, -1]]), dev([[1, -1, -1], [2, 3, -1]])
    p = L.page_plan(lens, new, a, free, count, 16, 30)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = L.page_plan(lens, new, b, free, count, 16, 30, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    again = L.page_plan(lens, new, a, free, count, 16, 30, out=p)
    assert again.slots.data_ptr() == p.slots.data_ptr()
    for x, y in zip(p, q):
        assert torch.equal(x, y)
    assert torch.equal(a, b)
    with pytest.raises(ValueError, match="new_lens"):
        L.page_plan(lens, new[:1], a, free, count, 16, 30)
    with pytest.raises(TypeError, match="table"):
        L.page_plan(lens, new, a.t().contiguous().t(), free, count, 16, 30)


@pytest.mark.gpu
def test_empty_list_of_free_pages():
    """Requests that stay within the pages they hold are granted, the others are
    not; an empty tensor has no address."""
    table = np.arange(12).reshape(4, 3)
    for count in (0, 5):
        L = _run([4, 16, 30, 0], [3, 1, 2, 0], table, np.zeros(0, dtype=np.int32), count, 16, 8)
        assert L.last_device_error() == 0
