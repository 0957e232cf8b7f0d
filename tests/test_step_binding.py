"""The Python entry points of the operators of a step check what they are given before
any pointer is taken: tensors of another device, of other shapes and types. (No GPU:
host tensors that say to be on one.)"""
import pytest
import torch

import draft_lm_head_gb300 as L
from draft_lm_head_gb300 import serving


class On(torch.Tensor):
    """A host tensor that says to be on the first GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


class Elsewhere(torch.Tensor):
    """And on the second."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def _t(*shape, dtype=torch.float32, kind=On):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def _i(*shape, kind=On):
    return _t(*shape, dtype=torch.int32, kind=kind)


def _calls():
    bf = torch.bfloat16
    ok = dict(q=_t(3, 4, 64, dtype=bf), k=_t(3, 2, 64, dtype=bf), pos=_i(3), turns=_t(32, dtype=torch.int64), kc=_t(5, 16, 2, 64, dtype=bf),
              w=_t(5, 16, 2), table=_i(2, 4), lens=_i(2), cu=_i(3), lse=_t(3, 4), p=_t(3, 50), tok=_i(3), r=_t(3), u=_t(2), ids=_i(3, 8),
              cq=_t(3, 8), kept=_i(2, 6), free=_i(9), count=_i(1))
    return ok, dict(
        rotary=(lambda a: L.rotary(a["q"], a["k"], a["pos"], a["turns"]), "q k pos turns"),
        verify_tree=(lambda a: L.verify_tree(a["p"], a["tok"], a["tok"], a["cu"], a["r"], a["u"], 2, cand_ids=a["ids"], cand_q=a["cq"]),
                     "p tok cu r u ids cq"),
        cache_keep=(lambda a: L.cache_keep([a["kc"], a["w"]], a["table"], a["kept"], first=a["lens"]), "kc w table kept lens"),
        page_release=(lambda a: L.page_release(a["lens"], a["lens"], a["table"], a["free"], a["count"], 16, cu=a["cu"]),
                      "lens table free count cu"),
        cache_weights=(lambda a: L.cache_weights(a["q"], a["kc"], a["table"], a["lens"], a["cu"], a["lse"], a["w"]),
                       "q kc table lens cu lse w"),
        cache_select=(lambda a: L.cache_select(a["w"], a["table"], a["lens"], 4), "w table lens"))


NAMES = ["rotary", "verify_tree", "cache_keep", "page_release", "cache_weights", "cache_select"]


@pytest.fixture(autouse=True)
def _first_gpu(monkeypatch):
    from draft_lm_head_gb300 import _memory, build, step
    build.build()
    monkeypatch.setattr(serving, "_current_device", lambda: 0)
    host = lambda shape, dtype, device, stream: torch.zeros(shape, dtype=dtype).as_subclass(On)
    monkeypatch.setattr(step, "result", host)
    monkeypatch.setattr(step, "scratch", lambda ws, nbytes, device, stream: torch.zeros(1 << 21, dtype=torch.uint8))
    monkeypatch.setattr(step, "_weights_bytes", lambda device, S: 0)

    class Lib:  # reached with all checks passed
        def __getattr__(self, name):
            return lambda *a: 0
    monkeypatch.setattr(step, "load", lambda: Lib())
    monkeypatch.setattr(step, "stream_handle", lambda stream, device: 0)


@pytest.mark.parametrize("name", NAMES)
def test_good_calls_reach_the_library(name):
    ok, calls = _calls()
    calls[name][0](ok)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device(name):
    ok, calls = _calls()
    call, args = calls[name]
    for a in args.split():
        bad = dict(ok)
        bad[a] = ok[a].as_subclass(torch.Tensor).clone().as_subclass(Elsewhere)
        with pytest.raises((ValueError, TypeError)):
            call(bad)


SHAPES = dict(
    rotary=dict(k=(3, 2, 32), pos=(2,)), verify_tree=dict(tok=(4,), cu=(3, 1), r=(2,), u=(3,), ids=(3, 7), cq=(2, 8)),
    cache_keep=dict(w=(5, 16, 3), table=(3, 4), kept=(2, 3, 6), lens=(3,)), page_release=dict(table=(3, 4), count=(2,), cu=(4,)),
    cache_weights=dict(kc=(5, 16, 2, 32), table=(3, 4), lens=(3,), cu=(4,), lse=(3, 3), w=(5, 16, 4)), cache_select=dict(table=(3, 4), lens=(1,)))


@pytest.mark.parametrize("name", NAMES)
def test_other_shapes_and_types(name):
    ok, calls = _calls()
    call, args = calls[name]
    wrong = [(a, torch.zeros(shape, dtype=ok[a].dtype)) for a, shape in SHAPES[name].items()]
    for a in args.split():
        if not (name == "cache_keep" and a in ("kc", "w")):  # (moves rows of any type)
            wrong += [(a, ok[a].as_subclass(torch.Tensor).to(t)) for t in (torch.float64, torch.int16)]
    for a, x in wrong:
        with pytest.raises((ValueError, TypeError)):
            call(dict(ok, **{a: x.as_subclass(On)}))


def test_candidates_of_no_column():
    """An empty tensor has no address: it must not pass for children that are given."""
    ok, calls = _calls()
    with pytest.raises(ValueError, match="candidate"):
        calls["verify_tree"][0](dict(ok, ids=_i(3, 0), cq=_t(3, 0)))
