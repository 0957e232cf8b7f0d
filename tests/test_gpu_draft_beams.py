"""The drafting example: every beam's score is that of its tokens when each is
read again from the start, by plain attention over the whole sequence in fp64.

The states are bf16: each of the layer's results (q, k, v, o and the sum behind
them) is rounded to 2^-8 of its value, in the example as here, and one that falls
to the other side of a rounding moves a logit by a few hundredths at this model's
sizes (logits of about unit spread, d = 256); 0.1 a token is allowed."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _state(model, tokens):
    """The layer's result at the last of the tokens, rounded as the example does."""
    import torch
    H, Hk, D = model.heads, model.kv_heads, model.dim
    x = model.embed[torch.tensor(tokens, device="cuda")]
    qkv = (x @ model.qkv).view(-1, H + 2 * Hk, D)
    q = qkv[-1, :H].double()
    k, v = (qkv[:, H + i * Hk:H + (i + 1) * Hk].double().repeat_interleave(H // Hk, 1) for i in (0, 1))
    p = torch.softmax((k * q).sum(-1) * D ** -0.5, 0)
    o = (p[..., None] * v).sum(0).to(torch.bfloat16)
    return x[-1:] + o.reshape(1, H * D) @ model.out


@pytest.mark.parametrize("beams,steps,page", [(1, 3, 16), (4, 6, 16), (3, 20, 32)])
def test_scores_of_the_beams(beams, steps, page):
    import torch
    from gpu_util import lib
    L = lib()
    import draft_beams
    model = draft_beams.Drafter()
    rng = np.random.default_rng(beams)
    prompts = [rng.integers(0, model.n, n).tolist() for n in (1, 16, 37, 64)]
    tokens, scores = draft_beams.draft(model, prompts, beams, steps, page)
    assert L.last_device_error() == 0
    tokens, scores = tokens.cpu().numpy(), scores.cpu().numpy()
    assert np.isfinite(scores).all() and np.all(np.diff(scores, axis=1) <= 0)
    for s, prompt in enumerate(prompts):
        assert len({tuple(t) for t in tokens[s]}) == beams  # no beam twice
        for b in range(beams):
            seq, total = list(prompt), 0.0
            for t in tokens[s, b]:
                ids, logits = model.candidates(_state(model, seq))
                where = (ids[0] == int(t)).nonzero()
                if not len(where):  # a candidate at the edge of its tile, the other way round here
                    total = None
                    break
                total += torch.log_softmax(logits[0].double(), 0)[where[0, 0]].item()
                seq.append(int(t))
            if total is not None:
                assert abs(total - scores[s, b]) <= 0.1 * steps, (s, b, total, scores[s, b])
