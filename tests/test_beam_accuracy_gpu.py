"""How near two beams' continuations may be for selection to order them: a row's sum of exponentials is formed in 32 bits."""
import math

import pytest
import torch

from selectivelib import select64
from test_beam_gpu import logits_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def accuracy(V):
    """How far a row's log sum may be off.  A term e^d, d = l - top: d is rounded, multiplied with a rounded constant and
    rounded, 3 |d| 2^-24, and its exponential off by 2^-22.  With the terms' shares p of the sum that makes 2^-22 + 3 H 2^-24,
    H = sum p |d| <= 1 + log V.  Additions: 16 values a lane and chunk (9), the lanes, warps and runs (5 + 4 + 7), and at every
    chunk of 4096 values the sum so far times an exponential where the maximum rises (8 with its addition)."""
    return 2.0**-22 + (3 * (1 + math.log(V)) + 25 + 8 * (-(-V // 4096))) * 2.0**-24


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [61, 5003, 131072])
@pytest.mark.parametrize("scale", [0.1, 1.0, 4.0])
def test_accuracy_of_scores(cuda_lib, dt, V, scale):
    """Scores that cancel their beam's best logarithm: what is left shows the log sum's error at its own size."""
    G, W = 24, 4
    logits, _ = logits_of(G, W, V, dt, seed=V, scale=scale)
    x = logits.double()
    first = torch.log_softmax(x, -1).amax(-1)
    scores = (-first).float()
    best, parents, tokens = cuda_lib.la_beam_select(logits, scores, k=1)
    # the chosen one, in 64 bits, is within twice the accuracy of the best, and its score within the accuracy
    total = scores.double() + first
    chosen = total.gather(1, parents.long())
    assert (total.amax(1) - chosen[:, 0]).max() <= 2 * accuracy(V)
    at = x.gather(1, parents.long()[..., None].expand(-1, -1, V)).log_softmax(-1).gather(2, tokens.long()[..., None])[:, 0, 0]
    exact = scores.double().gather(1, parents.long())[:, 0] + at
    assert (best[:, 0].double() - exact).abs().max() <= accuracy(V) + 2.0**-24 * exact.abs().max()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [61, 5003, 131072])
def test_near_scores_of_different_beams(cuda_lib, dt, V):
    """Beams whose best continuations are apart by a little more than twice the accuracy come out in their order."""
    G, W = 32, 8
    logits, _ = logits_of(G, W, V, dt, seed=V + 1, scale=1.0)
    logits[..., 7] = 12.0  # the best, by far: the k best are one of each beam
    first = torch.log_softmax(logits.double(), -1)[..., 7]
    g = torch.Generator(device="cuda").manual_seed(V)
    order = torch.rand(G, W, generator=g, device="cuda").argsort(-1)
    # scores around 0.5: a step of fp32 there is 2^-24
    gap = 2 * accuracy(V) + 2.0**-23
    scores = (order * gap - 0.5 - first).float()
    best, parents, tokens = cuda_lib.la_beam_select(logits, scores)
    _, p, t = select64(logits, scores, W)
    assert torch.equal(parents, p) and torch.equal(tokens, t)
    assert torch.equal(parents.long(), order.argsort(-1, descending=True))
