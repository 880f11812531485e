"""Selection where some lanes of every warp take the path for infinities and NaN while other warps raise the bound."""
import pytest
import torch

from selectivelib import select64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [4, 33, 64])
@pytest.mark.parametrize("odd", [NAN, INF])
def test_lanes_that_go_apart(cuda_lib, dt, k, odd):
    """Odd values in some lanes' places of every chunk, logits that rise along the row (every chunk has new
    candidates and a new bound), several runs' worth of chunks."""
    G, W, V = 2, 3, 70001
    g = torch.Generator(device="cuda").manual_seed(k)
    logits = torch.randn(G, W, V, generator=g, device="cuda") + torch.linspace(0, 8, V, device="cuda")
    # (infinities share the probability, and all others are as far below as 64 bits tell: enough of them for every k)
    logits[:, :, 3 :: 601 if odd == odd else 56] = odd
    logits, scores = logits.to(dt), -torch.rand(G, W, generator=g, device="cuda")
    for _ in range(3):
        best, parents, tokens = cuda_lib.la_beam_select(logits, scores, k=k)
        ref, p, t = select64(logits, scores, k)
        assert torch.equal(parents, p) and torch.equal(tokens, t)
        assert torch.equal(best.isneginf(), ref.isneginf())
