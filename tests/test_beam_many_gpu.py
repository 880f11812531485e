"""Reordering of many beams at once."""
import pytest
import torch

from test_beam_gpu import reorder

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("G,W", [(160, 8), (40, 33), (25, 64), (700, 2)])
def test_reorder_of_many_beams(cuda_lib, G, W):
    """More pieces of rows than 8 an SM, so that a block takes its piece in every pool: pools of several row sizes, some with
    nothing in a piece, one of several pieces and a part."""
    g = torch.Generator(device="cuda").manual_seed(G)
    n = G * W + 5
    pools = [torch.randn(n, 24, generator=g, device="cuda").to(BF16), torch.randn(n, 20004, generator=g, device="cuda"),
             torch.randint(0, 255, (n, 16), generator=g, device="cuda", dtype=torch.uint8),
             torch.randn(n, 8196, generator=g, device="cuda")]
    for i in range(3):
        slots = torch.randperm(n, generator=g, device="cuda")[: G * W].reshape(G, W).int()
        parents = torch.randint(W, (G, W), generator=g, device="cuda").int()
        if i == 1:
            parents.fill_(W - 1)
        if i == 2:
            parents[:, ::3] = -1
            slots[::2, 0] = -1
        reorder(cuda_lib, pools, slots, parents)
