"""A kernel launched at a large, a small and again the large shared-memory size."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_large_small_large(cuda_lib):
    gamma = [0.5]
    for d in (128, 32, 128):
        q, k, v = (torch.randn(1, 1, 70, d, device="cuda") for _ in range(3))
        out, S = cuda_lib.la_retention(q, k, v, gamma)
        ref = torch.zeros(d, d, device="cuda", dtype=torch.float64)
        for t in range(70):
            ref = 0.5 * ref + k[0, 0, t].double()[:, None] * v[0, 0, t].double()[None]
        assert (S[0, 0].double() - ref).abs().max() <= 1e-4
