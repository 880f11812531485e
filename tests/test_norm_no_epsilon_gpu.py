"""Gradient of the group norm without an epsilon, at token counts that leave rows of a block's last turn unused."""
import pytest
import torch

from gatedlib import norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("B,H,N,d", [(1, 3, 5, 64), (3, 3, 7, 32), (1, 16, 37, 128), (1, 1, 1, 128), (7, 5, 13, 32)])
def test_sums_without_epsilon(cuda_lib, B, H, N, d, gate, dt):
    gen = torch.Generator(device="cuda").manual_seed(B + H + N + d)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy = r(B, H, N, d).to(dt), r(B, N, H * d).to(dt)
    g, w, b = (r(B, N, H * d).to(dt) if gate else None), r(H * d), r(H * d)
    got = [t for t in cuda_lib.la_group_norm_backward(x, dy, g, w, b, eps=0.0) if t is not None]
    leaves = [t.double().requires_grad_() for t in (x, g, w, b) if t is not None]
    args = iter(leaves)
    y = norm64(next(args), next(args) if gate else None, next(args), next(args), eps=0.0)
    for t, ref in zip(got, torch.autograd.grad(y, leaves, dy.double())):
        assert torch.isfinite(t).all()
        # as for the other gradients: 2^-15 of the largest value, one rounding more in bf16
        tol = 2.0**-15 * ref.abs().amax() + (2.0**-8 * ref.abs() if t.dtype == torch.bfloat16 else 0.0)
        assert ((t.double() - ref).abs() - tol).max().item() <= 0
