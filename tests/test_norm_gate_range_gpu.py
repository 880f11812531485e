"""silu of the gate and its derivative, value by value, from the most negative gates to the largest.

weight = 0 and bias = dy = 1 leave y = g s and dgate = s + g s (1 - s), s = 1 / (1 + e^-g), alone.  e^-g comes
from 2^x of a product with log2 e: the product is off by 2^-24 and its constant by 2^-26 relative, so e^-g by
1.25 |g| 2^-24 < |g| 2^-23, and by 2^-22 of the instruction.  That reaches s with the factor 1 - s; the addition
(2^-24), the reciprocal (2^-23) and up to three roundings of products (2^-24 each) come on top: s and g s are good to
2^-21 + |g| 2^-23 (1 - s), and s (1 - s), which has e^-g once more, to 2^-21 + |g| 2^-22 + 2^-22 of itself, where it
still counts.  An s below 2^-126 becomes zero.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def gates(dt):
    small = torch.linspace(-120, 120, 4801, dtype=torch.float64)
    far = torch.tensor([1e3 + 0.3, 1e4 + 0.6, 12345.678, 1e5 + 0.4, 2.0**24, 2.0**24 + 6, 1e9, 1e20, 1e30, 3e38], dtype=torch.float64)
    g = torch.cat([small, far, -far, torch.tensor([0.0, -0.0, 1e-30, -1e-30], dtype=torch.float64)]).to(dt)
    n = -(-g.numel() // 128) * 128
    return torch.cat([g, g.new_zeros(n - g.numel())]).cuda().reshape(1, -1, 128)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_every_gate(cuda_lib, dt):
    gate = gates(dt)
    N = gate.shape[1]
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 1, N, 128, generator=gen, device="cuda").to(dt)
    w, b = torch.zeros(128, device="cuda"), torch.ones(128, device="cuda")
    y = cuda_lib.la_group_norm(x, gate, w, b)
    dgate = cuda_lib.la_group_norm_backward(x, torch.ones_like(gate), gate, w, b)[1]
    g = gate.double()
    s, one_less = torch.sigmoid(g), torch.sigmoid(-g)
    rel = 2.0**-21 + g.abs() * one_less * 2.0**-23
    flush = (1 + g.abs()) * 2.0**-126
    rounding = 2.0**-8 if dt == torch.bfloat16 else 0.0
    ref = g * s
    assert ((y.double() - ref).abs() <= (rel + rounding) * ref.abs() + flush * (g < -80)).all()
    ref = s + g * s * one_less
    tol = rel * s + (2 * rel + 2.0**-22 + g.abs().clamp(max=200) * 2.0**-22) * (g * s * one_less).abs()
    bad = (dgate.double() - ref).abs() > tol + rounding * ref.abs() + flush * (g < -80)
    assert not bad.any(), (gate[bad][:8].tolist(), dgate[bad][:8].tolist(), ref[bad][:8].tolist())
