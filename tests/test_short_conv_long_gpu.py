"""Sums over tokens of the convolution's gradient at sizes whose runs of tokens are long, and many columns and rows."""
import pytest
import torch

from selectivelib import slope

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_long_sums(cuda_lib):
    """Every token adds (1 + 2^-7)^2, a multiple of 2^-14, so sums below 2^10 are exact and every addition to one beyond 2^11
    loses it.  In runs of 512 tokens only the sums over runs are rounded, 2^-24 at each addition: 1024 runs in chains of 32, and 10
    to join the chains."""
    B, N, D, K, one = 64, 8192, 2048, 4, 1 + 2.0**-7
    x = torch.full((B, N, D), one, dtype=BF16, device="cuda")
    w = torch.ones(D, K, device="cuda")
    _, dw, db = cuda_lib.la_short_conv_backward(x, w, x, bias=torch.zeros(D, device="cuda"), silu=False)
    for j in range(K):
        want = B * (N - (K - 1 - j)) * one * one
        off = (dw[:, j].double() / want - 1).abs().max().item()
        assert off <= 42 * 2.0**-24, f"dw[{j}]: {off:.3g}"
    off = (db.double() / (B * N * one) - 1).abs().max().item()
    assert off <= 42 * 2.0**-24, f"db: {off:.3g}"


@pytest.mark.parametrize("dt", [F32, BF16])
def test_weights_of_a_long_sequence(cuda_lib, dt):
    """dweight and dbias of a million tokens against sums in 64 bits, taken in parts."""
    N, D, K = 2**20 + 77, 1032, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, N, D, generator=g, device="cuda").to(dt)
    dout = torch.randn(1, N, D, generator=g, device="cuda").to(dt)
    w, b = torch.randn(D, K, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    _, dw, db = cuda_lib.la_short_conv_backward(x, w, dout, bias=b)
    ref, size = torch.zeros(D, K + 1, dtype=torch.float64, device="cuda"), torch.zeros(D, K + 1, dtype=torch.float64, device="cuda")
    part = 1 << 14
    for t in range(0, N, part):
        m = min(part, N - t)
        xp = x[0, max(0, t - (K - 1)) : t + m].double()
        xp = torch.nn.functional.pad(xp, (0, 0, m + K - 1 - xp.shape[0], 0))
        u = sum(xp[j : j + m] * w[:, j].double() for j in range(K)) + b.double()
        gg = dout[0, t : t + m].double() * slope(u)
        for j in range(K + 1):
            v = gg * xp[j : j + m] if j < K else gg
            ref[:, j] += v.sum(0)
            size[:, j] += v.abs().sum(0)
    # a term: its slope, from u with K + 1 roundings of values up to 40 (2^-24 each), 2^-17; a sum: chains of at most 2^10
    # additions in a run and 2^10 over the runs, 2^-13
    tol = size * (2.0**-17 + 2.0**-13)
    assert ((dw.double() - ref[:, :K]).abs() <= tol[:, :K]).all()
    assert ((db.double() - ref[:, K]).abs() <= tol[:, K]).all()
