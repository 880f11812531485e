"""Sums over long sequences in the gradient of the selective scan."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_long_sums_of_the_scan(cuda_lib):
    """dD and ddt_bias over rows of 65536 tokens, one segment each.

    Every token adds (1 + 2^-7)^2, a multiple of 2^-14: a sum below 2^10 is exact, one beyond 2^11 loses it at every addition.
    What is exact in chains of 32 additions, and in sums of 2^11 of those (multiples of 2^-9 below 2^13), is rounded only where
    the sixteen rows of a chunk (15), and the table's rows (8 + 3 + 7), are added: 2^-24 each."""
    B = torch.cuda.get_device_properties(0).multi_processor_count
    N, D, ds, one = 65536, 64, 8, 1 + 2.0**-7
    x = torch.full((B, N, D), one, dtype=BF16, device="cuda")
    dt = torch.ones_like(x)
    A = torch.full((D, ds), -1e30, device="cuda")  # forgets at once: ddt = x (dout C . B)
    Bm = torch.zeros(B, N, ds, dtype=BF16, device="cuda")
    Bm[..., 3] = 1
    _, _, _, _, _, dD, _, dbias = cuda_lib.la_selective_scan_backward(
        x, dt, A, Bm, Bm, x, D=torch.zeros(D, device="cuda"), dt_bias=torch.zeros(D, device="cuda"), softplus=False)
    want = B * N * one * one
    for got, name in ((dD, "dD"), (dbias, "ddt_bias")):
        off = (got.double() / want - 1).abs().max().item()
        assert off <= 33 * 2.0**-24, f"{name}: {off:.3g}"
