"""States that grow (negative steps, A > 0) in sequences of several segments, whose decays are joined as one factor each.

Inputs are powers of two wherever a growth of many orders is concerned, so that the results are known without the bounds of
the token-by-token forms (which such a growth takes beyond any use)."""
import pytest
import torch

from selectivelib import make, scan64, scan_grad64, within
from test_selective_gpu import grads, run

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def still(N, D, ds, dt, step, A):
    """x = 0, no gate, no skip; one step everywhere."""
    d = make(1, N, D, ds, F32, seed=1, gate=False, skip=False, bias=False)
    d["softplus"], d["x"] = False, torch.zeros_like(d["x"])
    d["dt"] = torch.full_like(d["dt"], step)
    d["A"] = torch.full_like(d["A"], A)
    d["Bm"], d["Cm"], d["dout"] = torch.ones_like(d["Bm"]), torch.ones_like(d["Cm"]), torch.zeros_like(d["dout"])
    return {k: v.to(dt) if k in ("x", "dt", "Bm", "Cm", "dout") else v for k, v in d.items()}


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("step,A", [(-0.125, -8.0), (0.125, 8.0)])
@pytest.mark.parametrize("N", [600, 2100])
def test_nothing_grows_to_nothing(cuda_lib, dt, ds, step, A, N):
    """A state of zero stays zero whatever it is multiplied with; what comes in late grows from there.  e^{delta A} = e a
    token: a segment's decay is far beyond 2^128."""
    D, late = 24, N - 10
    d = still(N, D, ds, dt, step, A)
    d["x"][0, late] = 1.0
    out, S = run(cuda_lib, d)
    assert out[0, :late].eq(0).all()
    cut = {k: v[:, late:].contiguous() if k in ("x", "dt", "Bm", "Cm", "dout") else v for k, v in d.items()}
    ref, bound, refS, boundS, _ = scan64(cut)
    within(out[:, late:], ref, bound, "out")
    within(S, refS, boundS, "S")
    # the state's gradient, from the other end: the only gradient comes in at token 9
    d["x"].zero_()
    d["dout"][0, 9] = 1.0
    cut = {k: v[:, :10].contiguous() if k in ("x", "dt", "Bm", "Cm", "dout") else v for k, v in d.items()}
    got, ref = grads(cuda_lib, d), scan_grad64(cut)
    for n in ("dx", "ddt", "dB", "dC"):
        assert got[n][:, 10:].eq(0).all(), n
        within(got[n][:, :10].contiguous(), *ref[n], n)
    for n in ("dA", "dS0"):
        within(got[n], *ref[n], n)


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("ds", [8, 64])
@pytest.mark.parametrize("A", [100.0, 160.0, 230.0])
def test_a_small_state_grows_far(cuda_lib, ds, A, late):
    """A state of 2^-116 doubles A times over one half of 512 tokens, beyond what one fp32 factor holds, and is still a
    number; the state's gradient the same way back."""
    N, D, first = 512, 8, 2.0**-116
    d = still(N, D, ds, F32, 1 / 256, A * 0.6931471805599453)
    d["dt"][0, slice(256) if late else slice(256, None)] = 0.0
    # the exponent A log2 e: three roundings of A doublings; each of 256 tokens 2^-22 for its exponential, and 2^-22 for
    # the roundings of its exponent and product
    tol = 256 * 2.0**-21 + 4 * A * 2.0**-24
    _, S = run(cuda_lib, d | {"S0": torch.full((1, D, ds), first, device="cuda")})
    assert S.isfinite().all() and (S.double() / (first * 2.0**A) - 1).abs().max() < tol
    g = grads(cuda_lib, d | {"dS": torch.full((1, D, ds), first, device="cuda")})
    assert (g["dS0"].double() / (first * 2.0**A) - 1).abs().max() < tol


@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("gate,skip,bias", [(True, True, True), (False, False, False)])
def test_steps_of_either_sign_over_segments(cuda_lib, ds, gate, skip, bias):
    """Steps of either sign whose sum stays small: states within 2^50 throughout are compared token by token."""
    d = make(2, 700, 32, ds, F32, seed=ds, gate=gate, skip=skip, bias=bias, state=True)
    d["softplus"], d["dt"] = False, d["dt"] * 0.03
    d["dt_bias"] = None if d["dt_bias"] is None else torch.full_like(d["dt_bias"], 0.004)
    out, S = run(cuda_lib, d)
    ref, bound, refS, boundS, (*_, kept) = scan64(d)
    grad, got = scan_grad64(d), grads(cuda_lib, d)
    ok = torch.stack([hb for _, hb, _ in kept]).amax((0, 1, 3)) < 2.0**50
    assert ok.any()
    within(out[..., ok], ref[..., ok], bound[..., ok], "out")
    within(S[:, ok], refS[:, ok], boundS[:, ok], "S")
    for n, x in got.items():
        if x is None or n in ("dB", "dC"):
            continue
        cut = (lambda t: t[ok]) if x.shape[0] == 32 else (lambda t: t[:, ok]) if n == "dS0" else (lambda t: t[..., ok])
        within(cut(x), *map(cut, grad[n]), n)
