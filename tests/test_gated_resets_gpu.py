"""A decay of -inf is a cut: nothing before it is read behind it, whatever the decays behind it and the states hold."""
import pytest
import torch

from gatedlib import absolute, backward64, forward64, make, within
from test_gated_gpu import BF16, CASES, F32, NAN, tensor_core

pytestmark = pytest.mark.gpu
INF = float("inf")


def same(a, b, name):
    assert torch.equal(a, b), name


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("N,at,grow", [(300, 140, 141), (300, 30, 31), (20, 5, 6), (2600, 140, 300), (2600, 1290, 1300)])
def test_growth_behind_a_reset(cuda_lib, dt, dk, dv, N, at, grow):
    """Two decays of +40 behind a reset, a large state before it; keys of zero in between keep the results in range."""
    if N > 300 and dt == F32:
        N, at, grow = 700, 140, 300
    d = make(1, 2, N, dk, dv, dt, seed=at, state=True, scale=0.0)
    d["S0"] *= 1e25
    d["g"][:, :, at] = -INF
    d["k"][:, :, at:grow + 1] = 0
    d["g"][:, :, grow:grow + 2] = 40.0
    tc = tensor_core(dt, dk, dv)
    S = d["S0"].clone()
    out, _ = cuda_lib.la_gated_with_state(d["q"], d["k"], d["v"], d["g"], S)
    ref, refS, _ = forward64(**d)
    abso, absS, _ = forward64(**absolute(d))
    within(out, ref, abso, dt, "out", pair=tc, steps=2)
    within(S, refS, absS, F32, "S", pair=tc)
    got = cuda_lib.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"], S0=d["S0"], dS=d["dS"], need_state_grad=True)
    for name, x, r, a in zip(("dq", "dk", "dv", "dg", "dS0"), got, backward64(**d), backward64(**absolute(d))):
        within(x, r, a, dt, name, pair=tc, steps=2)


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("N,at", [(20, 0), (20, 7), (300, 0), (300, 31), (300, 150), (1500, 0), (1500, 200)])
def test_state_that_is_not_finite(cuda_lib, dt, dk, dv, bad, N, at):
    """From a reset on, results are those of a start from zeros, bit for bit; so are gradients up to one."""
    L = cuda_lib
    d = make(2, 2, N, dk, dv, dt, seed=N + at, state=True)
    d["g"][:, :, at] = -INF
    d["S0"].zero_()
    args = [d[n] for n in ("q", "k", "v", "g")]
    S, T = d["S0"].clone(), torch.full_like(d["S0"], bad)
    NaN = T.clone()
    want, _ = L.la_gated_with_state(*args, S)
    got, _ = L.la_gated_with_state(*args, T)
    same(got[:, :, at:], want[:, :, at:], "out")
    same(T, S, "S")
    grads = lambda S0, dS: L.la_gated_backward(*args, d["dout"], S0=S0, dS=dS, need_state_grad=True)  # noqa: E731
    ref, x = grads(d["S0"], d["dS"]), grads(NaN, d["dS"])
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), x, ref):
        cut = at if n in ("dq", "dg") else 0
        same(a[:, :, cut:], b[:, :, cut:], n)
    x = grads(d["S0"], NaN)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), x, ref):
        end = {"dk": at, "dv": at, "dg": at + 1}.get(n, b.shape[2])
        same(a[:, :, :end], b[:, :, :end], n)
    assert L.device_status() == 0


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("bad", [NAN, INF])
def test_step_on_a_slot_that_was_never_written(cuda_lib, dt, dk, dv, bad):
    d = make(3, 2, 1, dk, dv, dt, seed=2)
    d["g"][:2] = -INF
    pool = torch.full((4, 2, dk, dv), bad, device="cuda")
    pool[1] = 0
    one = [d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    slots = torch.tensor([3, 0, 1], dtype=torch.int32, device="cuda")
    out = cuda_lib.la_gated_decode_step(*one, pool, slots=slots)
    ref, refS, _ = forward64(**d)
    abso, absS, _ = forward64(**absolute(d))
    within(out, ref[:, :, 0], abso[:, :, 0], dt, "out")
    within(pool[slots.long()], refS, absS, F32, "S")
    assert not torch.isfinite(pool[2]).any()


def test_resets_of_every_kind_in_one_long_head(cuda_lib):
    """Many resets, some in a row, over several segments of a head; the sums of decays stay exact between them."""
    for D in (64, 128):
        d = make(1, 1, 2700, D, D, BF16, seed=3, state=True, scale=2.0**-9, resets=0.01)
        d["g"][0, 0, 700:1000] = -INF
        out, S = cuda_lib.la_gated_with_state(d["q"], d["k"], d["v"], d["g"], d["S0"].clone())
        ref, refS, _ = forward64(**d)
        abso, absS, _ = forward64(**absolute(d))
        within(out, ref, abso, BF16, "out", pair=True, steps=2)
        within(S, refS, absS, F32, "S", pair=True)
