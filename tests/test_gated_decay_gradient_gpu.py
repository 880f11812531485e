"""The decays' gradient held to its own terms: dg_t = e^{g_t} <S_{t-1}, R_t>, no allowance for its neighbours' size."""
import pytest
import torch

from gatedlib import absolute, backward64, make, within
from test_gated_gpu import BF16, CASES, F32, tensor_core

pytestmark = pytest.mark.gpu


def check(L, d, lengths=None):
    q, v = d["q"], d["v"]
    dg = L.la_gated_backward(q, d["k"], v, d["g"], d["dout"], S0=d["S0"], dS=d["dS"], lengths=lengths)[3]
    ref = backward64(**d, lengths=lengths)[3]
    own = backward64(**absolute(d), lengths=lengths)[3]
    within(dg, ref, own, F32, "dg", pair=tensor_core(q.dtype, q.shape[-1], v.shape[-1]))
    assert dg[torch.isneginf(d["g"])].eq(0).all(), "a reset token has a gradient"


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("state", [False, True])
def test_resets(cuda_lib, dt, dk, dv, state):
    d = make(2, 3, 300, dk, dv, dt, seed=5, state=state, resets=0.05)
    d["g"][0, 0, 126:131] = float("-inf")
    check(cuda_lib, d)


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("scale", [0.0, 0.3, 8.0, 40.0])
def test_from_weak_to_strong_decays(cuda_lib, dt, dk, dv, scale):
    check(cuda_lib, make(1, 4, 270, dk, dv, dt, seed=6, state=True, scale=scale))


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_one_strong_decay_among_weak_ones(cuda_lib, dt, dk, dv):
    """e^-25: the token's own pairs are 1e-11 of those on either side of it."""
    d = make(1, 2, 260, dk, dv, dt, seed=7, scale=0.02)
    for t in (1, 31, 32, 33, 40, 63, 64, 100, 127, 128, 140, 200, 259):
        d["g"][0, :, t] = -25.0
    check(cuda_lib, d)


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_padded(cuda_lib, dt, dk, dv):
    d = make(5, 2, 260, dk, dv, dt, seed=8, state=True, resets=0.03)
    check(cuda_lib, d, torch.tensor([260, 0, 1, 128, 77], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("N", [1, 2, 16, 17, 32, 33, 64, 96, 127])
def test_every_part_of_a_chunk(cuda_lib, N):
    for d in (64, 128):
        check(cuda_lib, make(1, 2, N, d, d, BF16, seed=N, resets=0.05))
