"""The gradient refuses to write the initial state's gradient over the initial state; over the upstream one it may.

Every call here is refused or has nothing to do: no pointer is read.
"""
import pytest

L = pytest.importorskip("causal_linear_attention_attn_gb300.linattn")

OK, INVALID = 0, 1
STATE = 2 * 64 * 64 * 4  # bytes of one batch row's states


def backward(S0, dS, dS0, N=8, dt=1):
    far = iter(range(1 << 30, 1 << 40, 1 << 24))
    q, k, v, g, dout, dq, dk, dv, dg, ws = (next(far) for _ in range(10))
    return L.lib.la_gated_backward(q, k, v, g, None, dout, S0, dS, dq, dk, dv, dg, dS0, 1, 2, N, 64, 64, dt, ws, 0, None)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("by", [0, 16, -16, STATE - 16, 16 - STATE])
def test_refused(dt, by):
    at = 1 << 20
    assert backward(at, None, at + by, dt=dt) == INVALID
    assert backward(at, at + 4 * STATE, at + by, dt=dt) == INVALID
    if by:  # over the upstream gradient only whole
        assert backward(None, at, at + by, dt=dt) == INVALID
        assert backward(at + 4 * STATE, at, at + by, dt=dt) == INVALID
