"""Refusals of the gated operators that need no GPU: every one returns before any CUDA call."""
import pytest
import torch

L = pytest.importorskip("causal_linear_attention_attn_gb300.linattn")

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 1 << 20  # aligned, never dereferenced


def gated(fn="la_gated", **kw):
    a = dict(q=P, k=P, v=P, g=P, lengths=None, out=P, S=P, B=1, H=2, N=8, dk=64, dv=64, dt=1, ws=P, bytes=1 << 40, stream=None)
    a.update(kw)
    return getattr(L.lib, fn)(*a.values())


@pytest.mark.parametrize("fn", ["la_gated", "la_gated_with_state"])
def test_prefill(fn):
    for name in ("q", "k", "v", "g", "out", "S"):
        assert gated(fn, **{name: None}) == INVALID
        assert gated(fn, **{name: P + (2 if name == "g" else 8)}) == MISALIGNED
    assert gated(fn, lengths=P + 2) == MISALIGNED
    assert gated(fn, ws=P + 4) == MISALIGNED
    for name in ("B", "H", "N", "dk"):
        assert gated(fn, **{name: -1}) == INVALID
    assert gated(fn, dk=48) == UNSUPPORTED and gated(fn, dv=256) == UNSUPPORTED and gated(fn, dt=2) == UNSUPPORTED
    assert gated(fn, B=1 << 20, H=1 << 20) == INVALID
    assert gated(fn, B=1 << 10, H=1 << 10, N=1 << 30) == INVALID
    assert gated(fn, B=0, q=None, S=None) == OK


def test_backward():
    names = ("q", "k", "v", "g", "lengths", "dout", "S0", "dS", "dq", "dk", "dv", "dg", "dS0")

    def call(**kw):
        a = dict.fromkeys(names, P) | dict(B=1, H=2, N=8, d_k=64, d_v=64, dt=1, ws=P, bytes=1 << 40, stream=None)
        a.update(kw)
        return L.lib.la_gated_backward(*a.values())

    for n in ("q", "k", "v", "g", "dout", "dq", "dk", "dv", "dg"):
        assert call(**{n: None}) == INVALID
    for n in names:
        assert call(**{n: P + 2}) == MISALIGNED
    assert call(d_k=16) == UNSUPPORTED and call(B=-1) == INVALID and call(H=0) == OK


def test_step():
    def call(**kw):
        a = dict(q=P, k=P, v=P, g=P, S=P, slots=P, out=P, B=2, H=2, n=4, dk=64, dv=64, dt=1, stream=None)
        a.update(kw)
        return L.lib.la_gated_decode_step(*a.values())

    for n in ("q", "k", "v", "g", "S", "out"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 2}) == MISALIGNED
    assert call(slots=None, n=1) == INVALID and call(n=-1) == INVALID
    assert call(dv=96) == UNSUPPORTED and call(B=0) == OK


def test_norm():
    def fwd(**kw):
        a = dict(x=P, gate=P, w=P, b=P, y=P, B=1, H=2, N=3, d=64, eps=1e-5, dt=1, stream=None)
        a.update(kw)
        return L.lib.la_group_norm(*a.values())

    def bwd(**kw):
        a = dict(x=P, dy=P, gate=P, w=P, b=P, dx=P, dgate=P, dw=P, db=P, B=1, H=2, N=3, d=64, eps=1e-5, dt=1, ws=P,
                 bytes=1 << 40, stream=None)
        a.update(kw)
        return L.lib.la_group_norm_backward(*a.values())

    for f in (fwd, bwd):
        assert f(x=None) == INVALID and f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(B=-1) == INVALID
        assert f(d=80) == UNSUPPORTED and f(dt=3) == UNSUPPORTED
        assert f(x=P + 8) == MISALIGNED and f(w=P + 4) == MISALIGNED
    assert fwd(y=None) == INVALID and fwd(N=0) == OK
    assert bwd(dgate=None) == INVALID and bwd(gate=None) == INVALID and bwd(dx=None) == INVALID and bwd(H=0) == OK


def test_workspace_of_nothing():
    assert L.lib.la_gated_workspace(0, 4, 128, 64, 64, 1, 0) == 0
    assert L.lib.la_gated_workspace(1, 4, 128, 60, 64, 1, 0) == 0
    assert L.lib.la_gated_workspace(1, 4, 128, 64, 64, 0, 1) > L.lib.la_gated_workspace(1, 4, 128, 64, 64, 0, 0) > 0
    assert L.lib.la_group_norm_workspace(1, 2, 0, 64) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        L.la_gated(q, q, q, torch.zeros(1, 2, 8))
    with pytest.raises(ValueError):
        L.la_gated(q[0], q, q, torch.zeros(1, 2, 8))
    with pytest.raises(TypeError):
        L.la_gated(q.double(), q, q, torch.zeros(1, 2, 8))
    with pytest.raises(ValueError):
        L.la_gated_with_state(q, q, q, torch.zeros(1, 2, 8), None)
    with pytest.raises(ValueError):
        L.la_group_norm(q)
    with pytest.raises(ValueError):
        L.la_gated_decode_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], torch.zeros(1, 2), q)
