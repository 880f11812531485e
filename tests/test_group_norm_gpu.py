"""The gated group norm and its gradient against 64 bits, and the layer's operators run together."""
import pytest
import torch

from gatedlib import EPS16, forward64, make, norm64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(B, H, N, d, dt, seed, gate=True, weight=True, bias=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return {"x": (r(B, H, N, d) * 3 + r(B, H, N, 1)).to(dt), "gate": (2 * r(B, N, H * d)).to(dt) if gate else None,
            "weight": r(H * d) if weight else None, "bias": r(H * d) if bias else None}, r(B, N, H * d).to(dt)


def close(got, ref, dt, name, rel=2.0**-17):
    """fp32: the statistics add d <= 128 terms in a tree and the rest is a few roundings and __expf (2^-21): 2^-17 of
    the row's largest value; bf16: one rounding more."""
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    tol = rel * ref.abs().amax() + (EPS16 * ref.abs() if got.dtype == BF16 else 0.0)
    off = ((got.double() - ref).abs() - tol).max().item() if ref.numel() else 0.0
    assert off <= 0, f"{name}: {off:.3g} beyond the bound"


SHAPES = [(1, 1, 1, 32), (2, 3, 5, 128), (1, 16, 37, 128), (3, 5, 64, 64), (1, 33, 9, 64), (2, 70, 3, 32), (1, 40, 50, 128),
          (256, 4, 1, 128), (2, 2, 4099, 64)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(cuda_lib, shape, dt):
    d, _ = inputs(*shape, dt, seed=sum(shape))
    close(cuda_lib.la_group_norm(**d), norm64(**d), dt, "y")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("have", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (1, 1, 1)])
def test_optional_arguments_and_gradient(cuda_lib, have, dt):
    d, dy = inputs(2, 6, 61, 64, dt, 9, *map(bool, have))
    close(cuda_lib.la_group_norm(**d), norm64(**d), dt, "y")
    check_grad(cuda_lib, d, dy, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(cuda_lib, shape, dt):
    d, dy = inputs(*shape, dt, seed=sum(shape) + 1)
    check_grad(cuda_lib, d, dy, dt)


def check_grad(L, d, dy, dt):
    leaves = {n: t.double().requires_grad_() for n, t in d.items() if t is not None}
    y = norm64(**leaves)
    grads = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), dy.double())))
    got = dict(zip(("x", "gate", "weight", "bias"), L.la_group_norm_backward(d["x"], dy, d["gate"], d["weight"], d["bias"])))
    for n, x in got.items():
        if d[n] is None:
            assert x is None
        else:
            # columns: sums of B N terms, fp32 chains of up to a few hundred: 2^-15 of their absolute sum's scale
            close(x, grads[n], dt, "d" + n, rel=2.0**-15)


def test_constant_rows_and_large_values(cuda_lib):
    """Rows without variance give the bias (eps alone under the root); large values do not overflow 32 bits."""
    x = torch.full((1, 2, 3, 64), 7.0, device="cuda")
    x[0, 1] = torch.randn(3, 64, device="cuda") * 1e15
    d = {"x": x, "gate": None, "weight": torch.full((128,), 2.0, device="cuda"), "bias": torch.arange(128.0, device="cuda")}
    y = cuda_lib.la_group_norm(**d)
    assert torch.equal(y[0, :, :64], d["bias"][None, :64].expand(3, 64))
    close(y, norm64(**d), F32, "y")


def test_gate_extremes(cuda_lib):
    """silu and its derivative at gates where e^-g overflows or vanishes."""
    d, dy = inputs(1, 1, 4, 128, F32, 3)
    d["gate"] = torch.linspace(-200, 200, 512, device="cuda").reshape(1, 4, 128).contiguous()
    close(cuda_lib.la_group_norm(**d), norm64(**d), F32, "y")
    check_grad(cuda_lib, d, dy, F32)


def test_no_tokens(cuda_lib):
    d, dy = inputs(2, 3, 0, 32, BF16, 1)
    assert cuda_lib.la_group_norm(**d).shape == (2, 0, 96)
    dx, dgate, dw, db = cuda_lib.la_group_norm_backward(d["x"], dy, d["gate"], d["weight"], d["bias"])
    assert dx.shape == d["x"].shape and dw.eq(0).all() and db.eq(0).all()


def test_same_from_run_to_run(cuda_lib):
    d, dy = inputs(2, 8, 3001, 128, BF16, 5)
    first = cuda_lib.la_group_norm_backward(d["x"], dy, d["gate"], d["weight"], d["bias"])
    for _ in range(3):
        again = cuda_lib.la_group_norm_backward(d["x"], dy, d["gate"], d["weight"], d["bias"])
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_layer_end_to_end(cuda_lib, dt):
    """Prefill, norm, gradient of both, then served tokens through the step and the norm, as one layer uses them."""
    L = cuda_lib
    B, H, N, dh = 2, 4, 333, 64
    d = make(B, H, N + 2, dh, dh, dt, seed=77)
    n, dy = inputs(B, H, N, dh, dt, 8)
    pre = {x: d[x][:, :, :N].contiguous() for x in ("q", "k", "v", "g")}
    out, S = L.la_gated(**pre)
    y = L.la_group_norm(out, n["gate"], n["weight"], n["bias"])
    dout, dgate, dw, db = L.la_group_norm_backward(out, dy, n["gate"], n["weight"], n["bias"])
    dq, dk, dv, dg = L.la_gated_backward(**pre, dout=dout)
    # the same in 64 bits, end to end
    leaves = [pre[x].double().requires_grad_() for x in ("q", "k", "v", "g")]
    o64 = quadratic64(*leaves)
    y64 = norm64(o64, n["gate"], n["weight"], n["bias"])
    ref = torch.autograd.grad(y64, leaves, dy.double())
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    bound = 1e-5 if dt == F32 else 2e-2  # bf16: out and dout are rounded to it between the operators
    assert rel(y, y64) <= bound
    for name, a, b in zip(("dq", "dk", "dv", "dg"), (dq, dk, dv, dg), ref):
        assert rel(a, b) <= bound, name
    full, _, _ = forward64(**d)
    for t in range(N, N + 2):
        o = L.la_gated_decode_step(*(d[x][:, :, t].contiguous() for x in ("q", "k", "v", "g")), S)
        yt = L.la_group_norm(o[:, :, None].contiguous(), None, n["weight"], n["bias"])
        assert rel(yt, norm64(full[:, :, t : t + 1], None, n["weight"], n["bias"])) <= bound


def quadratic64(q, k, v, g):
    """The pairwise definition, differentiable: out_i = sum_{j <= i} e^{g_{j+1} + .. + g_i} (q_i . k_j) v_j."""
    c = g.cumsum(-1)
    low = torch.ones(q.shape[2], q.shape[2], dtype=torch.bool, device=q.device).tril()
    w = torch.where(low, c[..., :, None] - c[..., None, :], float("-inf")).exp()
    return (q @ k.transpose(-1, -2) * w) @ v


def test_more_slabs_of_heads_than_blocks_fit(cuda_lib):
    """H = 20000 heads of 32 channels are 313 slabs: the gradient's column sums wait at a grid barrier for resident blocks only."""
    d, dy = inputs(1, 20000, 2, 32, BF16, 6)
    close(cuda_lib.la_group_norm(**d), norm64(**d), BF16, "y")
    check_grad(cuda_lib, d, dy, BF16)
