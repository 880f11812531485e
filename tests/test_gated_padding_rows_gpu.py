"""Padded batches through the layer: the rows behind a sequence's end that the binding allocates hold zeros."""
import pytest
import torch

from gatedlib import make

pytestmark = pytest.mark.gpu


def poison(numel, dtype):
    """Freed memory of that size, full of NaN, which the next allocation of the size takes."""
    t = torch.full((numel,), float("nan"), dtype=dtype, device="cuda")
    del t


@pytest.mark.parametrize("dt,D", [(torch.float32, 64), (torch.bfloat16, 128), (torch.bfloat16, 32)])
@pytest.mark.parametrize("state", [False, True])
def test_allocated_rows_and_the_norm_behind(cuda_lib, dt, D, state):
    L = cuda_lib
    B, H, N = 4, 2, 300
    d = make(B, H, N, D, D, dt, seed=17, state=state)
    lengths = torch.tensor([N, 0, 131, 1], dtype=torch.int32, device="cuda")
    dead = torch.arange(N, device="cuda") >= lengths[:, None]
    torch.cuda.empty_cache()
    poison(d["v"].numel(), dt)
    args = (d["q"], d["k"], d["v"], d["g"])
    out, S = L.la_gated_with_state(*args, d["S0"].clone(), lengths=lengths) if state else L.la_gated(*args, lengths=lengths)
    assert out[dead[:, None].expand(B, H, N)].eq(0).all()
    live = torch.full_like(out, float("nan"))
    if state:
        L.la_gated_with_state(*args, d["S0"].clone(), lengths=lengths, out=live)
    else:
        L.la_gated(*args, lengths=lengths, out=live)
    assert torch.equal(out, live.masked_fill(dead[:, None, :, None], 0))
    # the norm's gradient of a loss over the tokens that take part: padding rows add nothing
    gen = torch.Generator(device="cuda").manual_seed(3)
    gate, dy = (torch.randn(B, N, H * D, generator=gen, device="cuda").to(dt) for _ in range(2))
    dy.masked_fill_(dead[..., None], 0)
    w, b = torch.randn(H * D, generator=gen, device="cuda"), torch.randn(H * D, generator=gen, device="cuda")
    dx, dgate, dw, db = L.la_group_norm_backward(out, dy, gate, w, b)
    assert all(torch.isfinite(t).all() for t in (dx, dgate, dw, db))
    x = out.double().transpose(1, 2)
    h = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    u = dy.double() * gate.double() * torch.sigmoid(gate.double())
    for got, ref in ((dw, (u * h.reshape(B, N, H * D))[~dead].sum(0)), (db, u[~dead].sum(0))):
        assert (got.double() - ref).abs().max() <= 2.0**-15 * ref.abs().max()
    grads = L.la_gated_backward(*args, dx, S0=d["S0"], lengths=lengths)
    assert all(torch.isfinite(t).all() for t in grads)
