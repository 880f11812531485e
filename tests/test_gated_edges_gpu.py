"""Gated linear attention and the group norm at the ends of their ranges: rows of one chunk, and more than 2^31 elements."""
import pytest
import torch

from gatedlib import EPS16, absolute, backward64, forward64, make, norm64, within
from test_gated_gpu import BF16, CASES, F32, NAN, check_backward, check_forward, tensor_core

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("N", [1, 20, 32])
def test_padded_batch_of_one_chunk(cuda_lib, dt, dk, dv, state, N):
    lengths = torch.tensor([N, 0, N // 2, 1, -3, N + 5], dtype=torch.int32, device="cuda")
    d = make(6, 3, N, dk, dv, dt, seed=41 + N, state=state, resets=0.1)
    eff = lengths.clamp(0, N)
    dead = torch.arange(N, device="cuda") >= eff[:, None]
    clean = {n: None if t is None else t.clone() for n, t in d.items()}
    for n in ("q", "k", "v", "dout", "g"):
        d[n].masked_fill_(dead[:, None, :] if n == "g" else dead[:, None, :, None], NAN)
    check_forward(cuda_lib, clean, lengths)
    check_backward(cuda_lib, clean, lengths)
    grads = lambda x: cuda_lib.la_gated_backward(  # noqa: E731
        x["q"], x["k"], x["v"], x["g"], x["dout"], S0=x["S0"], dS=x["dS"], lengths=lengths, need_state_grad=True)
    for x, y in zip(grads(d), grads(clean)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("N", [20, 100])
def test_state_gradient_over_the_upstream_one(cuda_lib, N):
    """Through the C ABI: dS0 written over dS, on the path of one chunk a head and the one with a scan."""
    L = cuda_lib
    d = make(2, 3, N, 64, 32, F32, seed=95, state=True)
    want = L.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"], S0=d["S0"], dS=d["dS"], need_state_grad=True)
    got = [torch.empty_like(x) for x in want[:4]]
    dS = d["dS"].clone()
    need = L.lib.la_gated_workspace(2, 3, N, 64, 32, 0, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    p = L._ptr
    assert L.lib.la_gated_backward(p(d["q"]), p(d["k"]), p(d["v"]), p(d["g"]), None, p(d["dout"]), p(d["S0"]), p(dS),
                                   *map(p, got), p(dS), 2, 3, N, 64, 32, 0, p(ws), need,
                                   torch.cuda.current_stream().cuda_stream) == 0
    for x, y in zip((*got, dS), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dt,D,N", [(BF16, 128, 2**23 + 77), (F32, 32, 2**25 + 77)])
def test_more_elements_than_31_bits_count(cuda_lib, dt, D, N):
    """Resets near both ends make the first and last tokens' results independent of the millions between."""
    H, head, tail = 2, 200, 300
    new = lambda s: torch.empty(1, H, N, D, dtype=dt, device="cuda").normal_().mul_(s)  # noqa: E731
    q, k, v, dout = new(D**-0.25), new(D**-0.25), new(1.0), new(1.0)
    assert q.numel() > 2**31
    g = torch.full((1, H, N), -0.05, device="cuda")
    g[:, :, head] = g[:, :, N - tail] = float("-inf")
    tc = tensor_core(dt, D, D)
    out, S = cuda_lib.la_gated(q, k, v, g)
    parts = [{"S0": None, "dS": None} | {n: t[:, :, s].clone() for n, t in
             (("q", q), ("k", k), ("v", v), ("g", g), ("dout", dout))} for s in (slice(0, head), slice(N - tail, N))]
    for p, o in zip(parts, (out[:, :, :head], out[:, :, N - tail:])):
        within(o, forward64(**p)[0], forward64(**absolute(p))[0], dt, "out", pair=tc, steps=2)
    within(S, forward64(**parts[1])[1], forward64(**absolute(parts[1]))[1], dt, "S", pair=tc)
    # the norm behind it: the same rows in both layouts
    rows = [slice(0, 8), slice(N - 8, N)]
    gate = dout.view(1, N, H * D)
    y = cuda_lib.la_group_norm(out, gate)
    dx, dgate, *_ = cuda_lib.la_group_norm_backward(out, y, gate)
    for r in rows:
        x, t = out[:, :, r].double().requires_grad_(), gate[:, r].double().requires_grad_()
        ref = norm64(x, t)
        want = torch.autograd.grad(ref, (x, t), y[:, r].double())
        for a, b in ((y[:, r], ref), (dx[:, :, r], want[0]), (dgate[:, r], want[1])):
            off = (a.double() - b).abs() - 2.0**-15 * b.abs().amax() - (EPS16 * b.abs() if dt == BF16 else 0.0)
            assert off.max().item() <= 0
    del out, y, dx, dgate
    grads = cuda_lib.la_gated_backward(q, k, v, g, dout)
    for p, s in zip(parts, (slice(0, head), slice(N - tail, N))):
        ref, terms = backward64(**p), backward64(**absolute(p))
        for name, x, r, a in zip(("dq", "dk", "dv", "dg"), grads, ref, terms):
            if name == "dg":
                a = a + a.amax(-1, keepdim=True)
            within(x[:, :, s], r, a, dt, name, pair=tc, steps=2)
    assert cuda_lib.device_status() == 0


def test_pool_of_more_elements_than_31_bits_count(cuda_lib):
    H, D, slots = 32, 128, 4100
    pool = torch.zeros(slots, H, D, D, device="cuda")
    assert pool.numel() > 2**31
    d = make(2, H, 1, D, D, BF16, seed=5, state=True)
    at = torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda")
    pool[at.long()] = d["S0"]
    o = cuda_lib.la_gated_decode_step(*(d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")), pool, slots=at)
    ref, refS, _ = forward64(**d)
    abso, absS, _ = forward64(**absolute(d))
    within(o, ref[:, :, 0], abso[:, :, 0], BF16, "out")
    within(pool[at.long()], refS, absS, BF16, "S")
    assert pool[: slots - 1].count_nonzero() == pool[1].count_nonzero(), "a state outside the batch was touched"
