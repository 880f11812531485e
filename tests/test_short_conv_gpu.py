"""Short convolution, its gradient and step against the definition in 64 bits."""
import pytest
import torch

from selectivelib import conv64, conv_grad64, live_tokens, make_conv, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")
# (B, N, D): shorter than the window, borders of the four rows in flight and of runs of 16 tokens, many runs
SHAPES = [(1, 1, 8), (2, 2, 24), (1, 3, 16), (3, 4, 8), (1, 15, 40), (2, 16, 8), (1, 17, 264), (2, 131, 72), (1, 1000, 64)]


def run(L, d, lengths=None, **kw):
    out = torch.full_like(d["x"], NAN, memory_format=torch.contiguous_format)
    if d["S0"] is None:
        S = torch.full((d["x"].shape[0], d["w"].shape[1] - 1, d["x"].shape[2]), NAN, dtype=d["x"].dtype, device="cuda")
        return L.la_short_conv(d["x"], d["w"], bias=d["b"], silu=d["silu"], lengths=lengths, out=out, S=S, **kw)
    return L.la_short_conv_with_state(d["x"], d["w"], d["S0"].clone(), bias=d["b"], silu=d["silu"], lengths=lengths, out=out, **kw)


def grads(L, d, lengths=None):
    r = L.la_short_conv_backward(d["x"], d["w"], d["dout"], bias=d["b"], silu=d["silu"], S0=d["S0"], dS=d["dS"], lengths=lengths,
                                 need_state_grad=True)
    return dict(zip(("dx", "dw", "db", "dS0"), r))


def check(L, d, lengths=None):
    out, S = run(L, d, lengths)
    ref, bound, refS, _ = conv64(d, lengths)
    _, live = live_tokens(d["x"], lengths)
    assert out[~live].isnan().all(), "a padding row was written"
    within(out.masked_fill(~live[..., None], 0), ref, bound, "out")
    assert torch.equal(S.double(), refS)
    for n, x in grads(L, d, lengths).items():
        if x is not None:
            within(x, *conv_grad64(d, lengths)[n], n)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradient(cuda_lib, shape, K, dt):
    check(cuda_lib, make_conv(*shape, K, dt, seed=sum(shape) + K, state=(sum(shape) + K) % 2 == 1))


@pytest.mark.parametrize("silu,bias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_optional_parts(cuda_lib, silu, bias, K):
    d = make_conv(2, 70, 32, K, F32, seed=7, bias=bias, state=True)
    d["silu"] = silu
    assert (grads(cuda_lib, d)["db"] is None) == (not bias)
    check(cuda_lib, d)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("N", [3, 18, 300])
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(cuda_lib, dt, K, N, state):
    lengths = torch.tensor([0, 1, N // 2, 2, N, N + 9, -4], dtype=torch.int32, device="cuda")
    d = make_conv(7, N, 24, K, dt, seed=N + K, state=state)
    _, live = live_tokens(d["x"], lengths)
    dirty = d | {n: d[n].masked_fill(~live[..., None], NAN) for n in ("x", "dout")}
    check(cuda_lib, d, lengths)
    out, S = run(cuda_lib, dirty, lengths)
    o2, S2 = run(cuda_lib, d, lengths)
    assert torch.equal(S, S2) and torch.equal(out.nan_to_num(), o2.nan_to_num())
    for a, b in zip(grads(cuda_lib, dirty, lengths).values(), grads(cuda_lib, d, lengths).values()):
        assert torch.equal(a, b)
    fresh, _ = cuda_lib.la_short_conv(d["x"], d["w"], lengths=lengths)
    assert fresh[~live].eq(0).all(), "padding rows of an allocated output"


def test_large_values(cuda_lib):
    d = make_conv(1, 40, 16, 4, F32, seed=3)
    d["x"] *= 60
    check(cuda_lib, d)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_parts_of_wider_tensors(cuda_lib, dt):
    d = make_conv(3, 50, 40, 4, dt, seed=8, state=True)
    wide = torch.randn(3, 50, 80, device="cuda").to(dt)
    wide[..., 40:] = d["x"]
    e = d | {"x": wide[..., 40:]}
    for a, b in zip(run(cuda_lib, e), run(cuda_lib, d)):
        assert torch.equal(a, b)
    for a, b in zip(grads(cuda_lib, e).values(), grads(cuda_lib, d).values()):
        assert torch.equal(a, b) and a.is_contiguous()
    with pytest.raises(ValueError):
        cuda_lib.la_short_conv(wide.transpose(1, 2)[:, :, :40], d["w"])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_two_calls_are_one_and_the_steps_too(cuda_lib, dt, K):
    d = make_conv(3, 40, 2088, K, dt, seed=21)
    ref, bound, _, _ = conv64(d)
    part = lambda a, b: d | {"x": d["x"][:, a:b]}  # noqa: E731
    out, S = run(cuda_lib, {**part(0, 1), "x": d["x"][:, :1].contiguous()})  # shorter than the window
    out2, S = run(cuda_lib, {**part(1, 30), "x": d["x"][:, 1:30].contiguous(), "S0": S})
    within(torch.cat([out, out2], 1), ref[:, :30], bound[:, :30], "two parts")
    pool = torch.full((6, K - 1, 2088), NAN, dtype=dt, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for t in range(30, 40):
        o = cuda_lib.la_short_conv_step(d["x"][:, t], d["w"], pool, bias=d["b"], slots=slots)
        within(o, ref[:, t], bound[:, t], f"step {t}")
    assert torch.equal(pool[slots.long()], d["x"][:, 40 - K + 1 :])
    assert pool[[1, 3, 5]].isnan().all() and cuda_lib.device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_step_slots(cuda_lib, dt):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.randn(7, 72, generator=g, device="cuda").to(dt), torch.randn(72, 4, generator=g, device="cuda")
    pool = torch.randn(9, 3, 72, generator=g, device="cuda").to(dt)
    before = pool.clone()
    slots = torch.tensor([3, -1, 5, 3, 9, 8, -2], dtype=torch.int32, device="cuda")
    o = cuda_lib.la_short_conv_step(x, w, pool, slots=slots)
    assert cuda_lib.device_status() == 1 and cuda_lib.device_status() == 0
    assert o[[1, 3, 4, 6]].eq(0).all()
    for row, slot in ((0, 3), (2, 5), (5, 8)):
        assert torch.equal(pool[slot], torch.cat([before[slot, 1:], x[row : row + 1]]))
    rest = [0, 1, 2, 4, 6, 7]
    assert torch.equal(pool[rest], before[rest])
    cuda_lib.la_short_conv_step(x, w, pool)
    assert torch.equal(pool[:7, 2], x) and cuda_lib.device_status() == 0


def test_empty(cuda_lib):
    d = make_conv(2, 0, 16, 4, F32, seed=1, state=True)
    assert torch.equal(run(cuda_lib, d)[1], d["S0"])
    g = grads(cuda_lib, d)
    assert torch.equal(g["dS0"], d["dS"]) and g["dw"].eq(0).all() and g["db"].eq(0).all()
    assert run(cuda_lib, d | {"S0": None})[1].eq(0).all()
    e = make_conv(0, 5, 16, 4, F32, seed=1)
    assert run(cuda_lib, e)[0].numel() == 0 and grads(cuda_lib, e)["dw"].eq(0).all()


def test_graphs_and_repeats(cuda_lib):
    d = make_conv(2, 900, 24, 4, BF16, seed=31, state=True)
    want, want_g = run(cuda_lib, d), grads(cuda_lib, d)
    for _ in range(3):
        assert all(torch.equal(x, want_g[n]) for n, x in grads(cuda_lib, d).items())
    made = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made.append((g, run(cuda_lib, d), grads(cuda_lib, d)))
    streams = [torch.cuda.Stream() for _ in made]
    for (g, _, _), s in zip(made * 2, streams * 2):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for _, o, gr in made:
        assert all(torch.equal(a, b) for a, b in zip(o, want)) and all(torch.equal(x, want_g[n]) for n, x in gr.items())


def test_more_elements_than_31_bits_count(cuda_lib):
    N, D = 2**20 + 77, 2056
    x = torch.empty(1, N, D, dtype=BF16, device="cuda").normal_()
    dout = torch.empty(1, N, D, dtype=BF16, device="cuda").normal_()
    w = torch.randn(D, 4, device="cuda")
    assert x.numel() > 2**31
    out, S = cuda_lib.la_short_conv(x, w)
    dx, dw, _ = cuda_lib.la_short_conv_backward(x, w, dout)
    assert torch.equal(S[0], x[0, N - 3 :])
    d = {"x": x[:, N - 40 :].contiguous(), "w": w, "b": None, "silu": True, "dout": dout[:, N - 40 :].contiguous(), "S0": None, "dS": None}
    ref, bound, _, _ = conv64(d)
    within(out[:, N - 37 :], ref[:, 3:], bound[:, 3:], "tail")
    r, e = conv_grad64(d)["dx"]
    within(dx[:, N - 37 :], r[:, 3:], e[:, 3:], "dx tail")
