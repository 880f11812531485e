"""Selective scan, its gradient and step against the 64-bit recurrence, with bounds that follow it token by token."""
import pytest
import torch

from selectivelib import live_tokens, make, scan64, scan_grad64, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")
ARGS = ("x", "dt", "A", "Bm", "Cm")
OPTS = ("D", "z", "dt_bias", "softplus")

# (B, N, D, d_state): one token, borders of the chunks of 8, 16 and 32 tokens, channels that fill no block, long enough
# for several segments
SHAPES = [(1, 1, 8, 16), (2, 2, 24, 8), (1, 31, 64, 32), (2, 32, 40, 64), (1, 33, 72, 16), (3, 65, 16, 8), (1, 200, 136, 64),
          (2, 127, 64, 32), (1, 600, 72, 16), (2, 1100, 16, 8), (1, 530, 40, 64), (1, 777, 8, 32)]


def args(d):
    return [d[n] for n in ARGS], {n: d[n] for n in OPTS}


def run(L, d, lengths=None, out=None, **kw):
    a, o = args(d)
    if out is None:
        out = torch.full_like(d["x"], NAN, memory_format=torch.contiguous_format)
    if d["S0"] is None:
        S = torch.full((d["x"].shape[0], *d["A"].shape), NAN, device="cuda")
        return L.la_selective_scan(*a, **o, lengths=lengths, out=out, S=S, **kw)
    return L.la_selective_scan_with_state(*a, d["S0"].clone(), **o, lengths=lengths, out=out, **kw)


def check(L, d, lengths=None):
    out, S = run(L, d, lengths)
    ref, bound, refS, boundS, _ = scan64(d, lengths)
    _, live = live_tokens(d["x"], lengths)
    assert out[~live].isnan().all(), "a padding row was written"
    out = out.masked_fill(~live[..., None], 0)
    within(out, ref, bound, "out")
    within(S, refS, boundS, "S")


def grads(L, d, lengths=None):
    a, o = args(d)
    r = L.la_selective_scan_backward(*a, d["dout"], **o, S0=d["S0"], dS=d["dS"], lengths=lengths, need_state_grad=True)
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0"), r))


def check_grad(L, d, lengths=None):
    got, ref = grads(L, d, lengths), scan_grad64(d, lengths)
    for n, x in got.items():
        assert (x is None) == (n not in ref), n
        if x is not None:
            within(x, *ref[n], n)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradient(cuda_lib, shape, dt):
    d = make(*shape, dt, seed=sum(shape), state=sum(shape) % 2 == 1)
    check(cuda_lib, d)
    check_grad(cuda_lib, d)


PARTS = [(False, True, True), (True, False, False), (False, False, False), (True, True, True)]


@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("gate,skip,bias", PARTS)
@pytest.mark.parametrize("softplus", [True, False])
def test_optional_parts(cuda_lib, ds, gate, skip, bias, softplus):
    d = make(2, 70, 32, ds, F32, seed=ds, gate=gate, skip=skip, bias=bias, state=True)
    if not softplus:  # steps as they are
        d["softplus"], d["dt"] = False, d["dt"].abs() * 0.1
        d["dt_bias"] = None if d["dt_bias"] is None else d["dt_bias"].abs() * 0.05
    check(cuda_lib, d)
    check_grad(cuda_lib, d)


@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("gate,skip,bias", PARTS)
def test_steps_of_either_sign(cuda_lib, ds, gate, skip, bias):
    """Negative steps let a state grow: e^{|A| sum |delta|} passes float32's 2^128 in some channels here (|A| up to 30,
    steps around -0.1, 70 tokens), which have no value to compare then.  The others must not be touched by that; dB and
    dC, sums over all channels, cannot be compared."""
    d = make(2, 70, 32, ds, F32, seed=ds, gate=gate, skip=skip, bias=bias, state=True)
    d["softplus"], d["dt"] = False, d["dt"] * 0.1
    d["dt_bias"] = None if d["dt_bias"] is None else d["dt_bias"] * 0.05
    out, S = run(cuda_lib, d)
    ref, bound, refS, boundS, (*_, kept) = scan64(d)
    grad, got = scan_grad64(d), grads(cuda_lib, d)
    # the gradient of a state grows by the same factor from the other end, and the products of both reach 2^120
    ok = torch.stack([hb for _, hb, _ in kept]).amax((0, 1, 3)) < 2.0**50
    assert ok.any()
    within(out[..., ok], ref[..., ok], bound[..., ok], "out")
    within(S[:, ok], refS[:, ok], boundS[:, ok], "S")
    for n, x in got.items():
        if x is None or n in ("dB", "dC"):
            continue
        cut = (lambda t: t[ok]) if x.shape[0] == 32 else (lambda t: t[:, ok]) if n == "dS0" else (lambda t: t[..., ok])
        within(cut(x), *map(cut, grad[n]), n)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("N", [20, 300])
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(cuda_lib, dt, ds, N, state):
    """Rows of length 0, 1, inside a chunk, at its border, full, beyond N and below 0; the padding holds NaN and inf."""
    lengths = torch.tensor([0, 1, N // 2, 32, N, N + 9, -4], dtype=torch.int32, device="cuda")
    d = make(7, N, 24, ds, dt, seed=N + ds, state=state)
    dirty = dict(d)
    _, live = live_tokens(d["x"], lengths)
    for n in ("x", "dt", "Bm", "Cm", "z", "dout"):
        dirty[n] = d[n].masked_fill(~live[..., None], NAN)
    dirty["x"][2, N // 2 + 1] = float("inf")
    check(cuda_lib, d, lengths)
    check_grad(cuda_lib, d, lengths)
    out, S = run(cuda_lib, dirty, lengths)
    o2, S2 = run(cuda_lib, d, lengths)
    assert torch.equal(S, S2) and torch.equal(out.nan_to_num(), o2.nan_to_num())
    for a, b in zip(grads(cuda_lib, dirty, lengths).values(), grads(cuda_lib, d, lengths).values()):
        assert torch.equal(a, b)
    a, o = args(d)
    fresh, _ = cuda_lib.la_selective_scan(*a, **o, lengths=lengths)
    assert fresh[~live].eq(0).all(), "padding rows of an allocated output"


@pytest.mark.parametrize("ds", [16, 64])
def test_steep_and_vanishing_steps(cuda_lib, ds):
    """Steps from e^-60 to 40, decays from none to zero, gates far from zero."""
    d = make(1, 96, 16, ds, F32, seed=3, state=True)
    d["dt"][0, ::3] = -60.0
    d["dt"][0, 1::7] = 40.0
    d["A"][0] = 0.0
    d["A"][1] = -1e4
    d["z"][0, ::5] = -100.0
    d["z"][0, 1::5] = 60.0
    check(cuda_lib, d)
    check_grad(cuda_lib, d)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_parts_of_wider_tensors(cuda_lib, dt):
    d = make(3, 50, 40, 16, dt, seed=8, state=True)
    ref_out, ref_S = run(cuda_lib, d)
    ref = grads(cuda_lib, d)
    wide = torch.randn(3, 50, 2 * 40, device="cuda").to(dt)
    low = torch.randn(3, 50, 8 + 32, device="cuda").to(dt)
    wide[..., :40], wide[..., 40:], low[..., 8:24], low[..., 24:] = d["x"], d["z"], d["Bm"], d["Cm"]
    e = d | {"x": wide[..., :40], "z": wide[..., 40:], "Bm": low[..., 8:24], "Cm": low[..., 24:]}
    out, S = run(cuda_lib, e)
    assert torch.equal(out, ref_out) and torch.equal(S, ref_S)
    for n, x in grads(cuda_lib, e).items():
        assert torch.equal(x, ref[n]) and x.is_contiguous(), n
    with pytest.raises(ValueError):
        run(cuda_lib, d | {"x": d["x"].transpose(0, 1).contiguous().transpose(0, 1)})
    with pytest.raises(cuda_lib.LinAttnError):  # rows on no 16-byte border
        run(cuda_lib, d | {"x": torch.zeros(3, 50, 43, device="cuda", dtype=dt)[..., :40]})


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ds", [8, 16, 32, 64])
def test_two_calls_are_one_and_the_steps_too(cuda_lib, dt, ds):
    d = make(3, 90, 72, ds, dt, seed=21 + ds)
    cut, end = 37, 85
    part = lambda a, b: d | {n: d[n][:, a:b].contiguous() for n in ("x", "dt", "Bm", "Cm", "z", "dout")}  # noqa: E731
    ref, bound, _, _, (*_, kept) = scan64(d)
    out, S = run(cuda_lib, part(0, cut))
    out2, S = run(cuda_lib, part(cut, end) | {"S0": S})
    within(torch.cat([out, out2], 1), ref[:, :end], bound[:, :end], "two parts")
    pool = torch.full((6, 72, ds), NAN, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for t in range(end, 90):
        row = part(t, t + 1)
        one = {n: row[n][:, 0] for n in ("x", "dt", "Bm", "Cm", "z")}
        o = cuda_lib.la_selective_scan_step(one["x"], one["dt"], d["A"], one["Bm"], one["Cm"], pool, D=d["D"], z=one["z"],
                                            dt_bias=d["dt_bias"], slots=slots)
        within(o, ref[:, t], bound[:, t], f"step {t}")
    within(pool[slots.long()], kept[-1][0], kept[-1][2], "pool")
    assert pool[[1, 3, 5]].isnan().all() and cuda_lib.device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_step_slots(cuda_lib, dt):
    """Unused, repeated and bad slots leave every state alone but the first of each; no slots: row b on state b."""
    d = make(7, 1, 264, 16, dt, seed=2)
    one = [d["x"][:, 0], d["dt"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0]]
    pool = torch.randn(9, 264, 16, device="cuda")
    before = pool.clone()
    slots = torch.tensor([3, -1, 5, 3, 9, 8, -2], dtype=torch.int32, device="cuda")
    o = cuda_lib.la_selective_scan_step(*one, pool, D=d["D"], slots=slots)
    assert cuda_lib.device_status() == 1 and cuda_lib.device_status() == 0
    assert o[[1, 3, 4, 6]].eq(0).all()
    good = [0, 2, 5]
    ref, bound, S, Sb, _ = scan64(d | {"z": None, "dt_bias": None, "S0": before[[3, 0, 5, 0, 0, 8, 0]]})
    within(o[good], ref[good, 0], bound[good, 0], "out")
    within(pool[[3, 5, 8]], S[good], Sb[good], "S")
    rest = [0, 1, 2, 4, 6, 7]
    assert torch.equal(pool[rest], before[rest])
    pool = before.clone()
    cuda_lib.la_selective_scan_step(*one, pool, D=d["D"])
    ref, bound, S, Sb, _ = scan64(d | {"z": None, "dt_bias": None, "S0": before[:7]})
    within(pool[:7], S, Sb, "S without slots")
    assert torch.equal(pool[7:], before[7:]) and cuda_lib.device_status() == 0
    with pytest.raises(ValueError):
        cuda_lib.la_selective_scan_step(*one, pool[:6].contiguous())


@pytest.mark.parametrize("N", [40, 700])
def test_empty_and_passing_through(cuda_lib, N):
    d = make(2, 0, 16, 8, F32, seed=1, state=True)
    out, S = run(cuda_lib, d)
    assert out.numel() == 0 and torch.equal(S, d["S0"])
    g = grads(cuda_lib, d)
    assert torch.equal(g["dS0"], d["dS"]) and g["dA"].eq(0).all() and g["dD"].eq(0).all() and g["ddt_bias"].eq(0).all()
    assert run(cuda_lib, d | {"S0": None})[1].eq(0).all()
    e = make(0, 5, 16, 8, F32, seed=1)
    assert run(cuda_lib, e)[0].numel() == 0
    g = grads(cuda_lib, e)
    assert g["dA"].eq(0).all()
    # dS0 over dS, through the C ABI, with one segment and several
    d = make(2, N, 16, 8, F32, seed=5, state=True)
    want = grads(cuda_lib, d)
    L, p = cuda_lib, cuda_lib._ptr
    dS = d["dS"].clone()
    need = L.lib.la_selective_scan_workspace(2, N, 16, 8, 0, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = {n: torch.empty_like(want[n]) for n in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")}
    assert L.lib.la_selective_scan_backward(
        p(d["x"]), 16, p(d["dt"]), 16, p(d["A"]), p(d["Bm"]), 8, p(d["Cm"]), 8, p(d["D"]), p(d["z"]), 16, p(d["dt_bias"]), None,
        p(d["dout"]), p(d["S0"]), p(dS), *map(p, got.values()), p(dS), 2, N, 16, 8, 1, 0, p(ws), need,
        torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dS, want["dS0"]) and all(torch.equal(got[n], want[n]) for n in got)


def test_graphs_streams_and_repeats(cuda_lib):
    """The same bits from run to run, on another stream, and from two graphs that replay side by side."""
    d = make(2, 900, 24, 16, BF16, seed=31, state=True)
    want, want_S = run(cuda_lib, d)
    want_g = grads(cuda_lib, d)
    for _ in range(3):
        out, S = run(cuda_lib, d)
        assert torch.equal(out, want) and torch.equal(S, want_S)
        assert all(torch.equal(x, want_g[n]) for n, x in grads(cuda_lib, d).items())
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out, S = run(cuda_lib, d, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(out, want) and torch.equal(S, want_S)
    made = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made.append((g, run(cuda_lib, d), grads(cuda_lib, d)))
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        for (g, _, _), s in zip(made, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, (o, S), gr in made:
        assert torch.equal(o, want) and torch.equal(S, want_S)
        assert all(torch.equal(x, want_g[n]) for n, x in gr.items())
    assert cuda_lib.device_status() == 0


def test_more_elements_than_31_bits_count(cuda_lib):
    """Steps that forget everything near both ends make the first and last tokens' results independent of the others."""
    N, D, ds = 2**20 + 77, 2056, 8
    new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda").normal_()  # noqa: E731
    d = {"x": new(1, N, D), "dt": new(1, N, D).mul_(0.5).sub_(3), "Bm": new(1, N, ds), "Cm": new(1, N, ds),
         "A": -torch.rand(D, ds, device="cuda") - 0.5, "D": None, "z": None, "dt_bias": None, "softplus": True, "S0": None}
    assert d["x"].numel() > 2**31
    head, tail = 40, 50
    d["dt"][:, N - tail] = 4000.0
    a, o = args(d)
    out, S = cuda_lib.la_selective_scan(*a, **o)
    for s, name in ((slice(0, head), "head"), (slice(N - tail, N), "tail")):
        e = d | {n: d[n][:, s].contiguous() for n in ("x", "dt", "Bm", "Cm")}
        ref, bound, refS, boundS, _ = scan64(e)
        within(out[:, s], ref, bound, name)
    within(S, refS, boundS, "S")


def test_pool_of_more_elements_than_31_bits_count(cuda_lib):
    D, ds, slots = 8192, 64, 4100
    pool = torch.zeros(slots, D, ds, device="cuda")
    assert pool.numel() > 2**31
    d = make(2, 1, D, ds, BF16, seed=9, state=True)
    at = torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda")
    pool[at.long()] = d["S0"]
    one = [d["x"][:, 0], d["dt"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0]]
    o = cuda_lib.la_selective_scan_step(*one, pool, D=d["D"], z=d["z"][:, 0], dt_bias=d["dt_bias"], slots=at)
    ref, bound, S, Sb, _ = scan64(d)
    within(o, ref[:, 0], bound[:, 0], "out")
    within(pool[at.long()], S, Sb, "S")
    assert pool[: slots - 1].count_nonzero() == pool[1].count_nonzero(), "a state outside the batch was touched"


@pytest.mark.parametrize("ds", [8, 16, 32, 64])
@pytest.mark.parametrize("N", [1, 70, 600])
def test_components_that_forget_at_once(cuda_lib, ds, N):
    """A = -inf is e^{delta A} = 0 at every token with a step, as a very low A is, and none in the padding."""
    lengths = torch.tensor([N, N // 2, 0], dtype=torch.int32, device="cuda")
    d = make(3, N, 24, ds, F32, seed=ds + N, state=True)
    low, inf = dict(d, A=d["A"].clone()), dict(d, A=d["A"].clone())
    low["A"][::3, ::2], inf["A"][::3, ::2] = -1e38, -float("inf")
    for lens in (None, lengths):
        a, b = run(cuda_lib, low, lens), run(cuda_lib, inf, lens)
        assert torch.equal(a[0].nan_to_num(7.0), b[0].nan_to_num(7.0)) and torch.equal(a[1], b[1]) and b[1].isfinite().all()
        for n, x in grads(cuda_lib, inf, lens).items():
            assert x.isfinite().all(), n
            assert torch.equal(x, grads(cuda_lib, low, lens)[n]), n
    pools = [d["S0"].clone(), d["S0"].clone()]
    t = lambda e: ([e["x"][:, 0].contiguous(), e["dt"][:, 0].contiguous(), e["A"], e["Bm"][:, 0].contiguous(),  # noqa: E731
                    e["Cm"][:, 0].contiguous()], {"D": e["D"], "z": e["z"][:, 0].contiguous(), "dt_bias": e["dt_bias"]})
    outs = [cuda_lib.la_selective_scan_step(*t(e)[0], S, **t(e)[1]) for e, S in zip((low, inf), pools)]
    assert torch.equal(*outs) and torch.equal(*pools)
