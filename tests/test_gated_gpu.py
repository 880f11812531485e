"""Gated linear attention, its gradient and serving step against the 64-bit recurrence."""
import pytest
import torch

from gatedlib import absolute, backward64, forward64, make, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")

# (B, H, N, dk, dv): one token, chunk borders of every kernel (32 and 128 tokens) and one off them,
# unequal heads, long enough for several segments per head
SHAPES = [(1, 1, 1, 128, 128), (2, 3, 2, 64, 64), (1, 2, 31, 32, 64), (1, 1, 33, 128, 32), (1, 2, 127, 128, 128),
          (1, 2, 128, 64, 64), (2, 1, 129, 128, 128), (1, 3, 257, 64, 64), (2, 2, 300, 32, 32), (1, 1, 1100, 128, 128),
          (1, 1, 1027, 64, 64)]


def tensor_core(dt, dk, dv):
    return dt == BF16 and dk == dv and dk >= 64


def call(L, d, lengths=None, **kw):
    q, v = d["q"], d["v"]
    out = torch.full((*q.shape[:3], v.shape[-1]), NAN, dtype=q.dtype, device=q.device)
    if d["S0"] is None:
        S = torch.full((*q.shape[:2], q.shape[-1], v.shape[-1]), NAN, device=q.device)
        L.la_gated(q, d["k"], v, d["g"], lengths=lengths, out=out, S=S, **kw)
    else:
        S = d["S0"].clone()
        L.la_gated_with_state(q, d["k"], v, d["g"], S, lengths=lengths, out=out, **kw)
    return out, S


def check_forward(L, d, lengths=None):
    q, v = d["q"], d["v"]
    tc = tensor_core(q.dtype, q.shape[-1], v.shape[-1])
    out, S = call(L, d, lengths)
    a = absolute(d)
    ref, refS, _ = forward64(**d, lengths=lengths)
    abso, absS, _ = forward64(**a, lengths=lengths)
    if lengths is not None:
        dead = torch.arange(q.shape[2], device=q.device) >= lengths[:, None]
        dead = dead[:, None, :, None].expand_as(out)
        assert out[dead].isnan().all(), "a padding row was written"
        out = out.masked_fill(dead, 0)
    within(out, ref, abso, q.dtype, "out", pair=tc, steps=2)  # each weight or state rounded once, and its partner
    within(S, refS, absS, q.dtype, "S", pair=tc)
    assert L.device_status() == 0


def check_backward(L, d, lengths=None):
    q, v = d["q"], d["v"]
    tc = tensor_core(q.dtype, q.shape[-1], v.shape[-1])
    got = L.la_gated_backward(q, d["k"], v, d["g"], d["dout"], S0=d["S0"], dS=d["dS"], lengths=lengths,
                              need_state_grad=True)
    ref = backward64(**d, lengths=lengths)
    terms = backward64(**absolute(d), lengths=lengths)
    for name, x, r, a in zip(("dq", "dk", "dv", "dg", "dS0"), got, ref, terms):
        if name == "dg":
            # its parts are added over the chunk's pairs and across the border: terms of the neighbours' size
            a = a + a.amax(-1, keepdim=True)
        within(x, r, a, q.dtype, name, pair=tc, steps=2)
    assert L.device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(cuda_lib, shape, dt):
    check_forward(cuda_lib, make(*shape, dt, seed=sum(shape)))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(cuda_lib, shape, dt):
    check_backward(cuda_lib, make(*shape, dt, seed=sum(shape) + 1))


CASES = [(F32, 64, 32), (BF16, 64, 64), (BF16, 128, 128), (BF16, 32, 128)]


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_carried_state_and_resets(cuda_lib, dt, dk, dv):
    d = make(2, 3, 290, dk, dv, dt, seed=5, state=True, resets=0.02)
    d["g"][0, 0, 127:130] = float("-inf")  # resets around a chunk border
    d["g"][0, 1, 0] = float("-inf")
    d["g"][1, 2, -1] = float("-inf")
    check_forward(cuda_lib, d)
    check_backward(cuda_lib, d)


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("scale", [0.0, 3.0, 60.0, 400.0])
def test_decays_from_none_to_forgetting_at_once(cuda_lib, dt, dk, dv, scale):
    d = make(1, 2, 200, dk, dv, dt, seed=11, state=True, scale=scale)
    check_forward(cuda_lib, d)
    check_backward(cuda_lib, d)


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_every_token_resets(cuda_lib, dt, dk, dv):
    d = make(1, 2, 140, dk, dv, dt, seed=12, state=True, resets=1.1)
    check_forward(cuda_lib, d)
    check_backward(cuda_lib, d)


@pytest.mark.parametrize("dt,dk,dv", CASES)
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(cuda_lib, dt, dk, dv, state):
    """Rows of length 0, 1, inside a chunk, at its border, full, and beyond N; the padding holds NaN and inf."""
    N = 260
    lengths = torch.tensor([0, 1, 77, 128, N, N + 9, -4], dtype=torch.int32, device="cuda")
    d = make(7, 2, N, dk, dv, dt, seed=21, state=state)
    clean = {n: None if t is None else t.clone() for n, t in d.items()}
    eff = lengths.clamp(0, N)
    dead = torch.arange(N, device="cuda") >= eff[:, None]
    for n in ("q", "k", "v", "dout", "g"):
        d[n].masked_fill_(dead[:, None, :] if n == "g" else dead[:, None, :, None], NAN)
    d["v"][2, :, 200:] = float("inf")
    out, S = call(cuda_lib, d, lengths)
    o2, S2 = call(cuda_lib, clean, lengths)
    assert torch.equal(S, S2) and torch.equal(out.isnan(), o2.isnan())
    assert torch.equal(out.nan_to_num(), o2.nan_to_num())
    check_forward(cuda_lib, clean, eff)
    grads = lambda x: cuda_lib.la_gated_backward(  # noqa: E731
        x["q"], x["k"], x["v"], x["g"], x["dout"], S0=x["S0"], dS=x["dS"], lengths=lengths, need_state_grad=True)
    for x, y in zip(grads(d), grads(clean)):
        assert torch.equal(x, y)
    check_backward(cuda_lib, clean, eff)


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_empty(cuda_lib, dt, dk, dv):
    d = make(2, 2, 0, dk, dv, dt, seed=1, state=True)
    out, S = call(cuda_lib, d)
    assert out.numel() == 0 and torch.equal(S, d["S0"])
    *_, dS0 = cuda_lib.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"], dS=d["dS"], need_state_grad=True)
    assert torch.equal(dS0, d["dS"])
    d["S0"] = None
    assert call(cuda_lib, d)[1].eq(0).all()
    e = make(0, 2, 5, dk, dv, dt, seed=1)
    assert cuda_lib.la_gated(e["q"], e["k"], e["v"], e["g"])[0].numel() == 0


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_two_calls_are_one_and_the_steps_too(cuda_lib, dt, dk, dv):
    """A prompt cut in two continues from the state, and single tokens continue from that."""
    d = make(2, 3, 203, dk, dv, dt, seed=31)
    cut, end = 75, 200
    part = lambda a, b: {n: d[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "g")}  # noqa: E731
    out, S = cuda_lib.la_gated(**part(0, cut))
    out2, S = cuda_lib.la_gated_with_state(S=S, **part(cut, end))
    tc = tensor_core(dt, dk, dv)
    ref, refS, _ = forward64(**d)
    abso, absS, _ = forward64(**absolute(d))
    within(out, ref[:, :, :cut], abso[:, :, :cut], dt, "first part", pair=tc, steps=2)
    within(out2, ref[:, :, cut:end], abso[:, :, cut:end], dt, "second part", pair=tc, steps=2)
    pool = torch.full((5, 3, dk, dv), NAN, device="cuda")
    slots = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for t in range(end, 203):
        o = cuda_lib.la_gated_decode_step(*(d[n][:, :, t].contiguous() for n in ("q", "k", "v", "g")), pool, slots=slots)
        within(o, ref[:, :, t], abso[:, :, t], dt, f"token {t}", pair=tc)
    within(pool[slots.long()], refS, absS, dt, "pool", pair=tc)
    assert pool[[1, 2, 4]].isnan().all(), "a state outside the batch was touched"


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_step(cuda_lib, dt, dk, dv):
    d = make(4, 3, 1, dk, dv, dt, seed=dk + dv, state=True, resets=0.2)
    S = d["S0"].clone()
    one = [d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    o = cuda_lib.la_gated_decode_step(*one, S)
    ref, refS, _ = forward64(**d)
    abso, absS, _ = forward64(**absolute(d))
    within(o, ref[:, :, 0], abso[:, :, 0], dt, "out")
    within(S, refS, absS, dt, "S")


def test_step_bad_slots(cuda_lib):
    """Unused rows (negative) are silent; a slot out of range or given twice is skipped and reported."""
    d = make(6, 2, 1, 64, 64, BF16, seed=3)
    one = [d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    pool = torch.randn(4, 2, 64, 64, device="cuda")
    before = pool.clone()
    cuda_lib.device_status()

    def step(slots):
        pool.copy_(before)
        return cuda_lib.la_gated_decode_step(*one, pool, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))

    o = step([2, -1, 0, -7, 3, -1])
    assert cuda_lib.device_status() == 0
    assert o[[1, 3, 5]].eq(0).all() and o[[0, 2, 4]].ne(0).any(-1).all()
    assert torch.equal(pool[1], before[1]) and not torch.equal(pool[0], before[0])
    alone = pool.clone()
    o2 = step([2, 4, 0, 2, 3, 2147483647])  # 4 is past the pool, row 3 repeats row 0's slot
    assert cuda_lib.device_status() == 1 and cuda_lib.device_status() == 0
    assert torch.equal(o, o2) and torch.equal(pool, alone)


def test_long_batch_of_rows_with_a_repeat_far_back(cuda_lib):
    """The repeat check reaches past the first 256 rows."""
    B = 700
    d = make(B, 1, 1, 32, 32, F32, seed=4)
    one = [d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    pool = torch.randn(B, 1, 32, 32, device="cuda")
    slots = torch.randperm(B, device="cuda").to(torch.int32)
    slots[699] = slots[300]
    o = cuda_lib.la_gated_decode_step(*one, pool, slots=slots)
    assert cuda_lib.device_status() == 1
    assert o[699].eq(0).all() and o[300].ne(0).any()


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_gradient_against_differences(cuda_lib, dt, dk, dv):
    """The loss's change along a direction in the decays, by central differences in 64 bits."""
    d = make(1, 2, 150, dk, dv, dt, seed=41, state=True)
    *_, dg, dS0 = cuda_lib.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"], S0=d["S0"], dS=d["dS"],
                                             need_state_grad=True)

    def loss(g, S0):
        o, S, _ = forward64(d["q"], d["k"], d["v"], g, S0)
        return (o * d["dout"].double()).sum() + (S * d["dS"].double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(7)
    ug = torch.randn(d["g"].shape, generator=gen, device="cuda", dtype=torch.float64)
    uS = torch.randn(d["S0"].shape, generator=gen, device="cuda", dtype=torch.float64)
    h = 1e-5
    g, S0 = d["g"].double(), d["S0"].double()
    num = (loss(g + h * ug, S0 + h * uS) - loss(g - h * ug, S0 - h * uS)) / (2 * h)
    ana = (dg.double() * ug).sum() + (dS0.double() * uS).sum()
    size = (dg.double() * ug).norm() + (dS0.double() * uS).norm()
    # differences: h^2 times the third derivative, about 1e-9 here; results: 2^-15 of terms that partly cancel
    assert abs(num - ana) <= 1e-3 * size


def test_other_stream_and_graph(cuda_lib):
    """A call on a side stream, and forward plus gradient captured, replayed on new inputs beside a second graph."""
    L = cuda_lib
    sets = [make(1, 4, 700, 128, 128, BF16, seed=50 + i) for i in range(4)]

    def run(d):
        out, S = L.la_gated(d["q"], d["k"], d["v"], d["g"])
        return (out, S, *L.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"]))

    want = [[t.clone() for t in run(d)] for d in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = L.la_gated(sets[0]["q"], sets[0]["k"], sets[0]["v"], sets[0]["g"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    graphs = []
    for i in range(2):
        d = {n: None if t is None else t.clone() for n, t in sets[i].items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = run(d)
        graphs.append((g, d, r))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, (g, d, r) in enumerate(graphs):
        for n, t in sets[2 + i].items():
            if t is not None:
                d[n].copy_(t)
    torch.cuda.synchronize()
    for _ in range(3):  # both graphs in flight at once
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i, (_, _, r) in enumerate(graphs):
        for x, y in zip(r, want[2 + i]):
            assert torch.equal(x, y)


def test_results_do_not_change_from_run_to_run(cuda_lib):
    d = make(2, 5, 900, 64, 64, BF16, seed=60, state=True)
    run = lambda: (*call(cuda_lib, d), *cuda_lib.la_gated_backward(  # noqa: E731
        d["q"], d["k"], d["v"], d["g"], d["dout"], S0=d["S0"], dS=d["dS"], need_state_grad=True))
    first = run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, run()))


def test_many_heads(cuda_lib):
    """More (row, head) pairs than one launch dimension of 65535 holds."""
    d = make(70000, 1, 3, 32, 32, F32, seed=70)
    out, S = cuda_lib.la_gated(d["q"], d["k"], d["v"], d["g"])
    at = [0, 1, 65534, 65535, 65536, 69999]
    part = {n: None if t is None else t[at] for n, t in d.items()}
    ref, refS, _ = forward64(**part)
    abso, absS, _ = forward64(**absolute(part))
    within(out[at], ref, abso, F32, "out")
    within(S[at], refS, absS, F32, "S")
    dq = cuda_lib.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"])[0]
    within(dq[at], backward64(**part)[0], backward64(**absolute(part))[0], F32, "dq")


@pytest.mark.parametrize("d", [64, 128])
def test_segments_cut_by_lengths(cuda_lib, d):
    """Few heads: several segments each, of which rows fill all, one and a half, or a part of the first."""
    N = 2600 if d == 128 else 4100
    lengths = torch.tensor([N, 130, N // 2 + 77], dtype=torch.int32, device="cuda")
    x = make(3, 1, N, d, d, BF16, seed=91, state=True, resets=0.002)
    check_forward(cuda_lib, x, lengths)
    check_backward(cuda_lib, x, lengths)


def test_long_decays_and_segments(cuda_lib):
    """Decays of 2^-12 a token: the state before a segment carries thousands of tokens."""
    x = make(1, 2, 3000, 64, 64, BF16, seed=92, scale=2.0**-11)
    check_forward(cuda_lib, x)
    check_backward(cuda_lib, x)


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_offset_storage(cuda_lib, dt, dk, dv):
    """Tensors that start 16 but not 32 bytes, and decays that start 4 bytes, into their storage."""
    d = make(2, 2, 161, dk, dv, dt, seed=93, state=True)

    def shifted(t, by):
        if t is None:
            return None
        s = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
        s[by:] = t.reshape(-1)
        return s[by:].view(t.shape)

    by = 16 // torch.empty((), dtype=dt).element_size()
    e = {n: shifted(t, by if n in ("q", "k", "v", "dout") else 1 if n == "g" else 4) for n, t in d.items()}
    out = shifted(torch.zeros_like(d["v"]), by)
    S = shifted(d["S0"], 4)
    cuda_lib.la_gated_with_state(e["q"], e["k"], e["v"], e["g"], S, out=out)
    o2, S2 = call(cuda_lib, d)
    assert torch.equal(out, o2) and torch.equal(S, S2)
    grad = lambda x: cuda_lib.la_gated_backward(  # noqa: E731
        x["q"], x["k"], x["v"], x["g"], x["dout"], S0=x["S0"], dS=x["dS"], need_state_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(grad(e), grad(d)))
    with pytest.raises(cuda_lib.LinAttnError, match="MISALIGNED"):
        cuda_lib.la_gated(shifted(d["q"], 1), d["k"], d["v"], d["g"])


def test_gradient_written_to_unaligned_and_in_place_buffers(cuda_lib):
    """Through the C ABI: dq, dk, dv 16 bytes into their storage, and dS0 written over dS."""
    L = cuda_lib
    d = make(2, 2, 300, 128, 128, BF16, seed=94, state=True)
    want = L.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"], S0=d["S0"], dS=d["dS"], need_state_grad=True)
    bufs = [torch.full((d["q"].numel() + 8,), NAN, dtype=BF16, device="cuda")[8:] for _ in range(3)]
    dg, dS = torch.empty_like(d["g"]), d["dS"].clone()
    need = L.lib.la_gated_workspace(2, 2, 300, 128, 128, 1, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    p = L._ptr
    rc = L.lib.la_gated_backward(p(d["q"]), p(d["k"]), p(d["v"]), p(d["g"]), None, p(d["dout"]), p(d["S0"]), p(dS),
                                 *map(p, bufs), p(dg), p(dS), 2, 2, 300, 128, 128, 1, p(ws), need,
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for b, w in zip(bufs, want):
        assert torch.equal(b.view(w.shape), w)
    assert torch.equal(dg, want[3]) and torch.equal(dS, want[4])
    # a workspace that is too small is refused before anything runs
    assert L.lib.la_gated_backward(p(d["q"]), p(d["k"]), p(d["v"]), p(d["g"]), None, p(d["dout"]), None, None, *map(p, bufs),
                                   p(dg), None, 2, 2, 300, 128, 128, 1, p(ws), need - 1, None) == 1


def test_many_heads_on_the_tensor_cores(cuda_lib):
    d = make(70000, 1, 3, 64, 64, BF16, seed=71)
    out, S = cuda_lib.la_gated(d["q"], d["k"], d["v"], d["g"])
    at = [0, 1, 65534, 65535, 65536, 69999]
    part = {n: None if t is None else t[at] for n, t in d.items()}
    ref, refS, _ = forward64(**part)
    abso, absS, _ = forward64(**absolute(part))
    within(out[at], ref, abso, BF16, "out", pair=True, steps=2)
    within(S[at], refS, absS, BF16, "S", pair=True)
    dv = cuda_lib.la_gated_backward(d["q"], d["k"], d["v"], d["g"], d["dout"])[2]
    within(dv[at], backward64(**part)[2], backward64(**absolute(part))[2], BF16, "dv", pair=True, steps=2)


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_nan_decay_reaches_only_what_follows(cuda_lib, dt, dk, dv):
    d = make(1, 2, 200, dk, dv, dt, seed=95)
    d["g"][0, 1, 90] = NAN
    out, S = call(cuda_lib, d)
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(S[0, 0]).all()
    assert torch.isfinite(out[0, 1, :90]).all() and out[0, 1, 90:].isnan().all() and S[0, 1].isnan().all()


@pytest.mark.parametrize("dt,dk,dv", CASES)
def test_captured_on_two_streams_at_once(cuda_lib, dt, dk, dv):
    """Prefill, gradient, step and norm captured twice, both graphs in flight, against eager calls."""
    L = cuda_lib
    sets = [make(2, 3, 500, dk, dv, dt, seed=96 + i, state=True) for i in range(2)]
    gates = [torch.randn(2, 500, 3 * dv, device="cuda").to(dt) for _ in range(2)]
    w, b = torch.randn(3 * dv, device="cuda"), torch.randn(3 * dv, device="cuda")

    def run(d, gate):
        out, S = L.la_gated(d["q"], d["k"], d["v"], d["g"])
        y = L.la_group_norm(out, gate, w, b)
        dn = L.la_group_norm_backward(out, y, gate, w, b)
        gr = L.la_gated_backward(d["q"], d["k"], d["v"], d["g"], dn[0], dS=d["dS"], need_state_grad=True)
        o = L.la_gated_decode_step(*(d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")), S)
        return [out, S, y, *dn, *gr, o]

    want = [run(d, g) for d, g in zip(sets, gates)]
    torch.cuda.synchronize()
    graphs = []
    for d, g in zip(sets, gates):
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            r = run(d, g)
        graphs.append((G, r, torch.cuda.Stream()))
    for _ in range(5):
        for G, _, s in graphs:
            with torch.cuda.stream(s):
                G.replay()
    torch.cuda.synchronize()
    for (_, r, _), x in zip(graphs, want):
        assert all(torch.equal(a, c) for a, c in zip(r, x))
    assert L.device_status() == 0
