"""Beam selection and the reordering of states, and both behind a selective state space layer."""
import pytest
import torch

from selectivelib import reorder_slots, scan64, select64, silu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def same(L, logits, scores, k=None, finished=None, eos=0):
    k = logits.shape[1] if k is None else k
    best, parents, tokens = L.la_beam_select(logits, scores, k=k, finished=finished, eos=eos)
    ref, p, t = select64(logits, scores, k, finished, eos)
    assert torch.equal(parents, p) and torch.equal(tokens, t)
    assert torch.equal(best.isneginf(), ref.isneginf())
    live = ~ref.isneginf()
    # a row's logarithm is good to 2^-20 (fp32 exponentials, 2^-22 and |x - top| 2^-23 each), the score is rounded once
    assert ((best.double() - ref).abs()[live] <= 2.0**-19 + 2.0**-24 * ref.abs()[live]).all()
    return best, parents, tokens


def logits_of(G, W, V, dt, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(G, W, V, generator=g, device="cuda")).to(dt), -10 * torch.rand(G, W, generator=g, device="cuda")


# vocabularies off every border (16 bytes, a warp's and a block's share of a chunk), one value, several chunks and runs
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("G,W,V,k", [(1, 1, 1, 1), (3, 2, 5, 4), (2, 4, 33, 4), (5, 3, 1000, 6), (1, 8, 8192, 8), (2, 5, 8193, 5),
                                     (1, 4, 32003, 4), (2, 3, 100003, 64), (40, 16, 515, 16), (1, 64, 999, 64), (2, 33, 4097, 40),
                                     (700, 2, 9001, 2)])
def test_select(cuda_lib, G, W, V, k, dt):
    same(cuda_lib, *logits_of(G, W, V, dt, seed=V + k), k=k)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("k", [1, 8, 33, 64])
def test_ties(cuda_lib, dt, k):
    """All logits equal, two values only, identical beams: the lowest beam and token wins."""
    scores = torch.zeros(2, 4, device="cuda")
    for V in (70, 20001):
        same(cuda_lib, torch.zeros(2, 4, V, device="cuda", dtype=dt), scores, k=k)
        two = torch.zeros(2, 4, V, device="cuda", dtype=dt)
        two[:, :, ::3] = 1.0
        same(cuda_lib, two, scores, k=k)
        two[:, :, V // 2 :] = -0.0
        same(cuda_lib, two, scores, k=k)
        row, _ = logits_of(2, 1, V, dt, seed=5, scale=0.5)
        same(cuda_lib, row.expand(2, 4, V).contiguous(), scores, k=k)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [50, 30011])
def test_masks(cuda_lib, dt, V):
    logits, scores = logits_of(2, 4, V, dt, seed=V)
    m = logits.clone()
    m[:, :, : V - 7] = -INF  # seven tokens are left
    same(cuda_lib, m, scores)
    same(cuda_lib, m, scores, k=40)  # more than are left: -inf in order
    m[0, 2] = -INF  # a row with nothing left
    m[1] = -INF  # a group with nothing left
    same(cuda_lib, m, scores, k=40)
    m = logits.clone()
    m[0, 1, 3], m[0, 1, 9], m[1, 0, 5:20] = NAN, -INF, NAN
    m[1, 2] = NAN
    same(cuda_lib, m, scores, k=9)
    m[0, 0, 2], m[1, 3, 4], m[1, 3, 11] = INF, INF, INF  # infinite logits share the probability
    same(cuda_lib, m, scores, k=9)
    m = logits.clone()
    m[:, :, 1::2] = torch.finfo(dt).min  # a mask of the type's lowest value
    same(cuda_lib, m, scores, k=9)
    low = torch.full_like(logits, torch.finfo(dt).min)
    same(cuda_lib, low, scores, k=9)


def test_unused_and_finished_beams(cuda_lib):
    logits, scores = logits_of(3, 4, 3001, F32, seed=3)
    first = scores.clone()
    first[:, 1:] = -INF  # the first step: one beam is alive
    same(cuda_lib, logits, first)
    first[1, 0] = NAN
    same(cuda_lib, logits, first, k=9)
    done = torch.tensor([[True, False, True, False], [True] * 4, [False] * 4], device="cuda")
    for eos in (0, 2, 3000):
        same(cuda_lib, logits, scores, finished=done, eos=eos)
        same(cuda_lib, logits, scores, k=16, finished=done, eos=eos)
    first[0, 0] = -INF  # nothing is alive
    same(cuda_lib, logits, first, k=16, finished=done, eos=2)
    same(cuda_lib, logits[:, :, :2].contiguous(), scores, k=8, finished=done, eos=1)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_rows_of_a_wider_tensor(cuda_lib, dt):
    wide, scores = logits_of(3, 4, 1000, dt, seed=1)
    wide[..., 777:] = INF  # must not be looked at
    same(cuda_lib, wide[..., :777], scores)
    padded = torch.full((2, 3, 64), INF, device="cuda", dtype=dt)[:, :, :61]
    padded.copy_(torch.randn(2, 3, 61, device="cuda"))
    same(cuda_lib, padded, scores[:2, :3].contiguous())


def test_select_in_graphs_and_refusals(cuda_lib):
    logits, scores = logits_of(4, 4, 50001, BF16, seed=9)
    want = cuda_lib.la_beam_select(logits, scores)
    made = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made.append((g, cuda_lib.la_beam_select(logits, scores)))
    streams = [torch.cuda.Stream() for _ in made]
    for (g, _), s in zip(made * 3, streams * 3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for _, r in made:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert cuda_lib.la_beam_select(logits[:0], scores[:0])[0].shape == (0, 4)
    with pytest.raises(cuda_lib.LinAttnError):
        cuda_lib.la_beam_select(logits, scores, k=65)
    with pytest.raises(cuda_lib.LinAttnError):
        cuda_lib.la_beam_select(logits, scores, k=0)
    with pytest.raises(cuda_lib.LinAttnError):
        cuda_lib.la_beam_select(logits, scores, eos=50001)
    with pytest.raises(TypeError):
        cuda_lib.la_beam_select(logits, scores.double())
    with pytest.raises(ValueError):
        cuda_lib.la_beam_select(logits, scores[:, :3].contiguous())


def reorder(L, pools, slots, parents):
    want = [p.clone() for p in pools]
    new, moves = reorder_slots(slots, parents)
    for src, dst in moves:
        if src >= 0 and dst >= 0:
            for p in want:
                p[dst] = p[src]
    got = L.la_beam_reorder(pools, slots, parents)
    assert got.tolist() == new
    for a, b in zip(pools, want):
        assert torch.equal(a, b)
    assert L.device_status() == 0


@pytest.mark.parametrize("G,W", [(1, 1), (1, 4), (5, 3), (30, 8), (2, 33), (1, 64)])
def test_reorder(cuda_lib, G, W):
    g = torch.Generator(device="cuda").manual_seed(G * W)
    n = G * W + 3
    pools = [torch.randint(0, 1 << 30, (n, 3, 8), generator=g, device="cuda"),
             torch.randn(n, 2, 40, generator=g, device="cuda").to(BF16),
             torch.randn(n, 300, 32, generator=g, device="cuda"), torch.randn(n, 4, generator=g, device="cuda")]
    for i in range(4):
        slots = torch.randperm(n, generator=g, device="cuda")[: G * W].reshape(G, W).int()
        parents = torch.randint(W, (G, W), generator=g, device="cuda").int()
        if i == 1:
            parents = torch.arange(W, device="cuda").flip(0).int().repeat(G, 1)  # a permutation: nothing moves
        if i == 2:
            parents.zero_()
        if i == 3:
            parents[:, ::2] = -1  # new beams without a state
            slots[:, -1] = -1  # and an unused slot
        reorder(cuda_lib, pools, slots, parents)


def test_reorder_of_no_and_many_pools(cuda_lib):
    slots = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[1, 1, 0]], dtype=torch.int32, device="cuda")
    reorder(cuda_lib, [], slots, parents)
    reorder(cuda_lib, [torch.randn(3, 8, device="cuda") for _ in range(131)], slots, parents)
    pool = torch.randn(3, 8, device="cuda")
    want = pool.clone()
    want[1] = want[0]
    assert cuda_lib.la_beam_reorder(pool, slots, parents).tolist() == [[0, 1, 2]] and torch.equal(pool, want)
    empty = slots[:0]
    assert cuda_lib.la_beam_reorder([pool], empty, empty).shape == (0, 3)


def test_reorder_leaves_bad_beams_alone(cuda_lib):
    """Parents and slots out of range and slots that two beams share: no copy, every other beam's state follows it."""
    pool = torch.arange(10.0, device="cuda")[:, None].repeat(1, 4)
    def call(slots, parents):  # noqa: E306
        p = pool.clone()
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        new = cuda_lib.la_beam_reorder([p], t(slots), t(parents))
        status = cuda_lib.device_status()
        return new.tolist(), p[:, 0].tolist(), status

    base = list(range(10))
    new, got, status = call([[0, 1, 2]], [[0, 3, 0]])  # a parent too large
    assert status == 1 and new == [[0, 1, 2]] and got == [0, 1, 0] + base[3:]
    new, got, status = call([[0, 10, 2]], [[1, 1, 0]])  # copies from a slot that is not there
    assert status == 1 and new == [[10, 2, 0]] and got == base
    new, got, status = call([[0, 10, 2]], [[0, 0, 2]])  # copies to one
    assert status == 1 and new == [[0, 10, 2]] and got == base
    new, got, status = call([[0, 1], [1, 2]], [[0, 0], [0, 0]])  # slot 1 is read by the second group
    assert status == 1 and new == [[0, 1], [1, 2]] and got == [0, 1, 1] + base[3:]
    new, got, status = call([[4, 4, 5]], [[2, 2, 2]])
    assert status == 1 and got == base
    with pytest.raises(cuda_lib.LinAttnError):  # rows of 8 bytes
        cuda_lib.la_beam_reorder([torch.zeros(4, 2, device="cuda")], *(torch.zeros(1, 2, dtype=torch.int32, device="cuda"),) * 2)
    with pytest.raises(ValueError):
        cuda_lib.la_beam_reorder([pool, pool[:5]], *(torch.zeros(1, 2, dtype=torch.int32, device="cuda"),) * 2)
    with pytest.raises(ValueError):
        cuda_lib.la_beam_reorder([pool.t()], *(torch.zeros(1, 2, dtype=torch.int32, device="cuda"),) * 2)


def test_a_layer_served_by_beam_search(cuda_lib):
    """Prompt through convolution and scan, then steps on pools of states whose beams are selected and reordered; every
    hypothesis scored again from its whole token sequence in 64 bits."""
    L, G, W, V, D, ds, K, N, steps = cuda_lib, 3, 4, 61, 32, 16, 4, 9, 6
    g = torch.Generator(device="cuda").manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    E, w, b, A = r(V, D), r(D, K) * 0.5, r(D) * 0.1, -torch.exp(r(D, ds) * 0.3)
    Wd, Wb, Wc, Wz, Wo = (r(D, n) * D**-0.5 for n in (D, ds, ds, D, V))
    skip, bias = r(D), r(D) - 2
    prompt = torch.randint(V, (G, N), generator=g, device="cuda")

    def layer(tokens):  # all tokens of each row, [.., V] logits of the last, in 64 bits
        x = E.double()[tokens]
        xp = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
        u = silu(sum(xp[:, j : j + x.shape[1]] * w.double()[:, j] for j in range(K)) + b.double())
        d = {"x": u, "dt": u @ Wd.double(), "A": A, "Bm": u @ Wb.double(), "Cm": u @ Wc.double(), "D": skip, "dt_bias": bias,
             "z": x @ Wz.double(), "softplus": True, "S0": None}
        return scan64(d)[0][:, -1] @ Wo.double()

    x = E[prompt]
    u, conv = L.la_short_conv(x, w, bias=b)
    out, S = L.la_selective_scan(u, u @ Wd, A, u @ Wb, u @ Wc, D=skip, z=x @ Wz, dt_bias=bias)
    n = G * W + 2
    pools = [torch.full((n, K - 1, D), NAN, device="cuda"), torch.full((n, D, ds), NAN, device="cuda")]
    slots = torch.randperm(n, generator=g, device="cuda")[: G * W].reshape(G, W).int()
    pools[0][slots[:, 0].long()], pools[1][slots[:, 0].long()] = conv, S
    logits = (out[:, -1] @ Wo)[:, None].repeat(1, W, 1)
    scores = torch.full((G, W), -INF, device="cuda")
    scores[:, 0] = 0
    history = prompt[:, None].repeat(1, W, 1)
    for _ in range(steps):
        scores, parents, tokens = L.la_beam_select(logits, scores)
        slots = L.la_beam_reorder(pools, slots, parents)
        history = torch.cat([history.gather(1, parents.long()[..., None].expand(-1, -1, history.shape[2])), tokens.long()[..., None]], 2)
        x = E[tokens.long()].reshape(G * W, D)
        rows = slots.reshape(-1)
        u = L.la_short_conv_step(x, w, pools[0], bias=b, slots=rows)
        o = L.la_selective_scan_step(u, u @ Wd, A, u @ Wb, u @ Wc, pools[1], D=skip, z=x @ Wz, dt_bias=bias, slots=rows)
        logits = (o @ Wo).reshape(G, W, V)
    assert L.device_status() == 0
    rows = history.reshape(G * W, -1)
    total = torch.zeros(G * W, dtype=torch.float64, device="cuda")
    for t in range(N, N + steps):
        total += torch.log_softmax(layer(rows[:, :t]), -1).gather(1, rows[:, t : t + 1])[:, 0]
    ref = layer(rows)
    # fp32 products of 32 terms around the layer: far from 1e-4 of logits of size 10
    assert (logits.reshape(G * W, V).double() - ref).abs().max() < 1e-3
    assert (scores.reshape(-1).double() - total).abs().max() < 2e-3
    assert all(len({tuple(h) for h in history[i].tolist()}) == W for i in range(G)), "a hypothesis twice"


def test_a_serving_step_on_another_stream_and_in_a_graph(cuda_lib):
    """Selection, reordering and both steps: the same bits and pools on a given stream and replayed twice."""
    L, G, W, V, D, ds, K = cuda_lib, 2, 4, 5003, 40, 16, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    logits, scores, x, dt, Bm, Cm = r(G, W, V), r(G, W), r(G * W, D), r(G * W, D), r(G * W, ds), r(G * W, ds)
    w, A, n = r(D, K), -torch.exp(r(D, ds)), G * W + 1
    first = [r(n, K - 1, D), r(n, D, ds)]
    slots = torch.randperm(n, generator=g, device="cuda")[: G * W].reshape(G, W).int()

    def step(pools, stream=None):
        best, parents, tokens = L.la_beam_select(logits, scores, stream=stream)
        new = L.la_beam_reorder(pools, slots, parents, stream=stream)
        u = L.la_short_conv_step(x, w, pools[0], slots=new.reshape(-1), stream=stream)
        out = L.la_selective_scan_step(u, dt, A, Bm, Cm, pools[1], slots=new.reshape(-1), stream=stream)
        return [best, parents, tokens, new, u, out, *pools]

    want = step([p.clone() for p in first])
    pools, other = [p.clone() for p in first], torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = step(pools, stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(pools)
    for _ in range(2):
        for p, f in zip(pools, first):
            p.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert L.device_status() == 0
