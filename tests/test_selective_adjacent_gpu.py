"""Outputs that lie right behind inputs: all tensors of a call in one buffer, one behind the
other, give what separate ones give."""
import pytest
import torch

from selectivelib import make, make_conv

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Arena:
    """Tensors one behind the other (sizes are multiples of 16 bytes)."""

    def __init__(self, size=1 << 22):
        self.raw, self.used = torch.empty(size, dtype=torch.uint8, device="cuda"), 0

    def new(self, shape, dtype):
        n = torch.Size(shape).numel() * dtype.itemsize
        assert n % 16 == 0
        t = self.raw[self.used : self.used + n].view(dtype).view(shape)
        self.used += n
        return t

    def like(self, t):
        return self.new(t.shape, t.dtype)

    def copy(self, t):
        return None if t is None else self.like(t).copy_(t)


def stream():
    return torch.cuda.current_stream().cuda_stream


def test_scan_and_gradient(cuda_lib):
    L, p = cuda_lib, cuda_lib._ptr
    B, N, D, ds = 2, 70, 24, 16
    d = make(B, N, D, ds, BF16, seed=1, state=True)
    lengths = torch.tensor([70, 33, 0, 0], dtype=torch.int32, device="cuda")[:B]
    opts = {n: d[n] for n in ("D", "z", "dt_bias")}
    want, want_S = L.la_selective_scan_with_state(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["S0"].clone(), **opts, lengths=lengths)
    want_g = L.la_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dout"], **opts, S0=d["S0"], dS=d["dS"],
                                          lengths=lengths, need_state_grad=True)
    a = Arena()
    order = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")
    i = {n: a.copy(d[n]) for n in order}
    out, S, g = a.like(want).zero_(), a.copy(d["S0"]), [a.like(t) for t in want_g]
    dout, S0, dS = a.copy(d["dout"]), a.copy(d["S0"]), a.copy(d["dS"])
    args = (p(i["x"]), D, p(i["dt"]), D, p(i["A"]), p(i["Bm"]), ds, p(i["Cm"]), ds, p(i["D"]), p(i["z"]), D, p(i["dt_bias"]))
    ws = torch.empty(L.lib.la_selective_scan_workspace(B, N, D, ds, 1, 1) + 256, dtype=torch.uint8, device="cuda")
    assert L.lib.la_selective_scan_with_state(*args, p(lengths), p(out), p(S), B, N, D, ds, 1, 1, p(ws), ws.numel(), stream()) == 0
    dx, ddt, dA, dB, dC, dD, dz, dbias, dS0 = g
    assert L.lib.la_selective_scan_backward(*args, p(lengths), p(dout), p(S0), p(dS), p(dx), p(ddt), p(dA), p(dB), p(dC), p(dD), p(dz),
                                            p(dbias), p(dS0), B, N, D, ds, 1, 1, p(ws), ws.numel(), stream()) == 0
    assert torch.equal(out, want) and torch.equal(S, want_S)
    assert all(torch.equal(x, y) for x, y in zip(g, want_g))
    assert all(torch.equal(i[n], d[n]) for n in order) and torch.equal(S0, d["S0"]) and torch.equal(dS, d["dS"])


def test_conv_and_gradient(cuda_lib):
    L, p = cuda_lib, cuda_lib._ptr
    B, N, D, K = 2, 70, 24, 4
    d = make_conv(B, N, D, K, BF16, seed=2, state=True)
    want, want_S = L.la_short_conv_with_state(d["x"], d["w"], d["S0"].clone(), bias=d["b"])
    want_g = L.la_short_conv_backward(d["x"], d["w"], d["dout"], bias=d["b"], S0=d["S0"], dS=d["dS"], need_state_grad=True)
    a = Arena()
    x, w, b = (a.copy(d[n]) for n in ("x", "w", "b"))
    out, S, g = a.like(want), a.copy(d["S0"]), [a.like(t) for t in want_g]
    dout, S0, dS = (a.copy(d[n]) for n in ("dout", "S0", "dS"))
    ws = torch.empty(L.lib.la_short_conv_workspace(B, N, D, K) + 256, dtype=torch.uint8, device="cuda")
    assert L.lib.la_short_conv_with_state(p(x), D, p(w), p(b), None, p(out), p(S), B, N, D, K, 1, 1, stream()) == 0
    assert L.lib.la_short_conv_backward(p(x), D, p(w), p(b), None, p(dout), p(S0), p(dS), *map(p, g), B, N, D, K, 1, 1, p(ws),
                                        ws.numel(), stream()) == 0
    assert torch.equal(out, want) and torch.equal(S, want_S) and all(torch.equal(y, z) for y, z in zip(g, want_g))


def test_steps_selection_and_reordering(cuda_lib):
    L, p = cuda_lib, cuda_lib._ptr
    G, W, V, D, ds, K = 1, 4, 100, 24, 16, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    logits, scores, x, dt, A, Bm, Cm, w = r(G, W, V), r(G, W), r(W, D), r(W, D), -torch.exp(r(D, ds)), r(W, ds), r(W, ds), r(D, K)
    windows, states = r(W, K - 1, D), r(W, D, ds)
    slots = torch.tensor([[2, 0, 1, 3]], dtype=torch.int32, device="cuda")
    pools = [windows.clone(), states.clone()]
    best, parents, tokens = L.la_beam_select(logits, scores)
    new = L.la_beam_reorder(pools, slots, parents)
    u = L.la_short_conv_step(x, w, pools[0], slots=new.reshape(-1))
    o = L.la_selective_scan_step(u, dt, A, Bm, Cm, pools[1], slots=new.reshape(-1))
    a = Arena()
    logits, scores, x, dt, A, Bm, Cm, w, slots = (a.copy(t) for t in (logits, scores, x, dt, A, Bm, Cm, w, slots))
    got = [a.like(t) for t in (best, parents, tokens, new)]
    q = [a.copy(windows), a.copy(states)]
    u2, o2 = a.like(u), a.like(o)
    ws = torch.empty(L.lib.la_beam_select_workspace(G, W, W, V, 0) + 256, dtype=torch.uint8, device="cuda")
    assert L.lib.la_beam_select(p(logits), V, p(scores), None, *map(p, got[:3]), G, W, W, V, 0, 0, p(ws), ws.numel(), stream()) == 0
    at = (L._vp * 2)(*(t.data_ptr() for t in q))
    rows = (L._sz * 2)(*(t[0].nbytes for t in q))
    assert L.lib.la_beam_reorder(at, rows, 2, p(slots), p(got[1]), p(got[3]), G, W, W, stream()) == 0
    assert L.lib.la_short_conv_step(p(x), D, p(w), None, p(q[0]), p(got[3]), p(u2), W, W, D, K, 1, 0, stream()) == 0
    assert L.lib.la_selective_scan_step(p(u2), D, p(dt), D, p(A), p(Bm), ds, p(Cm), ds, None, None, 0, None, p(q[1]), p(got[3]), p(o2),
                                        W, W, D, ds, 1, 0, stream()) == 0
    assert all(torch.equal(y, z) for y, z in zip([*got, u2, o2, *q], [best, parents, tokens, new, u, o, *pools]))
    assert L.device_status() == 0
