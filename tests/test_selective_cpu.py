"""The 64-bit forms behind the GPU tests against differences, and the refusals, which return before any CUDA call."""
import pytest
import torch

from selectivelib import conv64, conv_grad64, make, make_conv, reorder_slots, scan64, scan_grad64, select64

F64 = torch.float64
L = pytest.importorskip("causal_linear_attention_attn_gb300.linattn")
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 1 << 20  # aligned, never dereferenced


def loss_of(fn, d, lengths):
    out, S = fn(d, lengths)[0], fn(d, lengths)[2]
    _, live = (None, None) if lengths is None else (0, torch.arange(out.shape[1]) < lengths[:, None])
    do = d["dout"] if live is None else d["dout"].masked_fill(~live[..., None], 0)
    return (out * do).sum() + ((S * d["dS"]).sum() if d["dS"] is not None else 0)


def differences(fn, d, key, lengths, eps=1e-6):
    t = d[key]
    g = torch.zeros_like(t)
    for i in range(t.numel()):
        v = t.flatten()[i].item()
        both = []
        for s in (eps, -eps):
            t.flatten()[i] = v + s
            both.append(loss_of(fn, d, lengths))
        t.flatten()[i] = v
        g.flatten()[i] = (both[0] - both[1]) / (2 * eps)
    return g


@pytest.mark.parametrize("gate,softplus,state,ragged", [(True, True, True, True), (False, False, False, False),
                                                         (True, True, False, False)])
def test_scan_gradient_formulas(gate, softplus, state, ragged):
    d = make(2, 5, 3, 2, F64, 3, gate=gate, state=state, device="cpu")
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    if not softplus:
        d["dt"], d["softplus"] = d["dt"].abs() * 0.3 + 2.5, False
    scan = lambda d, n: (lambda o: (o[0], o[1], o[2]))(scan64(d, n))  # noqa: E731
    n = torch.tensor([5, 2]) if ragged else None
    got = scan_grad64(d, n)
    names = {"dx": "x", "ddt": "dt", "dA": "A", "dB": "Bm", "dC": "Cm", "dD": "D", "ddt_bias": "dt_bias"}
    names |= {"dz": "z"} if gate else {}
    names |= {"dS0": "S0"} if state else {}
    for g, key in names.items():
        ref = differences(scan, d, key, n)
        assert (got[g][0] - ref).abs().max() < 1e-6 * (1 + ref.abs().max()), g


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("state", [False, True])
def test_conv_gradient_formulas(K, state):
    d = make_conv(2, 5, 3, K, F64, 4, state=state, device="cpu")
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    n = torch.tensor([5, 1])
    got = conv_grad64(d, n)
    for g, key in ({"dx": "x", "dw": "w", "db": "b"} | ({"dS0": "S0"} if state else {})).items():
        ref = differences(conv64, d, key, n)
        assert (got[g][0] - ref).abs().max() < 1e-6 * (1 + ref.abs().max()), g


def test_select_by_hand():
    logits = torch.log(torch.tensor([[[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]]))
    scores = torch.tensor([[0.0, 0.0]])
    best, parents, tokens = select64(logits, scores, 4)
    assert parents.tolist() == [[1, 0, 0, 0]] and tokens.tolist() == [[1, 0, 1, 2]]
    assert torch.allclose(best, torch.log(torch.tensor([[0.8, 0.5, 0.25, 0.25]], dtype=F64)))
    best, parents, tokens = select64(logits, scores, 2, torch.tensor([[True, False]]), 2)
    assert parents.tolist() == [[0, 1]] and tokens.tolist() == [[2, 1]] and best[0, 0] == 0


def test_reorder_by_hand():
    new, moves = reorder_slots(torch.tensor([[7, 3, 9, 1]]), torch.tensor([[2, 2, 0, 2]]))
    assert new == [[9, 3, 7, 1]] and moves == [(9, 3), (9, 1)]
    assert reorder_slots(torch.tensor([[4, 5]]), torch.tensor([[-1, 0]])) == ([[5, 4]], [])


def caller(fn, **defaults):
    def call(**kw):
        a = defaults | kw
        assert set(a) == set(defaults)
        return getattr(L.lib, fn)(*a.values())

    return call


@pytest.mark.parametrize("fn", ["la_short_conv", "la_short_conv_with_state"])
def test_conv_refusals(fn):
    call = caller(fn, x=P, ldx=64, w=P, b=P, lengths=None, out=P, S=P, B=1, N=8, D=64, K=4, silu=1, dt=1, stream=None)
    for n in ("x", "w", "out", "S"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 8}) == MISALIGNED
    assert call(lengths=P + 2) == MISALIGNED and call(b=P + 4) == MISALIGNED
    assert call(ldx=56) == INVALID and call(ldx=68) == MISALIGNED and call(ldx=1 << 40) == INVALID
    assert call(K=1) == UNSUPPORTED and call(K=5) == UNSUPPORTED and call(K=0) == INVALID
    assert call(D=60) == UNSUPPORTED and call(D=0) == INVALID and call(dt=2) == UNSUPPORTED
    assert call(B=-1) == INVALID and call(N=-1) == INVALID and call(B=0, x=None, S=None) == OK
    assert call(B=1 << 20, D=1 << 13) == INVALID


def test_conv_backward_refusals():
    names = ("dout", "S0", "dS", "dx", "dw", "db", "dS0")
    call = caller("la_short_conv_backward", x=P, ldx=64, w=P, b=P, lengths=None,
                  **{n: P + (i << 24) for i, n in enumerate(names)}, B=1, N=8, D=64, K=4, silu=1, dt=1, ws=P, bytes=1 << 40,
                  stream=None)
    for n in ("x", "w", "dout", "dx"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 8}) == MISALIGNED
    assert call(dS0=P + (1 << 24)) == INVALID and call(dS0=P + (2 << 24)) == INVALID  # over S0, over dS
    assert call(ws=P + 16) == MISALIGNED and call(dw=P + 2) == MISALIGNED
    assert call(ldx=60) == INVALID and call(K=7) == UNSUPPORTED


def test_conv_step_refusals():
    call = caller("la_short_conv_step", x=P, ldx=64, w=P, b=P, S=P, slots=P, out=P, B=2, n=4, D=64, K=4, silu=1, dt=1, stream=None)
    for n in ("x", "w", "S", "out"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 8}) == MISALIGNED
    assert call(slots=None, n=1) == INVALID and call(n=-1) == INVALID and call(slots=P + 2) == MISALIGNED
    assert call(B=0) == OK and call(ldx=0) == INVALID


SCAN = dict(x=P, ldx=64, delta=P, ldt=64, A=P, Bm=P, ldb=16, Cm=P, ldc=16, D=P, z=P, ldz=64, bias=P)
TAIL = dict(N=8, C=64, ds=16, softplus=1, dt=1)


def scan_common(call):
    for n in ("x", "delta", "A", "Bm", "Cm"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 8}) == MISALIGNED
    for n in ("D", "z", "bias"):
        assert call(**{n: P + 8}) == MISALIGNED
    for n, least in (("ldx", 64), ("ldt", 64), ("ldz", 64), ("ldb", 16), ("ldc", 16)):
        assert call(**{n: least - 8}) == INVALID and call(**{n: least + 4}) == MISALIGNED and call(**{n: 1 << 33}) == INVALID
    assert call(ds=12) == UNSUPPORTED and call(ds=128) == UNSUPPORTED and call(ds=0) == INVALID
    assert call(C=36) == UNSUPPORTED and call(dt=7) == UNSUPPORTED and call(B=-1) == INVALID
    assert call(C=1 << 26, ds=32, ldx=1 << 26, ldt=1 << 26, ldz=1 << 26) == INVALID  # a state of more than 31 bits count


@pytest.mark.parametrize("fn", ["la_selective_scan", "la_selective_scan_with_state"])
def test_scan_refusals(fn):
    call = caller(fn, **SCAN, lengths=None, out=P, S=P, B=1, **TAIL, ws=P, bytes=1 << 40, stream=None)
    scan_common(call)
    assert call(out=None) == INVALID and call(S=None) == INVALID and call(S=P + 4) == MISALIGNED
    assert call(ws=P + 16) == MISALIGNED and call(lengths=P + 1) == MISALIGNED and call(B=0, x=None, S=None) == OK


def test_scan_backward_refusals():
    names = ("dout", "S0", "dS", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dS0")
    call = caller("la_selective_scan_backward", **SCAN, lengths=None, **{n: P + (i << 24) for i, n in enumerate(names)}, B=1,
                  **TAIL, ws=P, bytes=1 << 40, stream=None)
    scan_common(call)
    for n in ("dout", "dx", "ddt", "dB", "dC", "dz"):
        assert call(**{n: None}) == INVALID
    assert call(z=None) == INVALID
    assert call(dS0=P + (1 << 24)) == INVALID and call(dS0=P + (2 << 24) + 64) == INVALID
    assert call(dA=P + 2) == MISALIGNED and call(dB=P + 8) == MISALIGNED


def test_scan_step_refusals():
    tail = {k: v for k, v in TAIL.items() if k != "N"}
    call = caller("la_selective_scan_step", **SCAN, S=P, slots=P, out=P, B=2, n=4, **tail, stream=None)
    scan_common(call)
    assert call(S=None) == INVALID and call(out=None) == INVALID and call(slots=None, n=1) == INVALID and call(B=0) == OK


def test_beam_refusals():
    call = caller("la_beam_select", logits=P, ld=100, scores=P, finished=P, best=P, parents=P, tokens=P, G=1, W=4, k=4, V=100,
                  eos=3, dt=1, ws=P, bytes=1 << 40, stream=None)
    for n in ("logits", "scores", "best", "parents", "tokens"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: P + 2}) == MISALIGNED
    assert call(k=0) == INVALID and call(k=65) == UNSUPPORTED and call(W=65, k=4) == UNSUPPORTED
    assert call(W=1, V=3, k=4, eos=0) == INVALID and call(eos=100) == INVALID and call(eos=-1) == INVALID
    assert call(ld=99) == INVALID and call(dt=2) == UNSUPPORTED and call(G=-1) == INVALID and call(G=0, logits=None) == OK
    assert L.lib.la_beam_select_workspace(0, 4, 4, 100, 1) == 0 < L.lib.la_beam_select_workspace(1, 4, 4, 100, 1)


def test_reorder_refusals():
    import ctypes

    def call(pools=(P,), rows=(64,), slots=P, parents=P + 4096, new=P + 8192, G=2, W=4, n=8):
        a = (ctypes.c_void_p * max(1, len(pools)))(*pools)
        r = (ctypes.c_size_t * max(1, len(rows)))(*rows)
        return L.lib.la_beam_reorder(a, r, len(pools), slots, parents, new, G, W, n, None)

    assert call(slots=None) == INVALID and call(parents=None) == INVALID and call(new=None) == INVALID
    assert call(new=P) == INVALID and call(new=P + 4096) == INVALID and call(W=65) == UNSUPPORTED and call(W=0) == INVALID
    assert call(pools=(P + 8,)) == MISALIGNED and call(rows=(24,)) == MISALIGNED and call(pools=(None,)) == INVALID
    assert call(G=0, slots=None) == OK and call(G=-1) == INVALID and call(n=-1) == INVALID and call(slots=P + 2) == MISALIGNED


def test_outputs_over_inputs_are_refused():
    """An output may lie right behind an input, not over a part of it (rows that are a part of wider ones included)."""
    far = lambda i: P + (i << 24)  # noqa: E731
    conv = caller("la_short_conv", x=P, ldx=128, w=far(1), b=None, lengths=None, out=far(2), S=far(3), B=2, N=8, D=64, K=4,
                  silu=1, dt=1, stream=None)
    size = 15 * 256 + 128
    for out in (P, P + size - 16, P - 2 * 8 * 128 + 16):
        assert conv(out=out) == INVALID
    step = caller("la_short_conv_step", x=P, ldx=64, w=far(1), b=None, S=far(2), slots=None, out=P, B=2, n=4, D=64, K=4,
                  silu=1, dt=1, stream=None)
    assert step() == INVALID
    apart = {n: far(i) for i, n in enumerate(("x", "delta", "A", "Bm", "Cm", "D", "z", "bias"))}
    scan = caller("la_selective_scan", **(SCAN | apart), lengths=None, out=far(9), S=far(10), B=1, **TAIL, ws=far(11),
                  bytes=1 << 40, stream=None)
    one = caller("la_selective_scan_step", **(SCAN | apart), S=far(9), slots=None, out=far(10), B=1, n=4,
                 **{k: v for k, v in TAIL.items() if k != "N"}, stream=None)
    for n in ("x", "delta", "Bm", "Cm", "z"):
        assert scan(out=apart[n]) == INVALID and one(out=apart[n]) == INVALID
    select = caller("la_beam_select", logits=P, ld=100, scores=far(1), finished=None, best=far(2), parents=far(3),
                    tokens=far(4), G=3, W=4, k=2, V=100, eos=3, dt=1, ws=far(5), bytes=1 << 40, stream=None)
    for n in ("best", "parents", "tokens"):
        assert select(**{n: far(1) + 44}) == INVALID and select(**{n: far(1) - 20}) == INVALID


def test_workspaces():
    w = L.lib.la_selective_scan_workspace
    assert w(0, 8, 64, 16, 1, 1) == 0 and w(1, 8, 60, 16, 1, 0) == 0 and w(1, 8, 64, 16, 1, 1) > 0
    assert L.lib.la_short_conv_workspace(1, 0, 64, 4) == 0 < L.lib.la_short_conv_workspace(1, 8, 64, 4)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(1, 8, 64)
    with pytest.raises(ValueError):
        L.la_short_conv(x, torch.zeros(64, 4))
    with pytest.raises(TypeError):
        L.la_short_conv(x.double(), torch.zeros(64, 4))
    with pytest.raises(ValueError):
        L.la_short_conv_with_state(x, torch.zeros(64, 4), None)
    with pytest.raises(ValueError):
        L.la_selective_scan(x[0], x, torch.zeros(64, 16), x, x)
    with pytest.raises(ValueError):
        L.la_selective_scan_with_state(x, x, torch.zeros(64, 16), x, x, None)
    with pytest.raises(ValueError):
        L.la_beam_select(x, torch.zeros(1, 8))
    with pytest.raises(ValueError):
        L.la_beam_reorder([x], torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32))
