"""Outputs over inputs or over each other, in the short convolution, the selective scan and beam search, are refused before any
CUDA call: no pointer is read."""
import ctypes

import pytest

L = pytest.importorskip("causal_linear_attention_attn_gb300.linattn")
INVALID = 1
P = 1 << 30
B, N, D, K, DS, SLOTS = 2, 8, 64, 4, 16, 5


def call(fn, names, spans, scalars, at):
    """fn with every tensor far from the others but those in `at`; names in the order of the arguments."""
    where = {n: P + (i << 24) for i, n in enumerate(spans)} | at
    values = where | scalars
    return getattr(L.lib, fn)(*(values[n] for n in names))


def pairs(outputs, inputs, allowed=()):
    for i, o in enumerate(outputs):
        for other in [*inputs, *outputs[:i]]:
            if (o, other) not in allowed:
                yield o, other


def check(fn, names, spans, outputs, scalars, allowed=()):
    """spans: bytes of each tensor (a multiple of 16 each).  An output at the other's start, over its last 16 bytes, and ending
    over its first 16."""
    inputs = [n for n in spans if n not in outputs]
    for o, other in pairs(outputs, inputs, allowed):
        base = P + (list(spans).index(other) << 24)
        for at in (base, base + spans[other] - 16, base - spans[o] + 16):
            assert call(fn, names.split(), spans, scalars, {o: at}) == INVALID, (fn, o, other, at - base)


SIZES = {"B": B, "N": N, "C": D, "K": K, "ds": DS, "n": SLOTS, "one": 1, "dt": 1, "none": None, "ldx": 2 * D, "ldt": D, "ldz": 3 * D,
         "ldb": DS, "ldc": 4 * DS, "ws": 1 << 20, "bytes": 1 << 40}


def span(rows, ld, width):
    return ((rows - 1) * ld + width) * 2


CONV = {"x": span(B * N, 2 * D, D), "w": D * K * 4, "b": D * 4, "lengths": 16}
WINDOW = B * (K - 1) * D * 2


@pytest.mark.parametrize("fn", ["la_short_conv", "la_short_conv_with_state"])
def test_conv(fn):
    spans = CONV | {"out": B * N * D * 2, "S": WINDOW}
    check(fn, "x ldx w b lengths out S B N C K one dt none", spans, ["out", "S"], SIZES)


def test_conv_backward():
    spans = CONV | {"dout": B * N * D * 2, "S0": WINDOW, "dS": WINDOW, "dx": B * N * D * 2, "dw": D * K * 4, "db": D * 4,
                    "dS0": WINDOW}
    check("la_short_conv_backward", "x ldx w b lengths dout S0 dS dx dw db dS0 B N C K one dt ws bytes none", spans,
          ["dx", "dw", "db", "dS0"], SIZES)


def test_conv_step():
    spans = {"x": span(B, 2 * D, D), "w": D * K * 4, "b": D * 4, "slots": 16, "S": SLOTS * (K - 1) * D * 2, "out": B * D * 2}
    check("la_short_conv_step", "x ldx w b S slots out B n C K one dt none", spans, ["S", "out"], SIZES)


def scan_spans(rows):
    return {"x": span(rows, 2 * D, D), "dt_": span(rows, D, D), "A": D * DS * 4, "Bm": span(rows, DS, DS), "Cm": span(rows, 4 * DS, DS),
            "D": D * 4, "z": span(rows, 3 * D, D), "bias": D * 4}


SCAN = "x ldx dt_ ldt A Bm ldb Cm ldc D z ldz bias "


@pytest.mark.parametrize("fn", ["la_selective_scan", "la_selective_scan_with_state"])
def test_scan(fn):
    spans = scan_spans(B * N) | {"lengths": 16, "out": B * N * D * 2, "S": B * D * DS * 4}
    check(fn, SCAN + "lengths out S B N C ds one dt ws bytes none", spans, ["out", "S"], SIZES)


def test_scan_backward():
    rows, state = B * N * D * 2, B * D * DS * 4
    spans = scan_spans(B * N) | {"lengths": 16, "dout": rows, "S0": state, "dS": state, "dx": rows, "ddt": rows, "dA": D * DS * 4,
                                 "dB": B * N * DS * 2, "dC": B * N * DS * 2, "dD": D * 4, "dz": rows, "dbias": D * 4, "dS0": state}
    outputs = ["dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dS0"]
    names = SCAN + "lengths dout S0 dS dx ddt dA dB dC dD dz dbias dS0 B N C ds one dt ws bytes none"
    check("la_selective_scan_backward", names, spans, outputs, SIZES, allowed=[("dS0", "dS")])
    at = P + (list(spans).index("dS") << 24)
    for by in (16, -16, state - 16):  # over the upstream gradient only whole
        assert call("la_selective_scan_backward", names.split(), spans, SIZES, {"dS0": at + by}) == INVALID
    for o in outputs[:-1]:  # and then it is an output all the same
        assert call("la_selective_scan_backward", names.split(), spans, SIZES, {"dS0": at, o: at}) == INVALID


def test_scan_step():
    spans = scan_spans(B) | {"slots": 16, "S": SLOTS * D * DS * 4, "out": B * D * 2}
    check("la_selective_scan_step", SCAN + "S slots out B n C ds one dt none", spans, ["S", "out"], SIZES)


def test_beam_select():
    G, W, k, V, ld = 4, 4, 4, 100, 104
    spans = {"logits": span(G * W, ld, V), "scores": G * W * 4, "finished": G * W, "best": G * k * 4, "parents": G * k * 4,
             "tokens": G * k * 4}
    scalars = {"ld": ld, "G": G, "W": W, "k": k, "V": V, "eos": 3, "dt": 1, "ws": 1 << 20, "bytes": 1 << 40, "none": None}
    check("la_beam_select", "logits ld scores finished best parents tokens G W k V eos dt ws bytes none", spans,
          ["best", "parents", "tokens"], scalars)


def test_beam_reorder():
    G, W, n, row = 4, 4, 20, 64
    size = G * W * 4
    base = {"slots": P, "parents": P + (1 << 24), "new": P + (2 << 24)}

    def reorder(pools, **at):
        a = (ctypes.c_void_p * len(pools))(*pools)
        r = (ctypes.c_size_t * len(pools))(*[row] * len(pools))
        where = base | at
        return L.lib.la_beam_reorder(a, r, len(pools), where["slots"], where["parents"], where["new"], G, W, n, None)

    free = P + (3 << 24)
    for other in ("slots", "parents"):
        for at in (base[other], base[other] + size - 4, base[other] - size + 4):
            assert reorder([free], new=at) == INVALID
    for other in base:
        for at in (base[other], base[other] + size - 16, base[other] - n * row + 16):
            assert reorder([free, at]) == INVALID, other
