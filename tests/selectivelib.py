"""Selective scan, short convolution and beam search in 64 bits, token by token, and the error bounds of their tests.

Bounds are elementwise and come from the same recurrences, run on absolute values (U = 2^-24 is half a step of float32):

* delta = softplus(v): v is rounded once, e^-|v| is off by |v| U + 2^-22 relative, the rest by 2^-22: relative (|v| + 4) 2^-22;
* a = e^{delta A}: exponent off by delta's error and three roundings, the exponential by 2^-22: relative
  |delta A| (delta's + 2^-22) + 2^-21;
* a state carries its predecessor's error times a, plus a's error times the predecessor, plus that of delta x B (delta's
  and four roundings) and of the sum: so long products of decays are bounded step by step, not by their length;
* silu and its slope: relative (|z| + 4) 2^-21 of z sigmoid(z), or of its slope's terms;
* sums: at most 2^7 additions one behind the other: 2^-17 of the sum of absolute values;
* a result in bfloat16: one rounding, 2^-8 of its value.
"""
import torch

U, SUM, EPS16 = 2.0**-24, 2.0**-17, 2.0**-8


def silu(x):
    return x * torch.sigmoid(x)


def slope(x):
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def live_tokens(x, lengths):
    n = torch.full((x.shape[0],), x.shape[1], device=x.device) if lengths is None else lengths.long().clamp(0, x.shape[1])
    return n, torch.arange(x.shape[1], device=x.device) < n[:, None]


def make(B, N, D, ds, dt, seed, gate=True, skip=True, bias=True, state=False, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    d = {"x": r(B, N, D).to(dt), "dt": r(B, N, D).to(dt), "A": -torch.exp(r(D, ds)), "Bm": r(B, N, ds).to(dt),
         "Cm": r(B, N, ds).to(dt), "D": r(D) if skip else None, "z": (2 * r(B, N, D)).to(dt) if gate else None,
         "dt_bias": r(D) - 2 if bias else None, "softplus": True, "dout": r(B, N, D).to(dt), "S0": None, "dS": None}
    if state:
        d["S0"], d["dS"] = r(B, D, ds), r(B, D, ds)
    return d


def _terms(d, lengths):
    """delta, x, B, C, z, dout in 64 bits (padding cleared) with the relative errors of delta and the gate."""
    n, live = live_tokens(d["x"], lengths)
    f = lambda k: d[k].double().masked_fill(~live[..., None], 0)  # noqa: E731
    v = d["dt"].double() + (0 if d["dt_bias"] is None else d["dt_bias"].double())
    delta = torch.logaddexp(v, torch.zeros_like(v)) if d["softplus"] else v
    delta = delta.masked_fill(~live[..., None], 0)
    rho = (v.abs() + 4) * 2.0**-22
    return n, live, v, delta, rho, f


def scan64(d, lengths=None):
    """out, S and their bounds; rows past a length are zero.  Also everything the gradient needs."""
    n, live, v, delta, rho, f = _terms(d, lengths)
    x, Bm, Cm, A = f("x"), f("Bm"), f("Cm"), d["A"].double()
    B, N, D = x.shape
    h = torch.zeros(B, D, A.shape[1], dtype=torch.float64, device=x.device) if d["S0"] is None else d["S0"].double()
    hb, he = h.abs(), torch.zeros_like(h)
    y, yb, ye, before, kept = [], [], [], [], []
    for t in range(N):
        a = (delta[:, t, :, None] * A).exp()
        ra = (delta[:, t, :, None] * A).abs() * (rho[:, t, :, None] + 2.0**-22) + 2.0**-21
        u = (delta[:, t] * x[:, t])[..., None] * Bm[:, t, None]
        before.append((h, hb, he, a, ra))
        on = live[:, t, None, None]
        new_b = a * hb + u.abs()
        new_e = a * he + ra * a * hb + (rho[:, t, :, None] + 4 * U) * u.abs() + U * new_b
        h, hb, he = torch.where(on, a * h + u, h), torch.where(on, new_b, hb), torch.where(on, new_e, he)
        kept.append((h, hb, he))
        c = Cm[:, t, None]
        y.append((h * c).sum(-1)), yb.append((hb * c.abs()).sum(-1)), ye.append((he * c.abs()).sum(-1))
    z3 = lambda l: torch.stack(l, 1) if l else torch.zeros_like(x)  # noqa: E731
    y, yb, ye = z3(y), z3(yb), z3(ye)
    if d["D"] is not None:
        y, yb = y + d["D"].double() * x, yb + (d["D"].double() * x).abs()
    ye = ye + SUM * yb
    out, oe = y, ye
    if d["z"] is not None:
        z = f("z")
        g = silu(z)
        out, oe = y * g, (ye + (z.abs() + 4) * 2.0**-21 * yb) * g.abs()
    return out, oe, h, he, (n, live, v, delta, rho, f, y, yb, ye, before, kept)


def scan_grad64(d, lengths=None):
    """{name: (gradient, bound)} from the formulas."""
    *_, hS, heS, (n, live, v, delta, rho, f, y, yb, ye, before, kept) = scan64(d, lengths)
    x, Bm, Cm, A, do = f("x"), f("Bm"), f("Cm"), d["A"].double(), f("dout")
    B, N, D = x.shape
    dy, rz = do, 2 * U
    r = {}
    if d["z"] is not None:
        z = f("z")
        rz = (z.abs() + 4) * 2.0**-21
        dy = do * silu(z)
        s = torch.sigmoid(z)
        parts = s * (1 + z.abs() * (1 - s))  # of the slope
        r["dz"] = (do * y * slope(z), do.abs() * (ye + rz * yb) * parts)
    rz = torch.as_tensor(rz, device=x.device).expand(B, N, D) if not isinstance(rz, torch.Tensor) else rz
    R = torch.zeros_like(hS) if d["dS"] is None else d["dS"].double()
    Rb, Re = R.abs(), torch.zeros_like(R)
    zero = torch.zeros_like
    dx, dxe, dd, dde = zero(x), zero(x), zero(x), zero(x)
    dB, dBe, dC, dCe = zero(Bm), zero(Bm), zero(Cm), zero(Cm)
    dA, dAe = zero(A), zero(A)
    for t in reversed(range(N)):
        on = live[:, t, None, None]
        (h, hb, he), (h0, h0b, h0e, a, ra) = kept[t], before[t]
        cd = Cm[:, t, None] * dy[:, t, :, None]
        G, Gb = R + cd, Rb + cd.abs()
        Ge = Re + rz[:, t, :, None] * cd.abs() + U * Gb
        e = dy[:, t, :, None].abs()
        dC[:, t] = (h * dy[:, t, :, None]).sum(1)
        dCe[:, t] = ((he + (rz[:, t, :, None] + SUM) * hb) * e).sum(1)
        u = (delta[:, t] * x[:, t])[..., None]
        dB[:, t] = (G * u).sum(1)
        dBe[:, t] = ((Ge + (rho[:, t, :, None] + SUM) * Gb) * u.abs()).sum(1)
        b = Bm[:, t, None]
        s1, s1b, s1e = (G * b).sum(-1), (Gb * b.abs()).sum(-1), (Ge * b.abs()).sum(-1)
        s1e = s1e + SUM * s1b
        w, wb = G * a * h0, Gb * a * h0b
        we = Ge * a * h0b + Gb * a * (h0e + ra * h0b) + 4 * U * wb
        s2, s2b = (w * A).sum(-1), (wb * A.abs()).sum(-1)
        s2e = (we * A.abs()).sum(-1) + SUM * s2b
        dt_ = delta[:, t]
        dx[:, t], dxe[:, t] = dt_ * s1, dt_.abs() * (s1e + (rho[:, t] + 2 * U) * s1b)
        dd[:, t] = x[:, t] * s1 + s2
        dde[:, t] = x[:, t].abs() * s1e + s2e + SUM * (x[:, t].abs() * s1b + s2b)
        dA += (w * dt_[..., None]).sum(0)
        dAe += ((we + (rho[:, t, :, None] + SUM) * wb) * dt_[..., None].abs()).sum(0)
        R, Rb = torch.where(on, a * G, R), torch.where(on, a * Gb, Rb)
        Re = torch.where(on, a * Ge + ra * a * Gb + U * a * Gb, Re)
    if d["D"] is not None:
        k = d["D"].double()
        dx, dxe = dx + k * dy, dxe + (k * dy).abs() * (rz + 4 * U)
        r["dD"] = ((dy * x).sum((0, 1)), ((rz + SUM) * (dy * x).abs()).sum((0, 1)))
    sig = torch.sigmoid(v) if d["softplus"] else torch.ones_like(v)
    ddt, ddte = dd * sig, (dde + (v.abs() + 4) * 2.0**-21 * dd.abs()) * sig
    ddt, ddte = (q.masked_fill(~live[..., None], 0) for q in (ddt, ddte))
    r |= {"dx": (dx, dxe), "ddt": (ddt, ddte), "dA": (dA, dAe), "dB": (dB, dBe), "dC": (dC, dCe), "dS0": (R, Re)}
    if d["dt_bias"] is not None:
        r["ddt_bias"] = (ddt.sum((0, 1)), (ddte + SUM * ddt.abs()).sum((0, 1)))
    return r


def within(got, ref, bound, name):
    assert got.shape == ref.shape, f"{name}: {tuple(got.shape)} for {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{name}: not finite"
    tol = bound + (EPS16 * (ref.abs() + bound) if got.dtype == torch.bfloat16 else 2 * U * ref.abs()) + 1e-36
    off = (got.double() - ref).abs() - tol
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{name}: {worst:.3g} beyond the bound (rms {ref.square().mean().sqrt().item():.3g})"


# ---- short convolution ---------------------------------------------------------------------------------------------
def make_conv(B, N, D, K, dt, seed, bias=True, state=False, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    d = {"x": r(B, N, D).to(dt), "w": r(D, K), "b": r(D) if bias else None, "silu": True, "dout": r(B, N, D).to(dt),
         "S0": None, "dS": None}
    if state:
        d["S0"], d["dS"] = r(B, K - 1, D).to(dt), r(B, K - 1, D).to(dt)
    return d


def conv64(d, lengths=None):
    """out, bound, S; and the padded inputs, u and its bound."""
    n, live = live_tokens(d["x"], lengths)
    x = d["x"].double().masked_fill(~live[..., None], 0)
    w, (B, N, D) = d["w"].double(), x.shape
    K = w.shape[1]
    S0 = torch.zeros(B, K - 1, D, dtype=torch.float64, device=x.device) if d["S0"] is None else d["S0"].double()
    xp = torch.cat([S0, x], 1)
    b = 0 if d["b"] is None else d["b"].double()
    u = sum((xp[:, j : j + N] * w[:, j] for j in range(K)), torch.zeros_like(x)) + b
    ub = sum((xp[:, j : j + N] * w[:, j]).abs() for j in range(K)) + (b.abs() if d["b"] is not None else 0)
    ue = (K + 1) * U * ub
    out, oe = u, ue
    if d["silu"]:  # |slope| <= 1.1
        out, oe = silu(u), 1.1 * ue + (u.abs() + 4) * 2.0**-21 * silu(u).abs()
    at = n[:, None] + torch.arange(K - 1, device=x.device)
    S = xp.gather(1, at[..., None].expand(-1, -1, D))
    mask = lambda t: t.masked_fill(~live[..., None], 0)  # noqa: E731
    return mask(out), mask(oe), S, (n, live, xp, u, ue)


def conv_grad64(d, lengths=None):
    _, _, _, (n, live, xp, u, ue) = conv64(d, lengths)
    w = d["w"].double()
    N, K = u.shape[1], w.shape[1]
    do = d["dout"].double().masked_fill(~live[..., None], 0)
    g, ge = do, torch.zeros_like(do)
    if d["silu"]:  # |the slope's derivative| <= 1/2
        s = torch.sigmoid(u)
        g, ge = do * slope(u), do.abs() * (ue / 2 + (u.abs() + 4) * 2.0**-21 * s * (1 + u.abs() * (1 - s)))
    dp, de = torch.zeros_like(xp), torch.zeros_like(xp)
    for j in range(K):
        dp[:, j : j + N] += g * w[:, j]
        de[:, j : j + N] += (ge + (K + 1) * U * g.abs()) * w[:, j].abs()
    if d["dS"] is not None:
        at = (n[:, None] + torch.arange(K - 1, device=u.device))[..., None].expand(-1, -1, u.shape[2])
        dp.scatter_add_(1, at, d["dS"].double())
        de.scatter_add_(1, at, U * d["dS"].double().abs())
    pad = lambda t: t.masked_fill(~live[..., None], 0)  # noqa: E731
    wins = [xp[:, j : j + N] for j in range(K)]
    dw = torch.stack([(g * q).sum((0, 1)) for q in wins], 1)
    dwe = torch.stack([((ge + SUM * g.abs()) * q.abs()).sum((0, 1)) for q in wins], 1)
    return {"dx": (pad(dp[:, K - 1 :]), pad(de[:, K - 1 :])), "dw": (dw, dwe),
            "db": (g.sum((0, 1)), (ge + SUM * g.abs()).sum((0, 1))), "dS0": (dp[:, : K - 1], de[:, : K - 1])}


# ---- beam search -----------------------------------------------------------------------------------------------------
def select64(logits, scores, k, finished=None, eos=0):
    """(scores, parents, tokens) by a stable sort of all continuations in 64 bits."""
    G, W, V = logits.shape
    x = logits.double()
    x = torch.where(x.isnan(), -torch.inf, x).clamp(max=torch.finfo(torch.float32).max)
    top = x.amax(-1, keepdim=True)
    x = x - torch.where(top == -torch.inf, 0.0, top)
    # (rows of whole kilobytes: equal rows have equal sums then, whatever order the library adds them in)
    x = x - torch.nn.functional.pad(x, (0, -V % 128), value=-torch.inf).exp().sum(-1, keepdim=True).log()
    s = scores.double()[..., None]
    s = torch.where(s.isnan(), -torch.inf, s)
    x = torch.where(x.isnan(), -torch.inf, x)
    total = s + x
    if finished is not None:
        only = torch.full((V,), -torch.inf, dtype=torch.float64, device=x.device)
        only[eos] = 0
        total = torch.where(finished[..., None], s + only, total)
    best, at = torch.sort(total.reshape(G, W * V), dim=-1, descending=True, stable=True)
    return best[:, :k], (at[:, :k] // V).int(), (at[:, :k] % V).int()


def reorder_slots(slots, parents):
    """New slots and the copies (from, to), in plain Python."""
    new, moves = [], []
    for have, of in zip(slots.tolist(), parents.tolist()):
        free, seen, row = [have[w] for w in range(len(have)) if w not in of], set(), []
        for p in of:
            ok = 0 <= p < len(have)
            if ok and p not in seen:
                row.append(have[p])
                seen.add(p)
            else:
                row.append(free.pop(0))
                if ok:
                    moves.append((have[p], row[-1]))
        new.append(row)
    return new, moves
