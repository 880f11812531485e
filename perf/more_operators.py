"""Workloads of the selective state space layer and of beam search over its states, with their plain forms.

Each case is one call of one operator (``beam`` makes the two calls of one beam search step).  ``run`` computes it in a
plain form (elementary torch operations in 32 bits, scores of beams in 64) or, with ``own`` set, through the library's
entry points.  Sizes follow the repository's configurations: 4 x 8192 tokens, 16 x 128 = 2048 channels, batches of 256.

Short convolution: u_t = bias + sum_{j<K} w_j x_{t-K+1+j} per channel, y = silu(u).
Selective scan: delta = softplus(dt + dt_bias), h_t = e^{delta A} h_{t-1} + delta x_t B_t, out = (C_t . h_t + D x_t) silu(z).
Beam selection: the k best of a group's W x V continuations by score + log-softmax(logits), ties to the lowest index.
Reordering: a beam's first child keeps its state's slot, the other children get copies in the slots that became free.
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # prompt processing of a batch of full-length prompts
        {"name": "scan_prefill_bf16", "op": "scan", "B": 4, "N": 8192, "D": 2048, "ds": 16, "dt": "bf16", "ragged": False,
         "state": False, "gate": True},
        # one long prompt of odd length that continues a cached state: few channels, many tokens
        {"name": "scan_long_state_bf16", "op": "scan", "B": 1, "N": 32749, "D": 1024, "ds": 16, "dt": "bf16",
         "ragged": False, "state": True, "gate": True},
        # a short prompt, 32-bit, where latency counts
        {"name": "scan_small_f32", "op": "scan", "B": 1, "N": 100, "D": 128, "ds": 8, "dt": "f32", "ragged": False,
         "state": False, "gate": False},
        # training step of the layer
        {"name": "scan_grad_bf16", "op": "scan_grad", "B": 4, "N": 4096, "D": 2048, "ds": 16, "dt": "bf16",
         "ragged": False, "state": False, "gate": True},
        # padded batch of odd sizes with a carried state (training in chunks), 32-bit
        {"name": "scan_grad_padded_f32", "op": "scan_grad", "B": 4, "N": 1021, "D": 520, "ds": 32, "dt": "f32",
         "ragged": True, "state": True, "gate": True},
        # one token for each served sequence
        {"name": "scan_step", "op": "scan_step", "B": 512, "D": 2048, "ds": 16, "dt": "bf16", "slots": 544},
        # the convolution in front of the scan: prompts, training, serving
        {"name": "conv_prefill_bf16", "op": "conv", "B": 4, "N": 8192, "D": 2048, "K": 4, "dt": "bf16", "ragged": True,
         "state": True},
        {"name": "conv_grad_bf16", "op": "conv_grad", "B": 4, "N": 8192, "D": 2048, "K": 4, "dt": "bf16", "ragged": False,
         "state": False},
        {"name": "conv_step", "op": "conv_step", "B": 256, "D": 2048, "K": 4, "dt": "bf16", "slots": 256},
        # the largest selection: many groups over a large vocabulary
        {"name": "select_bf16", "op": "select", "G": 64, "W": 8, "k": 8, "V": 131072, "dt": "bf16", "finished": False},
        # states of several layers follow their beams
        {"name": "reorder", "op": "reorder", "G": 64, "W": 8, "distinct": 5, "layers": 4, "D": 2048, "ds": 16, "K": 4,
         "slots": 544},
        # a whole beam search step of one sequence: selection and reordering, where latency counts
        {"name": "beam_small_f32", "op": "beam", "G": 1, "W": 4, "V": 32003, "dt": "f32", "finished": True, "layers": 2,
         "D": 512, "ds": 16, "K": 4, "slots": 6},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "scan_step", "conv", "conv_grad", "conv_step", "select",
                     "select", "reorder", "beam"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    D = 8 * _log_int(rng, 1, 256)
    ds = rng.choice([8, 16, 16, 32, 64])
    if op in ("scan", "scan_grad"):
        B = _log_int(rng, 1, 8)
        most = (4e8 if op == "scan" else 1.5e8) / (B * D * ds)
        return {"op": op, "B": B, "N": _log_int(rng, 1, max(2, min(int(most), 16384))), "D": D, "ds": ds, "dt": dt,
                "ragged": rng.random() < 0.4, "state": rng.random() < 0.5, "gate": rng.random() < 0.75}
    if op in ("conv", "conv_grad"):
        B = _log_int(rng, 1, 8)
        return {"op": op, "B": B, "N": _log_int(rng, 1, max(2, min(int(3e7 / (B * D)), 16384))), "D": D,
                "K": rng.choice([2, 3, 4]), "dt": dt, "ragged": rng.random() < 0.4, "state": rng.random() < 0.5}
    if op == "scan_step":
        B = _log_int(rng, 1, 256)
        return {"op": op, "B": B, "D": D, "ds": ds, "dt": dt, "slots": B + rng.randrange(0, 32)}
    if op == "conv_step":
        B = _log_int(rng, 1, 256)
        return {"op": op, "B": B, "D": D, "K": rng.choice([2, 3, 4]), "dt": dt, "slots": B + rng.randrange(0, 32)}
    G, W = _log_int(rng, 1, 48), _log_int(rng, 1, 16)
    V = _log_int(rng, 32, min(131072, int(3e7 / (G * W))))
    if op == "select":
        return {"op": op, "G": G, "W": W, "k": rng.choice([W, W, 2 * W, 1]), "V": V, "dt": dt,
                "finished": rng.random() < 0.5}
    slots = G * W + rng.randrange(0, 16)
    layers = _log_int(rng, 1, 4)
    D = min(D, 1024)
    if op == "reorder":
        return {"op": op, "G": G, "W": W, "distinct": rng.randint(1, W), "layers": layers, "D": D, "ds": ds, "K": 4,
                "slots": slots}
    return {"op": op, "G": G, "W": W, "V": V, "dt": dt, "finished": rng.random() < 0.5, "layers": layers, "D": D,
            "ds": 16, "K": 4, "slots": slots}


def _inputs(case, seed, device):
    """Projections' outputs ~ N(0, 1), steps delta around 1e-3 to 1e-1, A near -(1 .. ds), logits of a peaked softmax."""
    g = torch.Generator(device=device).manual_seed(int(seed) * 7919 + 29)
    op = case["op"]
    randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device=device)  # noqa: E731
    s = {"case": case}
    if op in ("select", "beam", "reorder"):
        G, W = case["G"], case["W"]
        if op != "reorder":
            s["logits"] = (3 * randn(G, W, case["V"])).to(DTYPES[case["dt"]])
            s["logits"][:, :, case["V"] // 3] = -math.inf  # a token that is never allowed
            s["scores"] = -20 * rand(G, W)
            s["eos"] = case["V"] - 1
            s["finished"] = rand(G, W) < 0.2 if case["finished"] else None
            s["k"] = case.get("k", W)
            if op == "select":
                return s
        else:  # `distinct` beams of each group survive, in random numbers and order
            alive = rand(G, W).argsort(-1)[:, : case["distinct"]]
            more = torch.randint(case["distinct"], (G, W - case["distinct"]), generator=g, device=device)
            of = torch.cat([alive, alive.gather(1, more)], 1).gather(1, rand(G, W).argsort(-1))
            s["parents"] = of.to(torch.int32).contiguous()
        s["slots"] = torch.randperm(case["slots"], generator=g, device=device)[: G * W].reshape(G, W).to(torch.int32)
        s["pools"] = []
        for _ in range(case["layers"]):
            s["pools"].append(randn(case["slots"], case["K"] - 1, case["D"]).to(torch.bfloat16))
            s["pools"].append(randn(case["slots"], case["D"], case["ds"]))
        return s
    dt, B, D = DTYPES[case["dt"]], case["B"], case["D"]
    lead = (B,) if op.endswith("step") else (B, case["N"])
    if op.startswith("conv"):
        K = case["K"]
        s["x"] = randn(*lead, 2 * D).to(dt)[..., :D]  # one half of the layer's input projection
        s["w"], s["b"] = randn(D, K) * K ** -0.5, 0.1 * randn(D)
        if op == "conv_grad":
            s["dout"] = randn(*lead, D).to(dt)
    else:
        ds = case["ds"]
        r = max(8, D // 16 // 8 * 8)
        low = randn(*lead, r + 2 * ds).to(dt)  # dt's factor, B and C come from one projection
        s["Bm"], s["Cm"] = low[..., r : r + ds], low[..., r + ds :]
        s["x"] = torch.nn.functional.silu(randn(*lead, D)).to(dt)
        s["dt"] = (0.5 * randn(*lead, D)).to(dt)
        step = torch.exp(rand(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
        s["A"] = -torch.exp(torch.log(torch.arange(1, ds + 1, device=device).float()) + 0.1 * randn(D, ds))
        s["D"] = 1 + 0.1 * randn(D)
        s["z"] = randn(*lead, 2 * D).to(dt)[..., D:] if case.get("gate", True) else None
        if op == "scan_grad":
            s["dout"] = randn(*lead, D).to(dt)
    if op.endswith("step"):
        s["slots"] = torch.randperm(case["slots"], generator=g, device=device)[:B].to(torch.int32)
        s["S"] = randn(case["slots"], D, case["ds"]) if op == "scan_step" else randn(case["slots"], case["K"] - 1, D).to(dt)
        return s
    N = case["N"]
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(N // 2, N + 1, (B,), generator=g, device=device, dtype=torch.int32)
        n[0] = N
        if B > 2:
            n[B - 1] = 0
        s["lengths"] = n
    shape = (B, case["K"] - 1, D) if op.startswith("conv") else (B, D, case["ds"])
    like = dt if op.startswith("conv") else torch.float32
    s["S0"] = randn(*shape).to(like) if case["state"] else None
    if op.endswith("grad"):
        s["dS"] = randn(*shape).to(like) if case["state"] else None
    else:
        s["out"] = torch.zeros(B, N, D, dtype=dt, device=device)  # rows past a sequence's end are left as they are
        s["S"] = torch.empty(shape, dtype=like, device=device)
    return s


def prepare(case, seed):
    return _inputs(case, seed, "cuda")


# --------------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------------
def _live(s, like):
    """Which tokens count, [B, N, 1], or None."""
    if s["lengths"] is None:
        return None
    return (torch.arange(like.shape[1], device=like.device) < s["lengths"][:, None])[..., None]


def _keep(live, x):
    return x if live is None else torch.where(live, x, torch.zeros_like(x))


def _silu(x):
    return x * torch.sigmoid(x)


def _silu_slope(x):
    e = torch.sigmoid(x)
    return e * (1 + x * (1 - e))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _window(s):
    """The inputs in 32 bits with the K - 1 before them: [B, N + K - 1, D]."""
    x = _keep(_live(s, s["x"]), s["x"].float())
    K = s["w"].shape[1]
    before = x.new_zeros(x.shape[0], K - 1, x.shape[2]) if s["S0"] is None else s["S0"].float()
    return torch.cat([before, x], 1)


def _ends(s):
    N = s["x"].shape[1]
    return torch.full((s["x"].shape[0],), N, device=s["x"].device) if s["lengths"] is None else s["lengths"].long()


def _plain_conv(s):
    xp, K, N = _window(s), s["w"].shape[1], s["x"].shape[1]
    u = s["b"] + sum(xp[:, j : j + N] * s["w"][:, j] for j in range(K))
    live = _live(s, s["x"])
    y = _silu(u)
    s["out"].copy_(y if live is None else torch.where(live, y, s["out"].float()))
    at = _ends(s)[:, None] + torch.arange(K - 1, device=xp.device)
    s["S"].copy_(xp.gather(1, at[..., None].expand(-1, -1, xp.shape[2])))
    return {"out": s["out"], "S": s["S"]}


def _plain_conv_grad(s):
    xp, K, N, dt = _window(s), s["w"].shape[1], s["x"].shape[1], s["x"].dtype
    live = _live(s, s["x"])
    u = s["b"] + sum(xp[:, j : j + N] * s["w"][:, j] for j in range(K))
    g = _keep(live, s["dout"].float() * _silu_slope(u))
    d = torch.zeros_like(xp)
    for j in range(K):
        d[:, j : j + N] += g * s["w"][:, j]
    if s["dS"] is not None:
        at = _ends(s)[:, None] + torch.arange(K - 1, device=xp.device)
        d.scatter_add_(1, at[..., None].expand(-1, -1, xp.shape[2]), s["dS"].float())
    dw = torch.stack([(g * xp[:, j : j + N]).sum((0, 1), dtype=torch.float64) for j in range(K)], 1).float()
    r = {"dx": _keep(live, d[:, K - 1 :]).to(dt), "dw": dw, "db": g.sum((0, 1), dtype=torch.float64).float()}
    if s["S0"] is not None:
        r["dS0"] = d[:, : K - 1].to(dt)
    return r


def _plain_conv_step(s):
    at = s["slots"].long()
    rows = torch.cat([s["S"][at].float(), s["x"].float()[:, None]], 1)  # [B, K, D]
    s["S"][at] = rows[:, 1:].to(s["S"].dtype)
    return {"out": _silu(s["b"] + (rows * s["w"].T).sum(1)).to(s["x"].dtype), "S": s["S"]}


def _terms(s):
    """delta, its argument, and the inputs in 32 bits with padding tokens cleared."""
    live = _live(s, s["x"])
    arg = s["dt"].float() + s["dt_bias"]
    f = lambda n: _keep(live, s[n].float())  # noqa: E731
    return live, arg, _keep(live, _softplus(arg)), f("x"), f("Bm"), f("Cm")


def _scan_chunk(a, b, h):
    """All states h_t = a_t h_{t-1} + b_t of a chunk [B, T, D, ds], by doubling."""
    b = torch.cat([(a[:, :1] * h[:, None] + b[:, :1]), b[:, 1:]], 1)
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], a[:, d:] * b[:, :-d] + b[:, d:]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _plain_scan(s):
    live, _, delta, x, Bm, Cm = _terms(s)
    N, ds = x.shape[1], Bm.shape[2]
    h = x.new_zeros(x.shape[0], x.shape[2], ds) if s["S0"] is None else s["S0"]
    y = torch.empty_like(x)
    for t in range(0, N, CHUNK):
        c = slice(t, t + CHUNK)
        a = torch.exp(delta[:, c, :, None] * s["A"])
        hs = _scan_chunk(a, (delta[:, c] * x[:, c])[..., None] * Bm[:, c, None, :], h)
        y[:, c] = (hs * Cm[:, c, None, :]).sum(-1)
        h = hs[:, -1]
    y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["out"].copy_(y if live is None else torch.where(live, y, s["out"].float()))
    s["S"].copy_(h)
    return {"out": s["out"], "S": s["S"]}


def _plain_scan_grad(s):
    live, arg, delta, x, Bm, Cm = _terms(s)
    N, ds, dt = x.shape[1], Bm.shape[2], s["x"].dtype
    dout = _keep(live, s["dout"].float())
    z = None if s["z"] is None else _keep(live, s["z"].float())
    dy = dout if z is None else dout * _silu(z)
    zero = x.new_zeros(x.shape[0], x.shape[2], ds)
    starts, h = [], zero if s["S0"] is None else s["S0"]
    for t in range(0, N, CHUNK):  # the state in front of each chunk
        c = slice(t, t + CHUNK)
        starts.append(h)
        a = torch.exp(delta[:, c, :, None] * s["A"])
        h = _scan_chunk(a, (delta[:, c] * x[:, c])[..., None] * Bm[:, c, None, :], h)[:, -1]
    G = zero if s["dS"] is None else s["dS"]  # gradient of the state behind the chunk
    y, dx, dd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dB, dC, dA = torch.empty_like(Bm), torch.empty_like(Cm), torch.zeros_like(s["A"], dtype=torch.float64)
    for i in reversed(range(len(starts))):
        c = slice(i * CHUNK, (i + 1) * CHUNK)
        a = torch.exp(delta[:, c, :, None] * s["A"])
        u = (delta[:, c] * x[:, c])[..., None]
        h = _scan_chunk(a, u * Bm[:, c, None, :], starts[i])
        y[:, c] = (h * Cm[:, c, None, :]).sum(-1)
        dC[:, c] = (h * dy[:, c, :, None]).sum(2)
        before = a * torch.cat([starts[i][:, None], h[:, :-1]], 1)
        # the same recurrence from the end: G_t = C_t dy_t + a_{t+1} G_{t+1}
        later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        g = _scan_chunk(later.flip(1), (Cm[:, c, None, :] * dy[:, c, :, None]).flip(1), G).flip(1)
        dB[:, c] = (g * u).sum(2)
        s1 = (g * Bm[:, c, None, :]).sum(-1)
        w = g * before
        dx[:, c] = delta[:, c] * s1
        dd[:, c] = x[:, c] * s1 + (w * s["A"]).sum(-1)
        dA += (w * delta[:, c, :, None]).sum((0, 1), dtype=torch.float64)
        G = a[:, 0] * g[:, 0]
    dx = dx + s["D"] * dy
    ddt = _keep(live, dd * torch.sigmoid(arg))
    r = {"dx": dx.to(dt), "ddt": ddt.to(dt), "dA": dA.float(), "dB": dB.to(dt), "dC": dC.to(dt),
         "dD": (dy * x).sum((0, 1), dtype=torch.float64).float()}
    if z is not None:
        r["dz"] = (dout * (y + s["D"] * x) * _silu_slope(z)).to(dt)
    r["ddt_bias"] = ddt.sum((0, 1), dtype=torch.float64).float()
    if s["S0"] is not None:
        r["dS0"] = G
    return r


def _plain_scan_step(s):
    at, x = s["slots"].long(), s["x"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["A"]) * s["S"][at] + (delta * x)[..., None] * s["Bm"].float()[:, None]
    s["S"][at] = h
    y = (h * s["Cm"].float()[:, None]).sum(-1) + s["D"] * x
    return {"out": (y * _silu(s["z"].float())).to(s["x"].dtype), "S": s["S"]}


def _plain_select(s):
    x = s["logits"].double()  # scores next to one another decide: 64 bits
    G, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    x = x - top
    x = s["scores"].double()[..., None] + (x - x.exp().sum(-1, keepdim=True).log())
    if s["finished"] is not None:  # a finished beam has one continuation, at no cost
        only = torch.full((V,), -math.inf, dtype=x.dtype, device=x.device)
        only[s["eos"]] = 0
        x = torch.where(s["finished"][..., None], s["scores"].double()[..., None] + only, x)
    best, at = torch.sort(x.reshape(G, W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, : s["k"]], at[:, : s["k"]]
    return {"scores": best.float(), "parents": (at // V).to(torch.int32), "tokens": (at % V).to(torch.int32)}


def _plain_reorder(s, parents):
    p, slots = parents.long(), s["slots"].long()
    W = p.shape[1]
    same = p[:, :, None] == p[:, None, :]
    first = ~(same & torch.ones(W, W, dtype=torch.bool, device=p.device).tril(-1)).any(-1)  # no earlier child of it
    has = (p[:, None, :] == torch.arange(W, device=p.device)[:, None]).any(-1)
    free = torch.sort(has.int(), dim=-1, stable=True).indices  # childless beams in order, then the others
    rank = (~first).int().cumsum(-1) - 1
    to = torch.where(first, slots.gather(1, p), slots.gather(1, free.gather(1, rank.clamp(min=0))))
    src, dst = slots.gather(1, p).flatten(), to.flatten()  # a kept row is copied to itself
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return {"slots": to.to(torch.int32), "pools": s["pools"]}


def _plain_beam(s):
    r = _plain_select(s)
    return r | _plain_reorder(s, r["parents"])


# --------------------------------------------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------------------------------------------
def _own(s):
    from causal_linear_attention_attn_gb300 import linattn as L

    op = s["case"]["op"]
    if op == "conv":
        if s["S0"] is None:
            L.la_short_conv(s["x"], s["w"], bias=s["b"], lengths=s["lengths"], out=s["out"], S=s["S"])
        else:
            s["S"].copy_(s["S0"])
            L.la_short_conv_with_state(s["x"], s["w"], s["S"], bias=s["b"], lengths=s["lengths"], out=s["out"])
        return {"out": s["out"], "S": s["S"]}
    if op == "conv_grad":
        r = L.la_short_conv_backward(s["x"], s["w"], s["dout"], bias=s["b"], S0=s["S0"], dS=s["dS"], lengths=s["lengths"],
                                     need_state_grad=s["S0"] is not None)
        return dict(zip(("dx", "dw", "db", "dS0"), r))
    if op == "conv_step":
        return {"out": L.la_short_conv_step(s["x"], s["w"], s["S"], bias=s["b"], slots=s["slots"]), "S": s["S"]}
    if op == "scan":
        kw = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "lengths": s["lengths"], "out": s["out"], "S": s["S"]}
        if s["S0"] is None:
            L.la_selective_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], **kw)
        else:
            s["S"].copy_(s["S0"])
            L.la_selective_scan_with_state(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], **kw)
        return {"out": s["out"], "S": s["S"]}
    if op == "scan_grad":
        r = L.la_selective_scan_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dout"], D=s["D"], z=s["z"],
                                         dt_bias=s["dt_bias"], S0=s["S0"], dS=s["dS"], lengths=s["lengths"],
                                         need_state_grad=s["S0"] is not None)
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")
        return {k: x for k, x in zip(names, r) if x is not None}
    if op == "scan_step":
        out = L.la_selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], D=s["D"], z=s["z"],
                                       dt_bias=s["dt_bias"], slots=s["slots"])
        return {"out": out, "S": s["S"]}
    r = {}
    parents = s.get("parents")
    if op != "reorder":
        best, parents, tokens = L.la_beam_select(s["logits"], s["scores"], k=s["k"], finished=s["finished"], eos=s["eos"])
        r = {"scores": best, "parents": parents, "tokens": tokens}
    if op != "select":
        r |= {"slots": L.la_beam_reorder(s["pools"], s["slots"], parents), "pools": s["pools"]}
    return r


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "reorder":
        return _plain_reorder(state, state["parents"])
    return {"conv": _plain_conv, "conv_grad": _plain_conv_grad, "conv_step": _plain_conv_step, "scan": _plain_scan,
            "scan_grad": _plain_scan_grad, "scan_step": _plain_scan_step, "select": _plain_select,
            "beam": _plain_beam}[op](state)


def work(case):
    op = case["op"]
    if op in ("select", "beam", "reorder"):
        G, W = case["G"], case["W"]
        r = {"bytes": 0, "flops": 0}
        if op != "reorder":
            e = 2 if case["dt"] == "bf16" else 4
            r = {"bytes": G * W * (e * case["V"] + 4) + 12 * G * case.get("k", W), "flops": 3 * G * W * case["V"]}
        if op != "select":
            row = case["layers"] * case["D"] * (2 * (case["K"] - 1) + 4 * case["ds"])
            # of independent children about (1 - 1/W)^W beams of a group have none
            copies = G * (W - case["distinct"]) if op == "reorder" else G * W * (1 - 1 / W) ** W
            r["bytes"] += 2 * copies * row + 12 * G * W
        return r
    e = 2 if case["dt"] == "bf16" else 4
    B, D = case["B"], case["D"]
    if op == "conv_step":
        return {"bytes": B * D * e * 2 * case["K"] + 4 * D * (case["K"] + 1), "flops": B * D * (2 * case["K"] + 6)}
    if op == "scan_step":
        ds = case["ds"]
        return {"bytes": B * (8 * D * ds + e * (4 * D + 2 * ds) + 4) + 4 * D * (ds + 2), "flops": B * D * (7 * ds + 20)}
    tokens = B * case["N"] * (0.7 if case["ragged"] and B > 2 else 0.85 if case["ragged"] else 1.0)
    grad = op.endswith("grad")
    if op.startswith("conv"):
        K = case["K"]
        state = B * (K - 1) * D * e
        extra = 4 * D * (K + 1) * (2 if grad else 1) + state * (3 * case["state"] if grad else 1 + case["state"])
        return {"bytes": tokens * D * e * (3 if grad else 2) + extra, "flops": tokens * D * (6 * K + 12 if grad else 2 * K + 6)}
    ds, gate = case["ds"], case["gate"]
    state = 4 * B * D * ds
    if not grad:
        return {"bytes": tokens * e * ((3 + gate) * D + 2 * ds) + state * (1 + case["state"]) + 4 * D * (ds + 2),
                "flops": tokens * D * (7 * ds + 20)}
    return {"bytes": tokens * e * ((5 + 2 * gate) * D + 4 * ds) + 3 * state * case["state"] + 8 * D * (ds + 2),
            "flops": tokens * D * (24 * ds + 40)}


# --------------------------------------------------------------------------------------------------------------
# 64 bits, token by token from the definitions
# --------------------------------------------------------------------------------------------------------------
def _exact_scan(s, states=False):
    d = lambda n: s[n].double()  # noqa: E731
    x, A, Bm, Cm = d("x"), d("A"), d("Bm"), d("Cm")
    delta = torch.logaddexp(d("dt") + d("dt_bias"), torch.zeros((), dtype=torch.float64, device=x.device))
    if s["lengths"] is not None:
        past = torch.arange(x.shape[1], device=x.device)[None] >= s["lengths"][:, None]
        delta, x = delta.masked_fill(past[..., None], 0), x.masked_fill(past[..., None], 0)
        Bm, Cm = Bm.masked_fill(past[..., None], 0), Cm.masked_fill(past[..., None], 0)
    h = torch.zeros(x.shape[0], *A.shape, dtype=torch.float64, device=x.device) if s["S0"] is None else d("S0")
    rows, kept = [], []
    for t in range(x.shape[1]):
        if states:
            kept.append(h)
        h = h * (delta[:, t, :, None] * A).exp() + (delta[:, t] * x[:, t])[..., None] * Bm[:, t, None]
        rows.append((h @ Cm[:, t, :, None])[..., 0])
    return torch.stack(rows, 1) + d("D") * x, h, kept, (delta, x, A, Bm, Cm)


def _exact_scan_grad(s):
    y, h, kept, (delta, x, A, Bm, Cm) = _exact_scan(s, states=True)
    d = lambda n: s[n].double()  # noqa: E731
    past = None
    if s["lengths"] is not None:
        past = (torch.arange(x.shape[1], device=x.device)[None] >= s["lengths"][:, None])[..., None]
    do = d("dout") if past is None else d("dout").masked_fill(past, 0)
    dy, r = do, {}
    if s["z"] is not None:
        z = d("z")
        e = (-z).exp()
        dy = do * z / (1 + e)
        r["dz"] = do * y * (1 + e + z * e) / (1 + e).square()
    R = torch.zeros_like(h) if s["dS"] is None else d("dS")
    dx, dd, dB, dC, dA = (torch.zeros_like(t) for t in (x, x, Bm, Cm, A))
    for t in reversed(range(x.shape[1])):
        R = R + dy[:, t, :, None] * Cm[:, t, None]
        dC[:, t] = torch.einsum("bdn,bd->bn", h, dy[:, t])
        dB[:, t] = torch.einsum("bdn,bd->bn", R, delta[:, t] * x[:, t])
        RB = torch.einsum("bdn,bn->bd", R, Bm[:, t])
        dx[:, t] = delta[:, t] * RB
        h = kept[t]
        R = R * (delta[:, t, :, None] * A).exp()
        dd[:, t] = x[:, t] * RB + (R * h * A).sum(-1)
        dA += (R * h * delta[:, t, :, None]).sum(0)
    ddt = dd / (1 + (-(d("dt") + d("dt_bias"))).exp())
    if past is not None:
        ddt = ddt.masked_fill(past, 0)
    r |= {"dx": dx + d("D") * dy, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (dy * x).sum((0, 1)),
          "ddt_bias": ddt.sum((0, 1))}
    if s["S0"] is not None:
        r["dS0"] = R
    return r


def _exact_conv(s, grad):
    w, b, x = s["w"].double(), s["b"].double(), s["x"].double()
    B, N, D = x.shape
    K = w.shape[1]
    n = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    S0 = torch.zeros(B, K - 1, D, dtype=torch.float64, device=x.device) if s["S0"] is None else s["S0"].double()
    zeros = torch.zeros_like
    out, S, dx, dw, db, dS0 = zeros(x), zeros(S0), zeros(x), zeros(w), zeros(b), zeros(S0)
    for i in range(B):
        seq = torch.cat([S0[i], x[i, : n[i]]]).T[:, None]  # [D, 1, K - 1 + n]
        S[i] = seq[:, 0, n[i] :].T
        dseq = zeros(seq)
        if n[i]:
            view = seq[:, 0].unfold(-1, K, 1)  # [D, n, K]
            u = (view * w[:, None]).sum(-1) + b[:, None]
            e = (-u).exp()
            out[i, : n[i]] = (u / (1 + e)).T
            if grad:
                g = s["dout"][i, : n[i]].double().T * (1 + e + u * e) / (1 + e).square()
                dw += (view * g[..., None]).sum(1)
                db += g.sum(1)
                for t in range(K):
                    dseq[:, 0, t : t + n[i]] += g * w[:, t : t + 1]
        if grad:
            if s["dS"] is not None:
                dseq[:, 0, n[i] :] += s["dS"][i].double().T
            dS0[i], dx[i, : n[i]] = dseq[:, 0, : K - 1].T, dseq[:, 0, K - 1 :].T
    if not grad:
        return {"out": out, "S": S}
    return {"dx": dx, "dw": dw, "db": db} | ({"dS0": dS0} if s["S0"] is not None else {})


def _exact_select(s):
    G, W, V = s["logits"].shape
    scores, parents, tokens = [], [], []
    for i in range(G):
        x = torch.log_softmax(s["logits"][i].double(), -1) + s["scores"][i].double()[:, None]
        if s["finished"] is not None:
            for w in s["finished"][i].nonzero()[:, 0].tolist():
                x[w] = -math.inf
                x[w, s["eos"]] = s["scores"][i, w].double()
        x = x.flatten()
        least = x.topk(s["k"]).values[-1]
        among = (x >= least).nonzero()[:, 0].tolist()  # all that could be chosen, ties to the lowest place
        vals = x[x >= least].tolist()
        order = sorted(range(len(among)), key=lambda j: (-vals[j], among[j]))[: s["k"]]
        scores.append([vals[j] for j in order])
        parents.append([among[j] // V for j in order])
        tokens.append([among[j] % V for j in order])
    t = lambda v, dt: torch.tensor(v, dtype=dt, device=s["logits"].device)  # noqa: E731
    return {"scores": t(scores, torch.float64), "parents": t(parents, torch.int32), "tokens": t(tokens, torch.int32)}


def _exact_reorder(s, parents):
    slots, moves = s["slots"].tolist(), []
    new = []
    for have, of in zip(slots, parents.tolist()):
        free = [have[w] for w in range(len(have)) if w not in of]
        seen, row = set(), []
        for p in of:
            row.append(free.pop(0) if p in seen else have[p])
            if p in seen:
                moves.append((have[p], row[-1]))
            seen.add(p)
        new.append(row)
    pools = [p.clone() for p in s["pools"]]
    for src, dst in moves:
        for p in pools:
            p[dst] = p[src]
    return {"slots": torch.tensor(new, dtype=torch.int32, device=s["slots"].device), "pools": pools}


def exact(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    op = case["op"]
    if op == "scan" and case["N"] > 40000 or op == "scan_grad" and case["B"] * case["N"] * case["D"] * case["ds"] > 1.2e9:
        return None
    s = _inputs(case, seed, device)
    if op == "scan":
        y, h, _, _ = _exact_scan(s)
        if s["z"] is not None:
            z = s["z"].double()
            y = y * z / (1 + (-z).exp())
        if s["lengths"] is not None:
            y = y.masked_fill((torch.arange(y.shape[1], device=device)[None] >= s["lengths"][:, None])[..., None], 0)
        return {"out": y, "S": h}
    if op == "scan_grad":
        return _exact_scan_grad(s)
    if op in ("conv", "conv_grad"):
        return _exact_conv(s, op == "conv_grad")
    if op == "conv_step":
        at, S = s["slots"].long(), s["S"].double()
        u = s["b"].double() + s["w"][:, -1].double() * s["x"].double()
        for j in range(S.shape[1]):
            u = u + s["w"][:, j].double() * S[at, j]
        S[at] = torch.cat([S[at, 1:], s["x"].double()[:, None]], 1)
        return {"out": u / (1 + (-u).exp()), "S": S}
    if op == "scan_step":
        s["S0"] = s["S"][s["slots"].long()]
        one = {k: v[:, None] for k, v in s.items() if k in ("x", "dt", "Bm", "Cm")}
        y, h, _, _ = _exact_scan(s | one | {"lengths": None})
        S = s["S"].double()
        S[s["slots"].long()] = h
        z = s["z"].double()
        return {"out": y[:, 0] * z / (1 + (-z).exp()), "S": S}
    if op == "select":
        return _exact_select(s)
    if op == "reorder":
        return _exact_reorder(s, s["parents"])
    r = _exact_select(s)
    return r | _exact_reorder(s, r["parents"])
