"""Workloads of the gated linear attention layer: prefill, its gradient, the serving step and the gated group norm.

Each case is one call of one operator.  ``run`` computes it in a plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library's entry points.  Sizes follow the repository's configurations
(4 x 16 x 8192 at d = 128, 8 x 16 x 4096 at d = 64, 1 x 2 x 256 at d = 32, decode over 256 x 32 heads).

Gated linear attention: S_t = e^{g_t} S_{t-1} + k_t v_t^T, out_t = q_t^T S_t, with a log decay g per token and head.
Group norm: y = ((x - mean) / sqrt(var + eps) * weight + bias) * silu(gate) per token over each head's channels.
"""
import math

import torch

own = False

EPS = 1e-5
LOG_ZERO = -200.0  # stands for log 0: e^-200 is zero in 32 bits
CHUNK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # prompt processing of a batch of full-length prompts
        {"name": "gated_prefill_bf16", "op": "gated", "B": 4, "H": 16, "N": 8192, "dk": 128, "dv": 128, "dt": "bf16",
         "ragged": False, "state": False},
        # one long prompt of odd length that continues a cached state
        {"name": "gated_long_state_bf16", "op": "gated", "B": 1, "H": 32, "N": 32749, "dk": 128, "dv": 128, "dt": "bf16",
         "ragged": False, "state": True},
        # padded batch of short prompts, one of them empty, small heads
        {"name": "gated_padded_bf16_d64", "op": "gated", "B": 8, "H": 16, "N": 1000, "dk": 64, "dv": 64, "dt": "bf16",
         "ragged": True, "state": True},
        # the smallest call, 32-bit, where latency counts
        {"name": "gated_small_f32", "op": "gated", "B": 1, "H": 2, "N": 256, "dk": 32, "dv": 32, "dt": "f32",
         "ragged": False, "state": False},
        # training step of the layer
        {"name": "gated_grad_bf16", "op": "gated_grad", "B": 4, "H": 16, "N": 8192, "dk": 128, "dv": 128, "dt": "bf16",
         "ragged": False, "state": False},
        # training on padded sequences with a carried state and a gradient of the final one
        {"name": "gated_grad_padded_d64", "op": "gated_grad", "B": 4, "H": 16, "N": 2049, "dk": 64, "dv": 64, "dt": "bf16",
         "ragged": True, "state": True},
        # 32-bit gradient at unequal head sizes
        {"name": "gated_grad_f32", "op": "gated_grad", "B": 2, "H": 4, "N": 333, "dk": 64, "dv": 32, "dt": "f32",
         "ragged": False, "state": True},
        # one token for each of 256 sequences, their states anywhere in a pool
        {"name": "step_batch_bf16", "op": "step", "B": 256, "H": 32, "dk": 128, "dv": 128, "dt": "bf16", "slots": 288},
        # one token for a few sequences: latency
        {"name": "step_few_bf16_d64", "op": "step", "B": 3, "H": 16, "dk": 64, "dv": 64, "dt": "bf16", "slots": 8},
        # the norm behind the prefill, and its gradient in training
        {"name": "norm_bf16", "op": "norm", "B": 4, "H": 16, "N": 8192, "d": 128, "dt": "bf16", "gate": True, "affine": True},
        {"name": "norm_grad_bf16", "op": "norm_grad", "B": 4, "H": 16, "N": 4096, "d": 128, "dt": "bf16", "gate": True,
         "affine": True},
        # the norm behind the serving step
        {"name": "norm_token_bf16", "op": "norm", "B": 256, "H": 32, "N": 1, "d": 128, "dt": "bf16", "gate": True,
         "affine": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "step", "norm", "norm_grad"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        B = _log_int(rng, 1, 256)
        return {"op": op, "B": B, "H": _log_int(rng, 1, 32), "dk": rng.choice([32, 64, 128]), "dv": rng.choice([32, 64, 128]),
                "dt": dt, "slots": B + rng.randrange(0, 32)}
    if op in ("norm", "norm_grad"):
        return {"op": op, "B": _log_int(rng, 1, 4), "H": _log_int(rng, 1, 16), "N": _log_int(rng, 1, 4096),
                "d": rng.choice([32, 64, 128]), "dt": dt, "gate": rng.random() < 0.75, "affine": rng.random() < 0.75}
    if rng.random() < 0.6:
        dk = dv = rng.choice([64, 128])
    else:
        dk, dv = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
    fast = dt == "bf16" and dk == dv and dk >= 64
    B, H = _log_int(rng, 1, 8), _log_int(rng, 1, 16)
    most = (400_000 if fast else 40_000) // (B * H)
    return {"op": op, "B": B, "H": H, "N": _log_int(rng, 1, max(2, min(most, 16384))), "dk": dk, "dv": dv, "dt": dt,
            "ragged": rng.random() < 0.4, "state": rng.random() < 0.5}


def _inputs(case, seed, device):
    """q, k ~ N(0, 1) d_k^-1/4, v ~ N(0, 1) and log decays whose scales differ by head, with a few resets."""
    g = torch.Generator(device=device).manual_seed(int(seed) * 7919 + 17)
    op, dt, B, H = case["op"], DTYPES[case["dt"]], case["B"], case["H"]
    randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        N, d = case["N"], case["d"]
        s["x"] = (randn(B, H, N, d) * torch.exp(randn(B, H, N, 1))).to(dt)
        s["gate"] = randn(B, N, H * d).to(dt) if case["gate"] else None
        s["weight"] = 1 + 0.1 * randn(H * d) if case["affine"] else None
        s["bias"] = 0.1 * randn(H * d) if case["affine"] else None
        s["dy"] = randn(B, N, H * d).to(dt) if op == "norm_grad" else None
        return s
    dk, dv = case["dk"], case["dv"]
    lead = (B, H) if op == "step" else (B, H, case["N"])
    s["q"], s["k"] = ((randn(*lead, dk) * dk ** -0.25).to(dt) for _ in range(2))
    s["v"] = randn(*lead, dv).to(dt)
    scale = 2.0 ** -(1 + torch.arange(H, device=device) % 8)
    x = torch.nn.functional.softplus(randn(*lead))
    s["g"] = -scale.reshape(1, H, *([1] * (len(lead) - 2))) * x
    reset = torch.rand(*lead, generator=g, device=device) < 1 / 512  # a new document within the sequence
    s["g"][reset] = -math.inf
    if op == "step":
        order = torch.randperm(case["slots"], generator=g, device=device)
        s["slots"] = order[:B].to(torch.int32)
        s["S"] = randn(case["slots"], H, dk, dv)
        return s
    N = case["N"]
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(N // 2, N + 1, (B,), generator=g, device=device, dtype=torch.int32)
        n[0] = N
        if B > 2:
            n[B - 1] = 0
        s["lengths"] = n
    s["S0"] = randn(B, H, dk, dv) if case["state"] else None
    if op == "gated":
        s["out"] = torch.zeros(B, H, N, dv, dtype=dt, device=device)  # rows past a sequence's end are left as they are
        s["S"] = torch.empty(B, H, dk, dv, device=device)
    else:
        s["dout"] = randn(B, H, N, dv).to(dt)
        s["dS"] = randn(B, H, dk, dv) if case["state"] else None
    return s


def prepare(case, seed):
    return _inputs(case, seed, "cuda")


# --------------------------------------------------------------------------------------------------------------
# plain forms: chunks of 128 tokens, all chunks at once; log decays summed in 64 bits, everything else in 32
# --------------------------------------------------------------------------------------------------------------
def _chunks(x, n):
    """[B, H, N, d] -> [B, H, n, CHUNK, d] in 32 bits, zeros behind the end."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - x.shape[2])).reshape(*x.shape[:2], n, CHUNK, x.shape[3])


def _masked(s):
    """Inputs in chunks, padding tokens cleared, and the decays' running sums inside and across chunks."""
    q, k, v, g = s["q"], s["k"], s["v"], s["g"].clamp(min=LOG_ZERO).double()
    do = s.get("dout")
    N, dev = q.shape[2], q.device
    if s["lengths"] is not None:
        live = (torch.arange(N, device=dev) < s["lengths"][:, None])[:, None, :]
        g = torch.where(live, g, torch.zeros_like(g))
        clear = lambda x: torch.where(live[..., None], x, torch.zeros_like(x))  # noqa: E731
        q, k, v, do = clear(q), clear(k), clear(v), None if do is None else clear(do)
    n = max(1, -(-N // CHUNK))
    c = torch.nn.functional.pad(g, (0, n * CHUNK - N)).reshape(*g.shape[:2], n, CHUNK).cumsum(-1)
    total = c[..., -1]
    return n, _chunks(q, n), _chunks(k, n), _chunks(v, n), None if do is None else _chunks(do, n), c, total, total.cumsum(-1)


def _decays(c):
    """e^{c_i - c_j} for j <= i in a chunk, else 0."""
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=c.device).tril()
    return torch.where(low, (c[..., :, None] - c[..., None, :]).float(), -torch.inf).exp()


def _states(k, v, c, total, across, n, S0):
    """State at each chunk's start and at the end: [B, H, n + 1, dk, dv]."""
    part = (k * (total[..., None] - c).exp().float()[..., None]).transpose(-1, -2) @ v
    lead = torch.nn.functional.pad(across, (1, 0))  # decay up to each chunk's start, and to the end
    below = torch.ones(n + 1, n, dtype=torch.bool, device=c.device).tril(-1)
    mix = torch.where(below, (lead[..., :, None] - across[..., None, :]).float(), -torch.inf).exp()
    S = (mix @ part.flatten(-2)).unflatten(-1, part.shape[-2:])
    return S if S0 is None else S + lead.exp().float()[..., None, None] * S0[:, :, None]


def _plain_gated(s):
    n, q, k, v, _, c, total, across = _masked(s)
    S = _states(k, v, c, total, across, n, s["S0"])
    o = ((q @ k.transpose(-1, -2)) * _decays(c)) @ v + c.exp().float()[..., None] * (q @ S[:, :, :-1])
    o = o.flatten(2, 3)[:, :, : s["q"].shape[2]]
    if s["lengths"] is None:
        s["out"].copy_(o)
    else:
        live = (torch.arange(o.shape[2], device=o.device) < s["lengths"][:, None])[:, None, :, None]
        s["out"].copy_(torch.where(live, o, s["out"].float()))
    s["S"].copy_(S[:, :, -1])
    return {"out": s["out"], "S": s["S"]}


def _plain_gated_grad(s):
    n, q, k, v, do, c, total, across = _masked(s)
    N, dt = s["q"].shape[2], s["q"].dtype
    S = _states(k, v, c, total, across, n, s["S0"])[:, :, :-1]
    # gradient of the state behind each chunk and of the initial one: the same sums from the end
    ec, ew = c.exp().float()[..., None], (total[..., None] - c).exp().float()[..., None]
    part = (q * ec).transpose(-1, -2) @ do
    lead = torch.nn.functional.pad(across, (1, 0))
    above = torch.ones(n + 1, n, dtype=torch.bool, device=c.device).triu()
    mix = torch.where(above, (lead[..., None, :-1] - lead[..., :, None]).float(), -torch.inf).exp()
    R = (mix @ part.flatten(-2)).unflatten(-1, part.shape[-2:])
    if s["dS"] is not None:
        R = R + (lead[..., -1:] - lead).exp().float()[..., None, None] * s["dS"][:, :, None]
    dS0, R = R[:, :, 0], R[:, :, 1:]
    D = _decays(c)
    P, dP = (q @ k.transpose(-1, -2)) * D, (do @ v.transpose(-1, -2)) * D
    dq_in = ec * (do @ S.transpose(-1, -2))
    dk_out = ew * (v @ R.transpose(-1, -2))
    dq = dq_in + dP @ k
    dk = dk_out + dP.transpose(-1, -2) @ q
    dv = ew * (k @ R) + P.transpose(-1, -2) @ do
    # dg_t sums the weights of all pairs (i, j) with j < t <= i: both in the chunk, one of them, or neither
    M = (P * (do @ v.transpose(-1, -2))).tril(-1)
    inside = (M.sum(-1) - M.sum(-2)).double().flip(-1).cumsum(-1).flip(-1)
    from_left = (q * dq_in).sum(-1).double().flip(-1).cumsum(-1).flip(-1)
    to_right = torch.nn.functional.pad((k * dk_out).sum(-1).double().cumsum(-1)[..., :-1], (1, 0))
    over = total.exp() * (S * R).flatten(-2).sum(-1).double()
    dg = (inside + from_left + to_right + over[..., None]).flatten(2)[:, :, :N]
    if s["lengths"] is not None:  # padding tokens have no part in anything
        dg = torch.where((torch.arange(N, device=dg.device) < s["lengths"][:, None])[:, None, :], dg, torch.zeros_like(dg))
    cut = lambda x: x.flatten(2, 3)[:, :, :N].to(dt)  # noqa: E731
    r = {"dq": cut(dq), "dk": cut(dk), "dv": cut(dv), "dg": dg.float()}
    if s["S0"] is not None:
        r["dS0"] = dS0
    return r


def _plain_step(s):
    at = s["slots"].long()
    k, v = s["k"].float(), s["v"].float()
    S = s["g"].exp()[..., None, None] * s["S"][at] + k[..., :, None] * v[..., None, :]
    s["S"][at] = S
    return {"out": (s["q"].float()[..., None, :] @ S)[..., 0, :].to(s["q"].dtype), "S": s["S"]}


def _heads_last(x):
    return x.float().permute(0, 2, 1, 3)  # [B, H, N, d] -> [B, N, H, d]


def _normed(x):
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _affine(s, xh):
    if s["weight"] is not None:
        xh = xh * s["weight"].reshape(xh.shape[2:]) + s["bias"].reshape(xh.shape[2:])
    return xh


def _plain_norm(s):
    xh, _ = _normed(_heads_last(s["x"]))
    y = _affine(s, xh).flatten(2)
    if s["gate"] is not None:
        g = s["gate"].float()
        y = y * (g * torch.sigmoid(g))
    return {"y": y.to(s["x"].dtype)}


def _plain_norm_grad(s):
    dt = s["x"].dtype
    xh, r = _normed(_heads_last(s["x"]))
    dy = s["dy"].float()
    out = {}
    if s["gate"] is not None:
        g = s["gate"].float()
        sig = torch.sigmoid(g)
        out["dgate"] = (dy * _affine(s, xh).flatten(2) * sig * (1 + g * (1 - sig))).to(dt)
        dy = dy * (g * sig)
    dy = dy.reshape(xh.shape)
    if s["weight"] is not None:
        out["dweight"] = (dy * xh).sum((0, 1), dtype=torch.float64).flatten().float()
        out["dbias"] = dy.sum((0, 1), dtype=torch.float64).flatten().float()
        dy = dy * s["weight"].reshape(xh.shape[2:])
    dx = r * (dy - dy.mean(-1, keepdim=True) - xh * (dy * xh).mean(-1, keepdim=True))
    out["dx"] = dx.permute(0, 2, 1, 3).contiguous().to(dt)
    return out


# --------------------------------------------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------------------------------------------
def _own(s):
    from causal_linear_attention_attn_gb300 import linattn as L

    op = s["case"]["op"]
    if op == "gated":
        if s["S0"] is None:
            L.la_gated(s["q"], s["k"], s["v"], s["g"], lengths=s["lengths"], out=s["out"], S=s["S"])
        else:
            s["S"].copy_(s["S0"])
            L.la_gated_with_state(s["q"], s["k"], s["v"], s["g"], s["S"], lengths=s["lengths"], out=s["out"])
        return {"out": s["out"], "S": s["S"]}
    if op == "gated_grad":
        r = L.la_gated_backward(s["q"], s["k"], s["v"], s["g"], s["dout"], S0=s["S0"], dS=s["dS"], lengths=s["lengths"],
                                need_state_grad=s["S0"] is not None)
        return dict(zip(("dq", "dk", "dv", "dg", "dS0"), r))
    if op == "step":
        return {"out": L.la_gated_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"]), "S": s["S"]}
    if op == "norm":
        return {"y": L.la_group_norm(s["x"], gate=s["gate"], weight=s["weight"], bias=s["bias"], eps=EPS)}
    r = L.la_group_norm_backward(s["x"], s["dy"], gate=s["gate"], weight=s["weight"], bias=s["bias"], eps=EPS)
    return {k: x for k, x in zip(("dx", "dgate", "dweight", "dbias"), r) if x is not None}


def run(state):
    if own:
        return _own(state)
    return {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "step": _plain_step, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad}[state["case"]["op"]](state)


def work(case):
    e = 2 if case["dt"] == "bf16" else 4
    op, B, H = case["op"], case["B"], case["H"]
    if op in ("norm", "norm_grad"):
        n = B * H * case["N"] * case["d"]
        tensors = 2 + case["gate"] if op == "norm" else 3 + 2 * case["gate"]
        vectors = (2 if op == "norm" else 4) * case["affine"] * H * case["d"]
        return {"bytes": e * tensors * n + 4 * vectors, "flops": (10 if op == "norm" else 25) * n}
    dk, dv = case["dk"], case["dv"]
    state = B * H * dk * dv
    if op == "step":
        return {"bytes": 8 * state + B * H * (e * (2 * dk + 2 * dv) + 4) + 4 * B, "flops": 5 * state}
    tokens = B * H * case["N"] * (0.7 if case["ragged"] and B > 2 else 0.85 if case["ragged"] else 1.0)
    if op == "gated":
        return {"bytes": tokens * (e * (2 * dk + 2 * dv) + 4) + 4 * state * (1 + case["state"]), "flops": 4 * tokens * dk * dv}
    return {"bytes": tokens * (e * (4 * dk + 3 * dv) + 8) + 4 * state * (3 * case["state"]), "flops": 10 * tokens * dk * dv}


# --------------------------------------------------------------------------------------------------------------
# 64 bits, token by token from the definitions
# --------------------------------------------------------------------------------------------------------------
def _exact_gated(s):
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    B, H, N, dk = q.shape
    a = s["g"].double().exp()
    live = None
    if s["lengths"] is not None:
        live = torch.arange(N, device=q.device) < s["lengths"][:, None]  # [B, N]
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device) if s["S0"] is None else s["S0"].double()
    rows = []
    for t in range(N):
        new = S * a[:, :, t, None, None] + k[:, :, t, :, None] * v[:, :, t, None, :]
        S = new if live is None else torch.where(live[:, t, None, None, None], new, S)
        rows.append((q[:, :, t, None, :] @ S)[:, :, 0])
    out = torch.stack(rows, 2)
    if live is not None:
        out = torch.where(live[:, None, :, None], out, torch.zeros_like(out))
    return out, S, a, live


def _exact_gated_grad(s):
    out, S, a, live = _exact_gated(s)
    q, k, v, do = (s[x].double() for x in ("q", "k", "v", "dout"))
    if live is not None:
        do = torch.where(live[:, None, :, None], do, torch.zeros_like(do))
    N = q.shape[2]
    R = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()
    end = (R * S).sum((-1, -2))
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(N)):
        new = R + q[:, :, t, :, None] * do[:, :, t, None, :]
        if live is None:
            dk[:, :, t], dv[:, :, t] = (new @ v[:, :, t, :, None])[..., 0], (k[:, :, t, None, :] @ new)[:, :, 0]
            R = new * a[:, :, t, None, None]
        else:
            m = live[:, t, None, None].double()
            dk[:, :, t], dv[:, :, t] = m * (new @ v[:, :, t, :, None])[..., 0], m * (k[:, :, t, None, :] @ new)[:, :, 0]
            R = torch.where(live[:, t, None, None, None], new * a[:, :, t, None, None], R)
    # a second sweep forward for the queries' gradient
    S = torch.zeros_like(R) if s["S0"] is None else s["S0"].double()
    dq = torch.zeros_like(q)
    for t in range(N):
        new = S * a[:, :, t, None, None] + k[:, :, t, :, None] * v[:, :, t, None, :]
        if live is not None:
            new = torch.where(live[:, t, None, None, None], new, S)
        S = new
        dq[:, :, t] = (S @ do[:, :, t, :, None])[..., 0]
    # scaling the state before token t scales every later read of it and of the tokens behind it
    each = (do * out).sum(-1) - (k * dk).sum(-1)
    dg = each.flip(-1).cumsum(-1).flip(-1) + end[..., None]
    if live is not None:
        dg = torch.where(live[:, None, :], dg, torch.zeros_like(dg))
    r = {"dq": dq, "dk": dk, "dv": dv, "dg": torch.where(a == 0, torch.zeros_like(dg), dg)}
    if s["S0"] is not None:
        r["dS0"] = R
    return r


def exact(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    op = case["op"]
    if op in ("gated", "gated_grad") and (case["N"] > 40000 or case["B"] * case["H"] * case["N"] * case["dk"] * case["dv"] > 4e10):
        return None
    s = _inputs(case, seed, device)
    if op == "gated":
        out, S, _, _ = _exact_gated(s)
        return {"out": out, "S": S}
    if op == "gated_grad":
        return _exact_gated_grad(s)
    if op == "step":
        at = s["slots"].long()
        pool = s["S"].double()
        new = pool[at] * s["g"].double().exp()[..., None, None]
        new = new + s["k"].double()[..., :, None] * s["v"].double()[..., None, :]
        pool[at] = new
        return {"out": (s["q"].double()[..., :, None] * new).sum(-2), "S": pool}
    x = s["x"].double()
    B, H, N, d = x.shape
    std = (x.var(-1, unbiased=False) + EPS).sqrt()[..., None]
    h = (x - x.mean(-1, keepdim=True)) / std
    w = torch.ones(H * d, dtype=torch.float64, device=device) if s["weight"] is None else s["weight"].double()
    b = torch.zeros(H * d, dtype=torch.float64, device=device) if s["bias"] is None else s["bias"].double()
    h = h.transpose(1, 2).reshape(B, N, H * d)
    act = torch.ones_like(h)
    if s["gate"] is not None:
        g = s["gate"].double()
        act = g / (1 + (-g).exp())
    if op == "norm":
        return {"y": (h * w + b) * act}
    dy = s["dy"].double()
    r = {}
    if s["gate"] is not None:
        e = (-g).exp()
        r["dgate"] = dy * (h * w + b) * (1 + e + g * e) / (1 + e).square()
    if s["weight"] is not None:
        r["dweight"], r["dbias"] = (dy * act * h).sum((0, 1)), (dy * act).sum((0, 1))
    u = (dy * act * w).reshape(B, N, H, d).transpose(1, 2)
    h = h.reshape(B, N, H, d).transpose(1, 2)
    r["dx"] = (u - u.mean(-1, keepdim=True) - h * (u * h).mean(-1, keepdim=True)) / std
    return r
