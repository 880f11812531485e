"""64-bit token-by-token gated linear attention and group norm, and the error bounds of their tests.

Every bound is elementwise, a number of rounding steps times the sum of the absolute values of the
terms that an output adds up (computed by the same recurrence on absolute values):

* fp32 paths: chains of at most 2^8 additions of products, each off by 2^-24 relative: 2^-16.
* results held in 32 bits that pass the tensor cores: operands that are not inputs go there as
  bf16 pairs, off by 2^-8 * 2^-8 = 2^-16 at most, plus the 2^-16 above: 2^-15.
* bf16 results: one rounding of the result, 2^-8 of its value, and on the tensor cores one rounding
  of each weight or state, 2^-8 of each term.
"""
import torch

EPS32, EPS_PAIR, EPS16 = 2.0**-16, 2.0**-15, 2.0**-8


def gates(gen, B, H, N, scale=0.3, resets=0.0, device="cuda"):
    """Log decays -scale * 2^-(h mod 4) * uniform(0, 2), a share of them -inf."""
    g = -scale * 2.0 ** -(torch.arange(H, device=device) % 4)[None, :, None] * 2 * torch.rand(
        B, H, N, generator=gen, device=device)
    g[torch.rand(B, H, N, generator=gen, device=device) < resets] = float("-inf")
    return g


def make(B, H, N, dk, dv, dt, seed, state=False, resets=0.0, scale=0.3, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    d = {"q": (r(B, H, N, dk) * dk**-0.25).to(dt), "k": (r(B, H, N, dk) * dk**-0.25).to(dt), "v": r(B, H, N, dv).to(dt),
         "g": gates(gen, B, H, N, scale, resets, device), "dout": r(B, H, N, dv).to(dt), "S0": None, "dS": None}
    if state:
        d["S0"], d["dS"] = r(B, H, dk, dv), r(B, H, dk, dv)
    return d


def forward64(q, k, v, g, S0=None, lengths=None, **_):
    """(out, final S, all states before each token) in 64 bits; rows past a length are zero."""
    q, k, v, a = q.double(), k.double(), v.double(), g.double().exp()
    B, H, N, dk = q.shape
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device) if S0 is None else S0.double().clone()
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.long().clamp(0, N)
    out, before = torch.zeros(B, H, N, v.shape[-1], dtype=torch.float64, device=q.device), []
    for t in range(N):
        live = (t < n)[:, None, None, None]
        before.append(S)
        new = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        S = torch.where(live, new, S)
        out[:, :, t] = torch.where(live[..., 0], torch.einsum("bhx,bhxc->bhc", q[:, :, t], S), 0.0)
    return out, S, before


def backward64(q, k, v, g, dout, S0=None, dS=None, lengths=None):
    """dq, dk, dv, dg, dS0 in 64 bits, dg from its definition e^{g_t} <S_{t-1}, R_t>."""
    _, S, before = forward64(q, k, v, g, S0, lengths)
    before = before + [S]
    q, k, v, a, do = q.double(), k.double(), v.double(), g.double().exp(), dout.double()
    B, H, N, _ = q.shape
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.long().clamp(0, N)
    R = torch.zeros_like(S) if dS is None else dS.double().clone()
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(a)
    for t in reversed(range(N)):
        live = (t < n)[:, None, None, None]
        Rt = R + q[:, :, t, :, None] * do[:, :, t, None, :]
        put = lambda x: torch.where(live[..., 0], x, 0.0)  # noqa: E731
        dq[:, :, t] = put(torch.einsum("bhxc,bhc->bhx", before[t + 1], do[:, :, t]))
        dk[:, :, t] = put(torch.einsum("bhxc,bhc->bhx", Rt, v[:, :, t]))
        dv[:, :, t] = put(torch.einsum("bhxc,bhx->bhc", Rt, k[:, :, t]))
        dg[:, :, t] = put((a[:, :, t, None, None] * before[t] * Rt).sum(-1))[..., :].sum(-1)
        R = torch.where(live, a[:, :, t, None, None] * Rt, R)
    return dq, dk, dv, dg, R


def absolute(d):
    return {n: (t.double().abs() if n != "g" and t is not None and t.is_floating_point() else t) for n, t in d.items()}


def within(got, ref, terms, dt, name, pair=False, steps=1):
    """|got - ref| within the bound of the module's docstring; `steps` roundings to bf16 per term."""
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if got.dtype == torch.bfloat16:
        tol = EPS16 * ref.abs() + (steps * EPS16 * 1.01 if pair else EPS32 * 1.01) * terms
    else:
        tol = (EPS_PAIR if pair else EPS32) * terms
    off = (got.double() - ref).abs() - tol
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 1e-30, f"{name}: {worst:.3g} beyond the bound (rms {ref.square().mean().sqrt().item():.3g})"


def norm64(x, gate=None, weight=None, bias=None, eps=1e-5):
    x = x.double().transpose(1, 2)  # [B, N, H, d]
    h = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + eps).sqrt()
    B, N, H, d = x.shape
    y = h.reshape(B, N, H * d)
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y if gate is None else y * gate.double() * torch.sigmoid(gate.double())
