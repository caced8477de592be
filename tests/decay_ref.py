"""64-bit references and inputs for the decay linear-attention tests.

Bounds (relative L2 of each (sequence, head) on its own, fixed before the first run):

* 16-bit outputs: three independent roundings to the 16-bit type reach an output (the
  decayed scores, the state as it is read, the output itself).  A rounding is off by 0.42
  of the unit roundoff in the root mean square, 1.7e-3 for bf16 and 2.1e-4 for f16, so that
  the three are at most sqrt(3) times that, 2.9e-3 and 3.6e-4: held to 2^-8 and 2^-11.  It
  takes some hundred independent roundings for that; the few scores of a sequence of one or
  two tokens can be off by a whole roundoff, 2^-8, on their own, and such sequences are
  judged together where there are many of them.
* 16-bit states: the state's own rounding, 1.7e-3 (bf16) or 2.1e-4 (f16), plus the f32 error
  below: held to 2.1e-3 and 2.7e-4.
* f32 states: sums of up to some thousand f32 products and decays exp(sum log g), whose
  exponent is known to about 2^-23 of its size (at most 100 where the decay counts): 1e-5.
"""
from __future__ import annotations

import torch

OUT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STATE = {torch.bfloat16: 2.1e-3, torch.float16: 2.7e-4, torch.float32: 1e-5}


def recurrence(q, k, v, g, scale, state, lengths):
    """S_t = g_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t in 64 bits, sequence by sequence.
    ``state``: [N, H, 128, 128] or None.  Returns (outputs [T, H, 128], states [N, H, 128, 128])."""
    H = max(q.shape[1], v.shape[1])
    q, k, v = (x.double().repeat_interleave(H // x.shape[1], dim=1) for x in (q, k, v))
    T = q.shape[0]
    g = torch.ones(T, H, dtype=torch.float64, device=q.device) if g is None else g.double().expand(T, H)
    out = torch.zeros(T, H, 128, dtype=torch.float64, device=q.device)
    last, t = [], 0
    for n, length in enumerate(lengths):
        s = torch.zeros(H, 128, 128, dtype=torch.float64, device=q.device) if state is None else state[n].double().clone()
        for t in range(t, t + length):
            s = g[t][:, None, None] * s + v[t][:, :, None] * k[t][:, None, :]
            out[t] = torch.einsum("hrc,hc->hr", s, q[t])
        t += bool(length)
        last.append(s)
    return scale * out, torch.stack(last) if last else torch.zeros(0, H, 128, 128, dtype=torch.float64, device=q.device)


def make(lengths, h_qk, h_v, dtype=torch.bfloat16, gate="token", seed=0, device="cuda"):
    """Queries, keys, values and gates of packed sequences: (q, k, v, g, cu_seqlens)."""
    gen = torch.Generator(device=device).manual_seed(seed)
    T, H = sum(lengths), max(h_qk, h_v)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device).to(dtype)

    q, k, v = normal(T, h_qk, 128), normal(T, h_qk, 128), normal(T, h_v, 128)
    if gate == "none":
        g = None
    elif gate == "head":
        g = torch.exp(-torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device=device) / H))
    elif gate == "slow":
        g = torch.exp(-0.001 * torch.rand(T, H, generator=gen, device=device))
    elif gate == "reset":  # a decay that drops everything at some tokens, and next to everything at others
        g = torch.exp(-0.05 * torch.rand(T, H, generator=gen, device=device))
        kind = torch.rand(T, H, generator=gen, device=device)
        g = torch.where(kind < 0.05, torch.zeros_like(g), torch.where(kind < 0.1, torch.full_like(g, 1e-30), g))
    else:
        g = torch.exp(-torch.exp(torch.rand(H, generator=gen, device=device) * 3 - 2)
                      * torch.nn.functional.softplus(torch.randn(T, H, generator=gen, device=device)))
    cu = torch.tensor([0] + list(lengths), device=device).cumsum(0).to(torch.int32)
    return q, k, v, g, cu


def states(slots, heads, dtype, seed=0, device="cuda", std=1.0):
    gen = torch.Generator(device=device).manual_seed(1000 + seed)
    return (torch.randn(slots, heads, 128, 128, generator=gen, device=device) * std).to(dtype)


def rel(a, b):
    a, b = a.double(), b.double()
    d = float(b.norm())
    return float((a - b).norm()) / d if d else float((a - b).norm())


def check(out, out_ref, state, state_ref, lengths, which=None):
    """Each (sequence, head) within its bounds; ``which``: the sequences to look at."""
    t = 0
    for n, length in enumerate(lengths):
        rows, t = slice(t, t + length), t + length
        if which is not None and n not in which:
            continue
        for h in range(out.shape[1]):
            if length:
                e = rel(out[rows, h], out_ref[rows, h])
                assert e <= OUT[out.dtype], ("output", n, h, e)
            if state is not None:
                e = rel(state[n, h], state_ref[n, h])
                assert e <= STATE[state.dtype], ("state", n, h, e)


def norm_rope(x, weight, offset, eps, cos_sin, positions, interleaved):
    """The norm and the rotation in 64 bits."""
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (weight.double() + offset)
    if cos_sin is None:
        return y
    R = cos_sin.shape[1]
    at = torch.arange(x.shape[0], device=x.device) if positions is None else positions.long()
    c, s = cos_sin.double()[at][:, None, :R // 2], cos_sin.double()[at][:, None, R // 2:]
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    z = y.clone()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., a] * s + y[..., b] * c
    return z


def table(places, R, device="cuda"):
    angle = torch.arange(places, dtype=torch.float64, device=device)[:, None] * 10000.0 ** (
        -torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    return torch.cat([angle.cos(), angle.sin()], 1).float()
