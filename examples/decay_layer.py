"""A decay linear-attention layer as a server runs it: prompts first, then one token at a time.

    python examples/decay_layer.py

The projection's output holds queries, keys and values side by side.  Each call norms and rotates
the queries and keys in place, then attends: prompts of any lengths through the chunked prefill,
which leaves every sequence's state in its slot of a pool, and each new token of a batch through
the step, which updates the slots in place.  The last lines compare tokens that came one by one
with the same tokens as part of one longer prompt.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_24_gb300 as gdn  # noqa: E402

D = 128


class DecayLayer:
    """Random weights; ``H_qk`` query/key heads, ``H_v`` value heads, one decay for each head."""

    def __init__(self, hidden=1024, H_qk=8, H_v=16, places=8192, slots=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).to(torch.bfloat16)

        self.H_qk, self.H_v, H = H_qk, H_v, max(H_qk, H_v)
        self.w_in = normal(hidden, (2 * H_qk + H_v) * D, std=hidden ** -0.5)
        self.w_out = normal(H * D, hidden, std=(H * D) ** -0.5)
        self.q_weight, self.k_weight = torch.ones(D, device=device), torch.ones(D, device=device)
        angle = torch.arange(places, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, D, 2, device=device, dtype=torch.float64) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.decay = torch.exp(-torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device=device) / H))
        self.pool = torch.zeros(slots, H, D, D, dtype=torch.bfloat16, device=device)

    def _qkv(self, x, positions):
        qkv = (x @ self.w_in).view(x.shape[0], -1, D)
        q, k, v = qkv.split([self.H_qk, self.H_qk, self.H_v], dim=1)
        gdn.qk_norm_rope(q, k, self.cos_sin, positions, self.q_weight, self.k_weight, q_out=q, k_out=k)
        return q, k, v

    def prompts(self, x, cu_seqlens, positions, slots):
        """Tokens ``x`` [T, hidden] of packed prompts; their states go to ``slots`` of the pool."""
        q, k, v = self._qkv(x, positions)
        out, _ = gdn.decay_linear_attention(q, k, v, self.decay, cu_seqlens=cu_seqlens, output_final_state=True,
                                            output_state=self.pool, state_indices=slots)
        return out.flatten(1) @ self.w_out

    def tokens(self, x, positions, slots):
        """One new token ``x`` [B, hidden] for each sequence, whose states are in ``slots``."""
        q, k, v = self._qkv(x, positions)
        out = gdn.decay_linear_step(q, k, v, self.pool, self.decay, state_indices=slots)
        return out.flatten(1) @ self.w_out


def main(lengths=(300, 17, 1, 129), steps=8):
    """Prompts and ``steps`` new tokens each; returns how far (2-norm of the difference over 2-norm)
    the new tokens' results are from those of the same tokens inside one long prompt each."""
    torch.manual_seed(1)
    layer, n = DecayLayer(), len(lengths)
    x = [torch.randn(length + steps, layer.w_in.shape[0], device="cuda").to(torch.bfloat16) for length in lengths]
    slots = torch.randperm(layer.pool.shape[0], device="cuda")[:n].to(torch.int32)

    def packed(parts):
        cu = torch.tensor([0] + [len(p) for p in parts], device="cuda").cumsum(0).to(torch.int32)
        return torch.cat(parts), cu, torch.cat([torch.arange(len(p), device="cuda") for p in parts])

    tokens, cu, positions = packed([p[:length] for p, length in zip(x, lengths)])
    layer.prompts(tokens, cu, positions, slots)
    place = torch.tensor(lengths, device="cuda")
    stepped = [layer.tokens(torch.stack([p[length + i] for p, length in zip(x, lengths)]), place + i, slots) for i in range(steps)]
    stepped = torch.stack(stepped, 1)   # [n, steps, hidden]

    tokens, cu, positions = packed(x)
    whole = layer.prompts(tokens, cu, positions, slots)
    whole = torch.stack([whole[int(cu[i + 1]) - steps:int(cu[i + 1])] for i in range(n)])
    assert gdn.device_status() == 0
    return float((stepped.float() - whole.float()).norm() / whole.float().norm())


if __name__ == "__main__":
    print("new tokens one by one against one prompt: %.2e apart" % main())
