"""A softmax-attention layer between linear ones, as a server runs it: a prefix that all requests share, then requests token by token.

    python examples/softmax_layer.py

Keys and values of all tokens live in the pages of one cache.  The prefix is written once; each request's tokens go to pages of
its own, which the layer takes from a free list as they fill up.  A new token of a batch takes two calls: norm, rotation and append,
then the attention over the request's pages and over the prefix, which is read once for the batch.  The last lines compare the result
with the same attention in plain torch.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_24_gb300 as gdn  # noqa: E402

D = 128


class SoftmaxLayer:
    """Random weights; ``H_q`` query heads, ``H_k`` key/value heads, pages of ``page`` tokens."""

    def __init__(self, hidden=1024, H_q=16, H_k=2, places=8192, pages=256, page=16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).to(torch.bfloat16)

        self.H_q, self.H_k, self.page = H_q, H_k, page
        self.w_in = normal(hidden, (H_q + 2 * H_k) * D, std=hidden ** -0.5)
        self.w_out = normal(H_q * D, hidden, std=(H_q * D) ** -0.5)
        self.q_weight, self.k_weight = torch.ones(D, device=device), torch.ones(D, device=device)
        angle = torch.arange(places, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, D, 2, device=device, dtype=torch.float64) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.k_cache, self.v_cache = (torch.zeros(pages, page, H_k, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.free = list(range(pages))[::-1]

    def append(self, x, positions, slots):
        """Queries of the tokens ``x`` [T, hidden]; their keys and values go to ``slots``."""
        q, k, v = (x @ self.w_in).view(x.shape[0], -1, D).split([self.H_q, self.H_k, self.H_k], dim=1)
        return gdn.norm_rope_append(q, k, v, self.k_cache, self.v_cache, slots, self.cos_sin, positions, self.q_weight, self.k_weight)

    def prefix(self, x):
        """Writes the tokens ``x`` that all requests begin with."""
        n = len(x)
        self.prefix_pages = torch.tensor([self.free.pop() for _ in range(-(-n // self.page))], dtype=torch.int32, device=x.device)
        self.prefix_length = n
        at = torch.arange(n, device=x.device)
        self.append(x, at, self.prefix_pages[at // self.page] * self.page + at % self.page)

    def requests(self, n, longest):
        """Tables for ``n`` requests of up to ``longest`` tokens each behind the prefix."""
        device = self.k_cache.device
        self.tables = [[] for _ in range(n)]
        self.page_table = torch.full((n, -(-longest // self.page)), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(n, dtype=torch.int32, device=device)
        self.length = 0

    def tokens(self, x):
        """One new token ``x`` [n, hidden] of each request."""
        if self.length % self.page == 0:   # every request is at the same place here: all of them need a page
            for i, table in enumerate(self.tables):
                table.append(self.free.pop())
                self.page_table[i, len(table) - 1] = table[-1]
        slots = self.page_table[:, self.length // self.page] * self.page + self.length % self.page
        self.length += 1
        self.lengths += 1
        q = self.append(x, torch.full((len(x),), self.prefix_length + self.length - 1, device=x.device), slots)
        out = gdn.paged_attention_step(q, self.k_cache, self.v_cache, self.page_table, self.lengths, prefix_pages=self.prefix_pages,
                                       prefix_length=self.prefix_length)
        return q, out, out.flatten(1) @ self.w_out


def main(n=5, prefix=300, steps=40):
    """``steps`` tokens of ``n`` requests behind a prefix; returns how far (2-norm of the difference over 2-norm) the last
    attention is from the same one in 64 bits."""
    torch.manual_seed(2)
    layer = SoftmaxLayer()
    hidden = layer.w_in.shape[0]
    layer.prefix(torch.randn(prefix, hidden, device="cuda").to(torch.bfloat16))
    layer.requests(n, steps)
    for _ in range(steps):
        q, out, _ = layer.tokens(torch.randn(n, hidden, device="cuda").to(torch.bfloat16))
    assert gdn.device_status() == 0
    worst = 0.0
    for i in range(n):
        pages = torch.cat([layer.prefix_pages.long(), torch.tensor(layer.tables[i], device="cuda")])
        at = torch.cat([torch.arange(prefix), -(-prefix // layer.page) * layer.page + torch.arange(steps)]).cuda()
        k, v = (c[pages].flatten(0, 1)[at].double().repeat_interleave(layer.H_q // layer.H_k, 1) for c in (layer.k_cache, layer.v_cache))
        weight = torch.softmax(torch.einsum("hd,jhd->hj", q[i].double(), k) * D ** -0.5, -1)
        want = torch.einsum("hj,jhd->hd", weight, v)
        worst = max(worst, float((out[i].double() - want).norm() / want.norm()))
    return worst


if __name__ == "__main__":
    print("attention over the cache and the prefix against plain torch: %.2e apart" % main())
