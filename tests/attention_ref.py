"""64-bit references and inputs for the tests of the paged cache and the attention over it.

Bounds, fixed before the first run.  With w the softmax weights and A = sum_j w_j |v_j|, an output of a 16-bit
type whose unit roundoff is u (2^-8 for bf16, 2^-11 for f16) is off by at most

* u |out|, its own rounding,
* u A, the weights' rounding to that type before they meet the values,
* 2 d A, where d is how far a score can be off: its 128 products are summed in f32 by the tensor cores,
  in eight steps of sixteen, each of which can lose 2^-23 of the sum of the products' sizes once for
  its own sixteen and once for the running sum: d = 2^-19 max_j |scale| sum_i |q_i k_ij|, and 2^-21 for the
  exponential on top,
* f16 only: 2^-25 |v_j| for every key whose weight lies below the normal range, and 2^-25 for the output.

The logarithm of the sum is off by d + 2^-21 and a rounding of 2^-23 |lse|.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def normal(*shape, dtype=torch.bfloat16, seed=0, std=1.0, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device=device) * std).to(dtype)


def cache(pages, page, heads, dtype=torch.bfloat16, layout="places", seed=0, fill=None, device="cuda"):
    """(k_cache, v_cache) [pages, page, heads, 128]: by places, by heads, or woven into one buffer."""
    def made(*shape, seed):
        return torch.full(shape, fill, dtype=dtype, device=device) if fill is not None else normal(*shape, dtype=dtype, seed=seed, device=device)

    if layout == "heads":
        return tuple(made(pages, heads, page, 128, seed=seed + i).transpose(1, 2) for i in range(2))
    if layout == "woven":
        both = made(pages, 2, page, heads, 128, seed=seed)
        return both[:, 0], both[:, 1]
    if layout == "side":   # key and value heads of a place side by side
        both = made(pages, page, 2 * heads, 128, seed=seed)
        return both[:, :, :heads], both[:, :, heads:]
    return tuple(made(pages, page, heads, 128, seed=seed + i) for i in range(2))


class Batch:
    """Queries, caches, page tables and lengths.  Places without a key hold ``junk``; table entries behind a length, too."""

    def __init__(self, lengths, tokens=1, h_q=4, h_k=2, page=16, prefix=0, dtype=torch.bfloat16, idx=torch.int32, layout="places",
                 junk=float("nan"), seed=0, std=1.0, spare=2):
        self.lengths_list, self.tokens, self.prefix, self.page = list(lengths), tokens, prefix, page
        n = len(self.lengths_list)
        need = [-(-x // page) for x in self.lengths_list]
        shared = -(-prefix // page)
        pool = shared + sum(need) + spare
        gen = torch.Generator().manual_seed(seed)
        place = torch.randperm(pool, generator=gen)
        self.q = normal(n * tokens, h_q, 128, dtype=dtype, seed=seed + 1, std=std)
        self.k_cache, self.v_cache = cache(pool, page, h_k, dtype, layout, fill=junk)
        self.prefix_pages = place[:shared].to(idx).cuda() if prefix else None
        self.table = torch.full((n, max(need + [1]) + 1), -7, dtype=idx)
        self.keys, at = [], shared   # of each sequence: (k, v) [length, h_k, 128]
        self.shared = (normal(prefix, h_k, 128, dtype=dtype, seed=seed + 2), normal(prefix, h_k, 128, dtype=dtype, seed=seed + 3))
        self._write(self.shared, place[:shared])
        for i, x in enumerate(self.lengths_list):
            pages = place[at:at + need[i]]
            at += need[i]
            self.table[i, :need[i]] = pages.to(idx)
            kv = normal(x, h_k, 128, dtype=dtype, seed=seed + 10 + 2 * i), normal(x, h_k, 128, dtype=dtype, seed=seed + 11 + 2 * i)
            self.keys.append(kv)
            self._write(kv, pages)
        self.table = self.table.cuda()
        self.lengths = torch.tensor(self.lengths_list, dtype=idx, device="cuda")

    def _write(self, kv, pages):
        j = torch.arange(kv[0].shape[0])
        for c, x in zip((self.k_cache, self.v_cache), kv):
            c[pages[j // self.page].cuda(), (j % self.page).cuda()] = x

    def run(self, **kw):
        import gated_delta_rule_24_gb300 as gdn
        kw = {"return_lse": True, **kw}
        return gdn.paged_attention_step(self.q, self.k_cache, self.v_cache, self.table, self.lengths, prefix_pages=self.prefix_pages,
                                        prefix_length=self.prefix, **kw)

    def reference(self, scale=None):
        return attend(self.q, self.keys, self.shared, self.tokens, scale)


def attend(q, keys, shared, tokens, scale=None):
    """(out, lse, room of out, room of lse) in 64 bits, sequence by sequence; rows without a key give 0 and -inf."""
    scale = 128 ** -0.5 if scale is None else scale
    unit, f16 = UNIT[q.dtype], q.dtype == torch.float16
    h_q, h_k = q.shape[1], shared[0].shape[1]
    g = h_q // h_k
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    room, lse_room = torch.zeros_like(out), torch.zeros_like(lse)
    for n, (k, v) in enumerate(keys):
        for i in range(tokens):
            seen = max(0, k.shape[0] - tokens + i + 1)
            kk, vv = (torch.cat([s, x[:seen]]).double().repeat_interleave(g, 1) for s, x in zip(shared, (k, v)))   # [keys, h_q, 128]
            row = n * tokens + i
            if not kk.shape[0]:
                continue
            x = q[row].double()
            s = scale * (kk * x).sum(-1)
            size = abs(scale) * (kk * x).abs().sum(-1).amax(0)   # [h_q]
            w = torch.softmax(s, 0)
            out[row] = torch.einsum("jh,jhd->hd", w, vv)
            lse[row] = torch.logsumexp(s, 0)
            a = torch.einsum("jh,jhd->hd", w, vv.abs())
            d = 2.0 ** -19 * size + 2.0 ** -21
            room[row] = unit * out[row].abs() + (unit + 2 * d[:, None]) * a
            if f16:
                room[row] += 2.0 ** -25 * (1 + vv.abs().sum(0))
            lse_room[row] = d + 2.0 ** -21 + 2.0 ** -23 * lse[row].abs()
    return out, lse, room, lse_room


def check(got, ref, rows=None):
    (out, lse), (want, want_lse, room, lse_room) = got, ref
    at = slice(None) if rows is None else rows
    off = (out[at].double() - want[at]).abs() / room[at].clamp_min(1e-300)
    assert not bool(out[at].isnan().any()) and bool((off <= 1).all()), ("out", float(off.nan_to_num(9e9).max()))
    if lse is not None:
        none = want_lse[at] == -math.inf
        assert bool((lse[at][none] == -math.inf).all())
        off = ((lse[at].double() - want_lse[at]).abs() / lse_room[at])[~none]
        assert not bool(lse[at].isnan().any()) and bool((off <= 1).all()), ("lse", float(off.max()))
