"""The operators of softmax attention layers between linear ones: cases, inputs, plain forms and exact results.

Three operators of one layer, as a serving program calls them:

* ``axes``: norm and rotation of query and key heads where a token has a position on each of
  several axes (time, height, width) and every pair of values turns by one of them;
* ``append``: the same for the new tokens' queries and keys, with the keys and values written
  to their places in a paged cache on the way;
* ``attend``: attention of each sequence's newest tokens over its pages of that cache, and over a
  long prefix that the whole batch shares, computed once for all.

``own`` false computes them with elementary torch operations in 32 bits; ``own`` true calls
the package's entry points.  Head dimension 128; query head ``h`` reads key/value head
``h / (h_q / h_k)``.
"""
import math
import random

import torch

own = False

D = 128        # head dimension
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
INTS = {"i32": torch.int32, "i64": torch.int64}
SIZE = {"bf16": 2, "f16": 2, "i32": 4, "i64": 8}
PLACES = 4096                      # of a table of cosines and sines where positions come from an image or a video
MOST_ROPE_HEADS = 65536 * 48       # (query + key) heads times tokens of the largest rotation
MOST_APPEND_HEADS = 16384 * 48     # (query + key + value) heads times tokens of the largest append
MOST_KEYS = 256 * 8192 * 4         # keys times key heads of the largest batch's own pages
MOST_SCORES = 256 * 32 * 32768     # scores with the shared prefix of the largest batch


def listed():
    return [
        # a few tokens of an image, fp16, neighbours paired, every third pair on one axis: all latency
        axes("axes_37_turns", tokens=37, h_q=6, h_k=2, kind="turns", interleaved=True, dtype="f16", idx="i32"),
        # one image among the prompt, half of each head rotated
        axes("axes_4099_half", tokens=4099, h_q=16, h_k=4, rotary=64, kind="blocks", weights=False),
        # a long video, slices of one qkv buffer
        axes("axes_65536", tokens=65536, h_q=32, h_k=16, kind="blocks", fused=True),
        # the newest token of a sequence that decodes alone
        append("append_1", seqs=1, tokens=1, h_q=16, h_k=2, page=16),
        # the newest tokens of a full batch, fp16, 64-bit places, some of the batch's rows padding
        append("append_997", seqs=997, tokens=1, h_q=32, h_k=8, page=64, dtype="f16", idx="i64", padded=27, fused=True),
        # prompts of a batch, no norm, positions on three axes, pages by heads
        append("append_16384", seqs=4, tokens=4096, h_q=32, h_k=8, page=16, kind="blocks", norm=False, heads_first=True, fused=True),
        # one short sequence decoding alone: all latency
        attend("attend_1x511", seqs=1, mean=511, h_q=8, h_k=1, page=16),
        # an odd batch of three tokens each (a draft's), fp16, odd lengths, an odd page size, pages by heads
        attend("attend_37_drafts", seqs=37, tokens=3, mean=1500, ragged=True, h_q=12, h_k=4, page=24, dtype="f16", idx="i64", heads_first=True),
        # one long document
        attend("attend_1x131072", seqs=1, mean=131072, h_q=16, h_k=2, page=64),
        # a full batch of long sequences, the largest
        attend("attend_256x8192", seqs=256, mean=8192, h_q=32, h_k=4, page=64),
        # a few questions about one long document
        attend("attend_8_on_100000", seqs=8, mean=300, ragged=True, h_q=32, h_k=4, page=32, prefix=100000),
        # a full batch behind one long prefix
        attend("attend_256_on_32768", seqs=256, mean=512, ragged=True, h_q=32, h_k=4, page=64, prefix=32768),
    ]


def axes(name=None, *, tokens, h_q, h_k, kind, rotary=128, interleaved=False, dtype="bf16", weights=True, fused=False, idx="i64"):
    """``kind``: the pairs in one block for each of the axes, or taking turns."""
    case = dict(op="axes", tokens=tokens, h_q=h_q, h_k=h_k, kind=kind, rotary=rotary, interleaved=interleaved, dtype=dtype,
                weights=weights, fused=fused, idx=idx)
    return case if name is None else dict(case, name=name)


def append(name=None, *, seqs, tokens, h_q, h_k, page, kind="one", rotary=128, interleaved=False, dtype="bf16", norm=True,
           fused=False, idx="i32", padded=0, heads_first=False):
    """``tokens`` new ones of each sequence; the last ``padded`` rows have no place.  ``heads_first``: the heads of a
    page one behind the other."""
    case = dict(op="append", seqs=seqs, tokens=tokens, h_q=h_q, h_k=h_k, page=page, kind=kind, rotary=rotary,
                interleaved=interleaved, dtype=dtype, norm=norm, fused=fused, idx=idx, padded=padded, heads_first=heads_first)
    return case if name is None else dict(case, name=name)


def attend(name=None, *, seqs, mean, h_q, h_k, page, tokens=1, ragged=False, prefix=0, dtype="bf16", idx="i32",
           heads_first=False, lens=1):
    """``mean``: tokens of a sequence in its own pages, the ``tokens`` new ones included; ``prefix``: those that all share."""
    case = dict(op="attend", seqs=seqs, tokens=tokens, mean=mean, ragged=ragged, h_q=h_q, h_k=h_k, page=page, prefix=prefix,
                dtype=dtype, idx=idx, heads_first=heads_first, lens=lens)
    return case if name is None else dict(case, name=name)


def log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["axes", "append", "attend", "attend"])
    common = dict(dtype=rng.choice(["bf16", "bf16", "f16"]), idx=rng.choice(["i32", "i64"]))
    h_k = rng.choice([1, 2, 3, 4, 8])
    h_q = h_k * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    turn = dict(rotary=rng.choice([32, 64, 96, 128, 128]), interleaved=rng.random() < 0.4, fused=rng.random() < 0.5)
    if op == "axes":
        return axes(tokens=log_int(rng, 1, MOST_ROPE_HEADS // (h_q + h_k) // 2), h_q=h_q, h_k=h_k, kind=rng.choice(["blocks", "turns"]),
                    weights=rng.random() < 0.8, **turn, **common)
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    common["heads_first"] = rng.random() < 0.3
    if op == "append":
        seqs = log_int(rng, 1, 1024)
        tokens = rng.choice([1, 1, log_int(rng, 1, max(1, MOST_APPEND_HEADS // (seqs * (h_q + 2 * h_k)) // 2))])
        return append(seqs=seqs, tokens=tokens, h_q=h_q, h_k=h_k, page=page, kind=rng.choice(["one", "one", "blocks", "turns"]),
                      norm=rng.random() < 0.7, padded=rng.randint(0, seqs * tokens // 4), **turn, **common)
    seqs, tokens = log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 4])
    mean = log_int(rng, tokens, max(tokens, min(131072, MOST_KEYS // (seqs * h_k) // 2)))
    prefix = log_int(rng, 1, min(131072, MOST_SCORES // (seqs * tokens * h_q) // 2)) if rng.random() < 0.5 else 0
    if prefix:
        mean = min(mean, 4096)
    return attend(seqs=seqs, tokens=tokens, mean=mean, ragged=rng.random() < 0.7, h_q=h_q, h_k=h_k, page=page, prefix=prefix,
                  lens=rng.randrange(1 << 20), **common)


def lengths(case):
    """Tokens of each sequence in its own pages: all ``mean``, or even draws up to twice that."""
    if not case["ragged"]:
        return [case["mean"]] * case["seqs"]
    rng = random.Random(case["lens"])
    return [rng.randint(case["tokens"], max(case["tokens"], 2 * case["mean"] - case["tokens"])) for _ in range(case["seqs"])]


def axis_of_pairs(case):
    """The axis that turns each of the rotary / 2 pairs: time the first quarter and height and width half of the rest
    each, or the three in turns.  None where tokens have a single position."""
    pairs = case["rotary"] // 2
    if case["kind"] == "one":
        return None
    if case["kind"] == "turns":
        return [i % 3 for i in range(pairs)]
    time = pairs // 4
    height = (pairs - time) // 2
    return [0] * time + [1] * height + [2] * (pairs - time - height)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, idx = TYPES[case["dtype"]], INTS[case["idx"]]
    h_q, h_k = case["h_q"], case["h_k"]

    def normal(*shape, std=1.0):
        made = torch.empty(shape, dtype=dtype, device="cuda")
        for part in made.view(-1).split(1 << 28):   # a cache of gigabytes is not made in 32 bits at once
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * std)
        return made

    def below(high, *shape):
        return torch.randint(high, shape, generator=gen, device="cuda")

    def cache(pages):
        if case["heads_first"]:
            return normal(pages, h_k, case["page"], D).transpose(1, 2)
        return normal(pages, case["page"], h_k, D)

    if case["op"] == "attend":
        lens, page = lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        shared = -(-case["prefix"] // page)
        pool = shared + sum(need) + 3
        place = torch.randperm(pool, generator=gen, device="cuda").to(idx)
        table = torch.full((case["seqs"], max(need)), -1, dtype=idx, device="cuda")   # no page behind a sequence's last
        at = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
        table[at] = place[shared:shared + sum(need)]
        return dict(case=case, q=normal(case["seqs"] * case["tokens"], h_q, D, std=2.0), k_cache=cache(pool), v_cache=cache(pool),
                    table=table, lengths=torch.tensor(lens, device="cuda").to(idx), longest=max(lens),
                    prefix_pages=place[:shared].contiguous() if shared else None)
    t = case["tokens"] if case["op"] == "axes" else case["seqs"] * case["tokens"]
    if case["fused"]:   # the projection's output: queries, keys and values side by side
        q, k, v = normal(t, h_q + 2 * h_k, D).split([h_q, h_k, h_k], dim=1)
    else:
        q, k, v = normal(t, h_q, D), normal(t, h_k, D), normal(t, h_k, D)
    r, pairs = case["rotary"], axis_of_pairs(case)
    places = PLACES if pairs else max(PLACES, 2 * case["tokens"])
    angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    made = dict(case=case, q=q, k=k, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), pair_axes=pairs)
    if pairs:   # frames of 24 x 32 patches, from some time on
        i = torch.arange(t, device="cuda")
        time = (i // 768 + below(PLACES - 256, 1)) % PLACES
        made["positions"] = torch.stack([time, i // 32 % 24, i % 32]).to(idx).contiguous()
    else:       # each sequence goes on where it is
        first = below(places - case["tokens"] + 1, case["seqs"], 1)
        made["positions"] = (first + torch.arange(case["tokens"], device="cuda")).reshape(-1).to(idx)
    weights = case["weights"] if case["op"] == "axes" else case["norm"]
    made["weights"] = [1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda") if weights else None for _ in range(2)]
    if case["op"] == "axes":
        return made
    n, page = case["seqs"], case["page"]   # each sequence's new tokens: from a random place of its first page on
    each = -(-(case["tokens"] + page - 1) // page)
    pool = n * each + 3
    own_pages = torch.randperm(pool, generator=gen, device="cuda")[:n * each].view(n, each)
    at = below(page, n, 1) + torch.arange(case["tokens"], device="cuda")
    slots = (own_pages.gather(1, at // page) * page + at % page).reshape(-1)
    if case["padded"]:
        slots[t - case["padded"]:] = -1
    return dict(made, v=v, slots=slots.to(idx), k_cache=cache(pool), v_cache=cache(pool))


def run(state):
    s, case = state, state["case"]
    if own:
        import gated_delta_rule_24_gb300 as gdn

        if case["op"] == "axes":
            return gdn.qk_norm_rope(s["q"], s["k"], s["cos_sin"], s["positions"], *s["weights"], interleaved=case["interleaved"],
                                    pair_axes=s["pair_axes"])
        if case["op"] == "append":
            q = gdn.norm_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["cos_sin"], s["positions"],
                                     *s["weights"], norm=case["norm"], interleaved=case["interleaved"], pair_axes=s["pair_axes"])
            return q, s["k_cache"], s["v_cache"]
        return gdn.paged_attention_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], prefix_pages=s["prefix_pages"],
                                        prefix_length=case["prefix"], return_lse=True)
    if case["op"] == "attend":
        return plain_attend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["longest"], s["prefix_pages"], case["prefix"],
                            case["tokens"])
    norm = case["op"] == "axes" or case["norm"]
    turned = [plain_turn(x, w, norm, s["cos_sin"], s["positions"], s["pair_axes"], case["interleaved"])
              for x, w in ((s["q"], s["weights"][0]), (s["k"], s["weights"][1]))]
    if case["op"] == "axes":
        return tuple(turned)
    slots, k, v = s["slots"].long(), turned[1], s["v"]
    if case["padded"]:
        there = slots >= 0
        slots, k, v = slots[there], k[there], v[there]
    at = torch.div(slots, case["page"], rounding_mode="floor"), slots % case["page"]
    s["k_cache"][at] = k
    s["v_cache"][at] = v
    return turned[0], s["k_cache"], s["v_cache"]


def plain_turn(x, weight, norm, cos_sin, positions, pair_axes, interleaved):
    r = cos_sin.shape[1]
    y = x.float()
    if norm:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        y = y * weight
    if pair_axes is None:
        cos, sin = cos_sin[positions][:, None].chunk(2, dim=-1)
    else:
        axis, pair = torch.tensor(pair_axes, device=x.device), torch.arange(r // 2, device=x.device)
        place = positions[axis].t()   # [tokens, pairs]
        cos, sin = cos_sin[place, pair][:, None], cos_sin[place, pair + r // 2][:, None]
    if interleaved:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def plain_attend(q, k_cache, v_cache, table, lengths, longest, prefix_pages, prefix, tokens):
    """All sequences at once, each padded to the longest; the prefix once for all rows."""
    n, h_q, h_k = lengths.shape[0], q.shape[1], k_cache.shape[2]
    g = h_q // h_k
    rows = q.float().mul(D ** -0.5).reshape(n, tokens, h_k, g, D).permute(0, 2, 1, 3, 4).reshape(n, h_k, tokens * g, D)

    def own_pages(cache):   # [n, h_k, longest, D]
        return cache[table.long()].flatten(1, 2)[:, :longest].permute(0, 2, 1, 3).float()

    def shared_pages(cache):   # [h_k, prefix, D]
        return cache[prefix_pages.long()].flatten(0, 1)[:prefix].permute(1, 0, 2).float()

    seen = lengths[:, None] - tokens + 1 + torch.arange(tokens, device=q.device)   # own keys that each token sees
    hidden = torch.arange(longest, device=q.device) >= seen.repeat_interleave(g, 1)[:, None, :, None]
    scores = (rows @ own_pages(k_cache).transpose(-1, -2)).masked_fill(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if prefix:
        together = rows.transpose(0, 1).reshape(h_k, n * tokens * g, D)
        more = together @ shared_pages(k_cache).transpose(-1, -2)
        top = torch.maximum(top, more.amax(-1, keepdim=True).view(h_k, n, tokens * g, 1).transpose(0, 1))
        more.sub_(top.transpose(0, 1).reshape(h_k, n * tokens * g, 1)).exp_()
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    out = scores @ own_pages(v_cache)
    if prefix:
        total = total + more.sum(-1, keepdim=True).view(h_k, n, tokens * g, 1).transpose(0, 1)
        out = out + (more @ shared_pages(v_cache)).view(h_k, n, tokens * g, D).transpose(0, 1)

    def by_token(x):
        return x.view(n, h_k, tokens, g, -1).permute(0, 2, 1, 3, 4).reshape(n * tokens, h_q, -1)

    return by_token(out / total).to(q.dtype), by_token(top + total.log())[..., 0].contiguous()


def work(case):
    b, h_q, h_k = SIZE[case["dtype"]], case["h_q"], case["h_k"]
    if case["op"] == "attend":
        lens, t = lengths(case), case["tokens"]
        keys = sum(lens) + case["prefix"]
        pages = sum(-(-n // case["page"]) for n in lens + [case["prefix"]])
        pairs = sum(t * n - t * (t - 1) // 2 for n in lens) + len(lens) * t * case["prefix"]
        return {"bytes": 2 * b * D * h_k * keys + len(lens) * t * h_q * (2 * b * D + 4) + SIZE[case["idx"]] * (pages + len(lens)),
                "flops": 4 * D * h_q * pairs}
    r, append_ = case["rotary"], case["op"] == "append"
    t = case["seqs"] * case["tokens"] if append_ else case["tokens"]
    real = t - case["padded"] if append_ else t
    values = (t * h_q + real * h_k) * D
    index = SIZE[case["idx"]] * t * ((1 if case["kind"] == "one" else 3) + (1 if append_ else 0))
    weights = 2 * D * 4 if (case["norm"] if append_ else case["weights"]) else 0
    # the table's places that the tokens turn by, each once
    table = 4 * r * (t if case["kind"] == "one" else min(t, 24 + 32 + t // 768 + 1))
    return {"bytes": 2 * b * (values + (real * h_k * D if append_ else 0)) + min(table, 4 * r * max(PLACES, 2 * t)) + index + weights,
            "flops": 4 * values + 3 * values * r // D}


def exact(case, seed):
    """The definitions in 64 bits: complex turns for the rotation, one sequence after the other for the attention."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        return exact_attend(s)
    q, k = (exact_turn(s, x, w) for x, w in ((s["q"], s["weights"][0]), (s["k"], s["weights"][1])))
    if case["op"] == "axes":
        return q, k
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    real = case["seqs"] * case["tokens"] - case["padded"]
    page, at = (x[:real].long() for x in torch.unravel_index(s["slots"][:real].long(), k_cache.shape[:2]))
    k_cache.index_put_((page, at), k[:real])
    v_cache.index_put_((page, at), s["v"][:real].double())
    return q, k_cache, v_cache


def exact_turn(s, x, weight):
    case = s["case"]
    r, pairs = case["rotary"], s["pair_axes"]
    y = x.double()
    if case["op"] == "axes" or case["norm"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6)
    if weight is not None:
        y = y * weight.double()
    at = s["positions"].long()
    by_axis = [s["cos_sin"].double()[p] for p in (at if pairs else at[None])]   # [tokens, r] for each axis
    table = torch.stack([torch.complex(by_axis[a][:, i], by_axis[a][:, r // 2 + i])
                         for i, a in enumerate(pairs or [0] * (r // 2))], 1)[:, None]
    two = y[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(two.contiguous()) * table)
    y[..., :r] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return y


def exact_attend(s):
    case = s["case"]
    h_q, h_k, t, page = case["h_q"], case["h_k"], case["tokens"], case["page"]
    out = torch.empty(case["seqs"] * t, h_q, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(case["seqs"] * t, h_q, dtype=torch.float64, device="cuda")

    def keys_of(cache, pages, n):
        return cache[pages.long()].double().reshape(-1, h_k, D)[:n]

    shared = [keys_of(c, s["prefix_pages"], case["prefix"]) for c in (s["k_cache"], s["v_cache"])] if case["prefix"] else None
    for i, n in enumerate(lengths(case)):
        pages = s["table"][i, :-(-n // page)]
        k, v = (keys_of(c, pages, n) for c in (s["k_cache"], s["v_cache"]))
        q = s["q"][i * t:(i + 1) * t].double().view(t, h_k, h_q // h_k, D) / math.sqrt(D)
        score = torch.einsum("thgd,lhd->hgtl", q, k)
        for j in range(t):
            score[:, :, j, n - t + 1 + j:] = -math.inf
        if shared:
            score = torch.cat([torch.einsum("thgd,lhd->hgtl", q, shared[0]), score], -1)
        weight = torch.softmax(score, -1)
        both = torch.einsum("hgtl,lhd->thgd", weight[..., case["prefix"]:], v)
        if shared:
            both = both + torch.einsum("hgtl,lhd->thgd", weight[..., :case["prefix"]], shared[1])
        out[i * t:(i + 1) * t] = both.reshape(t, h_q, D)
        lse[i * t:(i + 1) * t] = torch.logsumexp(score, -1).permute(2, 0, 1).reshape(t, h_q)
    return out, lse
