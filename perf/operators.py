"""The decay linear-attention operators: cases, inputs, plain forms and exact results.

Three operators of one layer, as a serving program calls them:

* ``rope``: RMS norm of every query and key head, then the position rotation, in one pass;
* ``prefill``: linear attention with a decay, over packed prompts
  (``S_t = g_t S_{t-1} + v_t k_t^T``, ``o_t = scale S_t q_t``), states from and to pools;
* ``step``: one token for each sequence through the same recurrence, states in place.

``own`` false computes them with elementary torch operations in 32 bits; ``own`` true calls
the package's entry points.  Head dimension 128; query/key head ``h / (H / H_qk)`` and
value head ``h / (H / H_v)`` belong to head ``h`` of ``H = max(H_qk, H_v)``.
"""
import math
import random

import torch

own = False

D = 128        # head dimension
CHUNK = 128    # tokens that the plain prefill takes at once
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INTS = {"i32": torch.int32, "i64": torch.int64}
MOST_TOKEN_HEADS = 2 * 65536 * 32   # of the largest prefill
MOST_ROPE_HEADS = 65536 * 48        # (query + key) heads times tokens of the largest rotation
MOST_STEP_BYTES = 1024 * 16 * D * D * 2   # of the states of the largest step


def listed():
    return [
        # one new token of one sequence: all latency
        rope("rope_1_token", tokens=1, h_q=16, h_k=16),
        # a batch of new tokens, half of each head rotated, neighbours paired, fp16, slices of one qkv buffer
        rope("rope_997_half", tokens=997, h_q=8, h_k=2, rotary=64, interleaved=True, dtype="f16", fused=True, idx="i32"),
        # a long prompt, slices of one qkv buffer
        rope("rope_65536", tokens=65536, h_q=32, h_k=16, fused=True),
        # the smallest prompt: one sequence, one head
        prefill("prefill_1x256", seqs=1, mean=256, h_qk=1, h_v=1, init="none", state="f32", gate="token"),
        # eight prompts of mixed lengths (an empty one among them), states carried in
        prefill("prefill_8_varlen", seqs=8, mean=1024, ragged=True, h_qk=4, h_v=8, init="f32", state="f32", gate="token"),
        # the usual batch: equal prompts, one decay for each head
        prefill("prefill_16x4096", seqs=16, mean=4096, h_qk=16, h_v=32, init="bf16", state="bf16", gate="head"),
        # one long prompt on few heads, in fp16
        prefill("prefill_1x32000_fp16", seqs=1, mean=32000, h_qk=8, h_v=8, init="none", state="f32", gate="head", dtype="f16"),
        # two very long prompts, the largest
        prefill("prefill_2x65536", seqs=2, mean=65536, h_qk=16, h_v=32, init="f32", state="f32", gate="token"),
        # many short prompts through a pool of states
        prefill("prefill_1024_short", seqs=1024, mean=136, ragged=True, h_qk=8, h_v=16, init="bf16", state="bf16",
                gate="token", spare=256, cu="i64"),
        # one sequence decoding alone
        step("step_1_row", rows=1, h_qk=16, h_v=32, state="f32", gate="head"),
        # an odd batch, fp16, 32-bit states
        step("step_37_fp16", rows=37, h_qk=3, h_v=6, state="f32", gate="token", dtype="f16", spare=13, idx="i64"),
        # a full batch out of a 16-bit pool
        step("step_1024_pool", rows=1024, h_qk=8, h_v=16, state="bf16", gate="token", spare=256),
    ]


def rope(name=None, *, tokens, h_q, h_k, rotary=128, interleaved=False, dtype="bf16", weights=True, fused=False, idx="i64"):
    case = dict(op="rope", tokens=tokens, h_q=h_q, h_k=h_k, rotary=rotary, interleaved=interleaved, dtype=dtype,
                weights=weights, fused=fused, idx=idx)
    return case if name is None else dict(case, name=name)


def prefill(name=None, *, seqs, mean, h_qk, h_v, init, state, gate, ragged=False, dtype="bf16", spare=-1, cu="i32", lens=1):
    """``spare`` >= 0: the states are slots of pools with so many more slots than sequences."""
    case = dict(op="prefill", seqs=seqs, mean=mean, ragged=ragged, h_qk=h_qk, h_v=h_v, init=init, state=state, gate=gate,
                dtype=dtype, spare=spare, cu=cu, lens=lens)
    return case if name is None else dict(case, name=name)


def step(name=None, *, rows, h_qk, h_v, state, gate, dtype="bf16", spare=-1, idx="i32"):
    case = dict(op="step", rows=rows, h_qk=h_qk, h_v=h_v, state=state, gate=gate, dtype=dtype, spare=spare, idx=idx)
    return case if name is None else dict(case, name=name)


def log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def heads(rng):
    h, ratio = rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([1, 1, 2, 2, 4])
    return (h, h * ratio) if rng.random() < 0.85 else (h * ratio, h)


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "step"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        h_q, h_k = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 8, 16])
        return rope(tokens=log_int(rng, 1, MOST_ROPE_HEADS // (h_q + h_k) // 2), h_q=h_q, h_k=h_k, rotary=rng.choice([32, 64, 96, 128, 128]),
                    interleaved=rng.random() < 0.4, dtype=dtype, weights=rng.random() < 0.8, fused=rng.random() < 0.5,
                    idx=rng.choice(["i32", "i64"]))
    h_qk, h_v = heads(rng)
    h = max(h_qk, h_v)
    gate = rng.choice(["token", "head", "head", "slow", "none"])
    state = rng.choice(["f32", "f32", "bf16", "f16"] if dtype == "f16" else ["f32", "bf16"])
    spare = rng.choice([-1, 0, 5, 64])
    if op == "step":
        most = MOST_STEP_BYTES // (h * D * D * (4 if state == "f32" else 2))
        return step(rows=log_int(rng, 1, min(1024, most)), h_qk=h_qk, h_v=h_v, state=state,
                    gate="token" if gate == "none" else gate, dtype=dtype, spare=spare, idx=rng.choice(["i32", "i64"]))
    seqs = log_int(rng, 1, min(1024, 16384 // h))
    mean = log_int(rng, 1, max(1, min(65536, MOST_TOKEN_HEADS // (seqs * h) // 2)))
    return prefill(seqs=seqs, mean=mean, ragged=rng.random() < 0.7, h_qk=h_qk, h_v=h_v, init=rng.choice(["none", state, state]),
                   state=state, gate=gate, dtype=dtype, spare=spare, cu=rng.choice(["i32", "i64"]), lens=rng.randrange(1 << 20))


def lengths(case):
    """Tokens of each sequence: all ``mean``, or even draws from 0 to twice that."""
    if not case["ragged"]:
        return [case["mean"]] * case["seqs"]
    rng = random.Random(case["lens"])
    return [rng.randint(0, 2 * case["mean"]) for _ in range(case["seqs"])]


def gates(kind, rows, h, gen):
    """Decay of the state by each token: one for each head, one for each token and head, or none."""
    if kind == "none":
        return None
    if kind == "head":   # a geometric ladder of memories, from one token to 256
        return torch.exp(-torch.pow(2.0, -8.0 * torch.arange(1, h + 1, device="cuda") / h))
    if kind == "slow":   # memories of thousands of tokens
        return torch.exp(-0.001 * torch.rand(rows, h, generator=gen, device="cuda"))
    a = torch.rand(h, generator=gen, device="cuda") * 3.0 - 2.0
    x = torch.randn(rows, h, generator=gen, device="cuda")
    return torch.exp(-torch.exp(a) * torch.nn.functional.softplus(x))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    dtype = TYPES[case["dtype"]]
    if case["op"] == "rope":
        t, h_q, h_k, r = case["tokens"], case["h_q"], case["h_k"], case["rotary"]
        if case["fused"]:   # the projection's output: queries, keys and as many values side by side
            qkv = normal(t, h_q + 2 * h_k, D, dtype=dtype)
            q, k = qkv[:, :h_q], qkv[:, h_q:h_q + h_k]
        else:
            q, k = normal(t, h_q, D, dtype=dtype), normal(t, h_k, D, dtype=dtype)
        places = max(4096, t)
        angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            10000.0, -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        at = torch.arange(t, device="cuda")   # prompts one after another, from an odd start
        at = (at + int(torch.randint(places, (1,), generator=gen, device="cuda"))) % places
        weight = [1.0 + normal(D, dtype=torch.float32, std=0.1) if case["weights"] else None for _ in range(2)]
        return dict(case=case, q=q, k=k, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                    positions=at.to(INTS[case["idx"]]), q_weight=weight[0], k_weight=weight[1])
    h_qk, h_v = case["h_qk"], case["h_v"]
    h = max(h_qk, h_v)
    if case["op"] == "step":
        rows = n = case["rows"]
    else:
        lens = lengths(case)
        rows, n = sum(lens), len(lens)
    slots = n + max(0, case["spare"])
    made = dict(case=case, q=normal(rows, h_qk, D, dtype=dtype), k=normal(rows, h_qk, D, dtype=dtype),
                v=normal(rows, h_v, D, dtype=dtype), g=gates(case["gate"], rows, h, gen), indices=None)
    idx = INTS[case["idx"]] if case["op"] == "step" else torch.int32
    if case["spare"] >= 0:
        made["indices"] = torch.randperm(slots, generator=gen, device="cuda")[:n].to(idx)
    if case["op"] == "step":
        made["state"] = normal(slots, h, D, D, dtype=TYPES[case["state"]])
        return made
    made["initial"] = None if case["init"] == "none" else normal(slots, h, D, D, dtype=TYPES[case["init"]])
    made["final"] = torch.zeros(slots, h, D, D, dtype=TYPES[case["state"]], device="cuda")
    made["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(INTS[case["cu"]])
    made["longest"] = max(lens)
    return made


def run(state):
    s = state
    if own:
        import gated_delta_rule_24_gb300 as gdn

        if s["case"]["op"] == "rope":
            return gdn.qk_norm_rope(s["q"], s["k"], s["cos_sin"], s["positions"], s["q_weight"], s["k_weight"],
                                    interleaved=s["case"]["interleaved"])
        if s["case"]["op"] == "prefill":
            return gdn.decay_linear_attention(s["q"], s["k"], s["v"], s["g"], initial_state=s["initial"], output_final_state=True,
                                              cu_seqlens=s["cu"], output_state=s["final"], state_indices=s["indices"])
        return gdn.decay_linear_step(s["q"], s["k"], s["v"], s["state"], s["g"], state_indices=s["indices"]), s["state"]
    if s["case"]["op"] == "rope":
        args = s["cos_sin"], s["positions"], s["case"]["interleaved"]
        return plain_rope(s["q"], s["q_weight"], *args), plain_rope(s["k"], s["k_weight"], *args)
    if s["case"]["op"] == "prefill":
        return plain_prefill(s["q"], s["k"], s["v"], s["g"], s["initial"], s["final"], s["indices"], s["cu"], s["longest"])
    return plain_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["indices"])


def plain_rope(x, weight, cos_sin, positions, interleaved):
    r = cos_sin.shape[1]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        y = y * weight
    cos, sin = cos_sin[positions][:, None].chunk(2, dim=-1)
    if interleaved:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def plain_prefill(q, k, v, g, initial, final, indices, cu, longest):
    """All chunks of all sequences at once, each sequence padded to whole chunks: within a chunk the decayed products
    of queries and keys, between chunks the states, joined by the matrix of decays from chunk to chunk."""
    rows, n = q.shape[0], cu.shape[0] - 1
    h = max(q.shape[1], v.shape[1])
    c = max(1, -(-longest // CHUNK))
    at = cu[:-1, None].long() + torch.arange(c * CHUNK, device=q.device)
    real = at < cu[1:, None]

    def padded(x):   # [rows, heads, 128] -> [n, H, chunks, CHUNK, 128]
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[torch.where(real, at, rows)].float()
        return x.repeat_interleave(h // x.shape[2], dim=2).reshape(n, c, CHUNK, h, D).permute(0, 3, 1, 2, 4)

    qp, kp, vp = padded(q), padded(k), padded(v)
    log_g = torch.zeros(rows + 1, h, device=q.device)
    if g is not None:
        log_g[:rows] = g.float().log()
    log_g = log_g[torch.where(real, at, rows)].reshape(n, c, CHUNK, h).permute(0, 3, 1, 2)
    upto = log_g.cumsum(-1)
    after = log_g.flip(-1).cumsum(-1).flip(-1) - log_g           # decays of the tokens behind each in its chunk
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    within = (upto[..., :, None] - upto[..., None, :]).masked_fill(~low, -math.inf).exp()
    out = (qp @ kp.transpose(-1, -2) * within) @ vp
    del within
    added = (vp * after.exp()[..., None]).transpose(-1, -2) @ kp   # [n, h, c, dv, dk]
    # state before chunk i = sum over j < i of (decays of the chunks between) added_j + (all decays before i) initial
    whole = upto[..., -1]
    total = torch.cat([torch.zeros_like(whole[..., :1]), whole.cumsum(-1)], -1)             # [n, h, c + 1]
    past = torch.ones(c + 1, c, dtype=torch.bool, device=q.device).tril(-1)
    join = (total[..., :, None] - total[..., None, 1:]).masked_fill(~past, -math.inf).exp()   # [n, h, c + 1, c]
    states = (join @ added.reshape(n, h, c, D * D)).reshape(n, h, c + 1, D, D)
    del added, join
    slots = torch.arange(n, device=q.device) if indices is None else indices.long()
    if initial is not None:
        states += total.exp()[..., None, None] * initial[slots].float()[:, :, None]
    out += upto.exp()[..., None] * (qp @ states[:, :, :c].transpose(-1, -2))
    out = (out * D ** -0.5).to(q.dtype).permute(0, 2, 3, 1, 4).reshape(n, c * CHUNK, h, D)
    final[slots] = states[:, :, c].to(final.dtype)
    return out[real], final


def plain_step(q, k, v, g, state, indices):
    h, dtype = max(q.shape[1], v.shape[1]), q.dtype
    q, k, v = (x.float().repeat_interleave(h // x.shape[1], dim=1) for x in (q, k, v))
    slots = torch.arange(q.shape[0], device=q.device) if indices is None else indices.long()
    s = state[slots].float()
    if g is not None:
        s = s * g.float()[..., None, None]
    s = s + v[..., :, None] * k[..., None, :]
    out = ((s * q[..., None, :]).sum(-1) * D ** -0.5).to(dtype)
    state[slots] = s.to(state.dtype)
    return out, state


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b = size[case["dtype"]]
    if case["op"] == "rope":
        t, r = case["tokens"], case["rotary"]
        values = t * (case["h_q"] + case["h_k"]) * D
        return {"bytes": 2 * b * values + t * r * 4 + t * size_of(case["idx"]) + (2 * D * 4 if case["weights"] else 0),
                "flops": 4 * values + 3 * values * r // D}
    h = max(case["h_qk"], case["h_v"])
    lens = [1] * case["rows"] if case["op"] == "step" else lengths(case)
    rows, n = sum(lens), len(lens)
    total = rows * (2 * case["h_qk"] + case["h_v"] + h) * D * b
    total += {"none": 0, "head": 4 * h}.get(case["gate"], 4 * rows * h)
    total += n * h * D * D * size[case["state"]]
    if case["op"] == "step":
        total += n * h * D * D * size[case["state"]]
    elif case["init"] != "none":
        total += n * h * D * D * size[case["init"]]
    return {"bytes": total, "flops": 5 * rows * h * D * D}   # the recurrence: decay, update and read-out


def size_of(kind):
    return {"i32": 4, "i64": 8}[kind]


def exact(case, seed):
    """The definitions in 64 bits: complex turns for the rotation, the recurrence token by token for the rest."""
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(exact_rope(s, x, w) for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])))
    h = max(case["h_qk"], case["h_v"])
    q, k, v = (s[x].double() for x in "qkv")
    q, k, v = (x[:, torch.arange(h, device="cuda") // (h // x.shape[1])] for x in (q, k, v))
    rows = q.shape[0]
    g = torch.ones(rows, h, dtype=torch.float64, device="cuda") if s["g"] is None else s["g"].double().expand(rows, h)
    pool = s["state"] if case["op"] == "step" else s["final"]
    lens = [1] * case["rows"] if case["op"] == "step" else lengths(case)
    n = len(lens)
    slots = list(range(n)) if s["indices"] is None else s["indices"].tolist()
    start = pool if case["op"] == "step" else s["initial"]
    state = torch.zeros(n, h, D, D, dtype=torch.float64, device="cuda") if start is None else start[slots].double()
    out = torch.zeros(rows, h, D, dtype=torch.float64, device="cuda")
    # longest first, so that the sequences still running are always the first ones
    order = sorted(range(n), key=lambda i: -lens[i])
    first, begin = [0] * n, 0
    for i, length in enumerate(lens):
        first[i], begin = begin, begin + length
    state = state[order].reshape(n * h, D, D)
    first_of = torch.tensor([first[i] for i in order], device="cuda")
    alive = n
    for t in range(max(lens)):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        at = first_of[:alive] + t
        part = state[:alive * h]
        part.mul_(g[at].reshape(-1, 1, 1)).baddbmm_(v[at].reshape(-1, D, 1), k[at].reshape(-1, 1, D))
        out[at] = torch.bmm(part, q[at].reshape(-1, D, 1)).reshape(alive, h, D)
    full = pool.double()
    full[[slots[i] for i in order]] = state.reshape(n, h, D, D)
    return out / math.sqrt(D), full


def exact_rope(s, x, weight):
    r = s["case"]["rotary"]
    y = x.double()
    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6)
    if weight is not None:
        y = y * weight.double()
    table = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :r // 2], table[:, r // 2:])[:, None]
    pairs = y[..., :r].unflatten(-1, (r // 2, 2)) if s["case"]["interleaved"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., :r] = (z if s["case"]["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return y
