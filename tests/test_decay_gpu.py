"""Decay linear attention (prefill and one-token step) against the 64-bit recurrence."""
import math

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def run_and_check(lengths, h_qk, h_v, dtype=BF, gate="token", state=F32, init=True, pool=None, seed=0, **kw):
    q, k, v, g, cu = R.make(lengths, h_qk, h_v, dtype, gate, seed)
    N, H = len(lengths), max(h_qk, h_v)
    slots = N if pool is None else pool
    s0 = R.states(slots, H, state, seed) if init else None
    idx = None
    if pool is not None:
        idx = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:N].cuda()
    final = torch.full((slots, H, 128, 128), 7.0, dtype=state, device="cuda")
    out, got = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu,
                                          output_state=final, state_indices=idx, **kw)
    assert got is final
    at = torch.arange(N) if idx is None else idx.cpu()
    o_ref, s_ref = R.recurrence(q, k, v, g, kw.get("scale") or SCALE, None if s0 is None else s0[at.cuda()], lengths)
    R.check(out, o_ref, final[at.cuda()], s_ref, lengths)
    rest = sorted(set(range(slots)) - set(at.tolist()))
    assert bool((final[rest] == 7.0).all())
    return out, final


@pytest.mark.parametrize("lengths", [[1], [2, 1], [63, 64, 65], [127, 128, 129], [0, 5, 0], [255, 0, 256, 257, 1],
                                     [700, 384]], ids=str)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_lengths(lengths, dtype):
    run_and_check(lengths, 2, 2, dtype, seed=sum(lengths))


@pytest.mark.parametrize("heads", [(1, 1), (1, 4), (2, 4), (4, 2), (3, 6), (6, 1)], ids=str)
@pytest.mark.parametrize("gate", ["token", "head", "slow", "reset", "none"])
def test_heads_and_gates(heads, gate):
    run_and_check([130, 17, 260], *heads, gate=gate, seed=heads[0])


@pytest.mark.parametrize("dtype,state", [(BF, F32), (BF, BF), (BF, HF), (HF, F32), (HF, BF), (HF, HF)], ids=str)
@pytest.mark.parametrize("init,pool", [(False, None), (True, None), (True, 9)])
def test_states(dtype, state, init, pool):
    run_and_check([1, 200, 0, 128, 300], 2, 4, dtype, "head", state, init, pool, seed=3)


def test_long_memory_and_scale():
    run_and_check([3000, 2049], 1, 2, gate="slow", seed=4, scale=0.25)
    run_and_check([1500], 1, 1, HF, gate="none", seed=5)


def test_mixed_state_types_and_no_final_state():
    q, k, v, g, cu = R.make([150, 20], 2, 2, seed=6)
    s0 = R.states(2, 2, BF, 6)
    final = torch.empty(2, 2, 128, 128, device="cuda")
    out, _ = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu,
                                        output_state=final)
    R.check(out, *(x for x in (R.recurrence(q, k, v, g, SCALE, s0, [150, 20])[0], final,
                               R.recurrence(q, k, v, g, SCALE, s0, [150, 20])[1])), [150, 20])
    only = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, cu_seqlens=cu)
    assert torch.equal(only, out)


def test_strides_and_gate_types():
    """q, k, v slices of one buffer, a strided output, a gate stored heads first, 64-bit offsets of 16-bit gates."""
    lengths, H = [140, 3, 129], 3
    T = sum(lengths)
    buf = torch.randn(T, 3 * H + 1, 128, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda").to(BF)
    q, k, v = buf[:, :H], buf[:, H:2 * H], buf[:, 2 * H:3 * H]
    _, _, _, g, cu = R.make(lengths, H, H, seed=7)
    for gate in (g.t().contiguous().t(), g.to(BF), g.to(HF)):
        wide = torch.full((T, 2 * H, 128), 3.0, dtype=BF, device="cuda")
        out = wide[:, 1::2]
        _, st = gdn.decay_linear_attention(q, k, v, gate, cu_seqlens=cu.long(), output=out, output_final_state=True)
        o_ref, s_ref = R.recurrence(q, k, v, gate.float(), SCALE, None, lengths)
        R.check(out, o_ref, st, s_ref, lengths)
        assert bool((wide[:, ::2] == 3.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_do_not_leak(bad):
    """Rows of one sequence share a tile with the next one's: infinities and NaN there stay there."""
    lengths = [100, 60, 129, 5]
    q, k, v, g, cu = R.make(lengths, 1, 2, seed=8)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None, lengths)
    for x in (q, k, v):
        x[100:160] = bad
    q[289:] = bad
    k[289:] = bad
    v[289:] = bad
    g[100:160] = float("nan")
    out, st = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu)
    R.check(out, o_ref, st, s_ref, lengths, which=(0, 2))
    assert not bool(torch.isfinite(out[100:160]).all())


def test_empty_batches():
    q, k, v, g, cu = R.make([0, 0], 2, 2, seed=9)
    s0 = R.states(2, 2, F32, 9)
    out, st = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    assert out.shape == (0, 2, 128) and torch.equal(st, s0)
    out, st = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu)
    assert not bool(st.any())
    out, st = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu[:1])
    assert st.shape[0] == 0


@pytest.mark.parametrize("state", [F32, BF], ids=["f32", "bf16"])
def test_empty_sequences_pass_states_through(state):
    lengths = [0, 40, 0]
    q, k, v, g, cu = R.make(lengths, 2, 2, seed=10)
    s0 = R.states(3, 2, state, 10)
    _, st = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(st[0], s0[0]) and torch.equal(st[2], s0[2])


def test_bad_bounds_and_slots_are_skipped():
    lengths = [70, 30, 200]
    q, k, v, g, cu = R.make(lengths, 2, 2, seed=11)
    s0 = R.states(5, 2, F32, 11)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, s0[[4, 1, 2]], lengths)
    for cu_bad, idx, bit in (([0, 70, 100, 301], [4, 1, 2], 1), ([0, 70, 100, 300], [4, 1, 5], 2),
                             ([0, 70, 100, 300], [4, 1, -1], 2), ([0, 70, 100, 99], [4, 1, 2], 1)):
        out, final = torch.zeros(300, 2, 128, dtype=BF, device="cuda"), torch.zeros_like(s0)
        gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, output_state=final, output=out,
                                   cu_seqlens=torch.tensor(cu_bad, device="cuda"), state_indices=torch.tensor(idx, device="cuda"))
        assert gdn.device_status() == bit
        R.check(out, o_ref, final[[4, 1, 2]], s_ref, lengths, which=(0, 1))
        assert not bool(out[100:].any()) and not bool(final[[0, 2, 3]].any())


def test_bits_do_not_depend_on_the_batch_or_the_run():
    lengths = [300, 77, 1025]
    q, k, v, g, cu = R.make(lengths, 2, 4, seed=12)
    kw = dict(output_final_state=True, batch_invariant=True)
    out, st = gdn.decay_linear_attention(q, k, v, g, cu_seqlens=cu, **kw)
    again, st2 = gdn.decay_linear_attention(q, k, v, g, cu_seqlens=cu, **kw)
    assert torch.equal(out, again) and torch.equal(st, st2)
    one, st1 = gdn.decay_linear_attention(q[377:], k[377:], v[377:], g[377:], cu_seqlens=torch.tensor([0, 1025], device="cuda"), **kw)
    assert torch.equal(one, out[377:]) and torch.equal(st1[0], st[2])


def test_streams_and_graphs():
    lengths = [260, 40]
    q, k, v, g, cu = R.make(lengths, 2, 2, seed=13)
    want, st_want = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, st = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(st, st_want)
    state = st_want.clone()
    row = (q[:2].clone(), k[:2].clone(), v[:2].clone())
    graph = torch.cuda.CUDAGraph()
    out, st = torch.empty_like(want), torch.empty_like(st_want)
    step_out = torch.empty(2, 2, 128, dtype=BF, device="cuda")
    with torch.cuda.graph(graph):
        gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu, output=out, output_state=st)
        gdn.decay_linear_step(*row, state, g[:2], output=step_out)
    for x in (q, k, v):
        x.copy_(torch.randn_like(x))
    graph.replay()
    R.check(out, *(R.recurrence(q, k, v, g, SCALE, None, lengths)[0], st, R.recurrence(q, k, v, g, SCALE, None, lengths)[1]), lengths)
    o_ref, s_ref = R.recurrence(*row, g[:2], SCALE, st_want, [1, 1])
    R.check(step_out, o_ref, state, s_ref, [1, 1])


# ------------------------------------------------------------------------------- one token


@pytest.mark.parametrize("rows", [1, 3, 37])
@pytest.mark.parametrize("heads", [(1, 1), (2, 4), (6, 3)], ids=str)
@pytest.mark.parametrize("dtype,state", [(BF, F32), (BF, BF), (HF, F32), (HF, HF), (HF, BF)], ids=str)
def test_step(rows, heads, dtype, state):
    q, k, v, g, _ = R.make([1] * rows, *heads, dtype, seed=rows)
    H, slots = max(heads), rows + 5
    pool = R.states(slots, H, state, rows)
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(rows))[:rows].cuda().to(torch.int32)
    before = pool.clone()
    out = gdn.decay_linear_step(q, k, v, pool, g, state_indices=idx)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, before[idx.long()], [1] * rows)
    R.check(out, o_ref, pool[idx.long()], s_ref, [1] * rows)
    rest = sorted(set(range(slots)) - set(idx.tolist()))
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("gate", ["head", "reset", "none"])
def test_step_gates_and_defaults(gate):
    q, k, v, g, _ = R.make([1] * 9, 2, 2, gate=gate, seed=20)
    pool = R.states(9, 2, F32, 20)
    before = pool.clone()
    out = gdn.decay_linear_step(q, k, v, pool, g, scale=0.5)
    R.check(out, *(R.recurrence(q, k, v, g, 0.5, before, [1] * 9)[0], pool, R.recurrence(q, k, v, g, 0.5, before, [1] * 9)[1]),
            [1] * 9)


def test_step_strides():
    """Slices of one projection, a pool with other data between its heads, a strided output."""
    B, H = 5, 2
    buf = torch.randn(B, 3 * H, 128, generator=torch.Generator(device="cuda").manual_seed(21), device="cuda").to(BF)
    q, k, v = buf[:, :H], buf[:, H:2 * H], buf[:, 2 * H:]
    _, _, _, g, _ = R.make([1] * B, H, H, seed=21)
    wide = R.states(B, 2 * H, BF, 21)
    pool, before = wide[:, ::2], wide.clone()
    out = torch.zeros(B, 2 * H, 128, dtype=BF, device="cuda")
    gdn.decay_linear_step(q, k, v, pool, g.t().contiguous().t(), output=out[:, 1::2])
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, before[:, ::2], [1] * B)
    R.check(out[:, 1::2], o_ref, pool, s_ref, [1] * B)
    assert torch.equal(wide[:, 1::2], before[:, 1::2]) and not bool(out[:, ::2].any())


def test_step_bad_slot_is_skipped():
    q, k, v, g, _ = R.make([1] * 3, 1, 2, seed=22)
    pool = R.states(4, 2, F32, 22)
    before = pool.clone()
    out = torch.zeros(3, 2, 128, dtype=BF, device="cuda")
    gdn.decay_linear_step(q, k, v, pool, g, state_indices=torch.tensor([3, 4, -1], device="cuda"), output=out)
    assert gdn.device_status() == 2
    o_ref, s_ref = R.recurrence(q[:1], k[:1], v[:1], g[:1], SCALE, before[3:], [1])
    R.check(out[:1], o_ref, pool[3:], s_ref, [1])
    assert torch.equal(pool[:3], before[:3]) and not bool(out[1:].any())
    assert gdn.decay_linear_step(q[:0], k[:0], v[:0], pool, g[:0]).shape == (0, 2, 128)


def test_prompt_then_steps_is_one_sequence():
    prompt, steps = [130, 1, 64], 3
    lengths = [n + steps for n in prompt]
    q, k, v, g, cu = R.make(lengths, 2, 2, gate="head", seed=23)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None, lengths)
    first = cu[:-1].tolist()
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(first, prompt)]).cuda()
    out, pool = gdn.decay_linear_attention(q[rows], k[rows], v[rows], g, output_final_state=True,
                                           cu_seqlens=torch.tensor([0, 130, 131, 195], device="cuda"))
    assert R.rel(out, o_ref[rows]) <= R.OUT[BF]
    for j in range(steps):
        at = torch.tensor([a + n + j for a, n in zip(first, prompt)], device="cuda")
        out = gdn.decay_linear_step(q[at], k[at], v[at], pool, g)
        assert R.rel(out, o_ref[at]) <= R.OUT[BF]
    assert R.rel(pool, s_ref) <= R.STATE[F32]


def test_offsets_past_32_bits():
    """Slots more than 2^31 elements into a pool, tokens more than 2^31 elements apart."""
    slots = (1 << 31) // (2 * 128 * 128) + 3
    pool = torch.empty(slots, 2, 128, 128, dtype=BF, device="cuda")
    idx = torch.tensor([slots - 1, 0], device="cuda")
    pool[idx] = R.states(2, 2, BF, 24)
    before = pool[idx].clone()
    q, k, v, g, cu = R.make([140, 2], 2, 2, seed=24)
    final = torch.empty_like(pool)
    out, _ = gdn.decay_linear_attention(q, k, v, g, initial_state=pool, output_state=final, output_final_state=True,
                                        cu_seqlens=cu, state_indices=idx)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, before, [140, 2])
    R.check(out, o_ref, final[idx], s_ref, [140, 2])
    out = gdn.decay_linear_step(q[:2], k[:2], v[:2], pool, g[:2], state_indices=idx)
    o_ref, s_ref = R.recurrence(q[:2], k[:2], v[:2], g[:2], SCALE, before, [1, 1])
    R.check(out, o_ref, pool[idx], s_ref, [1, 1])
    del final, pool
    far = 1 << 24   # elements between tokens: 142 of them span 2^31
    room = torch.empty(142 * far, dtype=BF, device="cuda")
    spread = [room.as_strided((142, 2, 128), (far, 128, 1), o) for o in (0, 256, 512)]
    for x, y in zip(spread, (q, k, v)):
        x.copy_(y)
    want = gdn.decay_linear_attention(q, k, v, g, cu_seqlens=cu)
    assert torch.equal(gdn.decay_linear_attention(*spread, g, cu_seqlens=cu), want)
    assert math.isfinite(float(want.float().sum()))


# ------------------------------------------------------------------------------- sequences cut into segments


@pytest.mark.parametrize("splits", [2, 3, 5, 8])
@pytest.mark.parametrize("dtype,state,init,pool", [(BF, F32, True, None), (BF, BF, True, 7), (HF, F32, False, None)], ids=str)
def test_segments(force_split, splits, dtype, state, init, pool):
    """Segments of whole chunks, some of them empty: every output and final state as uncut."""
    force_split(splits)
    run_and_check([1100, 0, 1, 129, 384], 2, 4, dtype, "head", state, init, pool, seed=30 + splits)


@pytest.mark.parametrize("gate", ["token", "slow", "reset", "none"])
def test_segments_and_gates(force_split, gate):
    force_split(4)
    run_and_check([900, 530], 1, 2, gate=gate, seed=40)


def test_segments_skip_bad_sequences(force_split):
    force_split(3)
    lengths = [400, 300, 500]
    q, k, v, g, cu = R.make(lengths, 1, 2, seed=41)
    s0 = R.states(3, 2, F32, 41)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, s0, lengths)
    out, final = torch.zeros(1200, 2, 128, dtype=BF, device="cuda"), torch.zeros_like(s0)
    gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, output_state=final, output=out,
                               cu_seqlens=cu, state_indices=torch.tensor([0, 3, 2], device="cuda"))
    assert gdn.device_status() == 2
    R.check(out, o_ref, final, s_ref, lengths, which=(0, 2))
    assert not bool(out[400:700].any()) and not bool(final[1].any())


def test_planned_segments():
    """Few heads and a long sequence: the library cuts it by itself, the same way every time."""
    assert gdn.gdn_decay_workspace_bytes(1, 2, 9000) > 0 and gdn.gdn_decay_workspace_bytes(64, 16, 64 * 256) == 0
    out, st = run_and_check([9000], 1, 2, gate="slow", seed=42)
    again, st2 = run_and_check([9000], 1, 2, gate="slow", seed=42)
    assert torch.equal(out, again) and torch.equal(st, st2)
    whole, _ = run_and_check([9000], 1, 2, gate="slow", seed=42, batch_invariant=True)
    assert R.rel(out, whole) <= R.OUT[BF]


def test_segments_in_a_graph():
    q, k, v, g, cu = R.make([9000], 2, 2, gate="head", seed=43)
    need = gdn.gdn_decay_workspace_bytes(1, 2, 9000)
    gdn.gdn_reserve_workspace(need)
    out, st = torch.empty(9000, 2, 128, dtype=BF, device="cuda"), torch.empty(1, 2, 128, 128, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu, output=out, output_state=st)
    for x in (q, k, v):
        x.copy_(torch.randn_like(x))
    graph.replay()
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None, [9000])
    R.check(out, o_ref, st, s_ref, [9000])


@pytest.mark.parametrize("splits", [1, 2])
def test_long_runs_of_empty_sequences(force_split, splits):
    """Rounds of empty sequences between others, as every CTA of a persistent grid meets them."""
    force_split(splits)
    lengths = [2] * 200 + [0] * 2000 + [130, 1] * 100
    q, k, v, g, cu = R.make(lengths, 1, 1, seed=50)
    s0 = R.states(len(lengths), 1, F32, 50)
    out, st = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, s0, lengths)
    assert gdn.device_status() == 0
    assert R.rel(out, o_ref) <= R.OUT[BF]
    assert max(R.rel(a, b) for a, b in zip(st, s_ref)) <= R.STATE[F32]
    empty = torch.tensor([n == 0 for n in lengths], device="cuda")
    assert torch.equal(st[empty], s0[empty])


@pytest.mark.parametrize("dtype,into,state", [(BF, F32, F32), (BF, BF, BF), (BF, BF, F32), (HF, F32, HF), (HF, None, BF)], ids=str)
@pytest.mark.parametrize("splits", [1, 2])
def test_more_units_than_sms(force_split, splits, dtype, into, state):
    """More (sequence, head) units than SMs, of very different lengths, some of them empty, states of every pair of types."""
    force_split(splits)
    lengths = [0, 900, 3, 640, 0, 0, 129, 512] * 3 + [2300, 0]
    q, k, v, g, cu = R.make(lengths, 4, 8, dtype, "token", 51)
    N, slots = len(lengths), len(lengths) + 4
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(51))[:N].cuda()
    s0 = None if into is None else R.states(slots, 8, into, 51)
    final = torch.full((slots, 8, 128, 128), 7.0, dtype=state, device="cuda")
    out, _ = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, output_state=final,
                                        cu_seqlens=cu, state_indices=idx)
    assert gdn.device_status() == 0
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None if s0 is None else s0[idx], lengths)
    R.check(out, o_ref, final[idx], s_ref, lengths)
    rest = sorted(set(range(slots)) - set(idx.tolist()))
    assert bool((final[rest] == 7.0).all())


@pytest.mark.parametrize("dtype,state", [(BF, F32), (HF, HF)], ids=str)
def test_segments_of_more_units_than_sms(force_split, dtype, state):
    """As above, cut in two: segments without chunks among the states that are made first, too."""
    force_split(2)
    lengths = [0, 1900, 3, 1640, 0, 0, 129, 1512] * 3 + [2300, 0]
    q, k, v, g, cu = R.make(lengths, 8, 8, dtype, "slow", 53)
    s0 = R.states(len(lengths), 8, state, 53)
    final = torch.full_like(s0, 7.0)
    out, _ = gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, output_state=final, cu_seqlens=cu)
    assert gdn.device_status() == 0
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, s0, lengths)
    R.check(out, o_ref, final, s_ref, lengths)


def test_more_units_than_sms_skip_bad_sequences():
    lengths = [300, 700] * 20
    q, k, v, g, cu = R.make(lengths, 2, 8, seed=52)
    s0 = R.states(40, 8, F32, 52)
    idx = torch.arange(40, device="cuda")
    idx[7], idx[33] = 40, -1
    out, final = torch.zeros(20000, 8, 128, dtype=BF, device="cuda"), torch.zeros_like(s0)
    gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, output_state=final, output=out,
                               cu_seqlens=cu, state_indices=idx)
    assert gdn.device_status() == 2
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, s0, lengths)
    R.check(out, o_ref, final, s_ref, lengths, which=[n for n in range(40) if n not in (7, 33)])
    for n in (7, 33):
        assert not bool(out[cu[n]:cu[n + 1]].any()) and not bool(final[n].any())


def test_example_layer():
    """The example's prompts and steps agree with one long prompt to what their 16-bit states and
    outputs allow: each step rounds the state to bf16 (1.7e-3), eight of them and the roundings on
    either side (2.9e-3 each) are within 1e-2 together."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decay_layer.py")
    spec = importlib.util.spec_from_file_location("decay_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main() <= 1e-2
