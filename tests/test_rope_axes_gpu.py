"""Rotation by positions on several axes, and the append of new keys and values to a paged cache, against the
formulas in 64 bits.  Bounds: those of the norm and rotation (test_norm_rope_gpu.py); what is only copied is equal."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A
from tests import decay_ref as R
from tests.test_norm_rope_gpu import close, normal

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def turn(x, weight, offset, eps, cos_sin, positions, interleaved, pair_axes=None, norm=True):
    """The norm (or none) and the rotation in 64 bits."""
    y = x.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (weight.double() + offset)
    if cos_sin is None:
        return y
    half = cos_sin.shape[1] // 2
    i = torch.arange(half, device=x.device)
    if pair_axes is None:
        at = (torch.arange(x.shape[0], device=x.device) if positions is None else positions.long())[:, None].expand(-1, half)
    else:
        at = positions.long()[torch.tensor(pair_axes, device=x.device)].t()
    c, s = cos_sin.double()[at, i][:, None], cos_sin.double()[at, i + half][:, None]
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = y.clone()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., a] * s + y[..., b] * c
    return z


def places(axes, tokens, most, seed, idx=torch.int64):
    return torch.randint(0, most, (axes, tokens), generator=torch.Generator().manual_seed(seed)).cuda().to(idx)


KINDS = {"turns": lambda n, a: [i % a for i in range(n)], "blocks": lambda n, a: [min(a - 1, i * a // n) for i in range(n)],
         "last": lambda n, a: [a - 1] * n, "odd_blocks": lambda n, a: [0 if i < 3 else min(a - 1, 1 + (i - 3) // 5) for i in range(n)]}


@pytest.mark.parametrize("rotary", [16, 32, 48, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_axes(rotary, interleaved, kind, axes):
    dtype = HF if axes % 2 else BF
    q, k, cs = normal(33, 5, 128, dtype=dtype, seed=1), normal(33, 2, 128, dtype=dtype, seed=2), R.table(500, rotary)
    pos, pair_axes = places(axes, 33, 500, 3, torch.int32 if axes < 3 else torch.int64), KINDS[kind](rotary // 2, axes)
    w = 1 + normal(2, 128, dtype=F32, seed=4, std=0.2)
    a, b = gdn.qk_norm_rope(q, k, cs, pos, w[0], w[1], interleaved=interleaved, pair_axes=pair_axes)
    close(a, turn(q, w[0], 0, 1e-6, cs, pos, interleaved, pair_axes))
    close(b, turn(k, w[1], 0, 1e-6, cs, pos, interleaved, pair_axes))


@pytest.mark.parametrize("tokens,h_q,h_k", [(1, 1, 1), (1, 16, 16), (2, 3, 0), (129, 32, 8), (1000, 2, 2), (7001, 16, 4)])
def test_one_axis_is_the_plain_rotation(tokens, h_q, h_k):
    """The same position on every axis: the bits of qk_norm_rope."""
    q, cs = normal(tokens, h_q, 128, seed=5), R.table(9000, 128)
    k = normal(tokens, h_k, 128, seed=6) if h_k else None
    pos = places(1, tokens, 9000, 7)
    want = gdn.qk_norm_rope(q, k, cs, pos[0])
    got = gdn.qk_norm_rope(q, k, cs, pos.expand(3, -1), pair_axes=KINDS["turns"](64, 3))
    assert torch.equal(got[0], want[0]) and (k is None or torch.equal(got[1], want[1]))


def test_axes_in_place_with_bad_positions():
    buf, cs = normal(65, 9, 128, seed=8), R.table(100, 64)
    before, q, k = buf.clone(), buf[:, :4], buf[:, 4:6]
    pos, pair_axes = places(3, 65, 100, 9), KINDS["blocks"](32, 3)
    pos[2, 10], pos[0, 64] = 100, -1
    a, b = (turn(x, None, 0, 1e-6, cs, pos.clamp(0, 99), False, pair_axes) for x in (q, k))
    gdn.qk_norm_rope(q, k, cs, pos, q_out=q, k_out=k, pair_axes=pair_axes)
    assert gdn.device_status() == 8
    good = [i for i in range(65) if i not in (10, 64)]
    close(q[good], a[good])
    close(k[good], b[good])
    assert torch.equal(buf[[10, 64]], before[[10, 64]]) and torch.equal(buf[:, 6:], before[:, 6:])


class Tokens:
    def __init__(self, tokens, h_q, h_k, page=16, dtype=BF, rotary=128, layout="places", idx=torch.int32, axes=0, spare=3, seed=0,
                 weights=True, fused=False):
        self.q, self.k, self.v = normal(tokens, h_q + 2 * h_k, 128, dtype=dtype, seed=seed).split([h_q, h_k, h_k], 1)
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.cs = R.table(600, rotary) if rotary else None
        self.pair_axes = KINDS["odd_blocks"](rotary // 2, axes) if axes else None
        self.pos = places(axes, tokens, 600, seed + 1, idx) if axes else places(1, tokens, 600, seed + 1, idx)[0] if rotary else None
        pages = -(-tokens // page) + spare
        self.k_cache, self.v_cache = A.cache(pages, page, h_k, dtype, layout, seed=seed + 2)
        self.page = page
        self.slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(seed + 3))[:tokens].to(idx).cuda()
        self.w = [1 + normal(128, dtype=F32, seed=seed + 4 + i, std=0.2) if weights else None for i in range(2)]

    def check(self, norm=True, interleaved=False, **kw):
        before = [c.clone() for c in (self.k_cache, self.v_cache)]
        w = self.w if norm else [None, None]
        q = gdn.norm_rope_append(self.q, self.k, self.v, self.k_cache, self.v_cache, self.slots, self.cs, self.pos, *w, norm=norm,
                                 interleaved=interleaved, pair_axes=self.pair_axes, **kw)
        real = self.slots >= 0
        at = self.slots[real].long() // self.page, self.slots[real].long() % self.page
        args = (self.cs, self.pos, interleaved, self.pair_axes, norm)
        close(q, turn(self.q, w[0], 0, 1e-6, *args))
        close(self.k_cache[at], turn(self.k, w[1], 0, 1e-6, *args)[real])
        assert torch.equal(self.v_cache[at], self.v[real])
        for c, b in zip((self.k_cache, self.v_cache), before):   # nothing else was touched
            b[at] = c[at]
            assert torch.equal(c, b)
        return q


@pytest.mark.parametrize("tokens,h_q,h_k", [(1, 1, 1), (1, 16, 2), (3, 5, 5), (37, 12, 4), (500, 32, 8), (5000, 16, 2)])
@pytest.mark.parametrize("layout", ["places", "heads", "woven", "side"])
def test_append(tokens, h_q, h_k, layout):
    i = tokens % 3
    Tokens(tokens, h_q, h_k, page=[16, 24, 64][i], layout=layout, dtype=[BF, HF, BF][i], idx=[torch.int32, torch.int64][i % 2],
           seed=20 + i, fused=tokens % 2 == 1).check(interleaved=i == 1)


@pytest.mark.parametrize("rotary", [0, 16, 64, 112, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("axes", [0, 3])
def test_append_turns(rotary, norm, axes):
    if axes and not rotary:
        pytest.skip("no rotation, no axes")
    for interleaved in (False, True):
        Tokens(41, 6, 3, page=7, rotary=rotary, axes=axes, seed=24, weights=norm).check(norm=norm, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_without_norm_what_does_not_turn_is_copied(dtype):
    """Infinities, the smallest numbers and values beside them, with a rotation of half a head and without one."""
    for rotary in (0, 64):
        t = Tokens(9, 2, 2, dtype=dtype, rotary=rotary, seed=25, weights=False)
        t.k[3, 0, 100], t.k[4, 1, 127], t.k[5, 1, 66] = float("inf"), float("-inf"), 1e-30 if dtype == BF else 6e-8
        t.q[6, 0, 99] = float("inf")
        q = gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, norm=False)
        at = t.slots.long() // t.page, t.slots.long() % t.page
        assert torch.equal(q[..., rotary:], t.q[..., rotary:]) and torch.equal(t.k_cache[at][..., rotary:], t.k[..., rotary:])
        assert bool(t.k_cache[at][..., :rotary].isfinite().all())


def test_values_keep_their_bits():
    t = Tokens(64, 2, 2, seed=26)
    t.v.view(torch.int16).copy_(torch.randint(-32768, 32768, t.v.shape, generator=torch.Generator().manual_seed(1)).to(torch.int16))
    gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos)
    at = t.slots.long() // t.page, t.slots.long() % t.page
    assert torch.equal(t.v_cache.view(torch.int16)[at], t.v.view(torch.int16))


@pytest.mark.parametrize("rotary", [0, 16, 64, 112])
@pytest.mark.parametrize("interleaved", [False, True])
def test_without_norm_what_does_not_turn_keeps_its_bits(rotary, interleaved):
    """Zeros of either sign, NaN of any kind and all else."""
    t = Tokens(64, 2, 2, rotary=rotary, seed=32, weights=False)
    random = torch.randint(-32768, 32768, (2, 64, 2, 128), generator=torch.Generator().manual_seed(2)).to(torch.int16)
    random[:, ::3, :, 1::2], random[:, 1::3, :, ::2] = -32768, 0
    for x, bits in zip((t.q, t.k), random.cuda()):
        x[..., rotary:].view(torch.int16).copy_(bits[..., rotary:])
    q = gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, norm=False, interleaved=interleaved)
    at = t.slots.long() // t.page, t.slots.long() % t.page
    for got, x in ((q, t.q), (t.k_cache[at], t.k)):
        assert torch.equal(got[..., rotary:].contiguous().view(torch.int16), x[..., rotary:].contiguous().view(torch.int16))


def test_padded_and_bad_slots():
    t = Tokens(40, 4, 2, seed=27, idx=torch.int64)
    t.slots[7], t.slots[30:] = -5, -1
    t.check()
    most = t.k_cache.shape[0] * t.page
    t.slots[3], t.slots[5] = most, 1 << 40
    before = [c.clone() for c in (t.k_cache, t.v_cache)]
    q = gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, *t.w)
    assert gdn.device_status() == 0x10
    close(q, turn(t.q, t.w[0], 0, 1e-6, t.cs, t.pos, False))
    assert all(torch.equal(c, b) for c, b in zip((t.k_cache, t.v_cache), before))   # the good ones hold the same again


def test_bad_positions_leave_rows_and_places():
    t = Tokens(20, 4, 2, seed=28)
    t.pos[4], t.pos[9] = 600, -1
    for c in (t.k_cache, t.v_cache):
        c.fill_(3.0)
    q = torch.full_like(t.q, 9.0)
    gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, *t.w, q_out=q)
    assert gdn.device_status() == 8
    good = [i for i in range(20) if i not in (4, 9)]
    close(q[good], turn(t.q, t.w[0], 0, 1e-6, t.cs, t.pos.clamp(0, 599), False)[good])
    assert bool((q[[4, 9]] == 9.0).all())
    at = t.slots.long() // t.page, t.slots.long() % t.page
    for c in (t.k_cache, t.v_cache):
        assert bool((c[at][[4, 9]] == 3.0).all()) and not bool((c[at][good] == 3.0).all(-1).any())


def test_in_place_streams_graphs_and_nothing():
    t = Tokens(50, 4, 2, seed=29, fused=True)
    args = (t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, *t.w)
    want = gdn.norm_rope_append(t.q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = t.k_cache.clone()
    side.wait_stream(torch.cuda.current_stream())
    t.k_cache.record_stream(side)
    got = gdn.norm_rope_append(t.q, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(t.k_cache, kept)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.norm_rope_append(t.q, *args, q_out=out)
    t.q.copy_(normal(50, 4, 128, seed=30))
    t.slots.copy_(t.slots.flip(0))
    graph.replay()
    close(out, turn(t.q, t.w[0], 0, 1e-6, t.cs, t.pos, False))
    at = t.slots.long() // t.page, t.slots.long() % t.page
    assert torch.equal(t.v_cache[at], t.v)
    fresh = gdn.norm_rope_append(t.q, *args)
    gdn.norm_rope_append(t.q, *args, q_out=t.q)
    assert torch.equal(t.q, fresh)
    none = gdn.norm_rope_append(t.q[:0], t.k[:0], t.v[:0], t.k_cache, t.v_cache, t.slots[:0], t.cs, t.pos[:0])
    assert none.shape == (0, 4, 128)


def test_offsets_past_32_bits():
    far = 1 << 24
    room = torch.empty(2 * 140 * far, dtype=BF, device="cuda")
    t = Tokens(300, 2, 1, seed=31, spare=120)
    pages = t.k_cache.shape[0]
    t.k_cache, t.v_cache = (room[i * 140 * far:].as_strided((pages, 16, 1, 128), (far, 128, 128, 1)) for i in range(2))
    w = t.w
    q = gdn.norm_rope_append(t.q, t.k, t.v, t.k_cache, t.v_cache, t.slots, t.cs, t.pos, *w)
    at = t.slots.long() // t.page, t.slots.long() % t.page
    close(q, turn(t.q, w[0], 0, 1e-6, t.cs, t.pos, False))
    close(t.k_cache[at], turn(t.k, w[1], 0, 1e-6, t.cs, t.pos, False))
    assert torch.equal(t.v_cache[at], t.v)
