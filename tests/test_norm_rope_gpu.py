"""The norm of query and key heads with the rotation, against the formula in 64 bits.

Bounds: the arithmetic is in f32 and every value is rounded once to the 16-bit type, so a
value is within half a unit of its type plus a few 2^-24 of the pair that it comes from:
2^-8 |y| (bf16) or 2^-11 |y| (f16), taken as one whole unit, plus 2^-20 of the pair's size;
below f16's normal range its spacing 2^-24 takes the unit's place.
"""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def normal(*shape, dtype=BF, seed=0, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std).to(dtype)


def close(got, ref):
    unit = 2.0 ** -8 if got.dtype == BF else 2.0 ** -11
    size = ref.abs().amax(-1, keepdim=True)
    room = unit * ref.abs() + 2.0 ** -20 * size + (2.0 ** -24 if got.dtype == HF else 0.0)
    bad = (got.double() - ref).abs() > room
    assert not bool(bad.any()), float(((got.double() - ref).abs() / room).max())


@pytest.mark.parametrize("rotary", [16, 32, 48, 64, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_rotary_sizes(rotary, interleaved, dtype):
    q, k = normal(33, 5, 128, dtype=dtype, seed=1), normal(33, 2, 128, dtype=dtype, seed=2)
    cs = R.table(500, rotary)
    pos = torch.randint(0, 500, (33,), generator=torch.Generator().manual_seed(3)).cuda()
    w = 1 + normal(2, 128, dtype=F32, seed=4, std=0.2)
    a, b = gdn.qk_norm_rope(q, k, cs, pos, w[0], w[1], interleaved=interleaved)
    close(a, R.norm_rope(q, w[0], 0, 1e-6, cs, pos, interleaved))
    close(b, R.norm_rope(k, w[1], 0, 1e-6, cs, pos, interleaved))


@pytest.mark.parametrize("tokens,h_q,h_k", [(1, 1, 1), (1, 16, 16), (2, 3, 1), (7, 1, 5), (129, 32, 8), (1000, 2, 2)])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64, None], ids=str)
def test_sizes_and_positions(tokens, h_q, h_k, idx):
    q, k, cs = normal(tokens, h_q, 128, seed=5), normal(tokens, h_k, 128, seed=6), R.table(1000, 128)
    pos = None if idx is None else torch.randint(0, 1000, (tokens,), generator=torch.Generator().manual_seed(7)).cuda().to(idx)
    a, b = gdn.qk_norm_rope(q, k, cs, pos)
    close(a, R.norm_rope(q, None, 0, 1e-6, cs, pos, False))
    close(b, R.norm_rope(k, None, 0, 1e-6, cs, pos, False))


@pytest.mark.parametrize("wtype", [F32, BF, HF], ids=str)
def test_weights_offset_eps(wtype):
    q, k, cs = normal(20, 3, 128, seed=8, std=0.01), normal(20, 3, 128, seed=9, std=30.0), R.table(20, 64)
    w = normal(128, dtype=wtype, seed=10, std=0.3)
    a, b = gdn.qk_norm_rope(q, k, cs, None, w, None, eps=1e-3, weight_offset=1.0)
    close(a, R.norm_rope(q, w, 1.0, 1e-3, cs, None, False))
    close(b, R.norm_rope(k, None, 1.0, 1e-3, cs, None, False))


def test_without_rotation_or_keys():
    q, w = normal(11, 4, 128, seed=11), normal(128, dtype=F32, seed=12)
    a, b = gdn.qk_norm_rope(q, q_weight=w)
    assert b is None
    close(a, R.norm_rope(q, w, 0, 1e-6, None, None, False))
    cs = R.table(11, 32)
    a, _ = gdn.qk_norm_rope(q, None, cs)
    close(a, R.norm_rope(q, None, 0, 1e-6, cs, None, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_slices_of_one_buffer(interleaved):
    buf = normal(65, 9, 128, seed=13)
    before, cs = buf.clone(), R.table(65, 128)
    q, k = buf[:, :4], buf[:, 4:6]
    want = gdn.qk_norm_rope(q, k, cs, interleaved=interleaved)
    got = gdn.qk_norm_rope(q, k, cs, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, 6:], before[:, 6:])


def test_strided_outputs_and_heads():
    buf, cs = normal(40, 8, 128, seed=14), R.table(40, 128)
    q, k = buf[:, ::2], buf[:, 1::4]
    room = torch.zeros(40, 8, 128, dtype=BF, device="cuda")
    gdn.qk_norm_rope(q, k, cs, q_out=room[:, 4:], k_out=room[:, 1:3])
    close(room[:, 4:], R.norm_rope(q, None, 0, 1e-6, cs, None, False))
    close(room[:, 1:3], R.norm_rope(k, None, 0, 1e-6, cs, None, False))
    assert not bool(room[:, 0].any()) and not bool(room[:, 3].any())


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_special_rows_stay_in_their_rows(dtype):
    q, cs = normal(6, 2, 128, dtype=dtype, seed=15), R.table(6, 128)
    q[1, 0] = 0.0
    q[2, 1, 5] = float("nan")
    q[3, 0, 7] = float("inf")
    q[4, 1] = 60000.0
    a, _ = gdn.qk_norm_rope(q, None, cs)
    ref = R.norm_rope(q, None, 0, 1e-6, cs, None, False)
    fine = torch.ones(6, 2, dtype=torch.bool, device="cuda")
    fine[2, 1] = fine[3, 0] = False
    close(a[fine], ref[fine])
    assert not bool(a[1, 0].any()) and bool(a[2, 1].isnan().all()) and not bool(torch.isfinite(a[3, 0]).all())


def test_bad_positions_leave_their_rows():
    q, k, cs = normal(5, 2, 128, seed=16), normal(5, 1, 128, seed=17), R.table(10, 128)
    pos = torch.tensor([3, 10, -1, 9, 0], device="cuda")
    a, b = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    gdn.qk_norm_rope(q, k, cs, pos, q_out=a, k_out=b)
    assert gdn.device_status() == 8
    good = [0, 3, 4]
    close(a[good], R.norm_rope(q[good], None, 0, 1e-6, cs, pos[good], False))
    close(b[good], R.norm_rope(k[good], None, 0, 1e-6, cs, pos[good], False))
    assert bool((a[[1, 2]] == 5.0).all()) and bool((b[[1, 2]] == 5.0).all())


def test_streams_graphs_and_nothing():
    q, k, cs = normal(50, 4, 128, seed=18), normal(50, 2, 128, seed=19), R.table(50, 128)
    want = gdn.qk_norm_rope(q, k, cs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.qk_norm_rope(q, k, cs, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = [torch.empty_like(q), torch.empty_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.qk_norm_rope(q, k, cs, q_out=out[0], k_out=out[1])
    q.copy_(normal(50, 4, 128, seed=20))
    graph.replay()
    close(out[0], R.norm_rope(q, None, 0, 1e-6, cs, None, False))
    empty = gdn.qk_norm_rope(q[:0], k[:0], cs)
    assert empty[0].shape == (0, 4, 128)


def test_offsets_past_32_bits():
    far = 1 << 24
    room = torch.empty(140 * far, dtype=BF, device="cuda")
    q = room.as_strided((140, 2, 128), (far, 128, 1))
    q.copy_(normal(140, 2, 128, seed=21))
    cs = R.table(140, 128)
    want, _ = gdn.qk_norm_rope(q, None, cs)
    close(want, R.norm_rope(q, None, 0, 1e-6, cs, None, False))
    gdn.qk_norm_rope(q, None, cs, q_out=q)
    assert torch.equal(q, want)
