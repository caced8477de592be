"""Attention of new tokens over a paged cache and a shared prefix, against the formula in 64 bits
(bounds: attention_ref.py)."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A

pytestmark = pytest.mark.gpu
BF, HF, I32, I64 = torch.bfloat16, torch.float16, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


SHAPES = {
    "one_key": dict(lengths=[1], h_q=1, h_k=1, page=8),
    "short": dict(lengths=[5], h_q=8, h_k=1),
    "ends": dict(lengths=[1, 15, 16, 17, 63, 64, 65, 127, 128, 129], h_q=4, h_k=2),
    "empty_among": dict(lengths=[0, 40, 0, 0, 200, 0], h_q=3, h_k=3, idx=I64),
    "all_empty": dict(lengths=[0, 0], h_q=2, h_k=1),
    "group_3": dict(lengths=[77, 300], h_q=6, h_k=2, page=24),
    "group_5": dict(lengths=[130], h_q=5, h_k=1, page=40, dtype=HF),
    "group_7": dict(lengths=[513, 2], h_q=14, h_k=2, page=32),
    "group_16": dict(lengths=[100, 257], h_q=16, h_k=1, page=64),
    "group_17": dict(lengths=[100, 257], h_q=34, h_k=2, page=64),
    "group_40": dict(lengths=[90, 31], h_q=40, h_k=1),
    "heads_1_to_1": dict(lengths=[250, 3, 90], h_q=8, h_k=8, page=128),
    "large_pages": dict(lengths=[700, 10], h_q=4, h_k=1, page=256, layout="heads"),
    "f16_by_heads": dict(lengths=[333, 64, 1], h_q=8, h_k=4, page=16, dtype=HF, layout="heads"),
    "woven": dict(lengths=[140, 222], h_q=8, h_k=2, layout="woven"),
    "side_by_side": dict(lengths=[140, 222], h_q=8, h_k=2, layout="side", dtype=HF),
    "two_tokens": dict(lengths=[2, 1, 0, 3, 100], tokens=2, h_q=4, h_k=2),
    "sixteen_tokens": dict(lengths=[16, 15, 40, 300], tokens=16, h_q=4, h_k=2, dtype=HF),
    "eighty_rows": dict(lengths=[300, 17, 5, 129], tokens=16, h_q=10, h_k=2, page=24),
    "heads_128": dict(lengths=[700, 0, 33], h_q=128, h_k=1, page=32, dtype=HF),
    "many_rows_long": dict(lengths=[9000, 64], tokens=3, h_q=24, h_k=1, page=64),
    "many": dict(lengths=[(37 * i) % 211 for i in range(300)], h_q=4, h_k=2),
    "hundreds": dict(lengths=[0 if 480 < i < 620 else (41 * i) % 83 for i in range(700)], h_q=3, h_k=1, page=8),
    "hundreds_behind_a_prefix": dict(lengths=[0 if 500 < i < 520 else (41 * i) % 83 for i in range(600)], tokens=2, h_q=2, h_k=1, prefix=90, page=8),
    "long": dict(lengths=[20011], h_q=8, h_k=2, page=64),
    "long_and_short": dict(lengths=[1, 12000, 3, 0, 7000, 8], h_q=8, h_k=1, page=16),
    "prefix_1": dict(lengths=[3, 0, 20], prefix=1),
    "prefix_odd": dict(lengths=[30, 0, 200], prefix=77, h_q=6, h_k=2, page=24),
    "prefix_alone": dict(lengths=[0, 0, 0], prefix=300),
    "prefix_tokens": dict(lengths=[3, 1, 0, 50], tokens=3, prefix=130, h_q=4, h_k=1, dtype=HF),
    "prefix_rows_128": dict(lengths=[20] * 16, prefix=500, h_q=16, h_k=2, page=32),
    "prefix_rows_257": dict(lengths=[(i * 29) % 90 for i in range(257)], prefix=1000, h_q=2, h_k=2, page=16),
    "prefix_rows_many": dict(lengths=[(i * 29) % 90 for i in range(100)], prefix=1511, h_q=14, h_k=2, page=64, idx=I64),
    "prefix_rows_f16": dict(lengths=[5 + i for i in range(70)], prefix=640, h_q=16, h_k=2, page=128, dtype=HF, layout="heads"),
    "prefix_of_blocks": dict(lengths=[40, 2, 0, 300], tokens=8, h_q=16, h_k=1, prefix=100, page=8),
    "prefix_rows_short": dict(lengths=[(i * 29) % 90 for i in range(60)], prefix=3, h_q=16, h_k=2, page=8),
    "prefix_rows_tokens": dict(lengths=[(i * 31) % 140 for i in range(40)], tokens=4, prefix=257, h_q=8, h_k=1, layout="woven"),
    "prefix_long": dict(lengths=[40, 60], prefix=20007, h_q=8, h_k=2, page=64),
    "prefix_long_rows": dict(lengths=[(i * 13) % 50 for i in range(64)], prefix=9001, h_q=16, h_k=2, page=16),
}


@pytest.mark.parametrize("name", SHAPES)
def test_shapes(name):
    b = A.Batch(seed=3, **SHAPES[name])
    A.check(b.run(), b.reference())


@pytest.mark.parametrize("junk", [float("inf"), float("-inf"), 65504.0, 0.0])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_places_without_a_key_are_not_seen(junk, dtype):
    b = A.Batch([100, 0, 33, 1], prefix=45, page=24, junk=junk, dtype=dtype, seed=4)
    A.check(b.run(), b.reference())
    b = A.Batch([9 + i for i in range(40)], prefix=345, page=24, h_q=16, h_k=2, junk=junk, dtype=dtype, seed=4)
    A.check(b.run(), b.reference())


@pytest.mark.parametrize("scale", [0.5, -0.2, 1e-4])
def test_scales(scale):
    for kw in (dict(lengths=[100, 3], prefix=20), dict(lengths=[9] * 40, prefix=300, h_q=16, h_k=2)):
        b = A.Batch(seed=5, **kw)
        A.check(b.run(scale=scale), b.reference(scale))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("rows", [2, 40])
def test_large_scores(dtype, rows):
    """Scores that grow along the keys, by far more than an exponential holds: the maximum moves in every tile."""
    b = A.Batch([200] * rows, prefix=700, h_q=16, h_k=2, dtype=dtype, seed=6, std=4.0)
    for k, _ in [b.shared] + b.keys:
        k.mul_(torch.linspace(0.1, 8.0, k.shape[0], device="cuda").view(-1, 1, 1).to(dtype))
    b._write(b.shared, b.prefix_pages.cpu())
    for i, kv in enumerate(b.keys):
        b._write(kv, b.table[i, :-(-200 // b.page)].cpu())
    A.check(b.run(), b.reference())


def test_equal_keys_share_alike():
    """All scores alike, in f16 with a long sequence: weights of 1 / 30000 are not lost."""
    b = A.Batch([30000], h_q=4, h_k=1, page=64, dtype=HF, seed=7, spare=0)
    b.q.zero_()
    A.check(b.run(), b.reference())


def test_infinities_and_nan_stay_with_their_sequence_and_head():
    for prefix in (0, 50):
        b = A.Batch([70, 80, 90], prefix=prefix, h_q=4, h_k=2, seed=8)
        page, at = int(b.table[1, 2]), 5   # key 37 of sequence 1
        b.v_cache[page, at, 1, 3] = float("nan")
        b.v_cache[page, at, 1, 4] = float("inf")
        out, lse = b.run()
        ref = b.reference()
        A.check((out, lse), ref, rows=[0, 2])
        A.check((out[:, :2], lse[:, :2]), tuple(x[:, :2] for x in ref))
        assert bool(out[1, 2:, 3].isnan().all()) and bool((out[1, 2:, 4] == float("inf")).all())
        good = [i for i in range(128) if i not in (3, 4)]
        A.check((out[1:2, 2:, good], None), tuple(x[1:2, 2:, good] if x.dim() == 3 else x for x in ref))
        b = A.Batch([70, 80, 90], prefix=prefix, h_q=4, h_k=2, seed=8)
        b.k_cache[int(b.table[1, 2]), 5, 1, 3] = float("nan")
        out, lse = b.run()
        A.check((out, lse), ref, rows=[0, 2])
        assert bool(out[1, 2:].isnan().all()) and bool(lse[1, 2:].isnan().all())


def test_strided_queries_outputs_and_lse():
    b = A.Batch([100, 60, 5], prefix=20, h_q=4, h_k=2, seed=9)
    wide = A.normal(3, 10, 128, seed=10)
    wide[:, 3:7] = b.q
    b.q = wide[:, 3:7]
    room = torch.full((3, 9, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((3, 6), 7.0, device="cuda")
    out, l2 = b.run(output=room[:, 1:8:2], lse=lse[:, 1:5])
    assert out.data_ptr() == room[:, 1].data_ptr() and l2.data_ptr() == lse[:, 1:].data_ptr()
    A.check((room[:, 1:8:2], lse[:, 1:5]), b.reference())
    assert bool((room[:, 0::2] == 7.0).all()) and bool((lse[:, [0, 5]] == 7.0).all())
    assert b.run(return_lse=False).shape == b.q.shape


@pytest.mark.parametrize("prefix", [0, 100])
def test_bad_lengths_and_pages_leave_their_rows(prefix):
    b = A.Batch([100, 60, 5, 77, 64], prefix=prefix, tokens=2, seed=11)
    ref, good = b.reference(), b.lengths.clone()

    def run():
        out, lse = torch.full_like(b.q, 9.0), torch.full(b.q.shape[:2], 9.0, device="cuda")
        return b.run(output=out, lse=lse)

    for sequence, bad in ((1, -1), (1, (b.table.shape[1]) * b.page + 1)):
        b.lengths.copy_(good)
        b.lengths[sequence] = bad
        got = run()
        assert gdn.device_status() == 0x40
        A.check(got, ref, rows=[0, 1, 4, 5, 6, 7, 8, 9])
        assert bool((got[0][2:4] == 9.0).all()) and bool((got[1][2:4] == 9.0).all())
    b.lengths.copy_(good)
    for bad in (-1, b.k_cache.shape[0], 1 << 30):
        kept = b.table[3, 1].clone()
        b.table[3, 1] = bad
        got = run()
        assert gdn.device_status() == 0x20
        A.check(got, ref, rows=[0, 1, 2, 3, 4, 5, 8, 9])
        assert bool((got[0][6:8] == 9.0).all()) and bool((got[1][6:8] == 9.0).all())
        b.table[3, 1] = kept
    A.check(run(), ref)


@pytest.mark.parametrize("rows", [3, 60])
def test_a_bad_prefix_page_leaves_all_rows(rows):
    b = A.Batch([20] * rows, prefix=300, h_q=16, h_k=2, seed=12, idx=I64)
    b.prefix_pages[7] = 1 << 40
    out, lse = torch.full_like(b.q, 9.0), torch.full(b.q.shape[:2], 9.0, device="cuda")
    b.run(output=out, lse=lse)
    assert gdn.device_status() == 0x20
    assert bool((out == 9.0).all()) and bool((lse == 9.0).all())


def test_more_prefix_pages_than_the_prefix_needs():
    b = A.Batch([20, 30], prefix=40, seed=13)
    b.prefix_pages = torch.cat([b.prefix_pages, torch.full((5,), -3, dtype=I32, device="cuda")])
    A.check(b.run(), b.reference())
    b.prefix = 0   # pages without a prefix
    ref = A.attend(b.q, b.keys, tuple(x[:0] for x in b.shared), 1)
    A.check(b.run(), ref)


def test_offsets_past_32_bits():
    far = 1 << 24
    room = torch.empty(2 * 140 * far, dtype=BF, device="cuda")   # pages 32 MiB apart: 4.7 GB a cache
    b = A.Batch([700, 900, 300], h_q=4, h_k=1, page=16, seed=14, spare=5)
    pages = b.k_cache.shape[0]
    assert pages >= 120
    for i, name in enumerate(("k_cache", "v_cache")):
        c = room[i * 140 * far:].as_strided((pages, 16, 1, 128), (far, 128, 128, 1))
        c.copy_(getattr(b, name))
        setattr(b, name, c)
    A.check(b.run(), b.reference())


def test_the_same_bits_every_time():
    for kw in (dict(lengths=[5000, 31, 900], prefix=0), dict(lengths=[(i * 29) % 90 for i in range(80)], prefix=3001, h_q=16, h_k=2)):
        b = A.Batch(seed=15, **kw)
        want = [x.clone() for x in b.run()]
        for _ in range(5):
            assert all(torch.equal(x, y) for x, y in zip(b.run(), want))


def test_streams_graphs_and_nothing():
    works = [A.Batch([4000 + 700 * i, 31, 900], prefix=[0, 333, 2000][i], h_q=16, h_k=2, seed=16 + 100 * i) for i in range(3)]
    want = [[x.clone() for x in b.run()] for b in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(10):
        got = [b.run(stream=s) for b, s in zip(works, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    b = works[2]
    gdn.gdn_reserve_workspace(gdn.gdn_paged_attention_workspace_bytes(3, 1, 16, 2, 2000))
    out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(output=out, lse=lse)
    for lengths in ([4000, 31, 900], [5, 4100, 0]):   # the captured call follows what its inputs hold
        b.lengths.copy_(torch.tensor(lengths))
        b.table.copy_(torch.randint(0, b.k_cache.shape[0], b.table.shape, generator=torch.Generator().manual_seed(2)))
        if lengths[1] > b.table.shape[1] * b.page:
            lengths[1] = b.table.shape[1] * b.page
            b.lengths[1] = lengths[1]
        b.k_cache.nan_to_num_(0.25)
        b.v_cache.nan_to_num_(0.5)
        graph.replay()
        flat = [c.flatten(0, 1) for c in (b.k_cache, b.v_cache)]
        keys = []
        for i, n in enumerate(lengths):
            j = torch.arange(n, device="cuda")
            at = b.table[i].long()[j // b.page] * b.page + j % b.page
            keys.append(tuple(c[at] for c in flat))
        j = torch.arange(b.prefix, device="cuda")
        at = b.prefix_pages.long()[j // b.page] * b.page + j % b.page
        A.check((out, lse), A.attend(b.q, keys, tuple(c[at] for c in flat), 1))
    none = gdn.paged_attention_step(b.q[:0], b.k_cache, b.v_cache, b.table[:0], b.lengths[:0])
    assert none.shape == (0, 16, 128)
    nothing = gdn.paged_attention_step(b.q, b.k_cache[:0], b.v_cache[:0], b.table[:, :0], torch.zeros_like(b.lengths), return_lse=True)
    assert not bool(nothing[0].any()) and bool((nothing[1] == float("-inf")).all())


def test_the_workspace_it_asks_for_is_enough():
    """A capture after the workspace of just these sizes was reserved."""
    for kw in (dict(lengths=[3000, 5], h_q=8, h_k=2), dict(lengths=[10] * 130, prefix=700, h_q=32, h_k=4), dict(lengths=[300] * 3, tokens=16, prefix=2000, h_q=20, h_k=1)):
        b = A.Batch(seed=17, **kw)
        want = [x.clone() for x in b.run()]
        torch.cuda.synchronize()
        gdn.load_library().gdn_shutdown()
        gdn.gdn_init(0)
        gdn.gdn_reserve_workspace(gdn.gdn_paged_attention_workspace_bytes(len(b.lengths_list), b.tokens, b.q.shape[1], b.k_cache.shape[2], b.prefix))
        out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.run(output=out, lse=lse)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_first_call_of_a_thread():
    import threading
    b, failed = A.Batch([300, 20], prefix=50, seed=18), []
    want = [x.clone() for x in b.run()]
    torch.cuda.synchronize()
    got = []

    def run():
        try:
            got.append(b.run())
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(x, y) for x, y in zip(got[0], want))
