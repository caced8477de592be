"""Attention whose weights are known exactly, over long sequences and prefixes: a tile or a part that is lost, met twice or taken from
elsewhere shows in every column.

Queries of zero make all scores 0 and all weights the same power of two, and small whole numbers as values make sums that f32
holds exactly (below 2^24).  What is left: the reciprocal of the count and the product with it, 2^-22 of the output at most together, and the
output's own rounding u.  The logarithm log n: log2f is off by 2^-23 of it, its sum with the base, the product with ln 2 and that constant by 2^-24 each: 2^-21 |lse| is
more than all of them, and 2^-21 is for n = 1.

A key whose score is 16 x 64 / sqrt(128) = 90 beside scores of 0 (weights of 2^-130, nothing beside its own) makes the output its value.
"""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A
from tests.test_attention_nonfinite_gpu import write_back

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def whole_numbers(b):
    gen = torch.Generator(device="cuda").manual_seed(90)
    for _, v in [b.shared] + b.keys:
        v.copy_(torch.randint(-8, 9, v.shape, generator=gen, device="cuda"))
    write_back(b)


def near(out, want, dtype):
    unit = A.UNIT[dtype]
    room = (unit + 2.0 ** -21) * want.abs() + (2.0 ** -25 if dtype == HF else 0.0)
    off = (out.double() - want).abs() - room
    assert bool((off <= 0).all()), float(off.max())


LONG = {
    "one": dict(lengths=[20011], h_q=8, h_k=2, page=64),
    "one_f16_pages_of_8": dict(lengths=[30000], h_q=4, h_k=1, page=8),
    "one_very_long": dict(lengths=[131072], h_q=8, h_k=1, page=64),
    "sixteen_rows": dict(lengths=[50021], h_q=16, h_k=1, page=128),
    "many_rows": dict(lengths=[7001, 30], tokens=4, h_q=40, h_k=2, page=16),
    "drafts": dict(lengths=[5000 + 300 * i for i in range(20)], tokens=3, h_q=4, h_k=2, page=24),
    "short": dict(lengths=[(37 * i) % 190 for i in range(700)], h_q=4, h_k=2, page=16),
    "prefix_of_2_rows": dict(lengths=[40], prefix=20007, h_q=4, h_k=2, page=64),
    "prefix_of_16_rows": dict(lengths=[40, 0, 70, 1], prefix=33333, h_q=8, h_k=2, page=16),
    "prefix_of_32_rows": dict(lengths=[300] * 8, prefix=100000, h_q=8, h_k=2, page=32),
    "prefix_of_128_rows": dict(lengths=[(13 * i) % 300 for i in range(16)], prefix=40009, h_q=16, h_k=2, page=64),
    "prefix_of_300_rows": dict(lengths=[(13 * i) % 300 for i in range(75)], prefix=20007, h_q=8, h_k=2, page=64),
    "prefix_of_600_rows": dict(lengths=[(13 * i) % 300 for i in range(150)], tokens=2, prefix=9001, h_q=4, h_k=2, page=8),
}


@TYPES
@pytest.mark.parametrize("name", LONG)
def test_means(dtype, name):
    b = A.Batch(dtype=dtype, seed=91, spare=0, **LONG[name])
    b.q.zero_()
    whole_numbers(b)
    out, lse = b.run()
    g = b.q.shape[1] // b.k_cache.shape[2]
    shared = b.shared[1].double().sum(0)
    for n, (_, v) in enumerate(b.keys):
        total = torch.cat([shared[None], shared + v.double().cumsum(0)])   # [keys seen, h_k, 128]
        for i in range(b.tokens):
            seen, row = max(0, len(v) - b.tokens + i + 1), n * b.tokens + i
            count = b.prefix + seen
            near(out[row], (total[seen] / max(1, count)).repeat_interleave(g, 0), dtype)
            want = torch.tensor(float(count), dtype=torch.float64).log()
            assert bool(((lse[row].double() - want).abs() <= 2.0 ** -21 * (1 + want.abs())).all() if count else (lse[row] == want).all())


@TYPES
def test_one_key_of_many_sequences(dtype):
    """Each of 300 sequences has its own such key: at tiles', warps' and pages' ends and all over."""
    places = [0, 1, 7, 8, 15, 16, 31, 47, 48, 63, 64, 65, 127, 128, 191, 192, 255, 256, 511, 512, 690, 699]
    places += [(97 * i) % 700 for i in range(300 - len(places))]
    b = A.Batch([700] * 300, h_q=4, h_k=2, page=16, dtype=dtype, seed=92)
    whole_numbers(b)
    b.q.zero_()
    b.q[..., 0] = 16.0
    for (k, v), at in zip(b.keys, places):
        k[:, :, 0] = 0.0
        k[at, :, 0] = 64.0
    write_back(b)
    out, _ = b.run()
    want = torch.stack([v[at].double().repeat_interleave(2, 0) for (_, v), at in zip(b.keys, places)])
    near(out, want, dtype)


@TYPES
@pytest.mark.parametrize("kw", [dict(lengths=[20011], h_q=8, h_k=2, page=64), dict(lengths=[6001], tokens=2, h_q=20, h_k=1, page=24),
                                dict(lengths=[30], prefix=20007, h_q=8, h_k=2, page=64),
                                dict(lengths=[5] * 10, prefix=20007, h_q=8, h_k=2, page=64), dict(lengths=[5] * 80, prefix=9001, h_q=8, h_k=2, page=16)],
                         ids=["own", "own_of_40_rows", "walk", "40_rows", "320_rows"])
def test_one_key_of_a_long_sequence(dtype, kw):
    """At 60 places in turn, workers' ends among them, wherever they lie."""
    b = A.Batch(dtype=dtype, seed=93, spare=0, **kw)
    whole_numbers(b)
    b.q.zero_()
    b.q[..., 0] = 16.0
    for k, _ in [b.shared] + b.keys:
        k[:, :, 0] = 0.0
    (k, v), pages = (b.shared, b.prefix_pages) if b.prefix else (b.keys[0], b.table[0])
    write_back(b)
    most = len(k) - (0 if b.prefix else b.tokens - 1)   # seen by all rows
    g = b.q.shape[1] // b.k_cache.shape[2]

    def put(at, x):
        b.k_cache[pages[at // b.page].long(), at % b.page, :, 0] = x

    for i in range(60):
        at = most - 1 if i == 0 else (i * 2 ** 20 // 59 * most >> 20) % most
        put(at, 64.0)
        out, _ = b.run()
        near(out, v[at].double().repeat_interleave(g, 0).expand(out.shape), dtype)
        put(at, 0.0)
