"""Infinities and NaN in keys and values that a draft's later tokens see and its earlier ones do not, and in a prefix of many rows.

What a row does not see leaves it within the bounds of attention_ref.py.  What it sees: an infinite or NaN value reaches its column
alone; a NaN key makes the row NaN, as does an infinite one whose score is +infinity; one whose score is -infinity has a weight
of zero, and the row is that of the other keys.
"""
import math

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def same(got, ref, what=""):
    """Finite where the reference is, within its bounds; else the same infinity, or NaN."""
    out, (want, _, room, _) = got.double(), ref
    good = want.isfinite()
    off = ((out - want).abs() / room.clamp_min(1e-300))[good]
    assert bool(out[good].isfinite().all()) and bool((off <= 1).all()), (what, float(off.nan_to_num(9e9).max()))
    assert bool((out[~good].isnan() == want[~good].isnan()).all()), what
    far = ~good & ~want.isnan()
    assert bool((out[far] == want[far]).all()), what


def write_back(b):
    if b.prefix:
        b._write(b.shared, b.prefix_pages.cpu().long())
    for i, kv in enumerate(b.keys):
        b._write(kv, b.table[i, :-(-len(kv[0]) // b.page)].cpu().long())


# Where the last tokens - 1 keys lie: in the first or the second eight of a warp's 16 keys, over both, over two warps, over two tiles.
LENGTHS = [1, 2, 5, 7, 8, 9, 10, 15, 16, 17, 18, 24, 25, 31, 33, 47, 48, 50, 62, 63, 64, 65, 66, 71, 80, 81, 100, 127, 128, 129, 130, 145, 191, 193, 200, 257]
DRAFTS = [(2, 4, 1), (2, 16, 2), (3, 4, 2), (3, 10, 2), (4, 2, 1), (16, 1, 1), (16, 2, 2), (16, 3, 1), (5, 20, 1)]


@TYPES
@pytest.mark.parametrize("page", [8, 24, 64])
@pytest.mark.parametrize("tokens,h_q,h_k", DRAFTS)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_values_that_later_tokens_see(dtype, page, tokens, h_q, h_k, value):
    """One such value in every key that some of the tokens do not see, each in a column of its own; none in head 0 where there are two."""
    b = A.Batch(LENGTHS, tokens=tokens, h_q=h_q, h_k=h_k, page=page, dtype=dtype, seed=80)
    for k, v in b.keys:
        for i in range(max(0, len(v) - tokens + 1), len(v)):
            v[i, h_k - 1, 5 + 7 * (len(v) - 1 - i)] = value
    write_back(b)
    out, lse = b.run()
    ref = b.reference()
    same(out, ref)
    assert h_k == 1 or bool(out[:, :h_q // 2].isfinite().all())
    A.check((torch.zeros_like(ref[0]), lse), (torch.zeros_like(ref[0]), ref[1], torch.ones_like(ref[0]), ref[3]))


@TYPES
@pytest.mark.parametrize("prefix", [37, 300])
def test_values_that_later_tokens_see_behind_a_prefix(dtype, prefix):
    for h_q, rows in ((4, 1), (16, len(LENGTHS))):   # by the walk, and by the tensor cores
        b = A.Batch(LENGTHS[-rows:], tokens=2, h_q=h_q, h_k=2, page=16, prefix=prefix, dtype=dtype, seed=81)
        for k, v in b.keys:
            v[-1, 1, 9] = INF
        write_back(b)
        out, _ = b.run()
        assert bool((out[1::2, h_q // 2:, 9] == INF).all()) and bool(out[::2].isfinite().all())
        same(out, b.reference())


@TYPES
@pytest.mark.parametrize("tokens,h_q,h_k", [(2, 4, 1), (3, 10, 2), (16, 2, 2), (16, 3, 1)])
@pytest.mark.parametrize("key", [INF, -INF, NAN])
def test_keys_that_later_tokens_see(dtype, tokens, h_q, h_k, key):
    """The last key of all but one, which the last two tokens see, at one place of head h_k - 1."""
    lengths = [x for x in LENGTHS if x > 1]
    b = A.Batch(lengths, tokens=tokens, h_q=h_q, h_k=h_k, dtype=dtype, seed=82)
    clean = b.reference()
    for k, v in b.keys:
        k[-1, h_k - 1, 77] = key
    write_back(b)
    out, lse = b.run()
    g = h_q // h_k
    for n, (k, v) in enumerate(b.keys):
        last, before = (n + 1) * tokens - 1, slice(n * tokens, (n + 1) * tokens - 1)
        same(out[before], tuple(x[before] for x in clean), ("not seen", n))
        same(out[last:last + 1, :h_q - g], tuple(x[last:last + 1, :h_q - g] for x in clean), ("another head", n))
        assert bool(lse[before][clean[1][before] > -INF].isfinite().all())
        without = A.attend(b.q[last:last + 1], [(k[:-1], v[:-1])], tuple(x[:0] for x in b.shared), 1)   # the row of the other keys
        for h in range(h_q - g, h_q):
            if key * float(b.q[last, h, 77]) == -INF:
                same(out[last, h], tuple(x[0, h] for x in without), ("no weight", n, h))
            else:
                assert bool(out[last, h].isnan().all()) and not bool(lse[last, h].isfinite())


PREFIXES = [dict(lengths=[9] * 5, h_q=16, h_k=2, prefix=300), dict(lengths=[(7 * i) % 40 for i in range(16)], h_q=16, h_k=2, prefix=1000),
            dict(lengths=[(7 * i) % 40 for i in range(20)], h_q=16, h_k=2, prefix=700, page=64), dict(lengths=[(7 * i) % 40 for i in range(33)], tokens=2, h_q=10, h_k=2, prefix=1537),
            dict(lengths=[3, 8], h_q=8, h_k=2, prefix=200)]
IDS = ["40_rows", "128_rows", "160_rows", "330_rows", "walk"]


@TYPES
@pytest.mark.parametrize("kw", PREFIXES, ids=IDS)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_values_of_a_prefix(dtype, kw, value):
    """In its first and its last keys and at tiles' ends, each in a column of its own of head 1."""
    b = A.Batch(dtype=dtype, seed=83, **kw)
    at = [0, 31, 32, 63, 64, 127, 128, b.prefix - 2, b.prefix - 1]
    for i, j in enumerate(at):
        b.shared[1][j, 1, 11 * i + 3] = value
    write_back(b)
    out, _ = b.run()
    ref = b.reference()
    assert int((~ref[0].isfinite()).sum()) == len(at) * out.shape[0] * out.shape[1] // 2
    same(out, ref)


@TYPES
@pytest.mark.parametrize("kw", PREFIXES, ids=IDS)
@pytest.mark.parametrize("key", [INF, -INF, NAN])
def test_keys_of_a_prefix(dtype, kw, key):
    """One at a time, in the first tile, at a tile's end and in the last one."""
    b = A.Batch(dtype=dtype, seed=84, **kw)
    clean, h = b.reference(), b.q.shape[1] // 2
    for at in (0, 127, b.prefix - 1):
        kept = b.shared[0][at].clone()
        b.shared[0][at, 1, 50] = key
        write_back(b)
        out, lse = b.run()
        same(out[:, :h], tuple(x[:, :h] for x in clean))
        none = key * b.q[:, h:, 50].float() == -INF
        assert bool(out[:, h:][~none].isnan().all()) and not bool(lse[:, h:][~none].isfinite().any())
        rest = [i for i in range(b.prefix) if i != at]
        without = A.attend(b.q, b.keys, tuple(x[rest] for x in b.shared), b.tokens)
        same(out[:, h:][none], tuple(x[:, h:][none] for x in without))
        b.shared[0][at] = kept


@TYPES
@pytest.mark.parametrize("kw", PREFIXES[:4] + [dict(lengths=[100, 3, 64], tokens=3, h_q=4, h_k=2), dict(lengths=[9000, 17], h_q=4, h_k=2)],
                         ids=IDS[:4] + ["own", "long"])
def test_scores_of_minus_infinity_alone(dtype, kw):
    """Rows that see keys, but none with a weight: zeros, and -infinity for the logarithm."""
    b = A.Batch(dtype=dtype, seed=85, **kw)
    for k, _ in [b.shared] + b.keys:
        k[:, :, 8] = INF
    b.q[..., 8] = -b.q[..., 8].abs() - 1
    b.q[0, 0, 8] = 1.0   # and one whose scores are all +infinity
    write_back(b)
    out, lse = b.run()
    if b.prefix or b.lengths_list[0] >= b.tokens:
        assert bool(out[0, 0].isnan().all())
    out[0, 0], lse[0, 0] = 0.0, -INF
    assert bool((out == 0).all()) and bool((lse == -INF).all())
