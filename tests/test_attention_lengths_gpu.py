"""Lengths that no page table holds are reported whatever else there is to do, and leave their rows."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def run(b, table, lengths, prefix):
    out, lse = torch.full_like(b.q, 9.0), torch.full(b.q.shape[:2], 9.0, device="cuda")
    gdn.paged_attention_step(b.q, b.k_cache, b.v_cache, table, lengths, prefix_pages=b.prefix_pages if prefix else None, prefix_length=prefix,
                             output=out, lse=lse, return_lse=True)
    return out, lse


@pytest.mark.parametrize("bad", [1, -1, 1 << 40])
@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("rows,h_q", [(3, 4), (40, 16), (3, 40)], ids=["few", "many", "wide"])
def test_a_table_without_columns(bad, prefix, rows, h_q):
    """Sequences without pages: every length but 0 is none.  40 rows of 8 heads take the prefix to the tensor cores."""
    b = A.Batch([0] * rows, prefix=prefix, h_q=h_q, h_k=2, idx=torch.int64, seed=70)
    ref, table = b.reference(), b.table[:, :0]
    lengths = torch.zeros_like(b.lengths)
    A.check(run(b, table, lengths, prefix), ref)
    assert gdn.device_status() == 0
    for at in (0, rows - 1):
        lengths.zero_()
        lengths[at] = bad
        got = run(b, table, lengths, prefix)
        assert gdn.device_status() == 0x40
        A.check(got, ref, rows=[i for i in range(rows) if i != at])
        assert bool((got[0][at] == 9.0).all()) and bool((got[1][at] == 9.0).all())


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("kw", [dict(h_q=4, h_k=2), dict(h_q=40, h_k=1), dict(h_q=4, h_k=2, tokens=4)], ids=["heads", "blocks", "tokens"])
def test_only_the_bad_ones(kw, prefix):
    """Far into a batch of more sequences than a warp, or the lengths that are kept, hold."""
    b = A.Batch([(7 * i) % 30 for i in range(600)], prefix=prefix, page=8, seed=71, **kw)
    ref, t = b.reference(), b.tokens
    for at in (0, 33, 599):
        lengths = b.lengths.clone()
        lengths[at] = b.table.shape[1] * b.page + 1
        got = run(b, b.table, lengths, prefix)
        assert gdn.device_status() == 0x40
        A.check(got, ref, rows=[i for i in range(600 * t) if i // t != at])
        rows = slice(at * t, at * t + t)
        assert bool((got[0][rows] == 9.0).all()) and bool((got[1][rows] == 9.0).all())


@pytest.mark.parametrize("rows,prefix", [(3, 0), (3, 40), (40, 40)], ids=["own", "walk", "tensor_cores"])
def test_a_cache_without_pages(rows, prefix):
    """Every page index is none then: reported, and the rows that need one are left."""
    b = A.Batch([5] * rows, prefix=prefix, h_q=16, h_k=2, seed=72)
    b.k_cache, b.v_cache = b.k_cache[:0], b.v_cache[:0]
    lengths = b.lengths.clone()
    lengths[0] = 0
    out, lse = run(b, b.table, lengths, prefix)
    assert gdn.device_status() == 0x20
    assert bool((out[1:] == 9.0).all()) and bool((lse[1:] == 9.0).all())
    assert bool((out[0] == (9.0 if prefix else 0.0)).all())


def test_a_hundred_thousand_sequences():
    """More than a thread counts at once, most of them empty."""
    n = 100_000
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    at = torch.randperm(n, generator=torch.Generator().manual_seed(73))[:3000].cuda()
    lengths[at] = torch.randint(1, 17, (3000,), generator=torch.Generator().manual_seed(74)).to(torch.int32).cuda()
    b = A.Batch([16] * 50, h_q=2, h_k=1, page=8, seed=75)
    table = b.table[torch.arange(n, device="cuda") % 50].contiguous()
    q = A.normal(n, 2, 128, seed=76)
    out, lse = gdn.paged_attention_step(q, b.k_cache, b.v_cache, table, lengths, return_lse=True)
    empty = lengths == 0
    assert not bool(out[empty].any()) and bool((lse[empty] == -float("inf")).all())
    keys = [tuple(x[:int(lengths[i])] for x in b.keys[int(i) % 50]) for i in at]
    A.check((out[at], lse[at]), A.attend(q[at], keys, tuple(x[:0] for x in b.shared), 1))
