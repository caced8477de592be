"""The own pages, and a prefix that is walked with them, keep more of a weight than the values' type holds where a sequence has up to 16
rows a key head and no prefix of more rows stands beside them.

Bounds, fixed before the first run.  With u, w, v, A and d as in attention_ref.py, a weight enters the sums as two numbers of the values'
type: the first is below it by a step of the type at most (2 u of it), the second is the rest, rounded (u of that): 2 u^2 of
the weight are lost, where rounding it once would lose u.  In f16 the rest is off by 2^-24 where it is small, beside a largest weight of 2^6
or more: 2^-30 |v_j| for every key; 2^-25 for the output.  What is left is 2 d A for the scores and u |out| for the output.
"""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import attention_ref as A

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


SHAPES = {
    "short": dict(lengths=[1, 2, 5, 15, 16, 17, 33, 63, 64, 65, 130], h_q=8, h_k=2),
    "sixteen_rows": dict(lengths=[40, 700, 1300], h_q=16, h_k=1, page=64),
    "sixteen_rows_of_tokens": dict(lengths=[300, 17, 129, 3], tokens=4, h_q=8, h_k=2, page=8),
    "drafts": dict(lengths=[(31 * i) % 400 for i in range(60)], tokens=3, h_q=6, h_k=2, page=24),
    "long": dict(lengths=[20011, 40], h_q=8, h_k=2, page=64),
    "walk": dict(lengths=[40, 0, 300], prefix=3001, h_q=4, h_k=1),
}


@pytest.mark.parametrize("std", [0.3, 1.0, 2.0])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("name", SHAPES)
def test_weights_keep_their_bits(name, dtype, std):
    b = A.Batch(dtype=dtype, seed=95, std=std, **SHAPES[name])
    out, lse = b.run()
    want, want_lse, room, lse_room = b.reference()
    u = A.UNIT[dtype]
    # attention_ref's room: u |out| + (u + 2 d) a, and in f16 2^-25 (1 + sum |v|); here 2 u^2 stands for that u, and 2^-30 for the 2^-25 of the values
    a, absolute = sums_of(b)
    room = room - (u - 2 * u * u) * a
    if dtype == HF:
        room -= (2.0 ** -25 - 2.0 ** -30) * absolute
    assert bool((room >= 0).all())
    off = (out.double() - want).abs() / room.clamp_min(1e-300)
    assert bool((off <= 1).all()), float(off.max())
    none = want_lse == -float("inf")
    assert bool(((lse.double() - want_lse).abs() <= lse_room)[~none].all())


def sums_of(b):
    """(sum_j w_j |v_j|, sum_j |v_j|) of every output, in 64 bits."""
    g, scale = b.q.shape[1] // b.k_cache.shape[2], 128 ** -0.5
    a = torch.zeros(b.q.shape, dtype=torch.float64, device="cuda")
    absolute = torch.zeros_like(a)
    for n, (k, v) in enumerate(b.keys):
        for i in range(b.tokens):
            seen, row = max(0, len(k) - b.tokens + i + 1), n * b.tokens + i
            kk, vv = (torch.cat([s, x[:seen]]).double().repeat_interleave(g, 1) for s, x in zip(b.shared, (k, v)))
            if len(kk):
                w = torch.softmax(scale * (kk * b.q[row].double()).sum(-1), 0)
                a[row] = torch.einsum("jh,jhd->hd", w, vv.abs())
                absolute[row] = vv.abs().sum(0)
    return a, absolute
