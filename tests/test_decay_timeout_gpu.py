"""A hand-off inside the decay prefill that does not come: the call ends, says so, and the next one is right."""
import time

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300.binding import DEVERR_TIMEOUT
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


@pytest.mark.parametrize("dtype,state", [(BF, BF), (BF, F32), (HF, F32)], ids=str)
@pytest.mark.parametrize("lengths,heads,splits", [([300, 1, 130], 2, 1), ([1400, 900], 2, 4), ([500, 0, 300] * 60, 4, 1),
                                                  ([900, 0, 700] * 40, 4, 2), ([40] * 90, 4, 1)],
                         ids=["uncut", "cut", "more_than_sms", "more_than_sms_cut", "short"])
def test_a_withheld_hand_off(force_split, dtype, state, lengths, heads, splits):
    force_split(splits)
    q, k, v, g, cu = R.make(lengths, heads, heads, dtype, "slow", seed=98)
    s0 = R.states(len(lengths), heads, state, 98)

    def call():
        return gdn.decay_linear_attention(q, k, v, g, initial_state=s0, output_final_state=True, cu_seqlens=cu)

    want = call()
    assert gdn.device_status() == 0
    gdn.testing_wait_limit(1_000_000, withhold_local_ready=True)
    try:
        start = time.perf_counter()
        call()
        assert gdn.device_status() == DEVERR_TIMEOUT
        assert time.perf_counter() - start < 5.0
    finally:
        gdn.testing_wait_limit(0)
    got = call()
    assert gdn.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
