"""A wait of the attention that runs out: the call returns, the device error word says so, and the next call is right."""
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
    gdn.testing_wait_limit(0)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("kw", [dict(lengths=[300, 20, 5000]), dict(lengths=[300, 20, 9], prefix=100),
                                dict(lengths=[9] * 60, prefix=3000, h_q=16, h_k=2)], ids=["own", "prefix", "prefix_rows"])
def test_a_wait_runs_out(kw):
    b = A.Batch(seed=40, **kw)
    ref = b.reference()
    A.check(b.run(), ref)
    gdn.testing_wait_limit(2000, withhold_local_ready=True)
    b.run()
    assert gdn.device_status() == gdn.binding.DEVERR_TIMEOUT
    gdn.testing_wait_limit(0)
    A.check(b.run(), ref)
