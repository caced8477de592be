"""Every entry point as the first CUDA call of its thread."""
import threading

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def calls():
    q, k, v, g, cu = R.make([140, 20], 2, 2, gate="slow", seed=90)
    out, state = torch.empty_like(v), torch.empty(2, 2, 128, 128, device="cuda")
    pool, beta = R.states(2, 2, torch.float32, 90), torch.full_like(g, 0.5)
    row = torch.empty(2, 2, 128, dtype=BF, device="cuda")
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    return {
        "decay_prefill": lambda: gdn.gdn_decay_prefill(q, k, v, g, 0.0, None, None, state, cu, False, out, 0),
        "decay_step": lambda: gdn.gdn_decay_step(q[:2], k[:2], v[:2], g[:2], 0.0, pool, None, row, 0),
        "norm_rope": lambda: gdn.gdn_qk_norm_rope(q, k, None, None, 0.0, 1e-6, None, None, False, q2, k2, 0),
        "chunk_prefill": lambda: gdn.gdn_chunk_prefill(q, k, v, g, beta, 0.0, None, None, state, cu, True, True, out, 0),
        "chunk_prefill_noalloc": lambda: gdn.gdn_chunk_prefill_noalloc(q, k, v, g, beta, 0.0, None, None, state, cu, True, True,
                                                                       out, error, 0),
        "decode_step": lambda: gdn.gdn_decode_step(q[:2], k[:2], v[:2], g[:2], beta[:2], 0.0, pool, None, True, row, 0),
    }


@pytest.mark.parametrize("name", ["decay_prefill", "decay_step", "norm_rope", "chunk_prefill", "chunk_prefill_noalloc", "decode_step"])
def test_first_call_of_a_thread(name):
    call, failed = calls()[name], []
    torch.cuda.synchronize()

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
