"""Host tensors handed to the decay operators: refused before anything runs, unless they are pinned."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding
from tests import decay_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["extension", "ctypes"], autouse=True)
def _way(request, monkeypatch, tmp_path):
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    if request.param == "ctypes":
        monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
        monkeypatch.setattr(binding, "_calls", binding._PyCall())
    yield
    assert gdn.device_status() == 0


def refused(call, *args, **kw):
    with pytest.raises(gdn.GdnError, match="host") as e:
        call(*args, **kw)
    assert e.value.status == 1


def test_refused():
    q, k, v, g, cu = R.make([9, 3], 2, 2, gate="head", seed=96)
    pool, table = R.states(12, 2, torch.float32, 96), R.table(20, 64)
    at = torch.arange(12, device="cuda")
    for i in range(4):
        args = [q, k, v, g]
        args[i] = args[i].cpu()
        refused(gdn.decay_linear_attention, *args, cu_seqlens=cu, output=torch.empty_like(v))
        refused(gdn.decay_linear_step, *args[:3], pool, args[3], output=torch.empty_like(v))
    refused(gdn.decay_linear_attention, q, k, v, g, cu_seqlens=cu.cpu())
    refused(gdn.decay_linear_attention, q, k, v, g, cu_seqlens=cu, initial_state=pool.cpu())
    refused(gdn.decay_linear_attention, q, k, v, g, cu_seqlens=cu, initial_state=pool, state_indices=at[:2].cpu())
    refused(gdn.decay_linear_attention, q, k, v, g, cu_seqlens=cu, output=torch.empty_like(v).cpu())
    refused(gdn.decay_linear_step, q, k, v, pool.cpu(), g)
    refused(gdn.decay_linear_step, q, k, v, pool, g, state_indices=at.cpu())
    refused(gdn.qk_norm_rope, q.cpu(), k, table)
    refused(gdn.qk_norm_rope, q, k, table.cpu())
    refused(gdn.qk_norm_rope, q, k, table, at.cpu())
    refused(gdn.qk_norm_rope, q, k, table, q_weight=torch.ones(128))


def test_pinned_tensors_are_read():
    q, k, v, g, cu = R.make([9, 3], 2, 2, gate="head", seed=97)
    want = gdn.decay_linear_attention(q, k, v, g, cu_seqlens=cu)
    pinned = cu.cpu().pin_memory()
    assert torch.equal(gdn.decay_linear_attention(q, k, v, g, cu_seqlens=pinned), want)
    torch.cuda.synchronize()
