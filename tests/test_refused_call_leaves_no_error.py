"""A call that fails because CUDA refused something says so itself, and does not leave the error behind for whoever asks CUDA next."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn


def last_error():
    """The error that CUDA's runtime would report next on this thread (the library and torch share one runtime)."""
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line)
    return ctypes.CDLL(path).cudaPeekAtLastError()


pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()


def test_a_workspace_that_does_not_fit():
    gdn.gdn_init(0)
    with pytest.raises(gdn.GdnError, match="out of memory") as e:
        gdn.gdn_reserve_workspace(1 << 50)
    assert e.value.status == 4 and last_error() == 0
    assert (torch.ones(3, device="cuda") + 1).tolist() == [2.0, 2.0, 2.0]
    gdn.gdn_reserve_workspace(1 << 20)
    q = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    cache = torch.randn(2, 8, 2, 128, device="cuda").to(torch.bfloat16)
    table, lengths = torch.arange(2, device="cuda").view(2, 1), torch.tensor([8, 3], device="cuda")
    assert bool(gdn.paged_attention_step(q, cache, cache.clone(), table, lengths).isfinite().all())
    assert gdn.device_status() == 0
