"""Sizes beyond what the decay operators count in 32 bits (no GPU: nothing valid is launched)."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    return gdn.load_library()


def tensor(dtype, shape, stride, at=1 << 40):
    d = binding.GdnTensor(data=at, dtype=binding._DTYPES[dtype], ndim=len(shape))
    for i, (n, s) in enumerate(zip(shape, stride)):
        d.shape[i], d.stride[i] = n, s
    return ctypes.byref(d)


@pytest.mark.parametrize("T,status", [((1 << 31) - 128, 2), ((1 << 31) - 65, 2)])
def test_tokens(lib, T, status):
    """Their last chunk of 128 would end beyond 2^31."""
    x = [tensor(torch.bfloat16, (T, 1, 128), (8, 128, 1), at=(i + 1) << 44) for i in range(4)]
    cu = tensor(torch.int64, (2,), (1,), at=1 << 50)
    assert lib.gdn_decay_prefill(*x[:3], None, 0.0, None, None, None, cu, 0, x[3], None) == status
    assert b"too many rows" in lib.gdn_last_error()
