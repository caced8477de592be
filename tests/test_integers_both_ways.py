"""Integers mean the same to the extension and by ctypes: those of other libraries are taken, and those that C does not hold are refused
(no GPU is needed: nothing valid is launched)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import test_attention_boundary as T

way = T.way


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()


def args(make, **changed):
    return {**make(), **changed, "stream": 0}


@pytest.mark.parametrize("prefix", [1 << 63, 1 << 64, (1 << 64) + 20, -(1 << 63) - 1, 1 << 200])
def test_a_prefix_that_c_does_not_hold(way, prefix):
    with pytest.raises(OverflowError):
        gdn.gdn_paged_attention_step(**args(T.attend_args, prefix_length=prefix))


@pytest.mark.parametrize("prefix", [20.0, "20"])
def test_a_prefix_that_is_no_integer(way, prefix):
    with pytest.raises(TypeError):
        gdn.gdn_paged_attention_step(**args(T.attend_args, prefix_length=prefix))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are host tensors: only for a machine without a GPU")
@pytest.mark.parametrize("integer", [np.int64, np.int32, lambda x: torch.tensor(x), bool])
def test_integers_of_other_libraries(way, integer):
    assert T.status(gdn.gdn_paged_attention_step, T.attend_args(), prefix_length=integer(1)) not in (0, T.INVALID, T.ALIAS)
    assert T.status(gdn.gdn_paged_attention_step, T.attend_args(), prefix_length=integer(0), prefix_pages=None) not in (0, T.INVALID, T.ALIAS)
    if integer is not bool:
        assert T.status(gdn.gdn_paged_attention_step, T.attend_args(), prefix_length=integer(33)) == T.INVALID
    for axes in ([integer(i % 2) for i in range(64)], tuple(integer(i % 2) for i in range(64))):
        assert T.status(gdn.gdn_qk_norm_rope_axes, T.axes_args(), pair_axes=axes) not in (0, T.INVALID, T.ALIAS)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are host tensors: only for a machine without a GPU")
def test_arrays_of_axes(way):
    for axes in (np.arange(64) % 3, torch.arange(64) % 3, range(0, 1), np.full(64, 3), np.full(64, -1)):
        good = len(axes) == 64 and 0 <= int(max(axes)) < 3 and int(min(axes)) >= 0
        got = T.status(gdn.gdn_qk_norm_rope_axes, T.axes_args(), pair_axes=axes)
        assert got not in (0, T.INVALID, T.ALIAS) if good else got == T.INVALID
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope_axes(**args(T.axes_args, pair_axes=np.zeros(64)))
