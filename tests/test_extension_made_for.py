"""The extension reads torch's objects at their places: it goes with one torch and one Python, and no other is loaded."""
import os
import sysconfig

import pytest
import torch

from gated_delta_rule_24_gb300 import binding, build
from tests import test_decay_boundary as B


@pytest.fixture(autouse=True)
def _lib():
    build.build()


def test_its_name_says_what_it_was_made_for():
    name = os.path.basename(build.PYCALL)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert binding._PYCALL_PATH == build.PYCALL


@pytest.mark.parametrize("what", ["torch", "commit", "python"])
def test_another_torch_or_python_asks_for_another_file(what, monkeypatch):
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "2.99.0+cu130")
    elif what == "commit":
        monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
    else:
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-nowhere")
    assert build.made_for() != build.MADE_FOR


def test_one_made_for_something_else_is_not_used(monkeypatch):
    """A file of the right name that was made for another torch: the calls go by ctypes."""
    if not os.path.exists(build.PYCALL):
        pytest.skip("the extension was not built")
    monkeypatch.setattr(binding, "_calls", binding._PyCall())
    assert type(binding._calls.qk_norm_rope).__name__ == "builtin_function_or_method"
    monkeypatch.setattr(binding, "_MADE_FOR", "another torch")
    monkeypatch.setattr(binding, "_calls", binding._PyCall())
    assert isinstance(binding._calls.qk_norm_rope.__self__, binding._ByCtypes)
    changed, want = B.ROPE[next(iter(B.ROPE))]
    import gated_delta_rule_24_gb300 as gdn
    assert B.status(gdn.gdn_qk_norm_rope, B.rope_args(), **changed) == want
