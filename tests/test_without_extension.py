"""The library and its binding on a machine where the small extension cannot be built or loaded."""
import os
import subprocess
import sys
import warnings

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding, build
from tests import test_decay_boundary as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.fixture
def missing(monkeypatch, tmp_path):
    """The binding as it starts, and no extension where it looks for one."""
    monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
    monkeypatch.setattr(binding, "_calls", binding._PyCall())


def test_the_library_loads_without_it():
    code = ("import sys; sys.path.insert(0, %r); from gated_delta_rule_24_gb300 import binding; "
            "binding._PYCALL_PATH = '/nowhere/gdn_pycall.so'; lib = binding.load_library(); "
            "assert lib.gdn_split_workspace_bytes(1, 1, 2) == 65536 and 'pycall' not in open('/proc/self/maps').read()" % ROOT)
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


@pytest.mark.parametrize("trouble", ["headers", "compiler"])
def test_the_library_builds_without_it(trouble, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "PYCALL", str(tmp_path / "gdn_pycall.so"))
    if trouble == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        def none(*args, **kw):
            raise FileNotFoundError("gcc")
        monkeypatch.setattr(build.subprocess, "run", none)
    with pytest.warns(UserWarning, match="host"):
        assert build.build() == build.LIB
    assert not os.path.exists(build.PYCALL)
    monkeypatch.undo()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build()


@pytest.mark.parametrize("case", B.PREFILL)
def test_prefill_refuses(missing, case):
    changed, want = B.PREFILL[case]
    assert B.status(gdn.gdn_decay_prefill, B.prefill_args(), **changed) == want


@pytest.mark.parametrize("case", B.STEP)
def test_step_refuses(missing, case):
    changed, want = B.STEP[case]
    assert B.status(gdn.gdn_decay_step, B.step_args(), **changed) == want


@pytest.mark.parametrize("case", B.ROPE)
def test_norm_rope_refuses(missing, case):
    changed, want = B.ROPE[case]
    assert B.status(gdn.gdn_qk_norm_rope, B.rope_args(), **changed) == want


def test_calls_refuse_what_is_no_tensor(missing):
    B.test_calls_refuse_what_is_no_tensor()


@pytest.mark.gpu
def test_the_same_results(missing):
    from tests import decay_ref as R
    gdn.gdn_init(0)
    q, k, v, g, cu = R.make([130, 20], 2, 4, gate="head", seed=95)
    table = R.table(200, 64)

    def run():
        pool = R.states(150, 4, torch.bfloat16, 95)
        return (*gdn.decay_linear_attention(q, k, v, g, cu_seqlens=cu, output_final_state=True, scale=0.5),
                gdn.decay_linear_step(q, k, v, pool, g), pool, *gdn.qk_norm_rope(q, k, table))

    by_ctypes = run()
    assert isinstance(binding._calls.decay_step.__self__, binding._ByCtypes)
    binding._calls = binding._PyCall()
    binding._PYCALL_PATH = build.PYCALL
    for a, b in zip(by_ctypes, run()):
        assert torch.equal(a, b)
    assert gdn.device_status() == 0
