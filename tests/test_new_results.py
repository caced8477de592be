"""Results that the extension allocates are asked about as the arguments are: where an input is allowed in pinned host memory, a
result made after it would lie in ordinary host memory, which may be gone when the kernel writes."""
import ctypes
import importlib.machinery
import importlib.util
import os
import shutil

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding, build

BF = torch.bfloat16


@pytest.fixture
def module(tmp_path):
    """The extension once more by itself, with C functions that do nothing, and ``known``, the tensors it is told are pinned."""
    build.build()
    if not os.path.exists(build.PYCALL):
        pytest.skip("the extension was not built")
    path = shutil.copy(build.PYCALL, tmp_path / "gdn_pycall.so")
    loader = importlib.machinery.ExtensionFileLoader("gdn_pycall", str(path))
    made = importlib.util.module_from_spec(importlib.util.spec_from_file_location("gdn_pycall", str(path), loader=loader))
    loader.exec_module(made)
    refuses = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 2)
    known = []

    def ask(t):
        if not any(t is x for x in known):
            raise gdn.GdnError(1, "a tensor is on the host")

    made.bind(ask, *[ctypes.cast(refuses, ctypes.c_void_p).value] * 6)
    made.kept = refuses, known
    yield made, known
    made.bind(None, *[0] * 6)


def rows(known, *shape, dtype=BF):
    known.append(torch.zeros(shape, dtype=dtype))
    return known[-1]


def test_rotation(module):
    module, known = module
    q, k = rows(known, 3, 4, 128), rows(known, 3, 2, 128)
    for args in ((q, k), (q, None)):
        with pytest.raises(gdn.GdnError, match="host"):
            module.new_qk_norm_rope(*args, None, None, 0.0, 1e-6, None, None, None, False)


def test_append(module):
    module, known = module
    q, k, v = rows(known, 3, 4, 128), rows(known, 3, 2, 128), rows(known, 3, 2, 128)
    caches = rows(known, 2, 8, 2, 128), rows(known, 2, 8, 2, 128)
    slots = rows(known, 3, dtype=torch.int32)
    with pytest.raises(gdn.GdnError, match="host"):
        module.new_norm_rope_append(q, k, v, None, None, 0.0, 1e-6, True, None, None, None, False, slots, *caches)


@pytest.mark.parametrize("with_lse", [False, True])
def test_attention(module, with_lse):
    module, known = module
    q, k, v = rows(known, 3, 4, 128), rows(known, 2, 8, 2, 128), rows(known, 2, 8, 2, 128)
    table, lengths = rows(known, 3, 1, dtype=torch.int32), rows(known, 3, dtype=torch.int32)
    with pytest.raises(gdn.GdnError, match="host"):
        module.new_paged_attention_step(q, k, v, table, lengths, 0.0, None, 0, with_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["extension", "ctypes"])
def test_pinned_queries(way, monkeypatch, tmp_path):
    """Refused without a result to write to, and read where there is one."""
    build.build()
    gdn.gdn_init(0)
    if way == "ctypes":
        monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
        monkeypatch.setattr(binding, "_calls", binding._PyCall())
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(BF)

    q, k, v, caches = normal(3, 4, 128), normal(3, 2, 128), normal(3, 2, 128), (normal(3, 8, 2, 128), normal(3, 8, 2, 128))
    slots, table = torch.arange(3, device="cuda"), torch.arange(3, device="cuda").view(3, 1)
    lengths = torch.tensor([5, 0, 8], device="cuda")
    cos_sin, positions = torch.ones(9, 32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    pinned = q.cpu().pin_memory()
    calls = [(lambda x, **kw: gdn.qk_norm_rope(x, **kw)[0], "q_out"),
             (lambda x, **kw: gdn.qk_norm_rope(x, None, cos_sin, positions, pair_axes=[0, 1] * 8, **kw)[0], "q_out"),
             (lambda x, **kw: gdn.norm_rope_append(x, k, v, *caches, slots, **kw), "q_out"),
             (lambda x, **kw: gdn.paged_attention_step(x, *caches, table, lengths, **kw), "output")]
    for call, result in calls:
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            with pytest.raises(gdn.GdnError, match="host") as e:
                call(pinned, **kw)
            assert e.value.status == 1
        want, out = call(q), torch.empty_like(q)
        call(pinned, **{result: out})
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    with pytest.raises(gdn.GdnError, match="host"):
        gdn.paged_attention_step(pinned, *caches, table, lengths, return_lse=True)
    with pytest.raises(gdn.GdnError, match="host"):   # a pinned k beside a q of the device
        gdn.qk_norm_rope(q, k.cpu().pin_memory())
    assert gdn.device_status() == 0
