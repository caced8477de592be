"""The operators of a softmax-attention layer one behind the other: prompts and new tokens appended, a prefix shared, steps by
themselves and captured into a graph."""
import importlib.util
import os

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding
from tests import attention_ref as A
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


class Layer:
    """``prompts`` tokens of each sequence behind a prefix; the last one is padding, with no tokens and no place."""

    def __init__(self, prompts, prefix, room, h_q=8, h_k=2, page=16, dtype=BF, layout="places", seed=0, axes=False):
        self.n, self.h_q, self.h_k, self.page, self.dtype, self.prefix = len(prompts), h_q, h_k, page, dtype, prefix
        width = -(-room // page)
        shared = -(-prefix // page)
        pool = torch.randperm(shared + self.n * width, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        self.k_cache, self.v_cache = A.cache(len(pool), page, h_k, dtype, layout, fill=float("nan"))
        self.prefix_pages, self.table = pool[:shared].contiguous() if prefix else None, pool[shared:].view(self.n, width)
        self.lengths = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.cs, self.seed = R.table(4096, 64), seed
        self.pair_axes = [i % 3 for i in range(32)] if axes else None
        self.w = 1 + A.normal(2, 128, dtype=torch.float32, seed=seed + 1, std=0.1)
        if prefix:
            at = torch.arange(prefix, device="cuda")
            self.append(prefix, at, self.prefix_pages[at // page] * page + at % page)
        for i, count in enumerate(prompts):
            if count:
                at = torch.arange(count, device="cuda")
                self.append(count, prefix + at, self.table[i, at // page] * page + at % page)
                self.lengths[i] = count

    def new(self, tokens):
        self.seed += 10
        return A.normal(tokens, self.h_q + 2 * self.h_k, 128, dtype=self.dtype, seed=self.seed, std=1.5)

    def turn(self, qkv, positions, slots):
        q, k, v = qkv.split([self.h_q, self.h_k, self.h_k], 1)
        if self.pair_axes:
            positions = torch.stack([positions, positions // 7, positions % 5])
        return gdn.norm_rope_append(q, k, v, self.k_cache, self.v_cache, slots, self.cs, positions, *self.w, pair_axes=self.pair_axes)

    def append(self, tokens, positions, slots):
        return self.turn(self.new(tokens), positions, slots)

    def places(self, tokens):
        """Positions and slots of each sequence's next tokens (none for the padding, the last one)."""
        at = (self.lengths[:, None] + torch.arange(tokens, device="cuda")).long()
        slots = self.table.gather(1, at // self.page).long() * self.page + at % self.page
        slots[-1] = -1
        return (self.prefix + at).reshape(-1), slots.reshape(-1)

    def attend(self, q, **kw):
        return gdn.paged_attention_step(q, self.k_cache, self.v_cache, self.table, self.lengths, prefix_pages=self.prefix_pages,
                                        prefix_length=self.prefix, return_lse=True, **kw)

    def held(self, pages, count):
        at = torch.arange(count, device="cuda")
        at = pages[at // self.page].long() * self.page + at % self.page
        return tuple(c.flatten(0, 1)[at] if c.is_contiguous() else c[at // self.page, at % self.page] for c in (self.k_cache, self.v_cache))

    def check(self, q, got, tokens):
        """Against the attention in 64 bits over what the caches hold, which were checked by themselves."""
        shared = self.held(self.prefix_pages, self.prefix) if self.prefix else (q.new_zeros(0, self.h_k, 128),) * 2
        keys = [self.held(self.table[i], int(self.lengths[i])) for i in range(self.n)]
        A.check(got, A.attend(q, keys, shared, tokens))


@pytest.mark.parametrize("kw", [dict(prefix=0), dict(prefix=77, page=24, dtype=HF, layout="heads"), dict(prefix=300, h_q=32, axes=True, layout="woven")],
                         ids=["alone", "prefix", "prefix_of_many_rows"])
@pytest.mark.parametrize("tokens", [1, 3])
def test_prompts_and_steps(kw, tokens):
    layer = Layer([50, 1, 130, 16, 0], room=200, seed=60, **kw)
    for _ in range(6):
        positions, slots = layer.places(tokens)
        q = layer.append(layer.n * tokens, positions, slots)
        layer.lengths[:-1] += tokens
        layer.check(q, layer.attend(q), tokens)


def test_steps_captured_into_a_graph():
    layer = Layer([50, 1, 130, 16, 0], prefix=300, room=200, h_q=32, seed=61)
    qkv, out = layer.new(layer.n), torch.empty(layer.n, 32, 128, dtype=BF, device="cuda")
    lse = torch.empty(layer.n, 32, device="cuda")
    kept = {}

    def step():
        positions, slots = layer.places(1)
        kept["q"] = layer.turn(qkv, positions, slots)
        layer.lengths[:-1] += 1
        layer.attend(kept["q"], output=out, lse=lse)

    gdn.gdn_reserve_workspace(gdn.gdn_paged_attention_workspace_bytes(layer.n, 1, 32, 2, 300))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()   # once before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        qkv.copy_(layer.new(layer.n))
        graph.replay()
    torch.cuda.synchronize()
    assert layer.lengths.tolist() == [71, 22, 151, 37, 0]
    layer.check(kept["q"], (out, lse), 1)


def test_the_same_results_by_ctypes(monkeypatch, tmp_path):
    def run():
        layer = Layer([40, 9, 0], prefix=33, room=60, seed=62, axes=True)
        positions, slots = layer.places(1)
        q = layer.append(3, positions, slots)
        layer.lengths[:-1] += 1
        turned = gdn.qk_norm_rope(q, q[:, :2], layer.cs, torch.stack([positions] * 3), pair_axes=layer.pair_axes)
        return (q, *layer.attend(q), *turned, layer.k_cache.nan_to_num(0.5))

    want = run()
    monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
    monkeypatch.setattr(binding, "_calls", binding._PyCall())
    got = run()
    assert isinstance(binding._calls.norm_rope_append.__self__, binding._ByCtypes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("way", ["extension", "ctypes"])
def test_host_tensors_are_refused(way, monkeypatch, tmp_path):
    if way == "ctypes":
        monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
        monkeypatch.setattr(binding, "_calls", binding._PyCall())
    layer = Layer([40, 9, 0], prefix=33, room=60, seed=63)
    positions, slots = layer.places(1)
    q, k, v = layer.new(3).split([8, 2, 2], 1)

    def refused(call, *args, **kw):
        with pytest.raises(gdn.GdnError, match="host") as e:
            call(*args, **kw)
        assert e.value.status == 1

    for i in range(8):
        args = [q, k, v, layer.k_cache, layer.v_cache, slots, layer.cs, positions]
        args[i] = args[i].cpu()
        refused(gdn.norm_rope_append, *args, q_out=torch.empty_like(q))
    for i in range(5):
        args = [q, layer.k_cache, layer.v_cache, layer.table, layer.lengths]
        args[i] = args[i].cpu()
        refused(gdn.paged_attention_step, *args, output=torch.empty_like(q))
    refused(gdn.paged_attention_step, q, layer.k_cache, layer.v_cache, layer.table, layer.lengths, prefix_pages=layer.prefix_pages.cpu(), prefix_length=33)
    refused(gdn.qk_norm_rope, q, k, layer.cs, torch.stack([positions] * 3).cpu(), pair_axes=[0] * 32)


def test_results_belong_to_the_stream_that_is_given():
    layer = Layer([40, 9, 0], prefix=33, room=60, seed=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    positions, slots = layer.places(1)
    qkv = layer.new(3)
    side.wait_stream(torch.cuda.current_stream())
    q, k, v = qkv.split([8, 2, 2], 1)
    turned = gdn.norm_rope_append(q, k, v, layer.k_cache, layer.v_cache, slots, layer.cs, positions, *layer.w, stream=side)
    with torch.cuda.stream(side):
        layer.lengths[:-1] += 1
    got = layer.attend(turned, stream=side)
    side.synchronize()
    layer.check(turned, got, 1)


def test_the_example_runs():
    spec = importlib.util.spec_from_file_location("softmax_layer", os.path.join(ROOT, "examples", "softmax_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(n=3, prefix=50, steps=20) < 2.0 ** -7   # the output's and the weights' rounding, 2^-8 each at most
    assert example.main(n=40, prefix=200, steps=3) < 2.0 ** -7
