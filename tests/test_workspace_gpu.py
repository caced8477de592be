"""The one workspace of a device, under calls on several streams, in graphs, and while it grows."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import workloads as W
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _fresh(force_split):
    from gated_delta_rule_24_gb300 import build
    build.build()
    torch.cuda.synchronize()
    gdn.load_library().gdn_shutdown()   # no workspace yet
    gdn.gdn_init(0)
    force_split(8)
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


class Decay:
    def __init__(self, tokens, heads, seed):
        self.q, self.k, self.v, self.g, self.cu = R.make([tokens], heads, heads, gate="slow", seed=seed)
        self.out = torch.empty(tokens, heads, 128, dtype=BF, device="cuda")
        self.state = torch.empty(1, heads, 128, 128, device="cuda")

    def run(self, stream=None):
        gdn.decay_linear_attention(self.q, self.k, self.v, self.g, output_final_state=True, cu_seqlens=self.cu,
                                   output=self.out, output_state=self.state, stream=stream)

    def bits(self):
        return self.out.clone(), self.state.clone()


class DeltaRule:
    def __init__(self, tokens, heads, seed):
        self.p = W.make_problem([tokens], heads, heads, gates="mamba", init=None, seed=seed, batch_invariant=False)
        for name in ("q", "k", "v", "g", "beta", "cu_seqlens"):
            setattr(self.p, name, getattr(self.p, name).cuda())
        self.out = torch.empty(tokens, heads, 128, dtype=BF, device="cuda")
        self.state = torch.empty(1, heads, 128, 128, dtype=self.p.state_dtype, device="cuda")

    def run(self, stream=None):
        gdn.run_problem(self.p, output=self.out, output_state=self.state, stream=stream)

    bits = Decay.bits


def alone(work):
    work.run()
    torch.cuda.synchronize()
    bits = work.bits()
    work.out.fill_(9)
    work.state.fill_(9)
    torch.cuda.synchronize()
    return bits


def same(work, bits):
    return all(torch.equal(a, b) for a, b in zip(work.bits(), bits))


@pytest.mark.parametrize("kinds", [(Decay, Decay), (Decay, DeltaRule), (DeltaRule, DeltaRule)], ids=["decay", "both", "delta"])
def test_streams_take_turns(kinds):
    """Calls on three streams, of sizes that leave SMs free for one another, have the bits they have alone."""
    works = [kinds[i % 2](6000 + 900 * i, 2, 70 + i) for i in range(3)]
    want = [alone(w) for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(20):
        for w, s in zip(works, streams):
            w.run(s)
    torch.cuda.synchronize()
    assert all(same(w, b) for w, b in zip(works, want))


def test_growth_waits_for_the_other_stream():
    works = [Decay(4096, heads, 75 + heads) for heads in (1, 2, 4, 8, 16, 32)]
    want = [alone(w) for w in works]
    gdn.load_library().gdn_shutdown()
    gdn.gdn_init(0)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for i, w in enumerate(works):   # each needs twice the workspace of the one before it
        w.run(b if i % 2 else a)
    torch.cuda.synchronize()
    assert all(same(w, bits) for w, bits in zip(works, want))


def test_a_graph_outlives_growth():
    small, large = Decay(4096, 2, 80), Decay(4096, 24, 81)
    gdn.gdn_reserve_workspace(gdn.gdn_decay_workspace_bytes(1, 2, 4096))
    want = alone(small)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        small.run()
    expected = alone(large)   # a larger workspace takes over
    taken = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(64)]   # whatever was freed is in use again
    for _ in range(3):
        small.out.fill_(9)
        small.state.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert same(small, want)
    assert all(bool((t == 3.0).all()) for t in taken)
    large.run()
    torch.cuda.synchronize()
    assert same(large, expected)


def test_threads_take_turns():
    import threading
    works = [Decay(5000 + 700 * i, 2, 85 + i) for i in range(3)]
    want = [alone(w) for w in works]
    errors = []

    def loop(w):
        try:
            gdn.testing_force_splits(8)   # a setting of the thread
            stream = torch.cuda.Stream()
            for _ in range(20):
                w.run(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(same(w, bits) for w, bits in zip(works, want))
