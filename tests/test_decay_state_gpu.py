"""What f32 states of the decay prefill hold after many tokens, against sums in 64 bits."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def summed(k, v, g, state=None):
    """The state behind one sequence, [H, 128, 128] in 64 bits: every token's product times the decays behind it."""
    T, H = v.shape[:2]
    logs = torch.zeros(T, H, dtype=torch.float64, device=v.device) if g is None else g.double().expand(T, H).log()
    behind = logs.flip(0).cumsum(0).flip(0) - logs
    s = torch.einsum("thr,thc->hrc", v.double() * behind.exp()[..., None], k.double())
    return s if state is None else s + logs.sum(0).exp()[:, None, None] * state.double()


def final_state(q, k, v, g, state=None, **kw):
    cu = torch.tensor([0, q.shape[0]], dtype=torch.int32, device="cuda")
    _, s = gdn.decay_linear_attention(q, k, v, g, initial_state=state, output_final_state=True, cu_seqlens=cu, **kw)
    assert s.dtype == F32
    return s


# A state that tokens of zeros pass over is multiplied by one decay a chunk: 2^x, with an error of up to two units in
# the last place, and the rounding of the product, half of one.  A unit is at most 2^-23 of the value.
UNITS = 3 * 2.0 ** -23
DECAYS = (1 - 2.0 ** -24, 1 - 1e-6, 0.99999, 0.9999)


@pytest.mark.parametrize("invariant", [True, False], ids=["uncut", "planned"])
@pytest.mark.parametrize("zeros", ["keys", "values"])
def test_tokens_of_zeros_only_decay(zeros, invariant):
    T, g = 64000, torch.tensor(DECAYS, device="cuda")
    q, k, v, _, _ = R.make([T], len(DECAYS), len(DECAYS), gate="none", seed=60)
    (k if zeros == "keys" else v)[1:] = 0
    got, want = final_state(q, k, v, g, batch_invariant=invariant)[0], summed(k, v, g)
    for h in range(len(DECAYS)):
        assert R.rel(got[h], want[h]) <= T / 128 * UNITS, (DECAYS[h], R.rel(got[h], want[h]))


def test_short_calls_of_zeros_only_decay():
    calls, g = 400, torch.tensor(DECAYS, device="cuda")
    q, k, v, _, _ = R.make([3], len(DECAYS), len(DECAYS), gate="none", seed=61)
    s0 = R.states(1, len(DECAYS), F32, 61)
    for n in (1, 3):
        s = s0
        for _ in range(calls):
            s = final_state(q[:n], torch.zeros_like(k[:n]), v[:n], g, s)
        want = s0.double() * (g.double() ** (n * calls))[:, None, None]
        for h in range(len(DECAYS)):
            assert R.rel(s[0, h], want[0, h]) <= calls * UNITS, (n, DECAYS[h], R.rel(s[0, h], want[0, h]))


# From here on the bound is that of f32 sums, whatever the number of tokens or calls (tests/decay_ref.py).


def each_head(got, want, what):
    for h in range(want.shape[0]):
        assert R.rel(got[h], want[h]) <= R.STATE[F32], (what, h, R.rel(got[h], want[h]))


@pytest.mark.parametrize("T,invariant", [(16000, True), (60000, True), (60000, False)], ids=["16000", "60000", "60000_planned"])
@pytest.mark.parametrize("gate", ["none", 1e-5, 5e-4, "slow", "token"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_long_sums(dtype, gate, T, invariant):
    """A number: one decay of exp(-gate) for all tokens."""
    q, k, v, g, _ = R.make([T], 2, 2, dtype, gate if isinstance(gate, str) else "none", seed=62)
    if not isinstance(gate, str):
        g = torch.exp(torch.full((2,), -gate, device="cuda"))
    s0 = R.states(1, 2, F32, 62)
    each_head(final_state(q, k, v, g, s0, batch_invariant=invariant)[0], summed(k, v, g, s0[0]), (gate, T))


@pytest.mark.parametrize("n", [1, 4, 8, 128])
@pytest.mark.parametrize("gate", [0.0, 5e-4, "slow"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_short_calls(dtype, gate, n):
    """4096 tokens, n a call, into one state."""
    T = 4096
    q, k, v, g, _ = R.make([T], 2, 2, dtype, gate if isinstance(gate, str) else "none", seed=63)
    if not isinstance(gate, str):
        g = torch.exp(torch.full((T, 2), -gate, device="cuda"))
    s = None
    for t in range(0, T, n):
        s = final_state(q[t:t + n], k[t:t + n], v[t:t + n], g[t:t + n], s)
    each_head(s[0], summed(k, v, g), (gate, n))


@pytest.mark.parametrize("invariant", [True, False], ids=["uncut", "planned"])
def test_sparse_keys(invariant):
    """One token in 700 has a key; between them nothing but decays."""
    T, g = 64000, torch.tensor(DECAYS, device="cuda")
    q, k, v, _, _ = R.make([T], len(DECAYS), len(DECAYS), gate="none", seed=64)
    k[torch.arange(T, device="cuda") % 700 != 5] = 0
    each_head(final_state(q, k, v, g, batch_invariant=invariant)[0], summed(k, v, g), "sparse")


@pytest.mark.parametrize("T,splits", [(5, 1), (700, 1), (3000, 1), (3000, 4)])
@pytest.mark.parametrize("std", [1e4, 1e-2, 1e-3, 1e-4, 1e-6])
def test_f16_values_of_any_size(force_split, std, T, splits):
    """f16 values far from 1, next to the smallest (2^-24) and the largest there are, also where the last tokens of
    a chunk are zeros and only decayed ones count, and with a first row of heads that is a thousand times larger."""
    force_split(splits)
    for gate in ("token", "slow", "none"):
        q, k, v, g, _ = R.make([T], 2, 2, HF, gate, seed=65)
        v = (v.float() * std).clamp(-6e4, 6e4).to(HF)
        each_head(final_state(q, k, v, g)[0], summed(k, v, g), (gate, "all"))
        v[:, 1, ::16] = (v[:, 1, ::16].float() * 1e3).clamp(-6e4, 6e4).to(HF)
        got, want = final_state(q, k, v, g)[0], summed(k, v, g)
        each_head(got, want, (gate, "rows"))
        small = torch.arange(128, device="cuda") % 16 != 0
        assert R.rel(got[1, small], want[1, small]) <= R.STATE[F32], (gate, R.rel(got[1, small], want[1, small]))
        v[torch.arange(T, device="cuda") % 128 > 118] = 0
        each_head(final_state(q, k, v, g)[0], summed(k, v, g), (gate, "zeros"))


@pytest.mark.parametrize("state,std", [(HF, 3.0), (HF, 1e-2), (BF, 3.0), (BF, 1e-2), (BF, 1e-5)], ids=str)
def test_f16_values_into_16_bit_states(state, std):
    q, k, v, g, cu = R.make([700], 2, 2, HF, "token", seed=66)
    v = (v.float() * std).to(HF)
    final = torch.empty(1, 2, 128, 128, dtype=state, device="cuda")
    gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu, output_state=final)
    want = summed(k, v, g)
    for h in range(2):
        assert R.rel(final[0, h], want[h]) <= R.STATE[state], (h, R.rel(final[0, h], want[h]))
