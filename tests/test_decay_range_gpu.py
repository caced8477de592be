"""f16 inputs near the ends of the range that include/gdn.h gives for the scores and the state."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from tests import decay_ref as R

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()
    gdn.gdn_init(0)
    yield
    assert gdn.device_status() == 0


def run(q, k, v, g, cu, **kw):
    out, state = gdn.decay_linear_attention(q, k, v, g, output_final_state=True, cu_seqlens=cu, **kw)
    return out, state


@pytest.mark.parametrize("sq,sk,sv", [(100.0, 100.0, 1e-4), (100.0, 1e-2, 1e-2), (1e-2, 100.0, 0.1)], ids=str)
def test_inside(sq, sk, sv):
    """Scores of up to 6e4 (a hundred thousand of them, each 1e4 times a normal number: 4.5e4 at most), and states of 1e-3."""
    lengths = [300, 130]
    q, k, v, g, cu = R.make(lengths, 2, 2, HF, "slow", seed=99)
    q, k, v = ((x.float() * s).to(HF) for x, s in ((q, sq), (k, sk), (v, sv)))
    out, state = run(q, k, v, g, cu)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None, lengths)
    R.check(out, o_ref, state, s_ref, lengths)


def test_outside():
    """Scores of 5e5: outputs overflow, the states do not, and the other head and sequence do not notice."""
    lengths = [300, 130]
    q, k, v, g, cu = R.make(lengths, 2, 2, HF, "slow", seed=100)
    v = (v.float() * 1e-3).to(HF)
    for x in (q, k):
        x[:300, 0] = (x[:300, 0].float() * 700).to(HF)
    out, state = run(q, k, v, g, cu)
    o_ref, s_ref = R.recurrence(q, k, v, g, SCALE, None, lengths)
    assert not bool(torch.isfinite(out[:300, 0]).all())
    R.check(out[:, 1:], o_ref[:, 1:], state[:, 1:], s_ref[:, 1:], lengths)
    R.check(out, o_ref, state, s_ref, lengths, which=(1,))
    assert R.rel(state[0, 0], s_ref[0, 0]) <= R.STATE[F32]
