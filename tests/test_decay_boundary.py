"""What the decay linear-attention entry points refuse, and how their arguments cross the C
ABI (these run on a machine without a GPU: nothing valid is launched)."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding

INVALID, UNSUPPORTED, ALIAS = 1, 2, 3
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def status(fn, args, **changed):
    a = dict(args, **changed)
    try:
        fn(**a, stream=0)
    except binding.GdnError as e:
        return e.status
    return 0


def prefill_args():
    return dict(q=z(10, 2, 128), k=z(10, 2, 128), v=z(10, 4, 128), g=torch.ones(10, 4), scale=0.0,
                initial_state=torch.zeros(2, 4, 128, 128), state_indices=None, output_state=torch.zeros(2, 4, 128, 128),
                cu_seqlens=torch.tensor([0, 4, 10], dtype=torch.int32), batch_invariant=False, output=z(10, 4, 128))


_s = torch.zeros(2, 4, 128, 128)
_o = z(10, 4, 128)
PREFILL = {
    "q_f32": (dict(q=torch.zeros(10, 2, 128)), UNSUPPORTED),
    "head_dim": (dict(q=z(10, 2, 64), k=z(10, 2, 64)), UNSUPPORTED),
    "q_none": (dict(q=None), INVALID),
    "q_2d": (dict(q=z(10, 128)), INVALID),
    "q_k_heads": (dict(k=z(10, 1, 128)), UNSUPPORTED),
    "k_rows": (dict(k=z(9, 2, 128)), UNSUPPORTED),
    "v_rows": (dict(v=z(9, 4, 128)), INVALID),
    "heads_not_a_multiple": (dict(v=z(10, 3, 128)), UNSUPPORTED),
    "mixed_dtypes": (dict(v=z(10, 4, 128, dtype=HF)), UNSUPPORTED),
    "inner_stride": (dict(q=z(10, 2, 256)[..., ::2]), INVALID),
    "odd_stride": (dict(q=z(10 * 260).as_strided((10, 2, 128), (260, 128, 1))), INVALID),
    "misaligned": (dict(q=z(10 * 256 + 8)[1:1 + 2560].view(10, 2, 128)), INVALID),
    "g_shape": (dict(g=torch.ones(10, 2)), INVALID),
    "g_i32": (dict(g=torch.ones(10, 4, dtype=torch.int32)), UNSUPPORTED),
    "scale_nan": (dict(scale=float("nan")), INVALID),
    "state_heads": (dict(initial_state=torch.zeros(2, 2, 128, 128)), INVALID),
    "state_k_major": (dict(initial_state=torch.zeros(2, 4, 128, 128).transpose(2, 3)), INVALID),
    "state_i32": (dict(output_state=torch.zeros(2, 4, 128, 128, dtype=torch.int32)), UNSUPPORTED),
    "few_slots": (dict(output_state=torch.zeros(1, 4, 128, 128)), INVALID),
    "few_slots_in": (dict(initial_state=torch.zeros(1, 4, 128, 128)), INVALID),
    "cu_none": (dict(cu_seqlens=None), INVALID),
    "cu_empty": (dict(cu_seqlens=torch.zeros(0, dtype=torch.int32)), INVALID),
    "cu_float": (dict(cu_seqlens=torch.tensor([0.0, 4.0, 10.0])), UNSUPPORTED),
    "indices_length": (dict(state_indices=torch.tensor([0, 1, 2])), INVALID),
    "output_none": (dict(output=None), INVALID),
    "output_dtype": (dict(output=z(10, 4, 128, dtype=HF)), UNSUPPORTED),
    "output_heads": (dict(output=z(10, 2, 128)), INVALID),
    "states_alias": (dict(initial_state=_s, output_state=_s), ALIAS),
    "output_is_v": (dict(v=_o, output=_o), ALIAS),
}


@pytest.mark.parametrize("case", PREFILL)
def test_prefill_refuses(case):
    changed, want = PREFILL[case]
    assert status(gdn.gdn_decay_prefill, prefill_args(), **changed) == want
    assert gdn.load_library().gdn_last_error()


def step_args():
    return dict(q=z(3, 2, 128), k=z(3, 2, 128), v=z(3, 4, 128), g=torch.ones(3, 4), scale=0.0,
                state=torch.zeros(3, 4, 128, 128), state_indices=None, output=z(3, 4, 128))


STEP = {
    "state_none": (dict(state=None), INVALID),
    "state_heads": (dict(state=torch.zeros(3, 2, 128, 128)), INVALID),
    "state_rows": (dict(state=torch.zeros(3, 4, 128, 256)[..., :128]), INVALID),
    "few_slots": (dict(state=torch.zeros(2, 4, 128, 128)), INVALID),
    "indices_length": (dict(state_indices=torch.tensor([0, 1])), INVALID),
    "indices_float": (dict(state_indices=torch.tensor([0.0, 1.0, 2.0])), UNSUPPORTED),
    "g_shape": (dict(g=torch.ones(4)), INVALID),
    "scale_inf": (dict(scale=float("inf")), INVALID),
    "output_rows": (dict(output=z(2, 4, 128)), INVALID),
    "q_f32": (dict(q=torch.zeros(3, 2, 128)), UNSUPPORTED),
}


@pytest.mark.parametrize("case", STEP)
def test_step_refuses(case):
    changed, want = STEP[case]
    assert status(gdn.gdn_decay_step, step_args(), **changed) == want


def test_step_refuses_a_state_that_holds_an_input():
    pool = torch.zeros(3, 4, 128, 128, dtype=BF)
    inside = pool.view(-1)[:3 * 2 * 128].view(3, 2, 128)
    assert status(gdn.gdn_decay_step, step_args(), state=pool, k=inside) == ALIAS
    assert status(gdn.gdn_decay_step, step_args(), state=pool, output=pool.view(-1)[:3 * 4 * 128].view(3, 4, 128)) == ALIAS


def rope_args():
    return dict(q=z(6, 4, 128), k=z(6, 2, 128), q_weight=torch.ones(128), k_weight=None, weight_offset=0.0, eps=1e-6,
                cos_sin=torch.zeros(10, 128), positions=None, interleaved=False, q_out=z(6, 4, 128), k_out=z(6, 2, 128))


_fused = z(6, 8, 128)
ROPE = {
    "q_none": (dict(q=None), INVALID),
    "k_without_out": (dict(k_out=None), INVALID),
    "out_without_k": (dict(k=None), INVALID),
    "weight_without_k": (dict(k=None, k_out=None, k_weight=torch.ones(128)), INVALID),
    "k_rows": (dict(k=z(5, 2, 128), k_out=z(5, 2, 128)), INVALID),
    "k_dtype": (dict(k=z(6, 2, 128, dtype=HF), k_out=z(6, 2, 128, dtype=HF)), UNSUPPORTED),
    "out_dtype": (dict(q_out=z(6, 4, 128, dtype=HF)), UNSUPPORTED),
    "out_shape": (dict(q_out=z(6, 3, 128)), INVALID),
    "head_dim": (dict(q=z(6, 4, 64), q_out=z(6, 4, 64)), UNSUPPORTED),
    "weight_size": (dict(q_weight=torch.ones(64)), INVALID),
    "weight_stride": (dict(q_weight=torch.ones(256)[::2]), INVALID),
    "weight_i32": (dict(q_weight=torch.ones(128, dtype=torch.int32)), UNSUPPORTED),
    "eps_negative": (dict(eps=-1.0), INVALID),
    "eps_nan": (dict(eps=float("nan")), INVALID),
    "offset_inf": (dict(weight_offset=float("inf")), INVALID),
    "rotary_odd": (dict(cos_sin=torch.zeros(10, 24)), UNSUPPORTED),
    "rotary_large": (dict(cos_sin=torch.zeros(10, 144)), UNSUPPORTED),
    "table_bf16": (dict(cos_sin=z(10, 128)), UNSUPPORTED),
    "table_transposed": (dict(cos_sin=torch.zeros(128, 16).t()), INVALID),
    "few_places": (dict(cos_sin=torch.zeros(5, 128)), INVALID),
    "positions_length": (dict(positions=torch.zeros(5, dtype=torch.int32)), INVALID),
    "positions_float": (dict(positions=torch.zeros(6)), UNSUPPORTED),
    "positions_alone": (dict(cos_sin=None, positions=torch.zeros(6, dtype=torch.int32)), INVALID),
    "out_over_part_of_q": (dict(q=_fused[:, :4], q_out=_fused[:, 1:5]), ALIAS),
    "out_over_k": (dict(k=_fused[:, :2], q_out=_fused[:, 1:5]), ALIAS),
    "outs_overlap": (dict(q_out=_fused[:, :4], k_out=_fused[:, 3:5]), ALIAS),
}


@pytest.mark.parametrize("case", ROPE)
def test_norm_rope_refuses(case):
    changed, want = ROPE[case]
    assert status(gdn.gdn_qk_norm_rope, rope_args(), **changed) == want


@pytest.mark.parametrize("fn,args,changed", [
    (gdn.gdn_decay_prefill, prefill_args, {}),
    (gdn.gdn_decay_prefill, prefill_args, dict(g=torch.ones(4).expand(10, 4))),
    (gdn.gdn_decay_step, step_args, {}),
    (gdn.gdn_qk_norm_rope, rope_args, {}),
    (gdn.gdn_qk_norm_rope, rope_args, dict(q=_fused[:, :4], k=_fused[:, 4:6], q_out=_fused[:, :4], k_out=_fused[:, 4:6])),
], ids=["prefill", "prefill_head_gate", "step", "rope", "rope_in_place"])
def test_valid_arguments_reach_the_device_check(fn, args, changed):
    """The counterpart of the refusals: good arguments pass every check of the arguments."""
    if torch.cuda.is_available():
        pytest.skip("the arguments are host tensors: only for a machine without a GPU")
    assert status(fn, args(), **changed) not in (0, INVALID, ALIAS)


def test_descriptors_match_the_struct():
    for t in (torch.zeros(3), torch.zeros(4, 6)[:, 1:3], z(2, 3, 4).transpose(0, 2), torch.zeros(1, 2, 3, 4),
              torch.ones(5).expand(7, 5), torch.tensor(1.0)):
        none, at = binding._descriptors.fill(None, t)
        assert none is None
        got, want = ctypes.cast(at, ctypes.POINTER(binding.GdnTensor)).contents, binding.describe(t)
        assert (got.data, got.dtype, got.ndim) == (want.data, want.dtype, want.ndim)
        assert list(got.shape)[:t.dim()] == list(t.shape) and list(got.stride)[:t.dim()] == list(t.stride())
    with pytest.raises(TypeError):
        binding._descriptors.fill(torch.zeros(2, dtype=torch.int8))
    with pytest.raises(ValueError):
        binding._descriptors.fill(torch.zeros(1, 1, 1, 1, 1))


def test_wrappers_ask_for_bounds():
    a = prefill_args()
    with pytest.raises(ValueError):
        gdn.decay_linear_attention(a["q"], a["k"], a["v"], a["g"])


def test_workspace_bytes_follow_the_plan():
    """A state and a decay for each segment but the last; nothing where units fill the SMs."""
    plan = gdn.gdn_decay_workspace_bytes
    assert plan(0, 4, 100, 152) == 0 and plan(4, 0, 100, 152) == 0 and plan(4, 4, 100, 0) == 0
    assert plan(512, 16, 512 * 4096, 152) == 0 and plan(1, 1, 256, 152) == 0
    for args in ((1, 8, 32000, 152), (2, 32, 131072, 152), (1, 1, 1 << 20, 152)):
        got = plan(*args)
        blocks, rest = divmod(got, 65536 + 4)
        assert rest == 0 and blocks % (args[0] * args[1]) == 0 and 1 <= blocks // (args[0] * args[1]) < args[3]
    try:
        gdn.testing_force_splits(3)
        assert plan(5, 4, 1000, 152) == 5 * 4 * 2 * (65536 + 4)
    finally:
        gdn.testing_force_splits(0)


def test_calls_refuse_what_is_no_tensor():
    a = dict(step_args(), stream=0)
    with pytest.raises(AttributeError):
        gdn.gdn_decay_step(**dict(a, q=[1.0]))
    with pytest.raises(TypeError):
        gdn.gdn_decay_step(**dict(a, scale="1"))
    with pytest.raises(TypeError):
        gdn.gdn_decay_step(**dict(a, state=torch.zeros(3, 4, 128, 128, dtype=torch.int8)))
    with pytest.raises(ValueError):
        gdn.gdn_decay_step(**dict(a, k=torch.zeros(1, 1, 1, 1, 1)))
    with pytest.raises(RuntimeError):  # GdnError: host tensors, or no GPU at all
        gdn.decay_linear_step(a["q"], a["k"], a["v"], a["state"], torch.ones(a["v"].shape[1]), stream=0)
