"""What the append and the attention over a paged cache refuse (these run on a machine without a GPU: nothing valid is launched)."""
import pytest
import torch

import gated_delta_rule_24_gb300 as gdn
from gated_delta_rule_24_gb300 import binding
from tests.attention_ref import cache
from tests.test_decay_boundary import ALIAS, BF, HF, INVALID, UNSUPPORTED, status, z

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_24_gb300 import build
    build.build()


@pytest.fixture(params=["extension", "ctypes"])
def way(request, monkeypatch, tmp_path):
    if request.param == "ctypes":
        monkeypatch.setattr(binding, "_PYCALL_PATH", str(tmp_path / "gdn_pycall.so"))
        monkeypatch.setattr(binding, "_calls", binding._PyCall())


def axes_args():
    return dict(q=z(6, 4, 128), k=z(6, 2, 128), q_weight=torch.ones(128), k_weight=None, weight_offset=0.0, eps=1e-6,
                cos_sin=torch.zeros(10, 128), positions=torch.zeros(3, 6, dtype=I32), pair_axes=[0, 1] * 32, interleaved=False,
                q_out=z(6, 4, 128), k_out=z(6, 2, 128))


AXES = {
    "no_table": (dict(cos_sin=None), INVALID),
    "no_positions": (dict(positions=None), INVALID),
    "one_dim": (dict(positions=torch.zeros(6, dtype=I32)), INVALID),
    "five_axes": (dict(positions=torch.zeros(5, 6, dtype=I32)), UNSUPPORTED),
    "no_axes": (dict(positions=torch.zeros(0, 6, dtype=I32)), UNSUPPORTED),
    "tokens": (dict(positions=torch.zeros(3, 5, dtype=I32)), INVALID),
    "strided": (dict(positions=torch.zeros(6, 3, dtype=I32).t()), INVALID),
    "float": (dict(positions=torch.zeros(3, 6)), UNSUPPORTED),
    "few_pairs": (dict(pair_axes=[0] * 63), INVALID),
    "no_pairs": (dict(pair_axes=[]), INVALID),
    "axis_3_of_3": (dict(pair_axes=[0] * 63 + [3]), INVALID),
    "axis_below": (dict(pair_axes=[-1] + [0] * 63), INVALID),
    "axis_far": (dict(pair_axes=[1 << 32] + [0] * 63), INVALID),
    "axis_far_below": (dict(pair_axes=[-(1 << 40)] + [0] * 63), INVALID),
    "out_over_positions": (dict(q_out=torch.zeros(6 * 4 * 128, dtype=BF).view(6, 4, 128)), None),
    "eps_nan": (dict(eps=float("nan")), INVALID),
}


@pytest.mark.parametrize("case", AXES)
def test_axes_refuses(way, case):
    changed, want = AXES[case]
    if want is None:
        room = torch.zeros(6 * 4 * 128, dtype=BF)
        changed, want = dict(q_out=room.view(6, 4, 128), positions=room.view(I32)[:18].view(3, 6)), ALIAS
    assert status(gdn.gdn_qk_norm_rope_axes, axes_args(), **changed) == want
    assert gdn.load_library().gdn_last_error()


def test_axes_are_integers(way):
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope_axes(**dict(axes_args(), pair_axes=None, stream=0))
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope_axes(**dict(axes_args(), pair_axes=[0] * 65, stream=0))
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope_axes(**dict(axes_args(), pair_axes=["0"] * 64, stream=0))
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope_axes(**dict(axes_args(), pair_axes=5, stream=0))


def append_args():
    k, v = cache(3, 16, 2, fill=0.0, device="cpu")
    return dict(q=z(6, 4, 128), k=z(6, 2, 128), v=z(6, 2, 128), q_weight=torch.ones(128), k_weight=None, weight_offset=0.0, eps=1e-6,
                norm=True, cos_sin=torch.zeros(10, 128), positions=None, pair_axes=None, interleaved=False,
                slots=torch.arange(6, dtype=I32), q_out=z(6, 4, 128), k_cache=k, v_cache=v)


_fused, _cache = z(6, 8, 128), z(3, 16, 2, 128)
_big = z(4 * 4096 * 2)
APPEND = {
    "q_none": (dict(q=None), INVALID),
    "k_none": (dict(k=None), INVALID),
    "v_none": (dict(v=None), INVALID),
    "slots_none": (dict(slots=None), INVALID),
    "out_none": (dict(q_out=None), INVALID),
    "k_cache_none": (dict(k_cache=None), INVALID),
    "v_cache_none": (dict(v_cache=None), INVALID),
    "v_dtype": (dict(v=z(6, 2, 128, dtype=HF)), UNSUPPORTED),
    "v_rows": (dict(v=z(5, 2, 128)), INVALID),
    "v_heads": (dict(v=z(6, 4, 128)), INVALID),
    "head_dim": (dict(v=z(6, 2, 64)), UNSUPPORTED),
    "cache_dtype": (dict(k_cache=z(3, 16, 2, 128, dtype=HF)), UNSUPPORTED),
    "cache_heads": (dict(k_cache=z(3, 16, 4, 128), v_cache=z(3, 16, 4, 128)), INVALID),
    "cache_shapes": (dict(k_cache=z(4, 16, 2, 128)), INVALID),
    "cache_head_dim": (dict(k_cache=z(3, 16, 2, 64)), UNSUPPORTED),
    "cache_3d": (dict(k_cache=z(48, 2, 128)), INVALID),
    "cache_inner": (dict(k_cache=z(3, 16, 2, 256)[..., ::2]), INVALID),
    "cache_stride": (dict(k_cache=z(3 * 16 * 260).as_strided((3, 16, 2, 128), (16 * 260, 260, 128, 1))), INVALID),
    "cache_misaligned": (dict(k_cache=z(3 * 16 * 256 + 8)[4:4 + 3 * 16 * 256].view(3, 16, 2, 128)), INVALID),
    "cache_pages_overlap": (dict(k_cache=z(3 * 16 * 256).as_strided((3, 16, 2, 128), (256, 256, 128, 1))), INVALID),
    "cache_heads_overlap": (dict(k_cache=z(3 * 16 * 256).as_strided((3, 16, 2, 128), (4096, 256, 64, 1))), INVALID),
    "cache_expanded": (dict(k_cache=z(1, 16, 2, 128).expand(3, 16, 2, 128)), INVALID),
    "no_places": (dict(k_cache=z(3, 0, 2, 128), v_cache=z(3, 0, 2, 128)), INVALID),
    "slots_length": (dict(slots=torch.arange(5, dtype=I32)), INVALID),
    "slots_float": (dict(slots=torch.zeros(6)), UNSUPPORTED),
    "slots_strided": (dict(slots=torch.arange(12, dtype=I32)[::2]), INVALID),
    "weight_without_norm": (dict(norm=False), INVALID),
    "pairs_without_positions": (dict(pair_axes=[0] * 64), INVALID),
    "pairs_without_table": (dict(cos_sin=None, pair_axes=[0] * 64), INVALID),
    "positions_2d_without_pairs": (dict(positions=torch.zeros(1, 6, dtype=I32)), INVALID),
    "few_places": (dict(cos_sin=torch.zeros(5, 128)), INVALID),
    "positions_alone": (dict(cos_sin=None, positions=torch.zeros(6, dtype=I32)), INVALID),
    "out_over_k": (dict(k=_fused[:, :2], q_out=_fused[:, 1:5]), ALIAS),
    "out_over_part_of_q": (dict(q=_fused[:, :4], q_out=_fused[:, 1:5]), ALIAS),
    "caches_are_one": (dict(k_cache=_cache, v_cache=_cache), ALIAS),
    "caches_overlap": (dict(k_cache=z(4, 16, 2, 128)[:3], v_cache=None), None),
    "cache_over_q": (dict(q=_cache.view(-1)[:6 * 512].view(6, 4, 128), k_cache=_cache), ALIAS),
    "cache_over_out": (dict(q_out=_cache.view(-1)[:6 * 512].view(6, 4, 128), v_cache=_cache), ALIAS),
    "cache_over_slots": (dict(slots=_cache.view(-1).view(I32)[:6], v_cache=_cache), ALIAS),
    "eps_negative": (dict(eps=-1.0), INVALID),
    "offset_inf": (dict(weight_offset=float("inf")), INVALID),
}


@pytest.mark.parametrize("case", APPEND)
def test_append_refuses(way, case):
    changed, want = APPEND[case]
    if want is None:
        four = z(4, 16, 2, 128)
        changed, want = dict(k_cache=four[:3], v_cache=four[1:]), ALIAS
    assert status(gdn.gdn_norm_rope_append, append_args(), **changed) == want
    assert gdn.load_library().gdn_last_error()


def _views(what):
    """Caches [3, 16, 2, 128] in one buffer that share no element, and some that do."""
    both, side = z(3, 2, 16, 2, 128), z(3, 16, 4, 128)
    return {
        "woven_by_pages": (both[:, 0], both[:, 1]),
        "woven_by_pages_turned": (both[:, 1], both[:, 0]),
        "side_by_side": (side[:, :, :2], side[:, :, 2:]),
        "every_other_head": (side[:, :, ::2], side[:, :, 1::2]),
        "by_heads": tuple(z(3, 2, 2, 16, 128)[:, i].transpose(1, 2) for i in range(2)),
        "woven_by_places": tuple(z(3, 16, 2, 2, 128)[:, :, i] for i in range(2)),
        "half_a_head_on": (_big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1)), _big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1), 64)),
        "a_page_on": (_big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1)), _big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1), 8192)),
        "a_place_on": (_big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1)), _big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1), 512)),
        "other_strides": (_big.as_strided((3, 16, 2, 128), (4096 * 2, 512, 256, 1)), _big.as_strided((3, 16, 2, 128), (4096, 256, 128, 1), 4096 * 2)),
    }[what]


@pytest.mark.parametrize("what,shared", [("woven_by_pages", False), ("woven_by_pages_turned", False), ("side_by_side", False),
                                         ("every_other_head", False), ("by_heads", False), ("woven_by_places", False),
                                         ("half_a_head_on", True), ("a_page_on", True), ("a_place_on", True), ("other_strides", True)])
def test_caches_of_one_buffer(what, shared):
    if torch.cuda.is_available():
        pytest.skip("the arguments are host tensors: only for a machine without a GPU")
    k, v = _views(what)
    got = status(gdn.gdn_norm_rope_append, append_args(), k_cache=k, v_cache=v)
    assert got == ALIAS if shared else got not in (0, INVALID, ALIAS)


def attend_args():
    k, v = cache(5, 16, 2, fill=0.0, device="cpu")
    return dict(q=z(6, 4, 128), k_cache=k, v_cache=v, page_table=torch.zeros(3, 2, dtype=I32), lengths=torch.zeros(3, dtype=I32),
                scale=0.0, prefix_pages=torch.zeros(2, dtype=I32), prefix_length=20, output=z(6, 4, 128), lse=torch.zeros(6, 4))


ATTEND = {
    "q_none": (dict(q=None), INVALID),
    "q_f32": (dict(q=torch.zeros(6, 4, 128)), UNSUPPORTED),
    "head_dim": (dict(q=z(6, 4, 64)), UNSUPPORTED),
    "q_dtype": (dict(q=z(6, 4, 128, dtype=HF)), UNSUPPORTED),
    "heads": (dict(q=z(6, 5, 128), output=z(6, 5, 128), lse=torch.zeros(6, 5)), UNSUPPORTED),
    "cache_none": (dict(v_cache=None), INVALID),
    "cache_shapes": (dict(v_cache=z(4, 16, 2, 128)), INVALID),
    "cache_expanded": (dict(v_cache=z(1, 16, 2, 128).expand(5, 16, 2, 128)), INVALID),
    "page_of_12": (dict(k_cache=z(5, 12, 2, 128), v_cache=z(5, 12, 2, 128)), UNSUPPORTED),
    "rows": (dict(q=z(7, 4, 128), output=z(7, 4, 128), lse=torch.zeros(7, 4)), INVALID),
    "no_sequences": (dict(page_table=torch.zeros(0, 2, dtype=I32), lengths=torch.zeros(0, dtype=I32)), INVALID),
    "17_tokens": (dict(q=z(51, 4, 128), output=z(51, 4, 128), lse=torch.zeros(51, 4)), UNSUPPORTED),
    "no_tokens": (dict(q=z(0, 4, 128), output=z(0, 4, 128), lse=torch.zeros(0, 4)), UNSUPPORTED),
    "table_none": (dict(page_table=None), INVALID),
    "table_rows": (dict(page_table=torch.zeros(2, 2, dtype=I32)), INVALID),
    "table_1d": (dict(page_table=torch.zeros(6, dtype=I32)), INVALID),
    "table_float": (dict(page_table=torch.zeros(3, 2)), UNSUPPORTED),
    "table_transposed": (dict(page_table=torch.zeros(2, 3, dtype=I32).t()), INVALID),
    "table_too_wide": (dict(page_table=torch.zeros(1, dtype=I32).expand(3, 1 << 27)), INVALID),
    "table_too_many_keys": (dict(page_table=torch.zeros(1 << 27, dtype=torch.int32).as_strided((3, 1 << 27), (0, 1))), UNSUPPORTED),
    "lengths_none": (dict(lengths=None), INVALID),
    "lengths_float": (dict(lengths=torch.zeros(3)), UNSUPPORTED),
    "scale_nan": (dict(scale=float("nan")), INVALID),
    "prefix_below": (dict(prefix_length=-1), INVALID),
    "prefix_without_pages": (dict(prefix_pages=None), INVALID),
    "prefix_too_long": (dict(prefix_length=33), INVALID),
    "prefix_far_too_long": (dict(prefix_length=1 << 40), UNSUPPORTED),
    "prefix_float": (dict(prefix_pages=torch.zeros(2)), UNSUPPORTED),
    "output_none": (dict(output=None), INVALID),
    "output_dtype": (dict(output=z(6, 4, 128, dtype=HF)), UNSUPPORTED),
    "output_heads": (dict(output=z(6, 3, 128)), INVALID),
    "output_expanded": (dict(output=z(6, 1, 128).expand(6, 4, 128)), INVALID),
    "output_rows_over_heads": (dict(output=z(9 * 128).as_strided((6, 4, 128), (128, 128, 1))), INVALID),
    "output_heads_over_rows": (dict(output=z(36 * 128).as_strided((6, 4, 128), (128, 3 * 128, 1))), INVALID),
    "lse_f16": (dict(lse=z(6, 4)), UNSUPPORTED),
    "lse_shape": (dict(lse=torch.zeros(4, 6)), INVALID),
    "lse_transposed": (dict(lse=torch.zeros(4, 6).t()), INVALID),
    "lse_expanded": (dict(lse=torch.zeros(1, 4).expand(6, 4)), INVALID),
    "output_is_q": (dict(q=_fused[:, :4], output=_fused[:, :4]), ALIAS),
    "output_in_cache": (dict(v_cache=z(5, 16, 2, 128), output=None), None),
}


@pytest.mark.parametrize("case", ATTEND)
def test_attention_refuses(way, case):
    changed, want = ATTEND[case]
    if want is None:
        v = z(5, 16, 2, 128)
        changed, want = dict(v_cache=v, output=v.view(-1)[:6 * 512].view(6, 4, 128)), ALIAS
    assert status(gdn.gdn_paged_attention_step, attend_args(), **changed) == want
    assert gdn.load_library().gdn_last_error()


def _off(*shape, dtype=I32):
    """Zeros that begin two bytes behind where an element may begin."""
    n = torch.zeros(shape, dtype=dtype).numel()
    return torch.frombuffer(bytearray(8 * n + 32), dtype=dtype, count=n, offset=2).view(shape)


@pytest.mark.parametrize("fn,args,name,tensor", [
    (gdn.gdn_qk_norm_rope_axes, axes_args, "positions", _off(3, 6)), (gdn.gdn_norm_rope_append, append_args, "slots", _off(6)),
    (gdn.gdn_norm_rope_append, append_args, "positions", _off(6, dtype=torch.int64)),
    (gdn.gdn_paged_attention_step, attend_args, "page_table", _off(3, 2)), (gdn.gdn_paged_attention_step, attend_args, "lengths", _off(3)),
    (gdn.gdn_paged_attention_step, attend_args, "prefix_pages", _off(2)), (gdn.gdn_paged_attention_step, attend_args, "lse", _off(6, 4, dtype=torch.float32)),
], ids=["axes_positions", "slots", "positions", "page_table", "lengths", "prefix_pages", "lse"])
def test_elements_off_their_places_are_refused(way, fn, args, name, tensor):
    assert tensor.data_ptr() % 4 == 2
    assert status(fn, args(), **{name: tensor}) == INVALID
    assert b"aligned" in gdn.load_library().gdn_last_error()


@pytest.mark.parametrize("fn,args", [(gdn.gdn_qk_norm_rope_axes, axes_args), (gdn.gdn_norm_rope_append, append_args),
                                     (gdn.gdn_paged_attention_step, attend_args)], ids=["axes", "append", "attention"])
def test_valid_arguments_reach_the_device_check(way, fn, args):
    if torch.cuda.is_available():
        pytest.skip("the arguments are host tensors: only for a machine without a GPU")
    assert status(fn, args()) not in (0, INVALID, ALIAS)


def test_workspace_bytes():
    need = gdn.gdn_paged_attention_workspace_bytes
    assert need(0, 1, 8, 2, 0, 152) == 0 and need(4, 1, 8, 0, 0, 152) == 0 and need(4, 1, 8, 2, 0, 0) == 0
    assert need(1, 1, 8, 2, 0, 152) <= need(1, 1, 8, 2, 100000, 152) <= need(64, 1, 8, 2, 100000, 152)
