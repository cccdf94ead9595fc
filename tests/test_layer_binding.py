"""What the Python binding of the operators around the finalize refuses by its own checks, without a GPU."""
import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mfr():
    sys.path.insert(0, ROOT)
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_finalize_residual_gb300 as m
    return m


def struct_of(mfr, pack):
    return {"_pack_route": mfr.layer._CRoute, "_pack_route_backward": mfr.layer._CRouteBackward,
            "_pack_dispatch": mfr.layer._CDispatch, "_pack_routed_backward": mfr.layer._CRoutedBackward,
            "_pack_head_norm": mfr.layer._CHeadNorm}[pack]


def field_types(c):
    for _, t in c._fields_:
        if hasattr(t, "_fields_"):
            yield from field_types(t)
        else:
            yield t


def field_values(s):
    for name, t in s._fields_:
        v = getattr(s, name)
        if hasattr(t, "_fields_"):
            yield from field_values(v)
        else:
            yield v


@pytest.mark.parametrize("pack", ["_pack_route", "_pack_route_backward", "_pack_dispatch", "_pack_routed_backward", "_pack_head_norm"])
def test_packed_arguments_lie_in_their_fields(mfr, pack):
    cls = struct_of(mfr, pack)
    values = [i + 1.5 if t is mfr.layer._F else i + 1 for i, t in enumerate(field_types(cls))]
    assert list(field_values(cls.from_buffer_copy(getattr(mfr.layer, pack)(*values)))) == values


@pytest.mark.parametrize("pack", ["_pack_route", "_pack_route_backward", "_pack_routed_backward", "_pack_head_norm"])
@pytest.mark.parametrize("bad", [1e39, -1e300, 10 ** 400, "1", None])
def test_numbers_beyond_their_type_are_refused(mfr, pack, bad):
    """scale, routed_scaling_factor, eps and rotary_scale are FP32 in the argument block."""
    types = list(field_types(struct_of(mfr, pack)))
    good = [1.0 if t is mfr.layer._F else 1 for t in types]
    getattr(mfr.layer, pack)(*good)
    for i, t in enumerate(types):
        if t is mfr.layer._F:
            with pytest.raises(ValueError):
                getattr(mfr.layer, pack)(*good[:i], bad, *good[i + 1:])


@pytest.mark.parametrize("query,good", [("moe_route_max_rows", (4, 2, 8, 16)), ("moe_route_workspace_bytes", (4000, 2, 8)),
                                        ("head_norm_rotary_workspace_bytes", (40, 4, 2, 64))])
def test_sizes_beyond_32_bits_are_refused(mfr, query, good):
    f = getattr(mfr, query)
    assert f(*good) > 0
    for i in range(len(good)):
        for bad in (good[i] + 2 ** 32, good[i] - 2 ** 32, 2 ** 31, 10 ** 30, 2.0, None):
            with pytest.raises(ValueError):
                f(*good[:i], bad, *good[i + 1:])


def test_empty_batch_with_a_bias_off_its_alignment_is_refused(mfr):
    """Without tokens the expert order is still written, by a kernel that reads the bias.  (The pointers are refused, not read.)"""
    a = mfr.layer._CRoute(T=0, E=64, K=8, logits_dtype=2, scale_dtype=2, score=0, num_groups=1, topk_groups=1, group_score=0,
                          renormalize=1, row_align=16, scale=1.0, logits_stride=64, bias=0x20002, perm_idx=0x50000,
                          row_route=0x60000, num_rows=1000, expert_offsets=0x70000, expert_counts=0x80000, flags=1)
    assert mfr.raw_library().moe_route(ctypes.byref(a), None) == -1
    assert "bias" in mfr.raw_library().moe_finalize_last_error().decode()
