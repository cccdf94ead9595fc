"""Host-side checks, without a GPU, of the operators around the finalize: exports, struct layouts, size queries, and
the refusal of every bad argument before any CUDA call (the pointers here are never dereferenced)."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import layer_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer.h")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")


@pytest.fixture(scope="module")
def mfr():
    sys.path.insert(0, ROOT)
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_finalize_residual_gb300 as m
    return m


def _structs(layer):
    return {"mfr_route_args": layer._CRoute, "mfr_route_backward_args": layer._CRouteBackward,
            "mfr_dispatch_args": layer._CDispatch, "mfr_routed_backward_args": layer._CRoutedBackward,
            "mfr_heads": layer._CHeads, "mfr_head_norm_args": layer._CHeadNorm}


def test_every_declared_symbol_is_exported(mfr):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert len(names) == 9, names
    lib = ctypes.CDLL(mfr.library_path())
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path, mfr):
    structs = _structs(mfr.layer)
    lines = [f'printf("{c} %zu\\n", sizeof({c}));' for c in structs]
    lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for c, s in structs.items() for f, _ in s._fields_]
    lines += [f'printf("{n} %d\\n", {n});' for n in ("MFR_FLAG_ZERO_PADDING", "MFR_FLAG_POSITIONS_64", "MFR_FLAG_PDL")]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_layer.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    c = dict(line.rsplit(" ", 1) for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, s in structs.items():
        assert int(c[name]) == ctypes.sizeof(s), name
        for f, _ in s._fields_:
            assert int(c[f"{name}.{f}"]) == getattr(s, f).offset, (name, f)
    assert [int(c[n]) for n in ("MFR_FLAG_ZERO_PADDING", "MFR_FLAG_POSITIONS_64", "MFR_FLAG_PDL")] == \
        [mfr.layer._ZERO_PADDING, mfr.layer._POSITIONS_64, mfr.layer._PDL]


@pytest.mark.parametrize("T,K,E,align", [(1, 1, 1, 1), (3, 2, 8, 16), (100, 8, 256, 128), (16384, 8, 256, 128), (5, 64, 64, 7),
                                         (0, 4, 16, 128)])
def test_max_rows_holds_and_is_reached(mfr, T, K, E, align):
    rows = mfr.moe_route_max_rows(T, K, E, align)
    g = np.random.default_rng(T)
    for spread in (1, 2, E):
        ids = np.array([g.permutation(max(K, min(E, spread * K)))[:K] for _ in range(T)], dtype=np.int64).reshape(T, K)
        assert ref.order(ids, E, align, rows)[2][-1] <= rows
    # one more route than a multiple in as many experts as there are routes for reaches it
    n = T * K
    counts = np.zeros(E, dtype=np.int64)
    counts[:min(E, n)] = 1
    if n > E:
        counts[0] += (n - E) // align * align
        left = n - counts.sum()
        counts[0] += left
    assert (-(-counts // align) * align).sum() <= rows
    if (n - min(E, n)) % align == 0:
        assert (-(-counts // align) * align).sum() == rows


def test_size_queries_refuse_bad_sizes(mfr):
    for args in ((-1, 1, 1, 1), (1, 0, 8, 1), (1, 65, 100, 1), (1, 9, 8, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                 (1 << 28, 8, 8, 1), (1 << 20, 8, 1024, 1 << 22)):
        with pytest.raises(mfr.MoEFinalizeError):
            mfr.moe_route_max_rows(*args)
    with pytest.raises(mfr.MoEFinalizeError):
        mfr.moe_route_workspace_bytes(1, 9, 8)
    for args in ((-1, 1, 1, 64), (1, 1, 1, 24), (1, 1, 1, 528), (1, -1, 1, 64)):
        with pytest.raises(mfr.MoEFinalizeError):
            mfr.head_norm_rotary_workspace_bytes(*args)


def _args(mfr, call):
    """A valid argument block of a call, with fake pointers."""
    L = mfr.layer
    if call == "moe_route":
        a = L._CRoute(T=1000, E=64, K=8, logits_dtype=2, scale_dtype=2, score=0, num_groups=8, topk_groups=4,
                      group_score=1, renormalize=1, row_align=16, scale=1.0, logits=0x10000, logits_stride=64,
                      bias=0x20000, expert_ids=0x30000, expert_scale=0x40000, perm_idx=0x50000, row_route=0x60000,
                      num_rows=10000, expert_offsets=0x70000, expert_counts=0x80000, workspace=0x90000,
                      workspace_bytes=1 << 20, flags=1)
    elif call == "moe_route_backward":
        a = L._CRouteBackward(T=100, E=64, K=8, logits_dtype=0, scale_dtype=2, score=1, renormalize=0, scale=1.0,
                              logits=0x10000, logits_stride=64, expert_ids=0x30000, d_scale=0x40000, d_logits=0x50000,
                              d_logits_stride=80, flags=1)
    elif call == "moe_dispatch_rows":
        a = L._CDispatch(T=100, K=8, row_bytes=512, num_rows=1000, x=0x10000, perm_idx=0x20000, row_route=0x30000,
                         rows=0x40000, flags=1)
    elif call == "moe_routed_backward":
        a = L._CRoutedBackward(T=100, H=256, K=8, act_dtype=0, scale_dtype=2, routed_scaling_factor=1.0, num_rows=1000,
                               gemm2_out=0x10000, perm_idx=0x20000, expert_scale=0x30000, row_route=0x40000,
                               d_out=0x50000, d_gemm2=0x60000, d_scale=0x70000, flags=1)
    else:
        h = lambda p: L._CHeads(p, 1024, 128)  # noqa: E731
        a = L._CHeadNorm(T=10, q_heads=4, k_heads=2, D=128, rot=64, style=0, act_dtype=0, eps=1e-6, rotary_scale=1.0,
                         q=h(0x10000), k=h(0x20000), q_out=h(0x30000), k_out=h(0x40000), d_q_out=h(0x50000),
                         d_k_out=h(0x60000), q_weight=0x70000, k_weight=0x80000, positions=0x90000, inv_freq=0xA0000,
                         d_q_weight=0xB0000, d_k_weight=0xC0000, workspace=0xD0000, workspace_bytes=1 << 24, flags=1)
    return a


HEADS_BAD = [dict(T=-1), dict(q_heads=-1), dict(q_heads=0, k_heads=0), dict(q_heads=70000), dict(D=0), dict(D=24), dict(D=528),
             dict(rot=-2), dict(rot=130), dict(rot=24), dict(style=2), dict(style=1, rot=63), dict(act_dtype=2),
             dict(flags=2), dict(flags=16), dict(q_weight=0x70008), dict(positions=None), dict(positions=0x90002),
             dict(flags=9, positions=0x90004), dict(inv_freq=None), dict(inv_freq=0xA0002)]
BAD = {
    "moe_route": [
        dict(T=-1), dict(T=1 << 28), dict(E=0), dict(E=1025), dict(K=0), dict(K=65), dict(E=6, K=8, num_groups=1, topk_groups=1),
        dict(logits_dtype=3), dict(scale_dtype=-1), dict(score=2), dict(num_groups=0), dict(num_groups=64, topk_groups=1),
        dict(num_groups=7), dict(topk_groups=0), dict(topk_groups=9), dict(group_score=2), dict(renormalize=2),
        dict(row_align=0), dict(logits_stride=63), dict(logits_stride=1 << 40), dict(flags=2), dict(flags=4),
        dict(num_rows=800), dict(num_rows=1 << 31), dict(row_align=1 << 30), dict(row_route=None),
        dict(expert_counts=None), dict(perm_idx=None), dict(expert_offsets=None), dict(workspace=None),
        dict(workspace_bytes=100), dict(workspace=0x90008), dict(logits=None), dict(expert_ids=None),
        dict(expert_scale=None), dict(logits=0x10002), dict(bias=0x20002), dict(expert_ids=0x30001),
        dict(perm_idx=0x50002), dict(expert_scale=0x40002)],
    "moe_route_backward": [
        dict(T=-1), dict(E=0), dict(E=2000), dict(K=0), dict(K=65), dict(E=4), dict(logits_dtype=3), dict(scale_dtype=3),
        dict(score=-1), dict(renormalize=-1), dict(logits_stride=60), dict(d_logits_stride=0), dict(logits=None),
        dict(expert_ids=None), dict(d_scale=None), dict(d_logits=None), dict(logits=0x10001), dict(d_logits=0x50001),
        dict(d_scale=0x40002), dict(expert_ids=0x30002), dict(flags=8)],
    "moe_dispatch_rows": [
        dict(T=-1), dict(K=0), dict(K=65), dict(row_bytes=0), dict(row_bytes=24), dict(row_bytes=1 << 21),
        dict(num_rows=-1), dict(num_rows=1 << 31), dict(x=None), dict(perm_idx=None), dict(rows=None), dict(x=0x10008),
        dict(rows=0x40008), dict(perm_idx=0x20001), dict(row_route=0x30002), dict(flags=2)],
    "moe_routed_backward": [
        dict(T=-1), dict(K=0), dict(K=65), dict(H=0), dict(H=12), dict(H=65536), dict(act_dtype=2), dict(scale_dtype=3),
        dict(num_rows=-1), dict(num_rows=1 << 31), dict(d_gemm2=None, d_scale=None), dict(gemm2_out=None),
        dict(d_out=None), dict(perm_idx=None), dict(gemm2_out=0x10008), dict(d_out=0x50004), dict(d_gemm2=0x60008),
        dict(d_scale=0x70002), dict(expert_scale=0x30002), dict(perm_idx=0x20002), dict(flags=4)],
    "moe_head_norm_rotary": HEADS_BAD,
    "moe_head_norm_rotary_backward": HEADS_BAD + [
        dict(workspace=None), dict(workspace_bytes=1000), dict(workspace=0xD0004), dict(d_q_weight=0xB0002)],
}


@pytest.mark.parametrize("call,over", [(c, o) for c, v in BAD.items() for o in v],
                         ids=lambda v: v if isinstance(v, str) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_bad_arguments_are_refused(mfr, call, over):
    a = _args(mfr, call)
    for k, v in over.items():
        setattr(a, k, v)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) in (-1, -2)
    assert mfr.raw_library().moe_finalize_last_error().decode() != ""


@pytest.mark.parametrize("call", ["moe_head_norm_rotary", "moe_head_norm_rotary_backward"])
@pytest.mark.parametrize("name", ["q", "k", "q_out", "k_out", "d_q_out", "d_k_out"])
@pytest.mark.parametrize("data,ts,hs", [(None, 1024, 128), (0x10008, 1024, 128), (0x10000, 1020, 128), (0x10000, 1024, 132),
                                        (0x10000, 1 << 31, 128), (0x10000, 64, 128), (0x10000, 1024, 0)])
def test_bad_heads_are_refused(mfr, call, name, data, ts, hs):
    if not call.endswith("backward") and name.startswith("d_"):
        pytest.skip("read by the backward call only")
    a = _args(mfr, call)
    setattr(a, name, mfr.layer._CHeads(data, ts, hs))
    overlapping = data == 0x10000 and ts in (64, 1024) and hs in (0, 128)
    if overlapping and name not in ("q_out", "k_out"):
        pytest.skip("an input may repeat its heads")
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) == -1


@pytest.mark.parametrize("call", list(BAD))
def test_null_arguments_are_refused(mfr, call):
    assert getattr(mfr.raw_library(), call)(None, None) == -1


@no_gpu
@pytest.mark.parametrize("call", list(BAD))
def test_valid_call_without_gpu_reports_cuda_error(mfr, call):
    a = _args(mfr, call)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) == -3


@pytest.mark.parametrize("call,over", [
    ("moe_route", dict(T=0, perm_idx=None, row_route=None, expert_offsets=None, expert_counts=None)),
    ("moe_route_backward", dict(T=0, logits=None)), ("moe_dispatch_rows", dict(T=0, row_route=None)),
    ("moe_dispatch_rows", dict(num_rows=0, rows=None)), ("moe_routed_backward", dict(T=0, row_route=None)),
    ("moe_head_norm_rotary", dict(T=0)), ("moe_head_norm_rotary_backward", dict(T=0, d_q_weight=None, d_k_weight=None))])
def test_empty_batch_is_a_no_op(mfr, call, over):
    a = _args(mfr, call)
    for k, v in over.items():
        setattr(a, k, v)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) == 0


def test_cpu_tensors_and_bad_choices_are_refused(mfr):
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        mfr.moe_route(x, 2)
    with pytest.raises(ValueError):
        mfr.moe_route(x[0], 2)
    with pytest.raises(ValueError):
        mfr.moe_route_backward(torch.zeros(4, 2), x, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mfr.moe_dispatch(x, torch.zeros(4, 2, dtype=torch.int32), 8)
    p = mfr.Partial(x.bfloat16(), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mfr.moe_finalize_routed_backward(x.bfloat16(), p)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError):
        mfr.head_norm_rotary(q, q, None, None, pos, freq)
    with pytest.raises(ValueError):
        mfr.head_norm_rotary_backward(q, q, q, q, None, None, pos, freq)


def test_reference_against_closed_forms():
    """The 64-bit reference itself: uniform logits, one expert, a bias that decides, groups, a known turn."""
    ids, s = ref.choose(np.zeros((1, 4)), 2, "softmax")
    assert ids.tolist() == [[0, 1]] and np.allclose(s, 0.25)
    ids, s = ref.choose(np.zeros((1, 4)), 2, "sigmoid", bias=np.array([0.0, 0.1, 0.0, 0.2]))
    assert ids.tolist() == [[3, 1]] and np.allclose(s, 0.5)
    x = np.array([[5.0, -9.0, 3.0, 2.9]])
    assert ref.choose(x, 1, "softmax", G=2, Gk=1)[0].tolist() == [[0]]
    assert ref.choose(x, 2, "sigmoid", G=2, Gk=1, top2=True)[0].tolist() == [[2, 3]]
    assert ref.choose(np.array([[np.nan, -np.inf, 1.0]]), 2, "softmax")[0].tolist() == [[2, -1]]
    assert np.allclose(ref.weights(x, np.array([[0, 2]]), s, "softmax", True, 2.0), 2 / (1 + np.exp([[-2.0, 2.0]])))
    v = torch.tensor([[[1.0, 0.0, 0.0, 0.0] * 4]], dtype=torch.float64)
    y = ref.head_norm(v, None, [1], torch.tensor([np.pi / 2], dtype=torch.float64), "interleaved", 0.0, 1.0)
    assert np.allclose(y[0, 0, :4], [0, 2, 0, 0])
    assert abs(np.sin(ref._angle(10 ** 12, 1.0)) - np.sin(np.longdouble(10 ** 12))) < 1e-9
