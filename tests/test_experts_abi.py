"""Host-side checks, without a GPU, of the experts' products: exports, struct layouts, size queries, the refusal of every bad
argument before any CUDA call (the pointers here are never dereferenced), and what the binding refuses by itself."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import experts_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_experts.h")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mfr():
    sys.path.insert(0, ROOT)
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_finalize_residual_gb300 as m
    return m


def _structs(x):
    return {"mfr_expert_matmul_args": (x._CExpertMatmul, x._pack_matmul),
            "mfr_expert_matmul_backward_args": (x._CExpertMatmulBackward, x._pack_matmul_backward),
            "mfr_swiglu_backward_args": (x._CSwigluBackward, x._pack_swiglu), "mfr_nvfp4_args": (x._CNvfp4, x._pack_nvfp4),
            "mfr_expert_matmul_nvfp4_args": (x._CExpertMatmulNvfp4, x._pack_matmul_nvfp4)}


def test_every_declared_symbol_is_exported_and_bound(mfr):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert len(names) == 9, names
    lib = ctypes.CDLL(mfr.library_path())
    for n in names:
        assert hasattr(lib, n), n
    assert set(mfr.experts.__all__) <= set(mfr.__all__) and all(hasattr(mfr, n) for n in mfr.experts.__all__)


def test_struct_layout_matches_header(tmp_path, mfr):
    structs = {k: v[0] for k, v in _structs(mfr.experts).items()}
    lines = [f'printf("{c} %zu\\n", sizeof({c}));' for c in structs]
    lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for c, s in structs.items() for f, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_experts.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    c = dict(line.rsplit(" ", 1) for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, s in structs.items():
        assert int(c[name]) == ctypes.sizeof(s), name
        for f, _ in s._fields_:
            assert int(c[f"{name}.{f}"]) == getattr(s, f).offset, (name, f)


def test_packed_arguments_lie_in_their_fields(mfr):
    for cls, pack in _structs(mfr.experts).values():
        values = list(range(1, len(cls._fields_) + 1))
        s = cls.from_buffer_copy(pack(*values))
        assert [getattr(s, n) for n, _ in cls._fields_] == values


def _args(mfr, call):
    """A valid argument block of a call, with fake pointers."""
    X = mfr.experts
    p = lambda i: 0x10000 * i  # noqa: E731
    if call == "moe_expert_matmul":
        return X._CExpertMatmul(E=8, n_in=64, n_out=128, act_dtype=0, gated=1, num_rows=1000, rows=p(1), rows_stride=72, weight=p(2),
                                weight_stride=64, weight_expert_stride=256 * 64, expert_offsets=p(3), expert_counts=p(4), out=p(5),
                                out_stride=128, gate_up=p(6), gate_up_stride=256, flags=5)
    if call == "moe_expert_matmul_backward":
        return X._CExpertMatmulBackward(E=8, n_in=64, n_out=128, act_dtype=0, d_weight_dtype=2, accumulate=1, num_rows=1000, rows=p(1),
                                        rows_stride=64, weight=p(2), weight_stride=64, weight_expert_stride=128 * 64, d_out=p(3),
                                        d_out_stride=128, expert_offsets=p(4), expert_counts=p(5), d_rows=p(6), d_rows_stride=64,
                                        d_weight=p(7), flags=5)
    if call == "moe_swiglu_backward":
        return X._CSwigluBackward(num_rows=1000, F=128, act_dtype=1, gate_up=p(1), gate_up_stride=256, d_out=p(2), d_out_stride=128,
                                  row_route=p(3), d_gate_up=p(4), d_gate_up_stride=256, out=p(5), out_stride=128, flags=1)
    if call == "moe_expert_matmul_nvfp4":
        return X._CExpertMatmulNvfp4(E=8, n_in=128, n_out=128, out_dtype=0, gated=1, num_rows=1000, codes=p(1), sf=p(2), weight_codes=p(3),
                                     weight_sf=p(4), alpha=p(5), expert_offsets=p(6), expert_counts=p(7), out=p(8), out_stride=128, workspace=p(9), workspace_bytes=1 << 24, flags=5)
    return X._CNvfp4(matrices=2, rows=100, H=64, act_dtype=0, sf_layout=1, x=p(1), x_stride=64, scale=p(2), row_route=p(3), codes=p(4),
                     sf=p(5), flags=1)


COMMON = [dict(E=0), dict(E=1025), dict(num_rows=-1), dict(num_rows=1 << 31), dict(expert_offsets=None), dict(expert_offsets=0x30002),
          dict(expert_counts=0x30001), dict(n_in=0), dict(n_in=1 << 17), dict(n_out=0), dict(n_out=4), dict(n_out=1 << 17), dict(flags=2),
          dict(flags=8)]
NVFP4 = [dict(matrices=0), dict(rows=-1), dict(rows=1 << 31), dict(matrices=1 << 25, rows=1 << 10), dict(matrices=1 << 25, rows=1), dict(H=0),
         dict(H=24), dict(H=1 << 17), dict(act_dtype=2), dict(sf_layout=2), dict(x=None), dict(x=0x10008), dict(x_stride=56), dict(x_stride=68),
         dict(scale=None), dict(scale=0x20002), dict(row_route=0x30002), dict(codes=None), dict(codes=0x40004), dict(sf=None),
         dict(sf=0x50008), dict(flags=4)]
BAD = {
    "moe_expert_matmul": COMMON + [
        dict(n_in=60), dict(act_dtype=2), dict(gated=2), dict(gated=0), dict(rows=None), dict(rows=0x10008), dict(rows_stride=56),
        dict(rows_stride=68), dict(rows_stride=1 << 32), dict(weight=None), dict(weight=0x20004), dict(weight_stride=56), dict(weight_stride=66),
        dict(weight_expert_stride=255 * 64), dict(weight_expert_stride=256 * 64 + 4), dict(weight_expert_stride=1 << 39), dict(out=None),
        dict(out=0x50008), dict(out_stride=120), dict(out_stride=132), dict(gate_up=0x60008), dict(gate_up_stride=248),
        dict(num_rows=(1 << 31) - 1, n_out=65536, out_stride=65536, gate_up=None, weight_expert_stride=1 << 24)],
    "moe_expert_matmul_backward": COMMON + [
        dict(n_in=60), dict(act_dtype=2), dict(d_weight_dtype=1), dict(accumulate=2), dict(d_weight_dtype=0), dict(d_rows=None, d_weight=None),
        dict(rows=None), dict(rows_stride=60), dict(weight=None), dict(weight_stride=60), dict(weight_expert_stride=64), dict(d_out=None),
        dict(d_out=0x30008), dict(d_out_stride=120), dict(d_rows=0x60004), dict(d_rows_stride=56), dict(d_weight=0x70008)],
    "moe_swiglu_backward": [
        dict(num_rows=-1), dict(num_rows=1 << 31), dict(F=0), dict(F=12), dict(F=1 << 17), dict(act_dtype=2), dict(gate_up=None),
        dict(gate_up=0x10008), dict(gate_up_stride=248), dict(d_out=None), dict(d_out_stride=100), dict(row_route=0x30002),
        dict(d_gate_up=0x40008), dict(d_gate_up_stride=128), dict(out=0x50002), dict(out_stride=120), dict(d_gate_up=None, out=None), dict(flags=4)],
    "moe_expert_matmul_nvfp4": COMMON + [
        dict(n_in=96), dict(n_out=64), dict(out_dtype=2), dict(gated=-1), dict(codes=None), dict(codes=0x10008), dict(sf=None), dict(sf=0x20002),
        dict(weight_codes=None), dict(weight_codes=0x30008), dict(weight_sf=None), dict(weight_sf=0x40008), dict(alpha=0x50002), dict(out=None),
        dict(out=0x80008), dict(out_stride=120), dict(workspace=None), dict(workspace=0x90008), dict(workspace_bytes=1000)],
    "moe_nvfp4_quantize": NVFP4,
    "moe_nvfp4_dequantize": NVFP4,
}


@pytest.mark.parametrize("call,over", [(c, o) for c, v in BAD.items() for o in v],
                         ids=lambda v: v if isinstance(v, str) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_bad_arguments_are_refused(mfr, call, over):
    a = _args(mfr, call)
    for k, v in over.items():
        setattr(a, k, v)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) in (-1, -2)
    assert mfr.raw_library().moe_finalize_last_error().decode() != ""


@pytest.mark.parametrize("call", list(BAD))
def test_null_arguments_are_refused(mfr, call):
    assert getattr(mfr.raw_library(), call)(None, None) == -1


@no_gpu
@pytest.mark.parametrize("call", list(BAD))
def test_valid_call_without_gpu_reports_cuda_error(mfr, call):
    a = _args(mfr, call)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) == -3


@pytest.mark.parametrize("call,over", [
    ("moe_expert_matmul", dict(num_rows=0, rows=None, out=None)), ("moe_expert_matmul_nvfp4", dict(num_rows=0, codes=None, sf=None)),
    ("moe_expert_matmul_backward", dict(num_rows=0, rows=None, d_out=None)), ("moe_swiglu_backward", dict(num_rows=0, gate_up=None)),
    ("moe_nvfp4_quantize", dict(rows=0, x=None, codes=None)), ("moe_nvfp4_dequantize", dict(rows=0, x=None, sf=None))])
def test_empty_batch_is_a_no_op(mfr, call, over):
    a = _args(mfr, call)  # (the weights' gradient adds nothing: accumulate)
    for k, v in over.items():
        setattr(a, k, v)
    assert getattr(mfr.raw_library(), call)(ctypes.byref(a), None) == 0


def test_scale_bytes(mfr):
    assert mfr.nvfp4_sf_bytes(3, 64) == 12 and mfr.nvfp4_sf_bytes(3, 80, "swizzled_128x4") == 128 * 8
    assert mfr.nvfp4_sf_bytes(129, 64, "swizzled_128x4", 5) == 5 * 256 * 4 and mfr.nvfp4_sf_bytes(0, 16) == 0
    for args in ((-1, 64), (1, 8), (1, 64, "row_major", 0)):
        with pytest.raises(mfr.MoEFinalizeError):
            mfr.nvfp4_sf_bytes(*args)
    for args in ((1, 64, "tiles"), (1 << 64, 64), (1, 1 << 40)):
        with pytest.raises(ValueError):
            mfr.nvfp4_sf_bytes(*args)


def test_nvfp4_workspace_bytes(mfr):
    assert mfr.moe_expert_matmul_nvfp4_workspace_bytes(8, 128, 64) == 0
    assert mfr.moe_expert_matmul_nvfp4_workspace_bytes(8, 1000, 128) == (1000 // 192 + 8) * 2 * 2 * 512
    for args in ((0, 8, 64), (8, -1, 64), (8, 8, 96), (8, (1 << 31) - 1, 65536)):
        with pytest.raises(mfr.MoEFinalizeError):
            mfr.moe_expert_matmul_nvfp4_workspace_bytes(*args)
    with pytest.raises(ValueError):
        mfr.moe_expert_matmul_nvfp4_workspace_bytes(1 << 40, 8, 64)


def test_cpu_tensors_and_wrong_shapes_are_refused(mfr):
    x, w, o = torch.zeros(4, 64, dtype=BF), torch.zeros(2, 128, 64, dtype=BF), torch.zeros(3, dtype=torch.int32)
    d, s = torch.zeros(4, 128, dtype=BF), torch.ones(1)
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8)  # noqa: E731
    for call in (lambda: mfr.moe_expert_matmul(x, w, o), lambda: mfr.moe_expert_matmul(x[0], w, o), lambda: mfr.moe_expert_matmul(x, w[0], o),
                 lambda: mfr.moe_expert_matmul(None, w, o), lambda: mfr.moe_expert_matmul(x, None, o),
                 lambda: mfr.moe_expert_matmul(x, w[:, :127], o, gated=True), lambda: mfr.moe_expert_matmul_backward(d, x, w, o),
                 lambda: mfr.moe_expert_matmul_backward(d, None, None, o), lambda: mfr.moe_expert_matmul_backward(d, x, None, o),
                 lambda: mfr.moe_expert_matmul_backward(d, x, w, o, accumulate=True), lambda: mfr.moe_swiglu_backward(x, d),
                 lambda: mfr.moe_swiglu_backward(None, d), lambda: mfr.moe_swiglu_backward(x, d[:, :127]),
                 lambda: mfr.nvfp4_quantize(x, s), lambda: mfr.nvfp4_quantize(x[0], s), lambda: mfr.nvfp4_quantize(x, s, sf_layout="tiles"),
                 lambda: mfr.nvfp4_dequantize(u8(4, 32), u8(4, 4), s), lambda: mfr.nvfp4_dequantize(u8(4, 32), u8(4, 4), s, dtype=torch.float32),
                 lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 32), u8(4, 4), u8(2, 128, 32), u8(2, 512), o),
                 lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 32), None, u8(2, 128, 32), u8(2, 512), o)):
        with pytest.raises(ValueError):
            call()


def test_reference_against_closed_forms():
    """The 64-bit reference itself: known codes and scales, tiles, a gate."""
    codes, sf = ref.quantize(torch.tensor([[6.0, -3.0, 0.25, 0.75, 5.0, 2.5] + [0.0] * 9 + [-0.0]]), 1.0)
    assert sf.tolist() == [[1.0]] and codes[0, :6].tolist() == [7, 13, 0, 2, 6, 4] and codes[0, 15] == 8
    assert ref.values(torch.tensor([0x7f, 0x80], dtype=torch.uint8)).tolist() == [-6.0, 6.0, 0.0, -0.0]
    assert ref.e4m3(torch.tensor([500.0, 17.0, 19.0, 2.0 ** -10, 2.0 ** -9], dtype=torch.float64)).tolist() == [448, 16, 20, 0, 2.0 ** -9]
    assert ref.tile_at(130, 5)[129, 4] == (1 * 2 + 1) * 512 + 16 and ref.tile_at(130, 5)[33, 2] == 16 + 4 + 2
    y, _ = ref.gate(torch.tensor([0.0, 1.0, -800.0], dtype=torch.float64), torch.tensor([3.0, 2.0, 1.0], dtype=torch.float64))
    assert torch.allclose(y, torch.tensor([0.0, 2 / (1 + 2.718281828459045 ** -1), 0.0], dtype=torch.float64))
