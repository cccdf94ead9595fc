"""What the experts' products refuse before any CUDA call, beyond the list of test_experts_abi.py: no GPU, and the pointers are never
dereferenced."""
import ctypes
import os
import sys

import pytest
import torch

from test_experts_abi import _args

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
MOST_ROWS = (1 << 31) - 1024


@pytest.fixture(scope="module")
def mfr():
    sys.path.insert(0, ROOT)
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_finalize_residual_gb300 as m
    return m


def _narrow(mfr, call, rows):
    """A call of so many rows and few columns, valid but for their number."""
    a = _args(mfr, call)
    a.num_rows = rows
    a.n_in, a.n_out = (64, 8) if call.endswith("nvfp4") else (8, 8)
    if call != "moe_expert_matmul_backward":
        a.gated = 0
    if call == "moe_expert_matmul":
        a.gate_up = None
    if call.endswith("nvfp4"):
        a.workspace_bytes = 1 << 40
    return a


@no_gpu
@pytest.mark.parametrize("call", ["moe_expert_matmul", "moe_expert_matmul_backward", "moe_expert_matmul_nvfp4"])
def test_the_most_rows(mfr, call):
    """Row numbers are rounded up to whole tiles in 32 bits: more rows than leave room for that are refused."""
    f = getattr(mfr.raw_library(), call)
    assert f(ctypes.byref(_narrow(mfr, call, MOST_ROWS)), None) == -3  # (no device)
    for rows in (MOST_ROWS + 1, (1 << 31) - 256, (1 << 31) - 1):
        assert f(ctypes.byref(_narrow(mfr, call, rows)), None) == -1
        assert "num_rows" in mfr.raw_library().moe_finalize_last_error().decode()


def test_the_most_rows_of_a_workspace(mfr):
    assert mfr.moe_expert_matmul_nvfp4_workspace_bytes(8, MOST_ROWS, 64) == (MOST_ROWS // 192 + 8) * 2 * 512
    with pytest.raises(mfr.MoEFinalizeError):
        mfr.moe_expert_matmul_nvfp4_workspace_bytes(8, MOST_ROWS + 1, 64)


@pytest.mark.parametrize("no_tensor", [None, 3, [1.0]])
def test_what_is_no_tensor_is_refused(mfr, no_tensor):
    u8, s = torch.zeros(4, 32, dtype=torch.uint8), torch.ones(1)
    for call in (lambda: mfr.nvfp4_quantize(no_tensor, s), lambda: mfr.nvfp4_dequantize(no_tensor, u8, s)):
        with pytest.raises(ValueError):
            call()
