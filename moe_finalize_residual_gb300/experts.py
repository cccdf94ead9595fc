"""The experts' products, between the dispatch and the finalize: matrix products grouped by expert with their gradients,
the gate's gradient, and NVFP4 quantisation with the product of NVFP4 rows and weights.

A thin binding over ``include/moe_experts.h``, in the manner of ``layer``: it checks and marshals arguments, and every
step runs in the library's kernels.  Rows are in expert order, as ``moe_route`` and ``moe_dispatch`` leave them, with
``expert_offsets`` and ``expert_counts`` on the device.  Outputs that are not passed in are allocated.  Every call takes
``stream`` (default: the tensors' device's current stream), ``pdl`` (programmatic dependent launch) and ``check`` (False
skips the tensors' checks; the library's own stay).  Gradients are explicit calls.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Tuple

import torch

from .layer import DTYPE, _I, _L, _P, _PDL, _U, _ZERO_PADDING, _check_tensor, _choice, _enqueue, _good, _packer, _ptr

__all__ = [
    "moe_expert_matmul", "moe_expert_matmul_backward", "moe_swiglu_backward", "nvfp4_quantize", "nvfp4_dequantize",
    "nvfp4_sf_bytes", "moe_expert_matmul_nvfp4", "moe_expert_matmul_nvfp4_workspace_bytes",
    "moe_expert_read_timeouts",
]

_SF_LAYOUT = {"row_major": 0, "swizzled_128x4": 1}
_ACT = (torch.bfloat16, torch.float16)


class _CExpertMatmul(ctypes.Structure):
    _fields_ = [("E", _I), ("n_in", _I), ("n_out", _I), ("act_dtype", _I), ("gated", _I), ("num_rows", _L), ("rows", _P),
                ("rows_stride", _L), ("weight", _P), ("weight_stride", _L), ("weight_expert_stride", _L),
                ("expert_offsets", _P), ("expert_counts", _P), ("out", _P), ("out_stride", _L), ("gate_up", _P),
                ("gate_up_stride", _L), ("flags", _U)]


class _CExpertMatmulBackward(ctypes.Structure):
    _fields_ = [("E", _I), ("n_in", _I), ("n_out", _I), ("act_dtype", _I), ("d_weight_dtype", _I), ("accumulate", _I),
                ("num_rows", _L), ("rows", _P), ("rows_stride", _L), ("weight", _P), ("weight_stride", _L),
                ("weight_expert_stride", _L), ("d_out", _P), ("d_out_stride", _L), ("expert_offsets", _P),
                ("expert_counts", _P), ("d_rows", _P), ("d_rows_stride", _L), ("d_weight", _P), ("flags", _U)]


class _CSwigluBackward(ctypes.Structure):
    _fields_ = [("num_rows", _L), ("F", _I), ("act_dtype", _I), ("gate_up", _P), ("gate_up_stride", _L), ("d_out", _P),
                ("d_out_stride", _L), ("row_route", _P), ("d_gate_up", _P), ("d_gate_up_stride", _L), ("out", _P),
                ("out_stride", _L), ("flags", _U)]


class _CNvfp4(ctypes.Structure):
    _fields_ = [("matrices", _I), ("rows", _L), ("H", _I), ("act_dtype", _I), ("sf_layout", _I), ("x", _P), ("x_stride", _L),
                ("scale", _P), ("row_route", _P), ("codes", _P), ("sf", _P), ("flags", _U)]


class _CExpertMatmulNvfp4(ctypes.Structure):
    _fields_ = [("E", _I), ("n_in", _I), ("n_out", _I), ("out_dtype", _I), ("gated", _I), ("num_rows", _L), ("codes", _P),
                ("sf", _P), ("weight_codes", _P), ("weight_sf", _P), ("alpha", _P), ("expert_offsets", _P),
                ("expert_counts", _P), ("out", _P), ("out_stride", _L), ("workspace", _P), ("workspace_bytes", _L),
                ("flags", _U)]


_pack_matmul, _pack_matmul_backward, _pack_swiglu = map(_packer, (_CExpertMatmul, _CExpertMatmulBackward, _CSwigluBackward))
_pack_nvfp4, _pack_matmul_nvfp4 = _packer(_CNvfp4), _packer(_CExpertMatmulNvfp4)

_lib = None
_raise_status = None


def _bind(lib, raise_status):
    """Called once by the package: the loaded library and its status check."""
    global _lib, _raise_status
    _lib, _raise_status = lib, raise_status
    for name in ("moe_expert_matmul", "moe_expert_matmul_backward", "moe_swiglu_backward", "moe_nvfp4_quantize",
                 "moe_nvfp4_dequantize", "moe_expert_matmul_nvfp4"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [_P, _P], ctypes.c_int
    lib.moe_expert_read_timeouts.argtypes, lib.moe_expert_read_timeouts.restype = [ctypes.POINTER(_U)], ctypes.c_int
    f = lib.moe_expert_matmul_nvfp4_workspace_bytes
    f.argtypes, f.restype = [_I, _L, _I], _L
    lib.moe_nvfp4_sf_bytes.argtypes, lib.moe_nvfp4_sf_bytes.restype = [_I, _L, _I, _I], _L


def _row_tensor(name, t, index, shape, act, check):
    """Pointer and row stride of a tensor [rows, n] whose rows may be apart."""
    try:
        s = t.stride()
    except AttributeError:
        raise ValueError(f"{name} must be a tensor") from None
    if check and not (t.dtype is act and t.get_device() == index and t.shape == shape and (s[1] == 1 or shape[1] == 1)):
        _check_tensor(name, t, torch.device("cuda", index), shape, act, contiguous=False)
        raise ValueError(f"the values of a row must be contiguous in {name}")
    return t.data_ptr(), s[0] if shape[0] > 1 else shape[1]


def _weight(t, index, act, check):
    """Sizes, pointer and strides of the experts' weights [E, n, n_in]."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError("weight must be [E, n, n_in]")
    E, n, n_in = t.shape
    try:
        s = t.stride()
    except AttributeError:
        raise ValueError(f"{name} must be a tensor") from None
    if check and not (t.dtype is act and t.get_device() == index and s[2] == 1):
        _check_tensor("weight", t, torch.device("cuda", index), None, act, contiguous=False)
        raise ValueError("the values of a row must be contiguous in weight")
    row = s[1] if n > 1 else n_in
    return E, n, n_in, (t.data_ptr(), row, s[0] if E > 1 else n * row)


def _act_tensor(name, t, index, shape):
    """A tensor of either 16-bit type, its rows apart or not."""
    if not (isinstance(t, torch.Tensor) and t.dtype in _ACT and t.get_device() == index and t.shape == shape):
        _check_tensor(name, t, torch.device("cuda", index), shape, _ACT, contiguous=False)


def _first(name, t, check):
    """Device index and type of the call's first tensor, which the others follow."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor [rows, n]")
    index = t.get_device()
    if check and (index < 0 or t.dtype not in _ACT):
        _check_tensor(name, t, t.device, None, _ACT, contiguous=False)
    return index, t.dtype


def _check_order(expert_offsets, expert_counts, index, E):
    if not _good(expert_offsets, index, (E + 1,), torch.int32):
        _check_tensor("expert_offsets", expert_offsets, torch.device("cuda", index), (E + 1,), torch.int32)
    if expert_counts is not None and not _good(expert_counts, index, (E,), torch.int32):
        _check_tensor("expert_counts", expert_counts, torch.device("cuda", index), (E,), torch.int32)


def moe_expert_matmul(rows: torch.Tensor, weight: torch.Tensor, expert_offsets: torch.Tensor,
                      expert_counts: Optional[torch.Tensor] = None, *, gated: bool = False,
                      gate_up: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, pdl: bool = True,
                      stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> torch.Tensor:
    """Each row of ``rows`` ([R, n_in], bf16 or fp16, in expert order) times its expert's ``weight`` ([E, n_out, n_in]):
    ``out[r, n] = sum_i rows[r, i] * weight[e, n, i]``, summed in FP32 and rounded once.

    With ``gated`` the weights are [E, 2 * n_out, n_in], the gate's rows first: ``out = g / (1 + exp(-g)) * u`` of the
    unrounded halves g and u; ``gate_up`` ([R, 2 * n_out]) takes them, rounded, for ``moe_swiglu_backward``.

    Expert e has the ``expert_counts[e]`` rows from ``expert_offsets[e]`` on (without counts: up to the next expert's), as
    ``moe_route`` writes both.  Rows of no expert are not used, whatever they hold; their rows of ``out`` and ``gate_up``
    are left as they were (zeros in an allocated ``out``).  Sizes are multiples of 8; rows and weights may be strided, by
    multiples of 8 elements."""
    index, act = _first("rows", rows, check)
    E, n, n_in, w = _weight(weight, index, act, check)
    R = rows.shape[0]
    if gated and n % 2:
        raise ValueError("a gated weight has 2 * n_out rows an expert")
    n_out = n // 2 if gated else n
    flags = _PDL if pdl else 0
    allocated = []
    if out is None:
        out = torch.empty(R, n_out, dtype=act, device=rows.device)
        allocated.append(out)
        if gate_up is None:  # (a caller's gate_up is left as it was: zeros for the allocated tensor alone)
            flags |= _ZERO_PADDING
        else:
            out.zero_()
    if check:
        _check_order(expert_offsets, expert_counts, index, E)
    g = (0, 0) if gate_up is None else _row_tensor("gate_up", gate_up, index, (R, n), act, check)
    args = _pack_matmul(E, n_in, n_out, DTYPE[act], 1 if gated else 0, R, *_row_tensor("rows", rows, index, (R, n_in), act, check),
                        *w, expert_offsets.data_ptr(), _ptr(expert_counts), *_row_tensor("out", out, index, (R, n_out), act, check),
                        *g, flags)
    _enqueue(_lib.moe_expert_matmul, args, index, stream, allocated)
    return out


def moe_expert_matmul_backward(d_out: torch.Tensor, rows: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                               expert_offsets: torch.Tensor, expert_counts: Optional[torch.Tensor] = None, *,
                               d_rows: Optional[torch.Tensor] = None, d_weight: Optional[torch.Tensor] = None,
                               want_d_rows: bool = True, want_d_weight: bool = True,
                               d_weight_dtype: Optional[torch.dtype] = None, accumulate: bool = False, pdl: bool = True,
                               stream: Optional[torch.cuda.Stream] = None, check: bool = True
                               ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradients of ``moe_expert_matmul`` without the gate, given that of its output ([R, n_out]): ``(d_rows, d_weight)``,
    each left out with its ``want_*`` False (then ``weight``, or ``rows``, may be None).  The first product's gradient takes
    ``moe_swiglu_backward``'s ``d_gate_up`` as its ``d_out``.

    ``d_weight`` ([E, n_out, n_in]) has the rows' type or, with ``d_weight_dtype`` or a tensor of it passed in, FP32; experts of
    no rows get zeros.  ``accumulate`` adds to an FP32 ``d_weight`` that is passed in.  Rows of no expert are not used, and
    their rows of ``d_rows`` are left as they were (zeros in an allocated one)."""
    index, act = _first("d_out", d_out, check)
    R, n_out = d_out.shape
    flags = _PDL if pdl else 0
    want_d_rows, want_d_weight = want_d_rows or d_rows is not None, want_d_weight or d_weight is not None
    if accumulate and d_weight is None:
        raise ValueError("accumulate needs a d_weight to add to")
    if want_d_rows and weight is None or want_d_weight and rows is None or rows is None and weight is None:
        raise ValueError("d_rows needs weight, and d_weight needs rows")
    try:
        E = expert_offsets.shape[0] - 1
    except (AttributeError, IndexError):
        raise ValueError("expert_offsets must be a tensor [E + 1]") from None
    w, x = (0, 0, 0), (0, 0)
    if weight is not None:
        We, Wn, n_in, w = _weight(weight, index, act, check)
        if check and (We, Wn) != (E, n_out):
            raise ValueError(f"weight is {list(weight.shape)}; [{E}, {n_out}, n_in] is wanted")
    if rows is not None:
        if check and (not isinstance(rows, torch.Tensor) or rows.dim() != 2):
            raise ValueError("rows must be a tensor [rows, n]")
        if weight is None:
            n_in = rows.shape[1]
        x = _row_tensor("rows", rows, index, (R, n_in), act, check)
    allocated = []
    dx, dw, dw_type = (0, 0), 0, act
    if want_d_rows:
        if d_rows is None:
            d_rows = torch.empty(R, n_in, dtype=act, device=d_out.device)
            allocated.append(d_rows)
            flags |= _ZERO_PADDING
        dx = _row_tensor("d_rows", d_rows, index, (R, n_in), act, check)
    if want_d_weight:
        if d_weight is None:
            dw_type = act if d_weight_dtype is None else d_weight_dtype
            if dw_type is not act and dw_type is not torch.float32:
                raise ValueError(f"d_weight_dtype {dw_type} is neither {act} nor torch.float32")
            d_weight = torch.empty(E, n_out, n_in, dtype=dw_type, device=d_out.device)
            allocated.append(d_weight)
        else:
            dw_type = getattr(d_weight, "dtype", None)
            if check and (d_weight_dtype is not None and dw_type is not d_weight_dtype
                          or not _good(d_weight, index, (E, n_out, n_in), dw_type)
                          or dw_type is not act and dw_type is not torch.float32):
                _check_tensor("d_weight", d_weight, d_out.device, (E, n_out, n_in), (act, torch.float32) if d_weight_dtype is None else d_weight_dtype)
        dw = d_weight.data_ptr()
    if check:
        _check_order(expert_offsets, expert_counts, index, E)
    args = _pack_matmul_backward(E, n_in, n_out, DTYPE[act], DTYPE[dw_type], 1 if accumulate else 0, R, *x, *w,
                                 *_row_tensor("d_out", d_out, index, (R, n_out), act, check), expert_offsets.data_ptr(),
                                 _ptr(expert_counts), *dx, dw, flags)
    _enqueue(_lib.moe_expert_matmul_backward, args, index, stream, allocated)
    return (d_rows if want_d_rows else None), (d_weight if want_d_weight else None)


def moe_swiglu_backward(d_out: Optional[torch.Tensor], gate_up: torch.Tensor, *, row_route: Optional[torch.Tensor] = None,
                        d_gate_up: Optional[torch.Tensor] = None, act: Optional[torch.Tensor] = None,
                        want_d_gate_up: bool = True, want_act: bool = True, pdl: bool = True,
                        stream: Optional[torch.cuda.Stream] = None, check: bool = True
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradient of the gate ``act = g / (1 + exp(-g)) * u`` to its inputs, the halves g and u of ``gate_up`` ([R, 2F], as
    ``moe_expert_matmul`` kept them), given that of its output ([R, F]); and ``act`` itself again, which the gradient of the
    second product's weights reads.  Returns ``(d_gate_up, act)``, each left out with its ``want_*`` False (``d_out`` may then be
    None for ``act`` alone).  With ``row_route`` (as ``moe_route`` wrote it) rows of no route are not read and get zeros.
    ``d_gate_up`` may be ``gate_up`` and ``act`` may be ``d_out``."""
    index, dt = _first("gate_up", gate_up, check)
    R, wide = gate_up.shape
    if wide % 2:
        raise ValueError("gate_up must be [rows, 2 * F]")
    F = wide // 2
    want_d_gate_up, want_act = want_d_gate_up or d_gate_up is not None, want_act or act is not None
    allocated = []
    d, dg, y = (0, 0), (0, 0), (0, 0)
    if want_d_gate_up:
        if d_out is None:
            raise ValueError("d_gate_up needs d_out")
        d = _row_tensor("d_out", d_out, index, (R, F), dt, check)
        if d_gate_up is None:
            d_gate_up = torch.empty(R, wide, dtype=dt, device=gate_up.device)
            allocated.append(d_gate_up)
        dg = _row_tensor("d_gate_up", d_gate_up, index, (R, wide), dt, check)
    if want_act:
        if act is None:
            act = torch.empty(R, F, dtype=dt, device=gate_up.device)
            allocated.append(act)
        y = _row_tensor("act", act, index, (R, F), dt, check)
    if check and row_route is not None and not _good(row_route, index, (R,), torch.int32):
        _check_tensor("row_route", row_route, gate_up.device, (R,), torch.int32)
    args = _pack_swiglu(R, F, DTYPE[dt], *_row_tensor("gate_up", gate_up, index, (R, wide), dt, check), *d, _ptr(row_route), *dg, *y,
                        _PDL if pdl else 0)
    _enqueue(_lib.moe_swiglu_backward, args, index, stream, allocated)
    return (d_gate_up if want_d_gate_up else None), (act if want_act else None)


# ----------------------------------------------------------------------------------------------------------------
# NVFP4
# ----------------------------------------------------------------------------------------------------------------

def nvfp4_sf_bytes(rows: int, H: int, sf_layout: str = "row_major", matrices: int = 1) -> int:
    """Bytes of the block scales of ``matrices`` matrices of ``rows`` rows of H values each."""
    layout = _choice(_SF_LAYOUT, "sf_layout", sf_layout)
    try:
        struct.pack("<iqi", matrices, rows, H)
    except struct.error as e:
        raise ValueError(f"a size is not an integer of its range: {e}") from None
    n = _lib.moe_nvfp4_sf_bytes(matrices, rows, H, layout)
    if n < 0:
        _raise_status(int(n))
    return int(n)


def _matrices(shape):
    """(matrices, rows, values) of [rows, n] or [matrices, rows, n]."""
    if len(shape) not in (2, 3):
        raise ValueError("a tensor [rows, n] or [matrices, rows, n] is wanted")
    return (1, *shape) if len(shape) == 2 else tuple(shape)


def _sf_shape(matrices, rows, H, layout, dims):
    """The shape of allocated scales: row-major ones follow the values, tiles are flat (for each matrix)."""
    if layout == 0:
        return (rows, H // 16) if dims == 2 else (matrices, rows, H // 16)
    tiles = -(-rows // 128) * 128 * -(-H // 64) * 4
    return (tiles,) if dims == 2 else (matrices, tiles)


def _check_nvfp4(codes, sf, scale, row_route, index, lead, rows, H, layout, matrices):
    dev = torch.device("cuda", index)
    if not _good(codes, index, (*lead, H // 2), torch.uint8):
        _check_tensor("codes", codes, dev, (*lead, H // 2), torch.uint8)
    if not _good(sf, index, None, sf.dtype if isinstance(sf, torch.Tensor) else None) or sf.dtype not in (torch.uint8, torch.float8_e4m3fn):
        _check_tensor("sf", sf, dev, None, (torch.uint8, torch.float8_e4m3fn))
    if H % 16 == 0 and sf.numel() != matrices * (rows * (H // 16) if layout == 0 else -(-rows // 128) * 128 * -(-H // 64) * 4):
        raise ValueError(f"sf holds {sf.numel()} scales; nvfp4_sf_bytes says how many are wanted")
    if scale is not None and not (_good(scale, index, None, torch.float32) and scale.numel() == 1):
        _check_tensor("scale", scale, dev, None, torch.float32)
        raise ValueError("scale must hold one value")
    if row_route is not None and not _good(row_route, index, lead, torch.int32):
        _check_tensor("row_route", row_route, dev, lead, torch.int32)


def _x(name, x, index, matrices, rows, H, check):
    """Pointer and row stride of [rows, H] (rows may be apart) or [matrices, rows, H] (without gaps)."""
    if x.dim() == 3:
        if check and not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return x.data_ptr(), H
    return _row_tensor(name, x, index, (rows, H), x.dtype, check)


def nvfp4_quantize(x: torch.Tensor, scale: torch.Tensor, *, sf_layout: str = "row_major",
                   row_route: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                   sf: Optional[torch.Tensor] = None, pdl: bool = True, stream: Optional[torch.cuda.Stream] = None,
                   check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """NVFP4 codes and block scales of ``x`` ([rows, H], or weights [E, n, H]; bf16 or fp16), as the finalize's NVFP4 output has
    them: blocks of 16 values, ``sf = e4m3(max|x| / 6 * scale)``, ``code = e2m1(x * (scale / sf))``, ``scale`` one FP32 value on
    the device.  A block with a NaN gets the scale NaN.

    Returns ``codes`` (uint8, two a byte, the even one in the low half) and ``sf`` (uint8): row-major beside the values, or with
    "swizzled_128x4" tiles of 128 rows x 4 blocks, for each matrix, with zeros behind its last row and block.
    ``moe_expert_matmul_nvfp4`` reads rows of the first kind and weights of the second.  With ``row_route`` rows of no route are
    not read and get zeros."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a tensor")
    matrices, rows, H = _matrices(x.shape)
    index, layout = x.get_device(), _choice(_SF_LAYOUT, "sf_layout", sf_layout)
    lead = tuple(x.shape[:-1])
    if check and (index < 0 or x.dtype not in _ACT):
        _check_tensor("x", x, x.device, None, _ACT, contiguous=False)
    allocated = []
    if codes is None:
        codes = torch.empty(*lead, H // 2, dtype=torch.uint8, device=x.device)
        allocated.append(codes)
    if sf is None:
        sf = torch.empty(_sf_shape(matrices, rows, H, layout, x.dim()), dtype=torch.uint8, device=x.device)
        allocated.append(sf)
    if check:
        if scale is None:
            raise ValueError("scale must be a tensor")
        _check_nvfp4(codes, sf, scale, row_route, index, lead, rows, H, layout, matrices)
    args = _pack_nvfp4(matrices, rows, H, DTYPE[x.dtype], layout, *_x("x", x, index, matrices, rows, H, check), scale.data_ptr(),
                       _ptr(row_route), codes.data_ptr(), sf.data_ptr(), _PDL if pdl else 0)
    _enqueue(_lib.moe_nvfp4_quantize, args, index, stream, allocated)
    return codes, sf


def nvfp4_dequantize(codes: torch.Tensor, sf: torch.Tensor, scale: torch.Tensor, *, sf_layout: str = "row_major",
                     row_route: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None, pdl: bool = True, stream: Optional[torch.cuda.Stream] = None,
                     check: bool = True) -> torch.Tensor:
    """The values that ``nvfp4_quantize``'s (or the finalize's) codes and scales stand for: ``code * (sf / scale)``, rounded to
    ``dtype`` (bf16 or fp16).  With ``row_route`` rows of no route are not read and get zeros."""
    if not isinstance(codes, torch.Tensor):
        raise ValueError("codes must be a tensor")
    matrices, rows, half = _matrices(codes.shape)
    H = 2 * half
    index, layout = codes.get_device(), _choice(_SF_LAYOUT, "sf_layout", sf_layout)
    lead = tuple(codes.shape[:-1])
    allocated = []
    if out is None:
        if dtype not in _ACT:
            raise ValueError(f"dtype {dtype} is not supported (bf16 or fp16)")
        out = torch.empty(*lead, H, dtype=dtype, device=codes.device)
        allocated.append(out)
    if check:
        if scale is None:
            raise ValueError("scale must be a tensor")
        if index < 0:
            _check_tensor("codes", codes, codes.device, None, torch.uint8)
        _check_nvfp4(codes, sf, scale, row_route, index, lead, rows, H, layout, matrices)
        _act_tensor("out", out, index, (*lead, H))
    args = _pack_nvfp4(matrices, rows, H, DTYPE[out.dtype], layout, *_x("out", out, index, matrices, rows, H, check), scale.data_ptr(),
                       _ptr(row_route), codes.data_ptr(), sf.data_ptr(), _PDL if pdl else 0)
    _enqueue(_lib.moe_nvfp4_dequantize, args, index, stream, allocated)
    return out


def moe_expert_matmul_nvfp4_workspace_bytes(E: int, rows: int, n_in: int) -> int:
    """Workspace of ``moe_expert_matmul_nvfp4`` (0 for few rows an expert)."""
    try:
        struct.pack("<iqi", E, rows, n_in)
    except struct.error as e:
        raise ValueError(f"a size is not an integer of its range: {e}") from None
    n = _lib.moe_expert_matmul_nvfp4_workspace_bytes(E, rows, n_in)
    if n < 0:
        _raise_status(int(n))
    return int(n)


_nvfp4_space = functools.lru_cache(maxsize=1024)(lambda E, rows, n_in: moe_expert_matmul_nvfp4_workspace_bytes(E, rows, n_in))


def moe_expert_matmul_nvfp4(codes: torch.Tensor, sf: torch.Tensor, weight_codes: torch.Tensor, weight_sf: torch.Tensor,
                            expert_offsets: torch.Tensor, expert_counts: Optional[torch.Tensor] = None, *,
                            alpha: Optional[torch.Tensor] = None, gated: bool = False, dtype: torch.dtype = torch.bfloat16,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, pdl: bool = True,
                            stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> torch.Tensor:
    """``moe_expert_matmul`` over NVFP4: rows ``codes`` ([R, n_in / 2] uint8) with row-major scales ``sf`` ([R, n_in / 16]) and
    weights ``weight_codes`` ([E, n, n_in / 2]) with their scales in tiles ``weight_sf``, all as ``nvfp4_quantize`` writes them
    (``moe_dispatch`` moves codes and row-major scales into expert order).  ``y = alpha[e] * sum (code * sf) * (code * sf)``, summed
    in FP32, before the gate and the one rounding to ``dtype`` (bf16 or fp16); ``alpha`` ([E] fp32, default ones) undoes the two
    global scales: 1 / (rows' scale * weights' scale).  n_in is a multiple of 64 and, with ``gated``, n_out one of 128.
    ``workspace`` (uint8, ``moe_expert_matmul_nvfp4_workspace_bytes``) must not be shared by calls that may run at the same time."""
    if not all(isinstance(t, torch.Tensor) for t in (codes, sf, weight_codes, weight_sf)) or codes.dim() != 2 or weight_codes.dim() != 3:
        raise ValueError("codes must be [rows, n_in / 2] and weight_codes [E, n, n_in / 2], with their scales")
    index = codes.get_device()
    R, half = codes.shape
    E, n, _ = weight_codes.shape
    if gated and n % 2:
        raise ValueError("a gated weight has 2 * n_out rows an expert")
    n_in, n_out = 2 * half, n // 2 if gated else n
    flags = _PDL if pdl else 0
    allocated = []
    if out is None:
        if dtype not in _ACT:
            raise ValueError(f"dtype {dtype} is not supported (bf16 or fp16)")
        out = torch.empty(R, n_out, dtype=dtype, device=codes.device)
        allocated.append(out)
        flags |= _ZERO_PADDING
    if check:
        if index < 0:
            _check_tensor("codes", codes, codes.device, None, torch.uint8)
        _check_nvfp4(codes, sf, None, None, index, (R,), R, n_in, 0, 1)
        _check_nvfp4(weight_codes, weight_sf, None, None, index, (E, n), n, n_in, 1, E)
        _check_order(expert_offsets, expert_counts, index, E)
        if alpha is not None and not _good(alpha, index, (E,), torch.float32):
            _check_tensor("alpha", alpha, codes.device, (E,), torch.float32)
        _act_tensor("out", out, index, (R, n_out))
    if workspace is not None:
        if check:
            _check_tensor("workspace", workspace, codes.device, None, torch.uint8)
        space = workspace.numel()
    else:
        space = _nvfp4_space(E, R, n_in)
        if space:
            workspace = torch.empty(space, dtype=torch.uint8, device=codes.device)
            allocated.append(workspace)
    args = _pack_matmul_nvfp4(E, n_in, n_out, DTYPE[out.dtype], 1 if gated else 0, R, codes.data_ptr(), sf.data_ptr(),
                              weight_codes.data_ptr(), weight_sf.data_ptr(), _ptr(alpha), expert_offsets.data_ptr(),
                              _ptr(expert_counts), *_row_tensor("out", out, index, (R, n_out), out.dtype, check),
                              _ptr(workspace) if space else 0, space, flags)
    _enqueue(_lib.moe_expert_matmul_nvfp4, args, index, stream, allocated)
    return out


def moe_expert_read_timeouts() -> int:
    """Waits of the products' kernels that ran out since the last call, on the current device and any of its streams (0 unless
    something is broken).  Synchronizes the device."""
    n = _U(0)
    status = _lib.moe_expert_read_timeouts(ctypes.byref(n))
    if status != 0:
        _raise_status(status)
    return int(n.value)
