"""The operators around the fused MoE finalize: expert routing, dispatch, the finalize's gradient, and the per-head
RMSNorm with position rotation of queries and keys.

A thin binding over ``include/moe_layer.h``, as the package's ``__init__`` is over ``moe_finalize.h``: it checks and
marshals arguments, and every step runs in the library's kernels.  Outputs that are not passed in are allocated.
Every call takes ``stream`` (default: the tensors' device's current stream), ``pdl`` (programmatic dependent launch)
and ``check`` (False skips the tensors' checks; the library's own stay).  Gradients are explicit calls.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import struct
import sys
from typing import Optional, Tuple

import torch

__all__ = [
    "Routing", "moe_route", "moe_route_max_rows", "moe_route_workspace_bytes", "moe_route_backward", "moe_dispatch",
    "moe_finalize_routed_backward", "head_norm_rotary", "head_norm_rotary_backward",
    "head_norm_rotary_workspace_bytes", "SCORE", "GROUP_SCORE", "ROTARY_STYLE",
]

_P, _I, _L, _F, _U = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_uint32

DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}
ROTARY_STYLE = {"half": 0, "interleaved": 1}
_PDL, _ZERO_PADDING, _POSITIONS_64 = 1, 4, 8


class _CRoute(ctypes.Structure):
    _fields_ = [("T", _I), ("E", _I), ("K", _I), ("logits_dtype", _I), ("scale_dtype", _I), ("score", _I),
                ("num_groups", _I), ("topk_groups", _I), ("group_score", _I), ("renormalize", _I), ("row_align", _I),
                ("scale", _F), ("logits", _P), ("logits_stride", _L), ("bias", _P), ("expert_ids", _P),
                ("expert_scale", _P), ("perm_idx", _P), ("row_route", _P), ("num_rows", _L), ("expert_offsets", _P),
                ("expert_counts", _P), ("workspace", _P), ("workspace_bytes", _L), ("flags", _U)]


class _CRouteBackward(ctypes.Structure):
    _fields_ = [("T", _I), ("E", _I), ("K", _I), ("logits_dtype", _I), ("scale_dtype", _I), ("score", _I),
                ("renormalize", _I), ("scale", _F), ("logits", _P), ("logits_stride", _L), ("expert_ids", _P),
                ("d_scale", _P), ("d_logits", _P), ("d_logits_stride", _L), ("flags", _U)]


class _CDispatch(ctypes.Structure):
    _fields_ = [("T", _I), ("K", _I), ("row_bytes", _L), ("num_rows", _L), ("x", _P), ("perm_idx", _P),
                ("row_route", _P), ("rows", _P), ("flags", _U)]


class _CRoutedBackward(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("K", _I), ("act_dtype", _I), ("scale_dtype", _I),
                ("routed_scaling_factor", _F), ("num_rows", _L), ("gemm2_out", _P), ("perm_idx", _P),
                ("expert_scale", _P), ("row_route", _P), ("d_out", _P), ("d_gemm2", _P), ("d_scale", _P),
                ("flags", _U)]


class _CHeads(ctypes.Structure):
    _fields_ = [("data", _P), ("token_stride", _L), ("head_stride", _L)]


class _CHeadNorm(ctypes.Structure):
    _fields_ = [("T", _I), ("q_heads", _I), ("k_heads", _I), ("D", _I), ("rot", _I), ("style", _I), ("act_dtype", _I),
                ("eps", _F), ("rotary_scale", _F), ("q", _CHeads), ("k", _CHeads), ("q_out", _CHeads),
                ("k_out", _CHeads), ("d_q_out", _CHeads), ("d_k_out", _CHeads), ("q_weight", _P), ("k_weight", _P),
                ("positions", _P), ("inv_freq", _P), ("d_q_weight", _P), ("d_k_weight", _P), ("workspace", _P),
                ("workspace_bytes", _L), ("flags", _U)]


_CODES = {_I: "i", _L: "q", _F: "f", _P: "Q", _U: "I"}


def _packer(cls):
    """Packs a structure's fields, nested ones in line: several times faster than filling a ctypes structure.  The format
    is the standard one, with the padding spelled out: the native one turns a float beyond FP32 into an infinity."""
    def fields(c, at):
        for name, t in c._fields_:
            offset = at + getattr(c, name).offset
            if issubclass(t, ctypes.Structure):
                yield from fields(t, offset)
            else:
                yield offset, t

    codes, end = "<", 0
    for offset, t in fields(cls, 0):
        codes += "x" * (offset - end) + _CODES[t]
        end = offset + ctypes.sizeof(t)
    packer = struct.Struct(codes + "x" * (ctypes.sizeof(cls) - end))
    assert packer.size == ctypes.sizeof(cls) and sys.byteorder == "little", cls

    def pack(*values):
        try:
            return packer.pack(*values)
        except (struct.error, OverflowError) as e:  # (OverflowError: a float beyond FP32)
            raise ValueError(f"an argument is not a number of its range: {e}") from None

    return pack


_pack_route, _pack_route_backward, _pack_dispatch = _packer(_CRoute), _packer(_CRouteBackward), _packer(_CDispatch)
_pack_routed_backward, _pack_head_norm = _packer(_CRoutedBackward), _packer(_CHeadNorm)

_lib = None
_raise_status = None
_current_device = torch.cuda.current_device
# the current stream's handle without a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _bind(lib, raise_status):
    """Called once by the package: the loaded library and its status check."""
    global _lib, _raise_status
    _lib, _raise_status = lib, raise_status
    for name in ("moe_route", "moe_route_backward", "moe_dispatch_rows", "moe_routed_backward",
                 "moe_head_norm_rotary", "moe_head_norm_rotary_backward"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [_P, _P], ctypes.c_int
    for name, n in (("moe_route_max_rows", 4), ("moe_route_workspace_bytes", 3),
                    ("moe_head_norm_rotary_workspace_bytes", 4)):
        f = getattr(lib, name)
        f.argtypes, f.restype = [_I] * n, _L


def _ptr(t):
    return 0 if t is None else t.data_ptr()


_INTS = {n: struct.Struct("<%di" % n).pack for n in (3, 4)}


def _size(query, *args) -> int:
    try:
        _INTS[len(args)](*args)  # (ctypes would keep the low 32 bits of a larger number)
    except struct.error as e:
        raise ValueError(f"a size is not a 32-bit integer: {e}") from None
    n = query(*args)
    if n < 0:
        _raise_status(int(n))
    return int(n)


def _choice(table, name, value):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} is {value!r}; one of {', '.join(table)} is wanted") from None


def _good(t, index, shape, dtype):
    """A contiguous tensor of this shape (None: any) and type (None: any of DTYPE) on this device."""
    try:
        return ((t.dtype is dtype or dtype is None and t.dtype in DTYPE) and t.get_device() == index
                and (shape is None or t.shape == shape) and t.is_contiguous())
    except AttributeError:  # None, or no tensor
        return False


def _check_tensor(name, t, device, shape, dtypes, contiguous=True):
    """``shape``: a tuple, or None.  ``dtypes``: a dtype or a container of them."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}; every tensor must be on {device} (a CUDA device)")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} is {list(t.shape)}; {list(shape)} is wanted")
    if t.dtype != dtypes if isinstance(dtypes, torch.dtype) else t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}; {dtypes if isinstance(dtypes, torch.dtype) else ', '.join(map(str, dtypes))} is wanted")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _enqueue(fn, args, index, stream, allocated):
    """Enqueue on ``stream`` with the tensors' device (``index``) current.  What the binding allocated on the current
    stream for use on another one is ordered behind the current stream's work, and recorded on the other, so that
    its memory is not given out again too early."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _enqueue(fn, args, index, stream, allocated)
    if stream is None:
        status = fn(args, _raw_stream(index))
    else:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}; the tensors are on cuda:{index}")
        current = torch.cuda.current_stream()
        if allocated and stream != current:
            stream.wait_stream(current)
            for t in allocated:
                t.record_stream(stream)
        status = fn(args, stream.cuda_stream)
    if status != 0:
        _raise_status(status)


# ----------------------------------------------------------------------------------------------------------------
# Routing
# ----------------------------------------------------------------------------------------------------------------

@dataclasses.dataclass
class Routing:
    """What ``moe_route`` writes.  ``perm_idx`` and ``expert_scale`` are those of a ``Partial``."""

    expert_ids: torch.Tensor                        # [T, K] int32, best first; -1 = no expert left to take
    expert_scale: torch.Tensor                      # [T, K] fp32/bf16/fp16 weights
    perm_idx: Optional[torch.Tensor] = None         # [T, K] int32: the row of route (t, k), or -1
    row_route: Optional[torch.Tensor] = None        # [rows] int32: the route t*K+k of a row, or -1
    expert_offsets: Optional[torch.Tensor] = None   # [E + 1] int32: where each expert's rows start
    expert_counts: Optional[torch.Tensor] = None    # [E] int32: routes of each expert


def moe_route_max_rows(T: int, K: int, E: int, row_align: int = 1) -> int:
    """The most rows that T*K routes fill when every expert's rows are padded to a multiple of ``row_align``."""
    return _size(_lib.moe_route_max_rows, T, K, E, row_align)


def moe_route_workspace_bytes(T: int, K: int, E: int) -> int:
    """Workspace of ``moe_route`` with the expert order (0 for small batches)."""
    return _size(_lib.moe_route_workspace_bytes, T, K, E)


_route_space = functools.lru_cache(maxsize=1024)(lambda T, K, E: moe_route_workspace_bytes(T, K, E))


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              num_groups: int = 1, topk_groups: int = 1, group_score: str = "max", renormalize: bool = True,
              scale: float = 1.0, scale_dtype: torch.dtype = torch.float32, row_align: int = 1, order: bool = True,
              out: Optional[Routing] = None, workspace: Optional[torch.Tensor] = None, pdl: bool = True,
              stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> Routing:
    """Choose ``top_k`` experts for each token and weigh them; with ``order``, sort the routes by expert.

    ``logits`` is [T, E] (fp32, bf16 or fp16; rows may be strided).  The score of an expert is its softmax or
    sigmoid; ``bias`` ([E] fp32) is added for the choice only.  With ``num_groups`` > 1 only the experts of the
    ``topk_groups`` best groups are taken, by a group's best choice score ("max") or the sum of its two best
    ("top2").  The weights are the scores, divided by their sum with ``renormalize``, times ``scale``.  Equal
    scores go to the lowest expert, and the order is decided as in 64 bits.  Experts with a logit of -inf or NaN
    are never taken; places left over get id -1, weight 0 and ``perm_idx`` -1, which the finalize skips.

    The expert order makes each expert's rows start at a multiple of ``row_align``.  ``out`` takes the outputs'
    buffers (``out.expert_offsets`` None: no order, whatever ``order`` says); ``row_route`` must hold at least
    ``moe_route_max_rows`` rows.  ``workspace`` must not be shared by calls that may run at the same time."""
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    index = logits.get_device()
    stride, inner = logits.stride()
    if check:
        if index < 0 or logits.dtype not in DTYPE:
            _check_tensor("logits", logits, logits.device, None, DTYPE, contiguous=False)
        if inner != 1 and E > 1:
            raise ValueError("the experts of a token must be contiguous in logits")
    allocated = []
    if out is None:
        dev = logits.device
        if scale_dtype not in DTYPE:
            raise ValueError(f"scale_dtype {scale_dtype} is not supported (fp32, bf16 or fp16)")
        out = Routing(torch.empty(T, top_k, dtype=torch.int32, device=dev),
                      torch.empty(T, top_k, dtype=scale_dtype, device=dev))
        allocated += [out.expert_ids, out.expert_scale]
        if order:
            out.perm_idx = torch.empty_like(out.expert_ids)
            out.row_route = torch.empty(moe_route_max_rows(T, top_k, E, row_align), dtype=torch.int32, device=dev)
            out.expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
            out.expert_counts = torch.empty(E, dtype=torch.int32, device=dev)
            allocated += [out.perm_idx, out.row_route, out.expert_offsets, out.expert_counts]
    ids, scales, perm, rows, offsets, counts = (out.expert_ids, out.expert_scale, out.perm_idx, out.row_route,
                                                out.expert_offsets, out.expert_counts)
    ordered = offsets is not None
    if check:
        shape = (T, top_k)
        if bias is not None and not _good(bias, index, (E,), torch.float32):
            _check_tensor("bias", bias, logits.device, (E,), torch.float32)
        if not (_good(ids, index, shape, torch.int32) and _good(scales, index, shape, None)):
            _check_tensor("expert_ids", ids, logits.device, shape, torch.int32)
            _check_tensor("expert_scale", scales, logits.device, shape, DTYPE)
        if ordered and not (_good(perm, index, shape, torch.int32) and _good(rows, index, None, torch.int32)
                            and _good(offsets, index, (E + 1,), torch.int32) and _good(counts, index, (E,), torch.int32)):
            _check_tensor("perm_idx", perm, logits.device, shape, torch.int32)
            _check_tensor("row_route", rows, logits.device, None, torch.int32)
            _check_tensor("expert_offsets", offsets, logits.device, (E + 1,), torch.int32)
            _check_tensor("expert_counts", counts, logits.device, (E,), torch.int32)
        if workspace is not None:
            _check_tensor("workspace", workspace, logits.device, None, torch.uint8)
    space = 0
    if ordered:
        if workspace is not None:
            space = workspace.numel()
        else:
            space = _route_space(T, top_k, E)
            if space:
                workspace = torch.empty(space, dtype=torch.uint8, device=logits.device)
                allocated.append(workspace)
        extra = (perm.data_ptr(), rows.data_ptr(), rows.numel(), offsets.data_ptr(), counts.data_ptr(),
                 workspace.data_ptr() if space else 0, space)
    else:
        extra = (0, 0, 0, 0, 0, 0, 0)
    args = _pack_route(T, E, top_k, DTYPE[logits.dtype], DTYPE[scales.dtype], _choice(SCORE, "score", score), num_groups,
                       topk_groups, _choice(GROUP_SCORE, "group_score", group_score), 1 if renormalize else 0, row_align,
                       scale, logits.data_ptr(), stride if T > 1 else E, 0 if bias is None else bias.data_ptr(),
                       ids.data_ptr(), scales.data_ptr(), *extra, _PDL if pdl else 0)
    _enqueue(_lib.moe_route, args, index, stream, allocated)
    return out


def moe_route_backward(d_scale: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor, *,
                       score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                       out: Optional[torch.Tensor] = None, pdl: bool = True,
                       stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> torch.Tensor:
    """The gradient of ``moe_route``'s weights to the logits ([T, E], the logits' dtype), the chosen experts held
    fixed.  ``score``, ``renormalize`` and ``scale`` are the forward call's; the bias and the groups only choose and
    have no gradient.  ``d_scale`` is [T, K] in any of the three types."""
    if logits.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("logits must be [T, E] and expert_ids [T, K]")
    T, E = logits.shape
    K = expert_ids.shape[1]
    index, act = logits.get_device(), logits.dtype
    allocated = []
    if out is None:
        out = torch.empty(T, E, dtype=act, device=logits.device)
        allocated.append(out)
    stride, inner = logits.stride()
    if check:
        dev, shape = logits.device, (T, K)
        if index < 0 or act not in DTYPE:
            _check_tensor("logits", logits, dev, None, DTYPE, contiguous=False)
        if not (_good(expert_ids, index, shape, torch.int32) and _good(d_scale, index, shape, None)):
            _check_tensor("expert_ids", expert_ids, dev, shape, torch.int32)
            _check_tensor("d_scale", d_scale, dev, shape, DTYPE)
        _check_tensor("out", out, dev, (T, E), act, contiguous=False)
        if E > 1 and (inner != 1 or out.stride(1) != 1):
            raise ValueError("the experts of a token must be contiguous in logits and out")
    args = _pack_route_backward(T, E, K, DTYPE[act], DTYPE[d_scale.dtype], _choice(SCORE, "score", score),
                                1 if renormalize else 0, scale, logits.data_ptr(), stride if T > 1 else E,
                                expert_ids.data_ptr(), d_scale.data_ptr(), out.data_ptr(), out.stride(0) if T > 1 else E,
                                _PDL if pdl else 0)
    _enqueue(_lib.moe_route_backward, args, index, stream, allocated)
    return out


# ----------------------------------------------------------------------------------------------------------------
# Dispatch and the finalize's gradient
# ----------------------------------------------------------------------------------------------------------------

def _rows_like(num_rows, like, row_route, allocated):
    """Rows in expert order: the kernel zeroes those of no route when it has ``row_route``, else they start as zeros."""
    make = torch.empty if row_route is not None else torch.zeros
    rows = make(num_rows, like.shape[1], dtype=like.dtype, device=like.device)
    allocated.append(rows)
    return rows


def moe_dispatch(x: torch.Tensor, perm_idx: torch.Tensor, num_rows: Optional[int] = None, *,
                 row_route: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, pdl: bool = True,
                 stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> torch.Tensor:
    """Copy each token's row ([T, n], any dtype, rows of a multiple of 16 bytes: activations, FP8 or NVFP4 codes,
    block scales) to the rows of its routes: ``out[perm_idx[t, k]] = x[t]``.  Routes outside the rows are skipped; no
    two routes may name the same row.  With ``row_route`` (as ``moe_route`` wrote it) the rows of no route are set to
    zero; without it they are left as they were, or zeros in an allocated output.  ``num_rows`` defaults to the
    length of ``row_route``.

    The gradient to ``x`` is ``moe_finalize_routed([Partial(d_rows, perm_idx)])``."""
    if perm_idx is None or x.dim() != 2 or perm_idx.dim() != 2:
        raise ValueError("x must be [T, n] and perm_idx [T, K]")
    index = x.get_device()
    T, n = x.shape
    if check and (index < 0 or not x.is_contiguous()):
        _check_tensor("x", x, x.device, None, x.dtype)
    allocated = []
    if out is None:
        if num_rows is None:
            if row_route is None:
                raise ValueError("num_rows, row_route or out must say how many rows there are")
            num_rows = row_route.shape[0]
        out = _rows_like(num_rows, x, row_route, allocated)
    rows = out.shape[0] if num_rows is None else num_rows
    K = perm_idx.shape[1]
    if check:
        if not (_good(out, index, (rows, n), x.dtype) and _good(perm_idx, index, (T, K), torch.int32)):
            _check_tensor("out", out, x.device, (rows, n), x.dtype)
            _check_tensor("perm_idx", perm_idx, x.device, (T, K), torch.int32)
        if row_route is not None and not _good(row_route, index, (rows,), torch.int32):
            _check_tensor("row_route", row_route, x.device, (rows,), torch.int32)
    args = _pack_dispatch(T, K, n * x.element_size(), rows, x.data_ptr(), perm_idx.data_ptr(), _ptr(row_route),
                          out.data_ptr(), _PDL if pdl else 0)
    _enqueue(_lib.moe_dispatch_rows, args, index, stream, allocated)
    return out


def moe_finalize_routed_backward(d_out: torch.Tensor, partial, *, routed_scaling_factor: float = 1.0,
                                 row_route: Optional[torch.Tensor] = None, d_gemm2: Optional[torch.Tensor] = None,
                                 d_scale: Optional[torch.Tensor] = None, want_d_gemm2: bool = True,
                                 want_d_scale: bool = True, pdl: bool = True,
                                 stream: Optional[torch.cuda.Stream] = None, check: bool = True
                                 ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradient of one partial of ``moe_finalize_routed`` to its GEMM2 rows and its expert scales, given the
    gradient ``d_out`` ([T, H]) of the finalized output; returns ``(d_gemm2, d_scale)`` (``want_*`` False leaves one
    out).  The gradient of ``shared_out`` is ``d_out`` itself, and every partial of a rank sum has the same ``d_out``.
    ``d_scale`` has the scales' dtype (fp32 where the partial has none).  No two routes may name the same row, and
    outputs overlap no input.  With ``row_route`` the rows of no route get zeros; without it they are left as they
    were, or zeros in an allocated output.  The residual addition and the RMSNorm of ``moe_finalize_fused`` have no
    gradient here: a program that trains through them gets ``d_out`` from its own norm's gradient."""
    x, perm, scale = partial.gemm2_out, partial.perm_idx, partial.expert_scale
    if perm is None or x is None or d_out.dim() != 2 or perm.dim() != 2 or x.dim() != 2:
        raise ValueError("d_out must be [T, H], gemm2_out [rows, H] and perm_idx [T, K]")
    T, H = d_out.shape
    K, rows = perm.shape[1], x.shape[0]
    index, act = d_out.get_device(), d_out.dtype
    sdt = torch.float32 if scale is None else scale.dtype
    allocated = []
    if d_gemm2 is None and want_d_gemm2:
        d_gemm2 = _rows_like(rows, x, row_route, allocated)
    if d_scale is None and want_d_scale:
        d_scale = torch.empty(T, K, dtype=sdt, device=d_out.device)
        allocated.append(d_scale)
    if check:
        dev, shape = d_out.device, (T, K)
        if index < 0 or (act is not torch.bfloat16 and act is not torch.float16) or not d_out.is_contiguous():
            _check_tensor("d_out", d_out, dev, None, (torch.bfloat16, torch.float16))
        if not (_good(x, index, (rows, H), act) and _good(perm, index, shape, torch.int32)):
            _check_tensor("gemm2_out", x, dev, (rows, H), act)
            _check_tensor("perm_idx", perm, dev, shape, torch.int32)
        if scale is not None and not _good(scale, index, shape, None):
            _check_tensor("expert_scale", scale, dev, shape, DTYPE)
        if row_route is not None and not _good(row_route, index, (rows,), torch.int32):
            _check_tensor("row_route", row_route, dev, (rows,), torch.int32)
        if d_gemm2 is not None and not _good(d_gemm2, index, (rows, H), act):
            _check_tensor("d_gemm2", d_gemm2, dev, (rows, H), act)
        if d_scale is not None and not _good(d_scale, index, shape, sdt):
            _check_tensor("d_scale", d_scale, dev, shape, sdt)
    args = _pack_routed_backward(T, H, K, DTYPE[act], DTYPE[sdt], routed_scaling_factor, rows, x.data_ptr(), perm.data_ptr(),
                                 _ptr(scale), _ptr(row_route), d_out.data_ptr(), _ptr(d_gemm2), _ptr(d_scale),
                                 _PDL if pdl else 0)
    _enqueue(_lib.moe_routed_backward, args, index, stream, allocated)
    return d_gemm2, d_scale


# ----------------------------------------------------------------------------------------------------------------
# Per-head norm and rotation
# ----------------------------------------------------------------------------------------------------------------

def _heads(name, t, index, shape, act, check):
    """Pointer and strides of a tensor of heads (those of a dimension of one are never used, whatever torch reports)."""
    s = t.stride()
    if check and not (t.dtype is act and t.get_device() == index and t.shape == shape and s[2] == 1):
        _check_tensor(name, t, torch.device("cuda", index), shape, act, contiguous=False)
        raise ValueError(f"the elements of a head must be contiguous in {name}")
    T, heads, D = shape
    return t.data_ptr(), s[0] if T > 1 else heads * D, s[1] if heads > 1 else D


def _head_shapes(q, k, q_weight, k_weight, positions, inv_freq, check):
    """Device index, type, and the shapes of the queries and the keys."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, heads, D] and k [T, kv_heads, D]")
    index, act = q.get_device(), q.dtype
    T, hq, D = shape = tuple(q.shape)
    if check:
        if index < 0 or (act is not torch.bfloat16 and act is not torch.float16):
            _check_tensor("q", q, q.device, None, (torch.bfloat16, torch.float16), contiguous=False)
        one = (D,)
        if q_weight is not None and not _good(q_weight, index, one, act):
            _check_tensor("q_weight", q_weight, q.device, one, act)
        if k_weight is not None and not _good(k_weight, index, one, act):
            _check_tensor("k_weight", k_weight, q.device, one, act)
        if not _good(positions, index, (T,), torch.int32):
            _check_tensor("positions", positions, q.device, (T,), (torch.int32, torch.int64))
        if not (inv_freq.dtype is torch.float32 and inv_freq.get_device() == index and inv_freq.dim() == 1 and inv_freq.is_contiguous()):
            _check_tensor("inv_freq", inv_freq, q.device, (inv_freq.numel(),), torch.float32)
    return index, act, shape, (T, k.shape[1], D)


def head_norm_rotary(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor],
                     k_weight: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, *,
                     eps: float = 1e-6, style: str = "half", rotary_scale: float = 1.0,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, pdl: bool = True,
                     stream: Optional[torch.cuda.Stream] = None, check: bool = True
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMSNorm of every head of ``q`` ([T, heads, D]) and ``k`` ([T, kv_heads, D]) with the weights ([D], or None),
    then the rotation of its first ``2 * len(inv_freq)`` elements by ``positions[t] * inv_freq[j]`` (times
    ``rotary_scale``); one rounding at the end.  "half" pairs elements i and i + rot/2, "interleaved" 2i and 2i + 1.
    D is a multiple of 16 up to 512; tokens and heads may be strided (views of a packed projection), by multiples of
    8 elements.

    ``positions`` is int32 or int64.  A negative position marks a padding token: its values do not matter, and its
    output rows are left as they were (zeros in an allocated output).  ``q_out`` and ``k_out`` may be ``q`` and ``k``."""
    flags = _PDL if pdl else 0
    if positions.dtype is torch.int64:
        flags |= _POSITIONS_64
    allocated = []
    index, act, sq, sk = _head_shapes(q, k, q_weight, k_weight, positions, inv_freq, check)
    if q_out is None and k_out is None:
        q_out = torch.empty(sq, dtype=act, device=q.device)
        k_out = torch.empty(sk, dtype=act, device=q.device)
        flags |= _ZERO_PADDING
        allocated += [q_out, k_out]
    elif q_out is None or k_out is None:
        raise ValueError("q_out and k_out are passed both or neither")
    args = _pack_head_norm(sq[0], sq[1], sk[1], sq[2], 2 * inv_freq.numel(), _choice(ROTARY_STYLE, "style", style), DTYPE[act],
                           eps, rotary_scale, *_heads("q", q, index, sq, act, check), *_heads("k", k, index, sk, act, check),
                           *_heads("q_out", q_out, index, sq, act, check), *_heads("k_out", k_out, index, sk, act, check),
                           0, 0, 0, 0, 0, 0, _ptr(q_weight), _ptr(k_weight), positions.data_ptr(), inv_freq.data_ptr(),
                           0, 0, 0, 0, flags)
    _enqueue(_lib.moe_head_norm_rotary, args, index, stream, allocated)
    return q_out, k_out


def head_norm_rotary_workspace_bytes(T: int, q_heads: int, k_heads: int, D: int) -> int:
    """Workspace of ``head_norm_rotary_backward`` when a weight gradient is asked."""
    return _size(_lib.moe_head_norm_rotary_workspace_bytes, T, q_heads, k_heads, D)


_head_space = functools.lru_cache(maxsize=1024)(lambda *sizes: head_norm_rotary_workspace_bytes(*sizes))


def head_norm_rotary_backward(d_q_out: torch.Tensor, d_k_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                              q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                              positions: torch.Tensor, inv_freq: torch.Tensor, *, eps: float = 1e-6,
                              style: str = "half", rotary_scale: float = 1.0, d_q: Optional[torch.Tensor] = None,
                              d_k: Optional[torch.Tensor] = None, d_q_weight: Optional[torch.Tensor] = None,
                              d_k_weight: Optional[torch.Tensor] = None, want_weights: bool = True,
                              workspace: Optional[torch.Tensor] = None, pdl: bool = True,
                              stream: Optional[torch.cuda.Stream] = None, check: bool = True):
    """The gradients of ``head_norm_rotary``, given those of its outputs and its inputs as they were before the
    call: ``(d_q, d_k, d_q_weight, d_k_weight)``, the weights' in FP32 ([D], summed over tokens and heads in a fixed
    order; None where the weight is None or ``want_weights`` is False).  Padding tokens add nothing to the weights'
    gradients, and their rows of ``d_q`` and ``d_k`` are set to zero.  ``d_q`` and ``d_k`` may be ``d_q_out`` and
    ``d_k_out``, or ``q`` and ``k``.  ``workspace`` must not be shared by calls that may run at the same time."""
    flags = _PDL if pdl else 0
    if positions.dtype is torch.int64:
        flags |= _POSITIONS_64
    allocated = []
    index, act, sq, sk = _head_shapes(q, k, q_weight, k_weight, positions, inv_freq, check)
    T, hq, D = sq
    if d_q is None and d_k is None:
        d_q = torch.empty(sq, dtype=act, device=q.device)
        d_k = torch.empty(sk, dtype=act, device=q.device)
        allocated += [d_q, d_k]
    elif d_q is None or d_k is None:
        raise ValueError("d_q and d_k are passed both or neither")
    if want_weights:
        if d_q_weight is None and q_weight is not None:
            d_q_weight = torch.empty(D, dtype=torch.float32, device=q.device)
            allocated.append(d_q_weight)
        if d_k_weight is None and k_weight is not None:
            d_k_weight = torch.empty(D, dtype=torch.float32, device=q.device)
            allocated.append(d_k_weight)
    if check:
        one = (D,)
        if d_q_weight is not None and not _good(d_q_weight, index, one, torch.float32):
            _check_tensor("d_q_weight", d_q_weight, q.device, one, torch.float32)
        if d_k_weight is not None and not _good(d_k_weight, index, one, torch.float32):
            _check_tensor("d_k_weight", d_k_weight, q.device, one, torch.float32)
    space, at = 0, 0
    if d_q_weight is not None or d_k_weight is not None:
        if workspace is None:
            space = _head_space(T, hq, sk[1], D)
            workspace = torch.empty(space, dtype=torch.uint8, device=q.device)
            allocated.append(workspace)
        else:
            if check:
                _check_tensor("workspace", workspace, q.device, None, torch.uint8)
            space = workspace.numel()
        at = workspace.data_ptr()
    args = _pack_head_norm(T, hq, sk[1], D, 2 * inv_freq.numel(), _choice(ROTARY_STYLE, "style", style), DTYPE[act], eps,
                           rotary_scale, *_heads("q", q, index, sq, act, check), *_heads("k", k, index, sk, act, check),
                           *_heads("d_q", d_q, index, sq, act, check), *_heads("d_k", d_k, index, sk, act, check),
                           *_heads("d_q_out", d_q_out, index, sq, act, check), *_heads("d_k_out", d_k_out, index, sk, act, check),
                           _ptr(q_weight), _ptr(k_weight), positions.data_ptr(), inv_freq.data_ptr(), _ptr(d_q_weight),
                           _ptr(d_k_weight), at, space, flags)
    _enqueue(_lib.moe_head_norm_rotary_backward, args, index, stream, allocated)
    return d_q, d_k, d_q_weight, d_k_weight
