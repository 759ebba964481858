"""4-bit matrices, their product, and the routing of tokens to experts: the
binding of include/moe_fp4.h.  Argument marshalling only, as in ``binding``:
every step runs in the library's CUDA kernels, on the current stream or the
one given, and nothing falls back.

    routing = moe_sort(ids, experts)                    # ids: tokens x top_k
    q = fp4_quantize(x, routing=routing)                # x's rows in expert order
    y = fp4_gemm_tn(q, weights)                         # weights: an Fp4Matrix of experts
    out = moe_combine(y, routing, gates)                # back in token order

Tensors given as `out` are written in place; without it one is allocated.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import binding as _b
from .binding import GEMM_OK, GemmError, LIB

EXPORTED = ("fp4_code_bytes", "fp4_scale_bytes", "fp4_quantize", "fp4_dequantize", "fp4_gemm_tn",
            "fp4_get_device_error", "moe_sort_workspace_bytes", "moe_sort", "moe_dispatch",
            "moe_dispatch_backward", "moe_combine", "moe_combine_backward")

TYPES = {torch.float16: 0, torch.bfloat16: 1}
FORMATS = {"nvfp4": 0, "mxfp4": 1}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
MAX_EXPERTS, MAX_TOP_K = 1024, 64


class _RoutingC(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("top_k", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("pairs", ctypes.c_void_p), ("ids", ctypes.c_void_p)]


class _MatrixC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("format", ctypes.c_int32),
                ("exponent", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("group_rows", ctypes.c_int64),
                ("offsets", ctypes.c_void_p)]


def _declare():
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    pr, pm, pu = ctypes.POINTER(_RoutingC), ctypes.POINTER(_MatrixC), ctypes.POINTER(ctypes.c_uint64)
    for name, args in {
            "fp4_code_bytes": [i64, i64, pu],
            "fp4_scale_bytes": [i64, i64, i32, i32, i32, pu],
            "fp4_quantize": [pm, vp, i64, i32, pr, vp],
            "fp4_dequantize": [vp, i32, pm, vp],
            "fp4_gemm_tn": [vp, i32, pm, pm, ctypes.c_float, vp],
            "fp4_get_device_error": [vp, ctypes.POINTER(ctypes.c_uint32)],
            "moe_sort_workspace_bytes": [i64, i32, i32, pu],
            "moe_sort": [vp, vp, vp, vp, i64, i32, i32, vp, ctypes.c_uint64, vp],
            "moe_dispatch": [vp, vp, i64, i64, i32, pr, vp],
            "moe_dispatch_backward": [vp, vp, i64, i32, pr, vp],
            "moe_combine": [vp, vp, vp, i64, i32, pr, vp],
            "moe_combine_backward": [vp, vp, vp, vp, vp, i64, i32, pr, vp]}.items():
        f = getattr(LIB, name)
        f.argtypes, f.restype = args, i32


_declare()


def _call(name: str, device: torch.device, *args):
    """The C function with the stream's device current."""
    if device.index is None or device.index == torch.cuda.current_device():
        rc = getattr(LIB, name)(*args)
    else:
        with torch.cuda.device(device):
            rc = getattr(LIB, name)(*args)
    if rc != GEMM_OK:
        raise GemmError(rc, name)


def _stream(stream, device: torch.device) -> int:
    return int((stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream)


def _matrix(x: torch.Tensor, what: str) -> None:
    """x is a CUDA matrix of a supported type with contiguous rows."""
    if x.dtype not in TYPES:
        raise TypeError(f"{what} must be float16 or bfloat16")
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{what}'s rows must be contiguous")


def _out(out, shape, dtype, device, what: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or not out.is_contiguous() \
            or out.device != device:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         "on the inputs' device")
    return out


def _row_stride(x: torch.Tensor) -> int:
    """Elements between rows (a tensor of one row may report any stride)."""
    return max(x.stride(0), x.shape[1]) if x.shape[0] > 1 else x.shape[1]


@dataclass
class Routing:
    """Where each slot (token, j) went: rows[token, j] is its row in expert order, pairs the
    inverse, and expert e has rows offsets[e] to offsets[e + 1] - 1.  Dropped slots have the
    rows from offsets[-1] on.  All int32, on the device."""
    offsets: torch.Tensor
    rows: torch.Tensor
    pairs: torch.Tensor
    ids: torch.Tensor

    @property
    def tokens(self) -> int:
        return self.ids.shape[0]

    @property
    def top_k(self) -> int:
        return self.ids.shape[1]

    @property
    def experts(self) -> int:
        return self.offsets.shape[0] - 1

    @property
    def slots(self) -> int:
        return self.ids.numel()

    def _c(self) -> _RoutingC:
        return _RoutingC(self.ids.shape[0], self.ids.shape[1], self.offsets.shape[0] - 1,
                         self.offsets.data_ptr(), self.rows.data_ptr(), self.pairs.data_ptr(),
                         self.ids.data_ptr())


class Fp4Matrix:
    """A matrix of 4-bit blocks in the layout of include/moe_fp4.h.

    codes: rows x (cols rounded up to 32) / 2 bytes.  scales: tiles x chunks x 512 bytes.
    group_rows: rows of each group (for weights of several experts, one expert's outputs; default:
    all rows are one group).  Instead, `routing` marks rows in expert order."""

    __slots__ = ("codes", "scales", "cols", "format", "exponent", "group_rows", "routing", "groups")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, *, cols: int,
                 format: str = "nvfp4", exponent: int = 0, group_rows: int | None = None,
                 routing: Routing | None = None):
        if format not in FORMATS:
            raise ValueError(f"unknown format {format!r}")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if not (codes.is_cuda and scales.is_cuda) or codes.device != scales.device:
            raise ValueError("codes and scales must be CUDA tensors on one device")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        pitch = (cols + 31) // 32 * 16
        if codes.dim() != 2 or codes.shape[1] != pitch:
            raise ValueError(f"codes must be rows x {pitch}, got {tuple(codes.shape)}")
        rows = codes.shape[0]
        if routing is not None:
            if group_rows is not None or rows != routing.slots:
                raise ValueError("a matrix in expert order has a row per slot and no group_rows")
            self.groups, group_rows = routing.experts, 0
            tiles = rows // 128 + self.groups
        else:
            group_rows = rows if group_rows is None else int(group_rows)
            if group_rows < 0 or (rows % group_rows if group_rows else rows):
                raise ValueError(f"{rows} rows are not whole groups of {group_rows}")
            self.groups = max(rows // group_rows, 1) if group_rows else 1
            tiles = self.groups * -(-group_rows // 128)
        need = tiles * -(-cols // 256) * (4 if format == "nvfp4" else 2) * 512
        if scales.numel() < need:
            raise ValueError(f"scales must have {need} bytes, got {scales.numel()}")
        self.codes, self.scales, self.cols = codes, scales, int(cols)
        self.format, self.exponent = format, int(exponent)
        self.group_rows, self.routing = group_rows, routing

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def _c(self) -> _MatrixC:
        return _MatrixC(self.codes.data_ptr(), self.scales.data_ptr(), self.codes.shape[0],
                        self.cols, FORMATS[self.format], self.exponent, self.groups, 0,
                        self.group_rows,
                        self.routing.offsets.data_ptr() if self.routing is not None else None)


def _bytes(name: str, *args) -> int:
    n = ctypes.c_uint64(0)
    rc = getattr(LIB, name)(*args, ctypes.byref(n))
    if rc != GEMM_OK:
        raise GemmError(rc, name)
    return int(n.value)


def fp4_scale_bytes(rows: int, cols: int, format: str = "nvfp4", groups: int = 1,
                    by_offsets: bool = False) -> int:
    """Bytes of an Fp4Matrix's scales."""
    return _bytes("fp4_scale_bytes", rows, cols, FORMATS[format], groups, int(by_offsets))


def fp4_quantize(x: torch.Tensor, *, format: str = "nvfp4", exponent: int = 0,
                 group_rows: int | None = None, routing: Routing | None = None,
                 out: Fp4Matrix | None = None, stream=None) -> Fp4Matrix:
    """x (rows x cols, float16 or bfloat16, rows contiguous) as an Fp4Matrix.

    With a routing, x has a row per token and the result a row per slot, in expert order."""
    _matrix(x, "x")
    if format not in FORMATS:
        raise ValueError(f"unknown format {format!r}")
    rows, cols = x.shape
    if routing is not None:
        if rows != routing.tokens:
            raise ValueError(f"x has {rows} rows, the routing {routing.tokens} tokens")
        if routing.offsets.device != x.device:
            raise ValueError("x and the routing are on different devices")
        rows = routing.slots
    if out is None:
        pitch = (cols + 31) // 32 * 16
        if routing is not None:
            tiles = rows // 128 + routing.experts
        else:
            g = rows if group_rows is None else int(group_rows)
            tiles = rows // g * -(-g // 128) if g > 0 else 0
        chunks = -(-cols // 256) * (4 if format == "nvfp4" else 2)
        out = Fp4Matrix(torch.empty((rows, pitch), dtype=torch.uint8, device=x.device),
                        torch.empty((tiles, chunks, 512), dtype=torch.uint8, device=x.device),
                        cols=cols, format=format, exponent=exponent, group_rows=group_rows,
                        routing=routing)
    elif out.rows != rows or out.cols != cols or out.format != format \
            or out.exponent != exponent or out.routing is not routing or out.device != x.device \
            or (group_rows is not None and out.group_rows != group_rows):
        raise ValueError("out does not fit x, the format or the groups")
    _call("fp4_quantize", x.device, ctypes.byref(out._c()), x.data_ptr(), _row_stride(x),
          TYPES[x.dtype], ctypes.byref(routing._c()) if routing is not None else None,
          _stream(stream, x.device))
    return out


def fp4_dequantize(q: Fp4Matrix, dtype: torch.dtype = torch.float16,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of q, rows x cols; rows of dropped slots are zero."""
    if dtype not in TYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    out = _out(out, (q.rows, q.cols), dtype, q.device, "out")
    _call("fp4_dequantize", q.device, out.data_ptr(), TYPES[dtype], ctypes.byref(q._c()),
          _stream(stream, q.device))
    return out


def fp4_gemm_tn(a: Fp4Matrix, b: Fp4Matrix, *, alpha: float = 1.0,
                dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """out[r] = alpha * a[r] @ b[g(r)]^T (fp32 accumulation): g(r) is the group of row r, so with
    activations in expert order each row meets its expert's weights; rows of dropped slots give
    zeros.  b has as many groups as a, each of b.group_rows outputs."""
    if dtype not in TYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    if a.device != b.device:
        raise ValueError("a and b are on different devices")
    out = _out(out, (a.rows, b.group_rows), dtype, a.device, "out")
    _call("fp4_gemm_tn", a.device, out.data_ptr(), TYPES[dtype], ctypes.byref(a._c()),
          ctypes.byref(b._c()), float(alpha), _stream(stream, a.device))
    return out


def fp4_get_device_error(stream=None) -> tuple[int, int]:
    """(status, raw word) of the stream's error word of fp4_gemm_tn; synchronises the stream."""
    raw = ctypes.c_uint32(0)
    rc = LIB.fp4_get_device_error(_b._stream_handle(stream), ctypes.byref(raw))
    return rc, int(raw.value)


def moe_sort(ids: torch.Tensor, experts: int, workspace: torch.Tensor | None = None,
             stream=None) -> Routing:
    """Slots sorted by expert.  ids: tokens x top_k int32; a number outside [0, experts) drops
    its slot.  The order within an expert is the slots' own."""
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 2 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 2-D CUDA tensor (tokens x top_k)")
    experts = int(experts)
    if not 1 <= experts <= MAX_EXPERTS or not 1 <= ids.shape[1] <= MAX_TOP_K:
        raise ValueError(f"1 to {MAX_EXPERTS} experts and 1 to {MAX_TOP_K} slots are supported")
    need = _bytes("moe_sort_workspace_bytes", ids.shape[0], ids.shape[1], experts)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=ids.device)
    elif workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != ids.device
                                    or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on ids's device")
    r = Routing(torch.empty(experts + 1, dtype=torch.int32, device=ids.device),
                torch.empty_like(ids),
                torch.empty(ids.numel(), dtype=torch.int32, device=ids.device), ids)
    _call("moe_sort", ids.device, r.offsets.data_ptr(), r.rows.data_ptr(), r.pairs.data_ptr(),
          ids.data_ptr(), ids.shape[0], ids.shape[1], experts,
          workspace.data_ptr() if workspace is not None else None,
          workspace.numel() if workspace is not None else 0, _stream(stream, ids.device))
    return r


def _by_token(x: torch.Tensor, routing: Routing, what: str) -> None:
    _matrix(x, what)
    if x.shape[0] != routing.tokens or x.device != routing.offsets.device:
        raise ValueError(f"{what} must have the routing's {routing.tokens} rows, on its device")


def _by_slot(y: torch.Tensor, routing: Routing, what: str) -> None:
    _matrix(y, what)
    if y.shape[0] != routing.slots or not y.is_contiguous() or y.device != routing.offsets.device:
        raise ValueError(f"{what} must be contiguous with the routing's {routing.slots} rows, "
                         "on its device")


def _weights(weights: torch.Tensor, routing: Routing) -> None:
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if weights.shape != routing.ids.shape or not weights.is_contiguous() \
            or weights.device != routing.offsets.device:
        raise ValueError("weights must be contiguous, of the routing's tokens x top_k, "
                         "on its device")


def moe_dispatch(x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """x's rows (a row per token) in expert order, a row per slot; zeros for dropped slots."""
    _by_token(x, routing, "x")
    out = _out(out, (routing.slots, x.shape[1]), x.dtype, x.device, "out")
    _call("moe_dispatch", x.device, out.data_ptr(), x.data_ptr(), _row_stride(x), x.shape[1],
          TYPES[x.dtype], ctypes.byref(routing._c()), _stream(stream, x.device))
    return out


def moe_dispatch_backward(grad_y: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """moe_dispatch's gradient: each token's sum over its kept slots."""
    _by_slot(grad_y, routing, "grad_y")
    out = _out(out, (routing.tokens, grad_y.shape[1]), grad_y.dtype, grad_y.device, "out")
    _call("moe_dispatch_backward", grad_y.device, out.data_ptr(), grad_y.data_ptr(),
          grad_y.shape[1], TYPES[grad_y.dtype], ctypes.byref(routing._c()),
          _stream(stream, grad_y.device))
    return out


def moe_combine(y: torch.Tensor, routing: Routing, weights: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's weighted sum of its kept slots' rows of y.  weights: tokens x top_k float32."""
    _by_slot(y, routing, "y")
    _weights(weights, routing)
    out = _out(out, (routing.tokens, y.shape[1]), y.dtype, y.device, "out")
    _call("moe_combine", y.device, out.data_ptr(), y.data_ptr(), weights.data_ptr(), y.shape[1],
          TYPES[y.dtype], ctypes.byref(routing._c()), _stream(stream, y.device))
    return out


def moe_combine_backward(grad_out: torch.Tensor, y: torch.Tensor, routing: Routing,
                         weights: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """moe_combine's gradients: (of y, of weights); zeros for dropped slots."""
    _by_token(grad_out, routing, "grad_out")
    _by_slot(y, routing, "y")
    _weights(weights, routing)
    if grad_out.dtype != y.dtype or grad_out.shape[1] != y.shape[1] \
            or not grad_out.is_contiguous():
        raise ValueError("grad_out must be contiguous, of y's type and width")
    grad_y = torch.empty_like(y)
    grad_w = torch.empty_like(weights)
    _call("moe_combine_backward", y.device, grad_y.data_ptr(), grad_w.data_ptr(),
          grad_out.data_ptr(), y.data_ptr(), weights.data_ptr(), y.shape[1], TYPES[y.dtype],
          ctypes.byref(routing._c()), _stream(stream, y.device))
    return grad_y, grad_w
