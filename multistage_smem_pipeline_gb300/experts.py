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

import torch

from . import binding as _b
from .binding import GEMM_OK, GemmError, LIB

EXPORTED = ("fp4_code_bytes", "fp4_scale_bytes", "fp4_quantize", "fp4_dequantize", "fp4_gemm_tn",
            "fp4_get_device_error", "moe_sort", "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward")

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


_FUNCTIONS = {}


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
            "moe_sort": [vp, vp, vp, vp, i64, i32, i32, vp],
            "moe_dispatch": [vp, vp, i64, i64, i32, pr, vp],
            "moe_dispatch_backward": [vp, vp, i64, i32, pr, vp],
            "moe_combine": [vp, vp, vp, i64, i32, pr, vp],
            "moe_combine_backward": [vp, vp, vp, vp, vp, i64, i32, pr, vp]}.items():
        f = getattr(LIB, name)
        f.argtypes, f.restype = args, i32
        _FUNCTIONS[name] = f


_declare()


_raw_stream = torch._C._cuda_getCurrentRawStream  # of a device index, without a Stream object
_current_device = torch._C._cuda_getDevice


def _call(name: str, x: torch.Tensor, stream, *args):
    """The C function on `stream` (default: the current one of x's device), with that device
    current."""
    index = x.get_device()
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        rc = _FUNCTIONS[name](*args, handle)
    else:
        with torch.cuda.device(index):
            rc = _FUNCTIONS[name](*args, handle)
    if rc:
        raise GemmError(rc, name)


def _matrix(x: torch.Tensor, what: str) -> int:
    """x's type number; x must be a CUDA matrix of a supported type with contiguous rows."""
    kind = TYPES.get(x.dtype)
    if kind is None:
        raise TypeError(f"{what} must be float16 or bfloat16")
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    if not x.is_contiguous() and x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    return kind


def _out(out, shape, dtype, device, what: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or not out.is_contiguous() \
            or out.device != device:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         "on the inputs' device")
    return out


def _row_stride(x: torch.Tensor, cols: int) -> int:
    """Elements between rows (a tensor of one row may report any stride)."""
    return max(x.stride(0), cols) if x.shape[0] > 1 else cols


class Routing:
    """Where each slot (token, j) went: rows[token, j] is its row in expert order, pairs the
    inverse, and expert e has rows offsets[e] to offsets[e + 1] - 1.  Dropped slots have the
    rows from offsets[-1] on.  All int32, on the device.  moe_sort makes one; a program with a
    router of its own can give the tensors itself."""

    __slots__ = ("ids", "tokens", "top_k", "experts", "slots", "device", "_buffer", "_offsets",
                 "_rows", "_pairs", "_c", "_ref")

    def __init__(self, offsets: torch.Tensor, rows: torch.Tensor, pairs: torch.Tensor,
                 ids: torch.Tensor):
        for t, what in ((offsets, "offsets"), (rows, "rows"), (pairs, "pairs"), (ids, "ids")):
            if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() \
                    or t.device != ids.device:
                raise ValueError(f"{what} must be a contiguous int32 CUDA tensor on ids's device")
        if ids.dim() != 2 or rows.shape != ids.shape or pairs.numel() != ids.numel() \
                or offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("ids and rows must be tokens x top_k, pairs as many, and offsets "
                             "experts + 1")
        self._offsets, self._rows, self._pairs, self._buffer = offsets, rows, pairs, None
        self._set(ids, offsets.numel() - 1, offsets.data_ptr(), rows.data_ptr(), pairs.data_ptr())

    def _set(self, ids, experts, offsets, rows, pairs):
        self.ids, self.experts, self.device = ids, experts, ids.device
        self.tokens, self.top_k = ids.shape
        self.slots = self.tokens * self.top_k
        self._c = _RoutingC(self.tokens, self.top_k, experts, offsets, rows, pairs, ids.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _empty(cls, ids: torch.Tensor, experts: int) -> "Routing":
        """Unwritten: one allocation for the three arrays, each on a 16-byte boundary; the
        tensors are made when they are asked for."""
        self = cls.__new__(cls)
        n, head = ids.numel() + 3 & ~3, experts + 4 & ~3
        self._buffer = torch.empty(head + 2 * n, dtype=torch.int32, device=ids.device)
        self._offsets = self._rows = self._pairs = None
        at = self._buffer.data_ptr()
        self._set(ids, experts, at, at + 4 * head, at + 4 * (head + n))
        return self

    @property
    def offsets(self) -> torch.Tensor:
        if self._offsets is None:
            self._offsets = self._buffer[:self.experts + 1]
        return self._offsets

    @property
    def rows(self) -> torch.Tensor:
        if self._rows is None:
            head = self.experts + 4 & ~3
            self._rows = self._buffer.as_strided((self.tokens, self.top_k), (self.top_k, 1), head)
        return self._rows

    @property
    def pairs(self) -> torch.Tensor:
        if self._pairs is None:
            head, n = self.experts + 4 & ~3, self.slots + 3 & ~3
            self._pairs = self._buffer[head + n:head + n + self.slots]
        return self._pairs


def _layout(rows: int, cols: int, form: str, group_rows: int | None, routing: Routing | None):
    """(groups, rows of a uniform group, bytes of a row's codes, tiles, chunks of a tile)."""
    if form not in FORMATS:
        raise ValueError(f"unknown format {form!r}")
    chunks = -(-cols // 256) * (4 if form == "nvfp4" else 2)
    pitch = (cols + 31) // 32 * 16
    if routing is not None:
        if group_rows is not None or rows != routing.tokens * routing.top_k:
            raise ValueError("a matrix in expert order has a row per slot and no group_rows")
        return routing.experts, 0, pitch, rows // 128 + routing.experts, chunks
    g = rows if group_rows is None else int(group_rows)
    if g < 0 or (rows % g if g else rows):
        raise ValueError(f"{rows} rows are not whole groups of {g}")
    groups = max(rows // g, 1) if g else 1
    return groups, g, pitch, groups * -(-g // 128), chunks


class Fp4Matrix:
    """A matrix of 4-bit blocks in the layout of include/moe_fp4.h.

    codes: rows x (cols rounded up to 32) / 2 bytes.  scales: tiles x chunks x 512 bytes.
    group_rows: rows of each group (for weights of several experts, one expert's outputs; default:
    all rows are one group).  Instead, `routing` marks rows in expert order."""

    __slots__ = ("rows", "cols", "format", "exponent", "group_rows", "routing", "groups", "device",
                 "_shape", "_buffer", "_codes", "_scales", "_c", "_ref")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, *, cols: int,
                 format: str = "nvfp4", exponent: int = 0, group_rows: int | None = None,
                 routing: Routing | None = None):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if not (codes.is_cuda and scales.is_cuda) or codes.device != scales.device:
            raise ValueError("codes and scales must be CUDA tensors on one device")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        if codes.dim() != 2:
            raise ValueError("codes must be a matrix")
        shape = _layout(codes.shape[0], cols, format, group_rows, routing)
        if codes.shape[1] != shape[2]:
            raise ValueError(f"codes must be rows x {shape[2]}, got {tuple(codes.shape)}")
        if scales.numel() < shape[3] * shape[4] * 512:
            raise ValueError(f"scales must have {shape[3] * shape[4] * 512} bytes, "
                             f"got {scales.numel()}")
        self._codes, self._scales, self._buffer, self.device = codes, scales, None, codes.device
        self._set(codes.shape[0], cols, format, exponent, routing, shape, codes.data_ptr(),
                  scales.data_ptr())

    def _set(self, rows, cols, form, exponent, routing, shape, codes, scales):
        self.rows, self.cols, self.format, self.exponent = rows, int(cols), form, int(exponent)
        self.groups, self.group_rows, self.routing, self._shape = shape[0], shape[1], routing, shape
        self._c = _MatrixC(codes, scales, rows, self.cols, FORMATS[form], self.exponent, shape[0],
                           0, shape[1], None if routing is None else routing._c.offsets)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _empty(cls, rows, cols, form, exponent, group_rows, routing, device) -> "Fp4Matrix":
        """Unwritten: one allocation for scales and codes; the tensors are made when asked for."""
        self = cls.__new__(cls)
        shape = _layout(rows, cols, form, group_rows, routing)
        scales = shape[3] * shape[4] * 512
        self._buffer = torch.empty(scales + rows * shape[2], dtype=torch.uint8, device=device)
        self._codes = self._scales = None
        self.device = device
        at = self._buffer.data_ptr()
        self._set(rows, cols, form, exponent, routing, shape, at + scales, at)
        return self

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            tiles, chunks = self._shape[3:]
            self._scales = self._buffer[:tiles * chunks * 512].view(tiles, chunks, 512)
        return self._scales

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            tiles, chunks = self._shape[3:]
            self._codes = self._buffer[tiles * chunks * 512:].view(self.rows, self._shape[2])
        return self._codes

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
    kind = _matrix(x, "x")
    rows, cols = x.shape
    if routing is not None:
        if rows != routing.tokens:
            raise ValueError(f"x has {rows} rows, the routing {routing.tokens} tokens")
        if routing.device != x.device:
            raise ValueError("x and the routing are on different devices")
        rows = routing.slots
    if out is None:
        out = Fp4Matrix._empty(rows, cols, format, exponent, group_rows, routing, x.device)
    elif out.rows != rows or out.cols != cols or out.format != format \
            or out.exponent != exponent or out.routing is not routing or out.device != x.device \
            or (group_rows is not None and out.group_rows != group_rows):
        raise ValueError("out does not fit x, the format or the groups")
    _call("fp4_quantize", x, stream, out._ref, x.data_ptr(), _row_stride(x, cols), kind,
          None if routing is None else routing._ref)
    return out


def fp4_dequantize(q: Fp4Matrix, dtype: torch.dtype = torch.float16,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of q, rows x cols; rows of dropped slots are zero."""
    if dtype not in TYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    out = _out(out, (q.rows, q.cols), dtype, q.device, "out")
    _call("fp4_dequantize", out, stream, out.data_ptr(), TYPES[dtype], q._ref)
    return out


def fp4_gemm_tn(a: Fp4Matrix, b: Fp4Matrix, *, alpha: float = 1.0,
                dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """out[r] = alpha * a[r] @ b[g(r)]^T (fp32 accumulation): g(r) is the group of row r, so with
    activations in expert order each row meets its expert's weights; rows of dropped slots give
    zeros.  b has as many groups as a, each of b.group_rows outputs."""
    kind = TYPES.get(dtype)
    if kind is None:
        raise TypeError("dtype must be float16 or bfloat16")
    if a.device != b.device:
        raise ValueError("a and b are on different devices")
    out = _out(out, (a.rows, b.group_rows), dtype, a.device, "out")
    _call("fp4_gemm_tn", out, stream, out.data_ptr(), kind, a._ref, b._ref, alpha)
    return out


def fp4_get_device_error(stream=None) -> tuple[int, int]:
    """(status, raw word) of the stream's error word of fp4_gemm_tn; synchronises the stream."""
    raw = ctypes.c_uint32(0)
    rc = LIB.fp4_get_device_error(_b._stream_handle(stream), ctypes.byref(raw))
    return rc, int(raw.value)


def moe_sort(ids: torch.Tensor, experts: int, stream=None) -> Routing:
    """Slots sorted by expert.  ids: tokens x top_k int32; a number outside [0, experts) drops
    its slot.  The order within an expert is the slots' own."""
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 2 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 2-D CUDA tensor (tokens x top_k)")
    experts = int(experts)
    if not 1 <= experts <= MAX_EXPERTS or not 1 <= ids.shape[1] <= MAX_TOP_K:
        raise ValueError(f"1 to {MAX_EXPERTS} experts and 1 to {MAX_TOP_K} slots are supported")
    r = Routing._empty(ids, experts)
    c = r._c
    _call("moe_sort", ids, stream, c.offsets, c.rows, c.pairs, c.ids, r.tokens, r.top_k, experts)
    return r


def _by_token(x: torch.Tensor, routing: Routing, what: str) -> int:
    kind = _matrix(x, what)
    if x.shape[0] != routing.tokens or x.device != routing.device:
        raise ValueError(f"{what} must have the routing's {routing.tokens} rows, on its device")
    return kind


def _by_slot(y: torch.Tensor, routing: Routing, what: str) -> int:
    kind = _matrix(y, what)
    if y.shape[0] != routing.slots or not y.is_contiguous() or y.device != routing.device:
        raise ValueError(f"{what} must be contiguous with the routing's {routing.slots} rows, "
                         "on its device")
    return kind


def _weights(weights: torch.Tensor, routing: Routing) -> None:
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if weights.shape != routing.ids.shape or not weights.is_contiguous() \
            or weights.device != routing.device:
        raise ValueError("weights must be contiguous, of the routing's tokens x top_k, "
                         "on its device")


def moe_dispatch(x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """x's rows (a row per token) in expert order, a row per slot; zeros for dropped slots."""
    kind = _by_token(x, routing, "x")
    hidden = x.shape[1]
    out = _out(out, (routing.slots, hidden), x.dtype, x.device, "out")
    _call("moe_dispatch", x, stream, out.data_ptr(), x.data_ptr(), _row_stride(x, hidden), hidden,
          kind, routing._ref)
    return out


def moe_dispatch_backward(grad_y: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """moe_dispatch's gradient: each token's sum over its kept slots."""
    kind = _by_slot(grad_y, routing, "grad_y")
    hidden = grad_y.shape[1]
    out = _out(out, (routing.tokens, hidden), grad_y.dtype, grad_y.device, "out")
    _call("moe_dispatch_backward", out, stream, out.data_ptr(), grad_y.data_ptr(), hidden, kind,
          routing._ref)
    return out


def moe_combine(y: torch.Tensor, routing: Routing, weights: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's weighted sum of its kept slots' rows of y.  weights: tokens x top_k float32."""
    kind = _by_slot(y, routing, "y")
    _weights(weights, routing)
    hidden = y.shape[1]
    out = _out(out, (routing.tokens, hidden), y.dtype, y.device, "out")
    _call("moe_combine", out, stream, out.data_ptr(), y.data_ptr(), weights.data_ptr(), hidden,
          kind, routing._ref)
    return out


def moe_combine_backward(grad_out: torch.Tensor, y: torch.Tensor, routing: Routing,
                         weights: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """moe_combine's gradients: (of y, of weights); zeros for dropped slots."""
    kind = _by_slot(y, routing, "y")
    if _by_token(grad_out, routing, "grad_out") != kind or grad_out.shape[1] != y.shape[1] \
            or not grad_out.is_contiguous():
        raise ValueError("grad_out must be contiguous, of y's type and width")
    _weights(weights, routing)
    grad_y = torch.empty_like(y)
    grad_w = torch.empty_like(weights)
    _call("moe_combine_backward", y, stream, grad_y.data_ptr(), grad_w.data_ptr(),
          grad_out.data_ptr(), y.data_ptr(), weights.data_ptr(), y.shape[1], kind, routing._ref)
    return grad_y, grad_w
