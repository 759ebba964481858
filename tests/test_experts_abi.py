"""Checks of include/moe_fp4.h that need no GPU: what it declares is exported,
and bad arguments are refused on the host before the device is touched."""
import ctypes
import os
import re

import pytest
import torch

from conftest import cuda_available

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_fp4.h")
P = [0x10000000 * (i + 1) for i in range(8)]   # never dereferenced


class RoutingC(ctypes.Structure):          # moe_routing_t
    _fields_ = [("tokens", ctypes.c_int64), ("top_k", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("ids", ctypes.c_void_p)]


class MatrixC(ctypes.Structure):           # fp4_matrix_t
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("format", ctypes.c_int32),
                ("exponent", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("group_rows", ctypes.c_int64),
                ("offsets", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def ex():
    """The binding, with the library's C functions declared as `LIB`."""
    from multistage_smem_pipeline_gb300 import build
    build.build()
    from multistage_smem_pipeline_gb300 import experts
    lib = ctypes.CDLL(build.LIB)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    pr, pm, pu = (ctypes.POINTER(t) for t in (RoutingC, MatrixC, ctypes.c_uint64))
    for name, args in {
            "fp4_code_bytes": [i64, i64, pu],
            "fp4_scale_bytes": [i64, i64, i32, i32, i32, pu],
            "fp4_quantize": [pm, vp, i64, i32, pr, vp],
            "fp4_dequantize": [vp, i32, pm, vp],
            "fp4_gemm_tn": [vp, i32, pm, pm, ctypes.c_float, vp],
            "fp4_gemm_tn_ex": [vp, i32, pm, pm, ctypes.c_float, ctypes.c_uint64, i32, vp],
            "moe_sort": [vp, vp, vp, i64, i32, i32, vp],
            "moe_pairs": [vp, pr, vp],
            "moe_dispatch": [vp, vp, i64, i64, i32, pr, vp],
            "moe_dispatch_backward": [vp, vp, i64, i32, pr, vp],
            "moe_combine": [vp, vp, vp, i64, i32, pr, vp],
            "moe_combine_backward": [vp, vp, vp, vp, vp, i64, i32, pr, vp]}.items():
        getattr(lib, name).argtypes = args
    experts.LIB = lib
    return experts


def test_header_and_library_agree(ex):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^int\s+((?:moe|fp4)_[a-z0-9_]+)\s*\(", text, flags=re.M))
    assert names == set(ex.EXPORTED)
    for n in names:
        assert hasattr(ex.LIB, n)


def test_package_exports(ex):
    import multistage_smem_pipeline_gb300 as pkg
    for n in ("Fp4Matrix", "Routing", "fp4_quantize", "fp4_gemm_tn", "moe_sort", "moe_combine"):
        assert getattr(pkg, n) is getattr(ex, n) and n in pkg.__all__


def routing(ex, tokens=10, top_k=2, experts=4, **kw):
    v = dict(offsets=P[4], rows=P[5], ids=P[7])
    v.update(kw)
    return RoutingC(tokens, top_k, experts, v["offsets"], v["rows"], v["ids"])


def matrix(ex, rows=64, cols=256, format=0, exponent=0, groups=1, group_rows=None, offsets=None,
           codes=P[0], scales=P[1], reserved=0):
    return MatrixC(codes, scales, rows, cols, format, exponent, groups, reserved,
                       rows // max(groups, 1) if group_rows is None else group_rows, offsets)


def test_sizes(ex):
    # 300 rows are 3 tiles; 1000 columns are 4 runs of 256: 4 (nv) or 2 (mx) chunks each
    assert ex.fp4_scale_bytes(300, 1000, "nvfp4") == 3 * 4 * 4 * 512
    assert ex.fp4_scale_bytes(300, 1000, "mxfp4") == 3 * 4 * 2 * 512
    assert ex.fp4_scale_bytes(300, 1000, "nvfp4", groups=100) == 100 * 16 * 512
    # by offsets: 300 / 128 tiles and one more for every group
    assert ex.fp4_scale_bytes(300, 256, "mxfp4", groups=7, by_offsets=True) == (2 + 7) * 2 * 512
    assert ex.fp4_scale_bytes(0, 0) == 0
    n = ctypes.c_uint64(0)
    assert ex.LIB.fp4_code_bytes(3, 33, ctypes.byref(n)) == 0 and n.value == 3 * 32
    E = 1
    assert ex.LIB.fp4_code_bytes(3, 33, None) == E
    for args in [(-1, 8, 0, 1, 0), (8, 2**23 + 1, 0, 1, 0), (8, 8, 2, 1, 0), (8, 8, 0, 0, 0),
                 (9, 8, 0, 2, 0), (8, 8, 0, 1025, 1), (8, 8, 0, 1, 2), (2**31, 8, 0, 1, 0)]:
        assert ex.LIB.fp4_scale_bytes(*args, ctypes.byref(n)) == E, args
    for args in [(-1, 2, 4), (10, 0, 4), (10, 65, 4), (10, 2, 0), (10, 2, 1025), (2**31, 1, 4)]:
        assert ex.LIB.moe_sort(P[0], P[1], P[3], *args, None) == E, args


def quantize(ex, m, x=P[2], ldx=256, type=0, r=None):
    return ex.LIB.fp4_quantize(ctypes.byref(m), x, ldx, type,
                               ctypes.byref(r) if r is not None else None, None)


def test_quantize_refusals(ex):
    E, MIS = 1, 2
    for m in [matrix(ex, rows=-1), matrix(ex, cols=-1), matrix(ex, format=2),
              matrix(ex, exponent=101), matrix(ex, exponent=-101),
              matrix(ex, format=1, exponent=1), matrix(ex, groups=0), matrix(ex, group_rows=63),
              matrix(ex, groups=3), matrix(ex, reserved=1), matrix(ex, codes=0),
              matrix(ex, scales=0)]:
        assert quantize(ex, m) == E
    m = matrix(ex)
    assert quantize(ex, m, x=0) == E
    assert quantize(ex, m, ldx=255) == E
    assert quantize(ex, m, type=2) == E
    assert quantize(ex, m, x=P[2] + 1) == MIS
    assert quantize(ex, matrix(ex, codes=P[0] + 8)) == MIS
    assert quantize(ex, matrix(ex, scales=P[1] + 4)) == MIS
    assert quantize(ex, m, x=P[0] + 64) == E                      # x overlaps the codes
    assert quantize(ex, m, x=P[1] + 16) == E                      # ... the scales
    assert quantize(ex, matrix(ex, scales=P[0] + 16)) == E        # codes overlap scales
    assert quantize(ex, matrix(ex, offsets=P[3])) == E            # offsets, but no routing
    r = routing(ex)
    by = dict(rows=20, groups=4, offsets=P[4], group_rows=0)
    assert quantize(ex, matrix(ex, **{**by, "rows": 21}), r=r) == E
    assert quantize(ex, matrix(ex, **{**by, "groups": 3}), r=r) == E
    assert quantize(ex, matrix(ex, **{**by, "offsets": P[3]}), r=r) == E
    assert quantize(ex, matrix(ex, **by), r=routing(ex, top_k=0)) == E
    assert quantize(ex, matrix(ex, **by), r=routing(ex, rows=0)) == E
    assert quantize(ex, matrix(ex, **by), r=routing(ex, ids=P[7] + 2)) == MIS
    # nothing to do: no device, no pointers
    assert quantize(ex, matrix(ex, rows=0, codes=0, scales=0), x=0) == 0


def test_dequantize_refusals(ex):
    E, MIS = 1, 2
    f = ex.LIB.fp4_dequantize
    m = matrix(ex)
    assert f(0, 0, ctypes.byref(m), None) == E
    assert f(P[2], 3, ctypes.byref(m), None) == E
    assert f(P[2] + 1, 0, ctypes.byref(m), None) == MIS
    assert f(P[0] - 16, 0, ctypes.byref(m), None) == E
    assert f(P[2], 0, None, None) == E
    assert f(0, 0, ctypes.byref(matrix(ex, cols=0, codes=0, scales=0)), None) == 0


def gemm(ex, a, b, d=P[2], type=0, alpha=1.0):
    return ex.LIB.fp4_gemm_tn(d, type, ctypes.byref(a), ctypes.byref(b), alpha, None)


def test_gemm_refusals(ex):
    E, MIS = 1, 2
    a, b = matrix(ex), matrix(ex, rows=128, codes=P[4], scales=P[5])
    assert gemm(ex, a, b, d=0) == E
    assert gemm(ex, a, b, d=P[2] + 1) == MIS
    assert gemm(ex, a, b, type=2) == E
    assert gemm(ex, a, b, alpha=float("nan")) == E
    assert gemm(ex, a, b, alpha=float("inf")) == E
    for inject in (-1, 2):
        assert ex.LIB.fp4_gemm_tn_ex(P[2], 0, ctypes.byref(a), ctypes.byref(b), 1.0, 0, inject,
                                     None) == E
    assert gemm(ex, a, b, d=P[0]) == E and gemm(ex, a, b, d=P[5] + 32) == E      # overlaps
    for other in [dict(cols=255), dict(format=1), dict(groups=2, rows=128),
                  dict(offsets=P[6], rows=128), dict(codes=0)]:
        assert gemm(ex, a, matrix(ex, **{**dict(codes=P[4], scales=P[5]), **other})) == E, other
    assert gemm(ex, matrix(ex, rows=0, codes=0, scales=0), b, d=0) == 0
    assert ex.LIB.fp4_gemm_tn(P[2], 0, None, ctypes.byref(b), 1.0, None) == E


def test_routing_refusals(ex):
    E, MIS, L = 1, 2, ex.LIB
    r = ctypes.byref(routing(ex))
    assert L.moe_sort(0, P[1], P[3], 10, 2, 4, None) == E
    assert L.moe_sort(P[0], 0, P[3], 10, 2, 4, None) == E
    assert L.moe_sort(P[0] + 2, P[1], P[3], 10, 2, 4, None) == MIS
    assert L.moe_sort(P[0], P[1], P[3], 10, 2, 1025, None) == E
    assert L.moe_sort(P[0], P[1], P[1] + 16, 10, 2, 4, None) == E
    assert L.moe_sort(P[0], P[0] + 16, P[3], 10, 2, 4, None) == E
    assert L.moe_pairs(0, r, None) == E and L.moe_pairs(P[5], r, None) == E
    assert L.moe_pairs(P[0] + 1, r, None) == MIS and L.moe_pairs(P[0], None, None) == E
    assert L.moe_dispatch(0, P[1], 64, 64, 0, r, None) == E
    assert L.moe_dispatch(P[0], P[1], 63, 64, 0, r, None) == E
    assert L.moe_dispatch(P[0], P[1], 64, -1, 0, r, None) == E
    assert L.moe_dispatch(P[0], P[1], 64, 64, 2, r, None) == E
    assert L.moe_dispatch(P[0] + 1, P[1], 64, 64, 0, r, None) == MIS
    assert L.moe_dispatch(P[0], P[0] + 128, 64, 64, 0, r, None) == E
    assert L.moe_dispatch(P[0], P[1], 64, 64, 0, None, None) == E
    assert L.moe_dispatch_backward(P[0], P[0], 64, 0, r, None) == E
    assert L.moe_combine(P[0], P[1], 0, 64, 0, r, None) == E
    assert L.moe_combine(P[0], P[1], P[2] + 2, 64, 0, r, None) == MIS
    assert L.moe_combine(P[0], P[0] + 2, P[2], 64, 0, r, None) == E
    assert L.moe_combine_backward(P[0], P[1], P[2], P[0] + 64, P[3], 64, 0, r, None) == E
    assert L.moe_combine_backward(P[0], P[1], P[2], P[3], 0, 64, 0, r, None) == E
    assert L.moe_combine_backward(P[0], P[1], 0, P[3], P[2], 64, 0, r, None) == E
    empty = ctypes.byref(routing(ex, tokens=0, offsets=0, rows=0, ids=0))
    assert L.moe_dispatch(0, 0, 64, 64, 0, empty, None) == 0
    assert L.moe_combine(0, 0, 0, 64, 0, empty, None) == 0
    assert L.moe_combine_backward(0, 0, 0, 0, 0, 64, 0, empty, None) == 0
    assert L.moe_combine_backward(0, 0, P[2], P[3], 0, 64, 0, r, None) == 0   # nothing asked for


@pytest.mark.skipif(cuda_available(), reason="checks the no-device error path")
def test_valid_calls_without_a_device_report_it(ex):
    bad = (3, 6)
    r = routing(ex)
    a, b = matrix(ex), matrix(ex, rows=128, codes=P[4], scales=P[5])
    assert quantize(ex, a) in bad
    assert gemm(ex, a, b) in bad
    assert ex.LIB.moe_sort(P[0], P[1], P[3], 10, 2, 4, None) in bad
    assert ex.LIB.moe_combine(P[0], P[1], P[2], 64, 0, ctypes.byref(r), None) in bad


def test_python_refusals_on_cpu_tensors(ex):
    x = torch.zeros(4, 32, dtype=torch.float16)
    with pytest.raises(ValueError):
        ex.fp4_quantize(x)
    with pytest.raises(TypeError):
        ex.fp4_quantize(x.float())
    with pytest.raises(ValueError):
        ex.Fp4Matrix(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8),
                     cols=32)
    with pytest.raises(ValueError):
        ex.Fp4Matrix(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8),
                     cols=32, format="fp4")
    with pytest.raises(ValueError):
        ex.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        ex.moe_sort(torch.zeros(4, 2), 4)


def test_gemm_refuses_a_scale_beyond_fp32(ex):
    """alpha 2^(exponents) is one fp32 factor: infinite, it would turn sums of zero into NaN."""
    E = 1
    none = dict(rows=0, codes=0, scales=0)      # valid, and nothing to launch
    for ea, eb, alpha, want in [(100, 100, 1.0, E), (100, 28, 1.0, E), (100, 27, 1.0, 0),
                                (100, 100, 2.0 ** -80, 0), (100, -100, 2.0 ** 127, 0),
                                (60, 0, -2.0 ** 68, E), (-100, -100, 1.0, 0)]:
        a, b = matrix(ex, exponent=ea, **none), matrix(ex, rows=128, exponent=eb, codes=P[4], scales=P[5])
        assert gemm(ex, a, b, alpha=alpha) == want, (ea, eb, alpha)


def test_rows_that_overlap_are_refused(ex):
    """The kernels step by the row's width at least: an expanded row would be read past its end."""
    row = torch.zeros(1, 32, dtype=torch.float16)
    windows = torch.zeros(64, dtype=torch.float16).unfold(0, 32, 8)
    for x in (row.expand(4, 32), windows, torch.zeros(1, 1, dtype=torch.float16).expand(4, 1)):
        with pytest.raises(ValueError, match="overlap"):
            ex.fp4_quantize(x)
