"""Outputs that overlap the weights or the routing's arrays are refused on the host, as those that
overlap a matrix are (no GPU needed: addresses are only compared)."""
import ctypes

import pytest

from test_experts_abi import P, ex, matrix, quantize, routing  # noqa: F401 (ex: the fixture)

E = 1
SLOTS = 4 * 20        # bytes of a routing's rows, ids or weights: 10 tokens x 2
OFFSETS = 4 * 5
OFF, ROWS = P[4], P[5]


def inside(first, size):
    """Addresses whose range begins in [first, first + size), at either end of it."""
    return [first, first + size - 4]


def arrays():
    return inside(OFF, OFFSETS) + inside(ROWS, SLOTS)


def test_row_movers(ex):  # noqa: F811
    r, L = ctypes.byref(routing(ex)), ex.LIB
    for at in arrays():
        assert L.moe_dispatch(at, P[1], 64, 64, 0, r, None) == E
        assert L.moe_dispatch_backward(at, P[1], 64, 0, r, None) == E
        assert L.moe_combine(at, P[1], P[2], 64, 0, r, None) == E
        assert L.moe_combine_backward(at, P[3], P[0], P[1], P[2], 64, 0, r, None) == E
        assert L.moe_combine_backward(P[3], at, P[0], P[1], P[2], 64, 0, r, None) == E
        assert L.moe_combine_backward(0, at, P[0], P[1], P[2], 64, 0, r, None) == E
        assert L.moe_pairs(at, r, None) == E


def test_weights_and_their_gradient(ex):  # noqa: F811
    r, L = ctypes.byref(routing(ex)), ex.LIB
    for at in inside(P[2], SLOTS):                    # P[2]: the weights
        assert L.moe_combine(at, P[1], P[2], 64, 0, r, None) == E
        assert L.moe_combine_backward(at, P[3], P[0], P[1], P[2], 64, 0, r, None) == E
        assert L.moe_combine_backward(P[3], at, P[0], P[1], P[2], 64, 0, r, None) == E
    rows = 10 * 64 * 2
    for at in inside(P[0], rows) + inside(P[1], 2 * rows) + inside(P[3], 2 * rows):
        # the weights' gradient in the output's, in the rows, in the rows' gradient
        assert L.moe_combine_backward(P[3], at, P[0], P[1], P[2], 64, 0, r, None) == E


def test_quantise_and_product(ex):  # noqa: F811
    r = routing(ex)
    by = dict(rows=20, groups=4, offsets=OFF, group_rows=0)
    for at in (OFF, ROWS, ROWS + 64):
        assert quantize(ex, matrix(ex, codes=at, **by), r=r) == E
        assert quantize(ex, matrix(ex, scales=at, **by), r=r) == E
    a = matrix(ex, **by)
    b = matrix(ex, rows=4 * 32, groups=4, codes=P[3], scales=P[6])
    for at in inside(OFF, OFFSETS):
        assert ex.LIB.fp4_gemm_tn(at, 0, ctypes.byref(a), ctypes.byref(b), 1.0, None) == E
        assert ex.LIB.fp4_dequantize(at, 0, ctypes.byref(a), None) == E


@pytest.mark.parametrize("call", ["dispatch", "combine", "backward", "quantize", "gemm"])
def test_apart_is_not_refused(ex, call):  # noqa: F811
    """The same calls with everything apart get as far as asking for a device (or run on nothing)."""
    r, L = routing(ex, tokens=0), ex.LIB
    by = dict(rows=0, groups=4, offsets=OFF, group_rows=0)
    b = matrix(ex, rows=4 * 32, groups=4, codes=P[3], scales=P[6])
    assert {"dispatch": lambda: L.moe_dispatch(P[0], P[1], 64, 64, 0, ctypes.byref(r), None),
            "combine": lambda: L.moe_combine(P[0], P[1], P[2], 64, 0, ctypes.byref(r), None),
            "backward": lambda: L.moe_combine_backward(P[3], P[6], P[0], P[1], P[2], 64, 0,
                                                       ctypes.byref(r), None),
            "quantize": lambda: quantize(ex, matrix(ex, **by), r=r),
            "gemm": lambda: L.fp4_gemm_tn(P[2], 0, ctypes.byref(matrix(ex, **by)), ctypes.byref(b),
                                          1.0, None)}[call]() == 0
