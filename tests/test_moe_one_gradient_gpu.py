"""moe_combine_backward through its C entry with one of the two gradients left out (GPU): the other
has the bits that it has when both are asked for, and nothing else is written."""
import ctypes

import pytest
import torch

from test_moe_gpu import make, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


class RoutingC(ctypes.Structure):          # moe_routing_t
    _fields_ = [("tokens", ctypes.c_int64), ("top_k", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("ids", ctypes.c_void_p)]


# aligned rows, unaligned ones, and unaligned ones with slots enough for the form of many
@pytest.mark.parametrize("tokens,top_k,hidden,first", [(33, 3, 128, 0), (33, 3, 131, 0), (33, 3, 128, 1),
                                                       (1300, 8, 131, 0), (1300, 8, 7, 3), (5, 2, 1, 0)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_one_gradient(lib, dtype, tokens, top_k, hidden, first):
    from multistage_smem_pipeline_gb300 import build
    call = ctypes.CDLL(build.LIB).moe_combine_backward
    vp = ctypes.c_void_p
    call.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(RoutingC), vp]
    experts = 7
    ids = to_gpu(make(tokens, tokens, top_k, experts, 0.1), torch.int32)
    r = lib.moe_sort(ids, experts)
    slots = tokens * top_k

    def rows(n, fill=None):
        """n rows that start `first` elements past a 16-byte boundary, and what surrounds them."""
        flat = torch.full((n * hidden + first + 8,), 7.25, dtype=dtype, device="cuda")
        part = flat[first:first + n * hidden].view(n, hidden)
        if fill is not None:
            part.copy_(fill)
        return flat, part

    _, grad = rows(tokens, torch.randn(tokens, hidden, device="cuda"))
    _, y = rows(slots, torch.randn(slots, hidden, device="cuda"))
    w = torch.rand(tokens, top_k, device="cuda")
    both_y, both_w = lib.moe_combine_backward(grad, y, r, w)
    c = RoutingC(tokens, top_k, experts, r.offsets.data_ptr(), r.rows.data_ptr(), ids.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    kind = 0 if dtype == torch.float16 else 1

    flat, only_y = rows(slots)
    assert call(only_y.data_ptr(), None, grad.data_ptr(), y.data_ptr(), w.data_ptr(), hidden, kind,
                ctypes.byref(c), stream) == 0
    assert torch.equal(only_y, both_y)
    assert (flat[:first] == 7.25).all() and (flat[first + slots * hidden:] == 7.25).all()

    only_w = torch.full((slots + 2,), 7.25, device="cuda")
    assert call(None, only_w[1:].data_ptr(), grad.data_ptr(), y.data_ptr(), w.data_ptr(), hidden, kind,
                ctypes.byref(c), stream) == 0
    assert only_w[0] == 7.25 and only_w[-1] == 7.25
    # the windows begin elsewhere without the rows' gradient: fp32 sums in another order
    bound = torch.zeros(slots, dtype=torch.float64, device="cuda")
    g = grad.double().repeat_interleave(top_k, dim=0)
    live = (r.rows.flatten() < r.offsets[-1])
    bound[live] = (g.abs() * y[r.rows.flatten().long()].double().abs()).sum(1)[live]
    err = (only_w[1:-1].double() - both_w.flatten().double()).abs()
    assert (err <= 2 * (hidden + 1) * 2.0 ** -24 * bound).all()
    assert not only_w[1:-1][~live].any()
