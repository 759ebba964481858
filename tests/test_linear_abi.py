"""Checks of include/linear.h and of its binding that need no GPU: what it declares is exported, bad
arguments are refused on the host before the device is touched, workspaces, and the choice of forms."""
import ctypes
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from conftest import cuda_available

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "linear.h")
P = [0x1000000000 * (i + 1) for i in range(12)]   # never dereferenced
E, MIS = 1, 2


class RoutingC(ctypes.Structure):          # moe_routing_t
    _fields_ = [("tokens", ctypes.c_int64), ("top_k", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("ids", ctypes.c_void_p)]


class LayerC(ctypes.Structure):            # linear_t
    _fields_ = [("rows", ctypes.c_int64), ("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("type", ctypes.c_int32), ("activation", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("routing", ctypes.POINTER(RoutingC))]


class OptionsC(ctypes.Structure):          # linear_options_t
    _fields_ = [("cta_pair", ctypes.c_int), ("tile", ctypes.c_int), ("split_k", ctypes.c_int),
                ("inject", ctypes.c_int), ("timeout_ns", ctypes.c_uint64)]


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import build
    build.build()
    from multistage_smem_pipeline_gb300 import experts
    lib = ctypes.CDLL(build.LIB)
    vp, i64, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64
    pl, po, pu = ctypes.POINTER(LayerC), ctypes.POINTER(OptionsC), ctypes.POINTER(u64)
    lib.linear_forward.argtypes = [vp, vp, pl, vp, vp, i64, vp, u64, po, vp]
    lib.linear_backward.argtypes = [vp, vp, vp, pl, vp, i64, vp, vp, u64, po, vp]
    lib.linear_forward_workspace.argtypes = [pl, po, pu]
    lib.linear_backward_workspace.argtypes = [vp, vp, vp, pl, vp, i64, pu]
    experts.LINEAR = lib
    return experts


def layer(rows=100, in_=64, out=80, type=0, activation=0, x=P[0], ldx=64, w=P[1], ldw=64, routing=None):
    return LayerC(rows, in_, out, type, activation, x, ldx, w, ldw, ctypes.pointer(routing) if routing else None)


def routing(tokens=50, top_k=2, experts=4, offsets=P[8], rows=P[9], ids=P[10]):
    return RoutingC(tokens, top_k, experts, offsets, rows, ids)


def forward(ex, l, out=P[2], preact=None, bias=None, residual=None, ldr=80, ws=None, ws_bytes=0, opt=None):
    return ex.LINEAR.linear_forward(out, preact, ctypes.byref(l) if l else None, bias, residual, ldr, ws, ws_bytes,
                                    ctypes.byref(opt) if opt else None, None)


def backward(ex, l, gx=P[2], gw=P[3], gb=None, grad=P[4], ldg=80, preact=None, ws=P[5], ws_bytes=1 << 30, opt=None):
    return ex.LINEAR.linear_backward(gx, gw, gb, ctypes.byref(l) if l else None, grad, ldg, preact, ws, ws_bytes,
                                     ctypes.byref(opt) if opt else None, None)


def test_header_and_library_agree(ex):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^int\s+(linear_[a-z0-9_]+)\s*\(", text, flags=re.M))
    assert names == set(ex.EXPORTED_LINEAR)
    for n in names:
        assert hasattr(ex.LINEAR, n)


def test_package_exports(ex):
    import multistage_smem_pipeline_gb300 as pkg
    for n in ("linear", "linear_backward", "moe_linear", "moe_linear_backward", "linear_query_config",
              "linear_get_device_error"):
        assert getattr(pkg, n) is getattr(ex, n) and n in pkg.__all__


BAD_LAYERS = [dict(rows=-1), dict(rows=2 ** 30 + 1), dict(in_=-1), dict(in_=2 ** 23 + 1), dict(out=-1),
              dict(out=2 ** 23 + 1), dict(type=2), dict(type=-1), dict(activation=5), dict(activation=-1)]


def test_forward_refusals(ex):
    assert forward(ex, None) == E
    for bad in BAD_LAYERS:
        assert forward(ex, layer(**bad)) == E, bad
    for bad in (dict(x=0), dict(w=0), dict(ldx=63), dict(ldw=63), dict(ldx=-64), dict(ldw=1 << 60)):
        assert forward(ex, layer(**bad)) == E, bad
    assert forward(ex, layer(), out=0) == E
    assert forward(ex, layer(x=P[0] + 1)) == MIS and forward(ex, layer(w=P[1] + 1)) == MIS
    assert forward(ex, layer(), out=P[2] + 1) == MIS and forward(ex, layer(), bias=P[3] + 1) == MIS
    assert forward(ex, layer(), preact=P[3] + 1) == MIS
    assert forward(ex, layer(), residual=P[3] + 1) == MIS
    assert forward(ex, layer(), residual=P[3], ldr=79) == E
    for overlap in (dict(out=P[0] + 64), dict(out=P[1] + 16), dict(preact=P[2] + 32), dict(preact=P[0]),
                    dict(bias=P[2] + 2), dict(residual=P[2]), dict(residual=P[3], preact=P[3] + 160)):
        assert forward(ex, layer(), **overlap) == E, overlap


def test_options_refused(ex):
    for bad in (dict(tile=48), dict(tile=64, split_k=3), dict(tile=64, split_k=0), dict(cta_pair=1, tile=128, split_k=1),
                dict(cta_pair=1, tile=256, split_k=2), dict(cta_pair=2, tile=256, split_k=1), dict(split_k=2),
                dict(cta_pair=1), dict(inject=2), dict(inject=-1), dict(tile=16, split_k=1)):
        o = OptionsC(**bad)
        assert forward(ex, layer(), opt=o) == E, bad
        assert backward(ex, layer(), opt=o) == E, bad


def test_routed_refusals(ex):
    r = routing()
    assert forward(ex, layer(routing=r, rows=99)) == E
    assert forward(ex, layer(routing=r), residual=P[3]) == E                 # rows in expert order have none
    assert forward(ex, layer(routing=r), out=P[8]) == E                      # over the offsets
    assert forward(ex, layer(routing=r), preact=P[9] + 8) == E
    assert backward(ex, layer(routing=r), gb=P[8] + 4) == E
    assert backward(ex, layer(routing=r), ws=P[8] & ~15, gb=P[6]) == E       # the workspace, over the offsets
    assert forward(ex, layer(routing=routing(experts=0))) == E
    assert forward(ex, layer(routing=routing(experts=1025))) == E
    assert forward(ex, layer(routing=routing(offsets=0))) == E
    assert forward(ex, layer(routing=routing(offsets=P[8] + 2))) == MIS
    assert forward(ex, layer(routing=routing(tokens=2 ** 30))) == E
    assert forward(ex, layer(routing=routing(experts=1024), out=2 ** 22, ldw=64)) == E   # experts x out


def test_backward_refusals(ex):
    assert backward(ex, None) == E
    for bad in BAD_LAYERS:
        assert backward(ex, layer(**bad)) == E, bad
    assert backward(ex, layer(), grad=0) == E and backward(ex, layer(), grad=P[4] + 1) == MIS
    assert backward(ex, layer(), ldg=79) == E
    assert backward(ex, layer(activation=2)) == E                            # no preact
    assert backward(ex, layer(activation=2), preact=P[6] + 1) == MIS
    assert backward(ex, layer(x=0)) == E and backward(ex, layer(w=0)) == E
    assert backward(ex, layer(x=P[0] + 1)) == MIS and backward(ex, layer(w=P[1] + 1)) == MIS
    for n in ("gx", "gw", "gb"):
        assert backward(ex, layer(), **{n: P[7] + 1}) == MIS, n
    for overlap in (dict(gx=P[3] + 16), dict(gx=P[4]), dict(gw=P[0] + 2), dict(gb=P[3] + 2), dict(gx=P[1])):
        assert backward(ex, layer(), **overlap) == E, overlap
    assert backward(ex, layer(activation=2), preact=P[3]) == E               # over grad_w
    assert backward(ex, layer(), gb=P[6], ws=0) == E and backward(ex, layer(), gb=P[6], ws_bytes=16) == E
    assert backward(ex, layer(), gb=P[6], ws=P[5] + 8) == MIS
    assert backward(ex, layer(), gb=P[6], ws=P[4] + 160) == E
    # a gradient that is not asked for needs nothing of its own
    assert backward(ex, layer(x=0, w=0), gx=None, gw=None) == 0
    assert backward(ex, layer(x=0, w=0, rows=0), gx=None, gw=None, grad=0) == 0


def test_nothing_to_do(ex):
    assert forward(ex, layer(rows=0, x=0), out=0) == 0
    assert forward(ex, layer(out=0, w=0), out=0) == 0
    r = routing(tokens=0, offsets=0, rows=0, ids=0)
    assert forward(ex, layer(rows=0, routing=r, x=0), out=0) == 0
    assert backward(ex, layer(rows=0, in_=0, x=0), grad=0, gw=None) == 0


def test_workspaces(ex):
    n = ctypes.c_uint64(7)

    def fwd(opt=None, **kw):
        assert ex.LINEAR.linear_forward_workspace(ctypes.byref(layer(**kw)), ctypes.byref(opt) if opt else None,
                                                  ctypes.byref(n)) == 0
        return n.value

    def bwd(gx=P[2], gw=P[3], gb=P[6], grad=P[4], ldg=80, **kw):
        assert ex.LINEAR.linear_backward_workspace(gx, gw, gb, ctypes.byref(layer(**kw)), grad, ldg, ctypes.byref(n)) == 0
        return n.value

    assert fwd() == 0
    assert fwd(x=P[0] + 2) == 100 * 64 * 2                 # copied to 16-byte rows
    assert fwd(ldx=65) == 100 * 64 * 2 and fwd(ldw=67) == 80 * 64 * 2
    assert fwd(in_=63, ldx=63, ldw=63) == (100 + 80) * 64 * 2
    assert fwd(rows=3, in_=63, ldx=63, ldw=63) == 0        # few rows are read as they are
    assert fwd(opt=OptionsC(tile=64, split_k=1), rows=3, in_=63, ldx=63, ldw=63) == (3 + 80) * 64 * 2
    assert fwd(rows=0, x=P[0] + 2) == 0
    assert bwd(gb=None) == 0                               # dz is grad_out
    assert bwd(gb=None, ldg=81) == 100 * 80 * 2
    assert bwd(gb=None, activation=1) == 100 * 80 * 2
    assert bwd(gx=None, gw=None, gb=None, activation=1) == 0
    assert bwd() == (100 // 32 + 1) * 80 * 4               # strips of 32 rows
    assert bwd(gw=None, gb=None, w=P[1] + 2) == 80 * 64 * 2 and bwd(gw=None, gb=None, x=P[0] + 2) == 0
    assert ex.LINEAR.linear_forward_workspace(ctypes.byref(layer()), None, None) == E
    assert ex.LINEAR.linear_forward_workspace(None, None, ctypes.byref(n)) == E
    assert ex.LINEAR.linear_forward_workspace(ctypes.byref(layer()), ctypes.byref(OptionsC(tile=5)), ctypes.byref(n)) == E
    assert ex.LINEAR.linear_backward_workspace(P[2], None, None, ctypes.byref(layer(type=3)), P[4], 80, ctypes.byref(n)) == E


def test_forms(ex):
    """Every form is some product's, and every size has one."""
    seen = set()
    for rows in (1, 2, 4, 7, 30, 100, 300, 1000, 8192, 100000):
        for out in (1, 60, 500, 2000, 14336):
            for hidden in (1, 64, 1000, 8192):
                for experts in (0, 1, 16, 64):
                    for product in ("forward", "grad_x", "grad_w"):
                        c = ex.linear_query_config(product, rows, hidden, out, experts)
                        seen.add((product, c["cta_pair"], c["tile"]))
                        assert c["ctas"] >= 1 and c["split_k"] in (1, 2, 4, 8)
                        assert c["tile"] > 8 or product == "forward"
                        assert not c["cta_pair"] or (c["tile"] == 256 and c["split_k"] == 1)
                        if c["split_k"] > 1 and c["tile"] > 8:
                            assert c["ctas"] <= 152        # clusters that share sums are there at once
    for product in ("forward", "grad_x", "grad_w"):
        for pair, tile in ((1, 256), (0, 64), (0, 128), (0, 256)):
            assert (product, pair, tile) in seen, (product, pair, tile)
    assert ("grad_w", 0, 32) not in seen and ("forward", 0, 32) in seen
    assert {("forward", 0, r) for r in (1, 2, 4, 8)} <= seen
    assert ex.linear_query_config("forward", 1, 4096, 14336)["tile"] == 1
    assert ex.linear_query_config("forward", 8192, 8192, 8192)["cta_pair"] == 1
    from multistage_smem_pipeline_gb300.binding import GemmError
    for bad in (("sideways", 1, 1, 1), ("forward", 0, 1, 1), ("forward", 1, 0, 1), ("forward", 1, 1, 2 ** 23 + 1),
                ("forward", 2 ** 30 + 1, 1, 1), ("forward", 1, 1, 1, 1025), ("grad_w", 1, 1, 2 ** 22, 1024)):
        with pytest.raises(GemmError):
            ex.linear_query_config(*bad)


@pytest.mark.skipif(cuda_available(), reason="checks the no-device error path")
def test_valid_calls_without_a_device_report_it(ex):
    assert forward(ex, layer()) in (3, 6)
    assert forward(ex, layer(routing=routing())) in (3, 6)
    assert backward(ex, layer(), gb=P[6]) in (3, 6)


# ------------------------------------------------------------------ the binding
def fake(*sizes, dtype=torch.float16, device="cuda:0"):
    with FakeTensorMode():
        return torch.empty(*sizes, dtype=dtype, device=device)


def fake_routing(ex, tokens=10, top_k=2, experts=4, device="cuda:0"):
    def ints(*sizes):
        return fake(*sizes, dtype=torch.int32, device=device)
    return ex.Routing(ints(experts + 1), ints(tokens, top_k), ints(tokens, top_k))


def test_binding_refusals(ex):
    x, w, r = fake(20, 64), fake(80, 64), fake_routing(ex)
    we = fake(4, 80, 64)
    refused = [
        lambda: ex.linear(x[:, :63], w), lambda: ex.linear(x, we), lambda: ex.linear(fake(20, 64, 1), w),
        lambda: ex.linear(x, w, activation="tanh"), lambda: ex.linear(x, w, fake(81)), lambda: ex.linear(x, w, fake(1, 80)),
        lambda: ex.linear(x, w, fake(160)[::2]), lambda: ex.linear(x, w, residual=fake(20, 81)),
        lambda: ex.linear(x, w, residual=fake(19, 80)), lambda: ex.linear(x, w, residual=fake(1, 80).expand(20, 80)),
        lambda: ex.linear(x.t(), w), lambda: ex.linear(x[:1].expand(20, 64), w), lambda: ex.linear(x, w.t()),
        lambda: ex.linear(x, fake(80, 64, device="cuda:1")), lambda: ex.linear(x, w, fake(80, device="cuda:1")),
        lambda: ex.linear(x, w, residual=fake(20, 80, device="cuda:1")), lambda: ex.linear(x, fake(80, 64, dtype=torch.bfloat16)),
        lambda: ex.linear(x, w, fake(80, dtype=torch.float32)), lambda: ex.linear(torch.zeros(4, 64, dtype=torch.float16), w),
        lambda: ex.moe_linear(x, r, w), lambda: ex.moe_linear(x, r, fake(3, 80, 64)), lambda: ex.moe_linear(fake(19, 64), r, we),
        lambda: ex.moe_linear(x, r, we, fake(80)), lambda: ex.moe_linear(x, r, we, fake(4, 81)),
        lambda: ex.moe_linear(x, r, fake(8, 80, 64)[::2]), lambda: ex.moe_linear(x, r, fake(4, 64, 80).transpose(1, 2)),
        lambda: ex.moe_linear(x, fake_routing(ex, device="cuda:1"), we),
        lambda: ex.linear_backward(fake(20, 81), x, w), lambda: ex.linear_backward(fake(19, 80), x, w),
        lambda: ex.linear_backward(fake(20, 80), x[:, :32], w), lambda: ex.linear_backward(fake(20, 80), x, w, activation="silu"),
        lambda: ex.linear_backward(fake(20, 80), x, w, activation="silu", preact=fake(20, 81)),
        lambda: ex.linear_backward(fake(20, 80), x, w, activation="silu", preact=fake(20, 88)[:, :80]),
        lambda: ex.linear_backward(fake(20, 80), x, w, activation="silu", preact=fake(20, 80, dtype=torch.bfloat16)),
        lambda: ex.linear_backward(fake(20, 80), None, w), lambda: ex.linear_backward(fake(20, 80), x, None),
        lambda: ex.linear_backward(fake(1, 80).expand(20, 80), x, w),
        lambda: ex.linear_backward(fake(20, 80), fake(20, 64, device="cuda:1"), w),
        lambda: ex.moe_linear_backward(fake(20, 80), x, r, w), lambda: ex.moe_linear_backward(fake(19, 80), x, r, we),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    for call in (lambda: ex.linear(fake(20, 64, dtype=torch.float32), w), lambda: ex.linear(x, fake(80, 64, dtype=torch.float32)),
                 lambda: ex.linear_backward(fake(20, 80, dtype=torch.float32), x, w)):
        with pytest.raises(TypeError):
            call()
