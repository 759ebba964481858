"""Linear layers through their C entries, every array inside a buffer of its own filled with NaNs (GPU):
what surrounds outputs and a workspace of exactly the reported size stays as it was, every element of
an output is written, and neither what surrounds the inputs nor what the workspace held matters."""
import ctypes

import pytest
import torch

import linear_reference as ref
from test_linear_abi import LayerC, OptionsC, RoutingC
from test_linear_gpu import FEW, FORMS, make, routing_of

pytestmark = pytest.mark.gpu

PATTERN = 0x7fa5          # a NaN of either type, as no kernel makes them
MARGIN = 4096             # elements before and behind
NAMES = ("out", "preact", "grad_x", "grad_w", "grad_bias")


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


@pytest.fixture(scope="module")
def c(lib):
    from multistage_smem_pipeline_gb300 import build
    c = ctypes.CDLL(build.LIB)
    vp, i64, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64
    pl, po, pu = ctypes.POINTER(LayerC), ctypes.POINTER(OptionsC), ctypes.POINTER(u64)
    c.linear_forward.argtypes = [vp, vp, pl, vp, vp, i64, vp, u64, po, vp]
    c.linear_backward.argtypes = [vp, vp, vp, pl, vp, i64, vp, vp, u64, po, vp]
    c.linear_forward_workspace.argtypes = [pl, po, pu]
    c.linear_backward_workspace.argtypes = [vp, vp, vp, pl, vp, i64, pu]
    return c


class Guarded:
    """`count` 16-bit elements, `shift` elements past a 16-byte boundary, with NaNs on both sides and in them."""

    def __init__(self, count, shift=0, values=None):
        self.whole = torch.full((count + shift + 2 * MARGIN,), PATTERN, dtype=torch.int16, device="cuda")
        self.inside = slice(MARGIN + shift, MARGIN + shift + count)
        if values is not None:
            self.whole[self.inside] = values.reshape(-1).view(torch.int16)
        self.before = self.whole.clone()

    @property
    def ptr(self):
        return self.whole.data_ptr() + 2 * self.inside.start

    def values(self, dtype, *sizes):
        return self.whole[self.inside].view(dtype).view(*sizes)

    def check(self, what, written):
        now, before = self.whole, self.before
        assert torch.equal(now[:self.inside.start], before[:self.inside.start]), what + ": written before it"
        assert torch.equal(now[self.inside.stop:], before[self.inside.stop:]), what + ": written behind it"
        if written:
            left = (now[self.inside] == PATTERN).sum().item()
            assert left == 0, f"{what}: {left} elements were not written"
        elif written is not None:
            assert torch.equal(now, before), what + ": an input was written"


def run(lib, c, rows, out, hidden, dtype, shift, form=None, counts=None, dropped=0, activation="gelu", gap=0):
    """Forward and backward; rows of x, w, grad_out and the residual are `gap` elements apart."""
    experts = None if counts is None else len(counts)
    m = make(rows, out, hidden, dtype, experts=experts, seed=61)
    routing, offsets, rc = None, None, None
    if counts is not None:
        routing, offsets = routing_of(lib, counts, dropped)
        rc = RoutingC(rows, 1, experts, routing.offsets.data_ptr(), routing.rows.data_ptr(), routing.ids.data_ptr())
    groups = experts or 1

    def spread(t, cols):
        t = t.reshape(-1, cols)
        wide = torch.full((t.shape[0], cols + gap), PATTERN, dtype=torch.int16, device="cuda")
        wide[:, :cols] = t.view(torch.int16)
        return wide

    x, w = spread(m["x"], hidden), spread(m["w"], hidden)
    grad, residual = spread(m["grad"], out), spread(m["residual"], out)
    i = {k: Guarded(v.numel(), shift, v) for k, v in
         dict(x=x, w=w, grad=grad, residual=residual, bias=m["bias"], z=m["z"]).items()}
    o = {"out": Guarded(rows * out, shift), "preact": Guarded(rows * out, shift), "grad_x": Guarded(rows * hidden, shift),
         "grad_w": Guarded(groups * out * hidden, shift), "grad_bias": Guarded(groups * out, shift)}
    act = ref.ACTIVATIONS.index(activation)
    layer = LayerC(rows, hidden, out, 0 if dtype == torch.float16 else 1, act, i["x"].ptr, hidden + gap, i["w"].ptr,
                   hidden + gap, ctypes.pointer(rc) if rc else None)
    opt = OptionsC(*form) if form else OptionsC()
    n = ctypes.c_uint64()
    stream = torch.cuda.current_stream().cuda_stream
    spaces = []

    def space():
        assert n.value % 2 == 0
        spaces.append(Guarded(n.value // 2))
        assert spaces[-1].ptr % 16 == 0
        return spaces[-1].ptr if n.value else None

    few = form is not None and form[1] <= 8
    assert c.linear_forward_workspace(ctypes.byref(layer), ctypes.byref(opt), ctypes.byref(n)) == 0
    with_residual = counts is None
    assert c.linear_forward(o["out"].ptr, o["preact"].ptr, ctypes.byref(layer), i["bias"].ptr,
                            i["residual"].ptr if with_residual else None, out + gap, space(), n.value, ctypes.byref(opt),
                            stream) == 0
    weight = form is None or form[1] != 32
    done = ["out", "preact"]
    if not few:
        gw = o["grad_w"].ptr if weight else None
        done += ["grad_x", "grad_bias"] + ["grad_w"] * weight
        z = None if activation == "none" else i["z"].ptr
        assert c.linear_backward_workspace(o["grad_x"].ptr, gw, o["grad_bias"].ptr, ctypes.byref(layer), i["grad"].ptr,
                                           out + gap, ctypes.byref(n)) == 0
        assert c.linear_backward(o["grad_x"].ptr, gw, o["grad_bias"].ptr, ctypes.byref(layer), i["grad"].ptr, out + gap, z,
                                 space(), n.value, ctypes.byref(opt), stream) == 0
    torch.cuda.synchronize()
    for k, g in i.items():
        g.check(k, False)
    for g in spaces:
        g.check("workspace", None)
    for k in NAMES:
        o[k].check(k, True if k in done else False)
    want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], m["residual"] if with_residual else None, activation, offsets)
    ref.check(o["out"].values(dtype, rows, out), want, err, "out")
    ref.check(o["preact"].values(dtype, rows, out), wz, zerr, "z")
    if not few:
        gx, gw, gb = ref.backward(m["grad"], m["x"], m["w"], None if activation == "none" else m["z"], activation, offsets)
        ref.check(o["grad_x"].values(dtype, rows, hidden), *gx, "grad_x")
        if weight:
            ref.check(o["grad_w"].values(dtype, *m["w"].shape), *gw, "grad_w")
        ref.check(o["grad_bias"].values(dtype, *m["bias"].shape), *gb, "grad_bias")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("rows,out,hidden", [(1, 1, 1), (1, 8, 8), (3, 5, 7), (17, 129, 65), (33, 72, 136), (130, 257, 77),
                                             (257, 264, 520), (511, 33, 1001)])
def test_dense(lib, c, rows, out, hidden, shift):
    for k, dtype in enumerate((torch.float16, torch.bfloat16)):
        run(lib, c, rows, out, hidden, dtype, shift)
        run(lib, c, rows, out, hidden, dtype, shift, activation="none", gap=8 if k else 3)


@pytest.mark.parametrize("form", FORMS + FEW)
def test_every_form(lib, c, form):
    dtype = (torch.float16, torch.bfloat16)[form[2] > 1]
    for rows, out, hidden, shift, gap in ((1, 1, 1, 1, 0), (131, 258, 204, 0, 4), (33, 135, 1001, 1, 0), (270, 40, 72, 0, 0)):
        run(lib, c, rows, out, hidden, dtype, shift, form=form, gap=gap, activation="silu")


@pytest.mark.parametrize("form", [None] + FORMS + FEW)
@pytest.mark.parametrize("counts,dropped", [((0, 3, 0, 0, 1), 4), ((16, 33, 130, 0, 65, 257), 7), ((0, 0, 0), 3), ((1,), 0)])
def test_experts(lib, c, form, counts, dropped):
    rows = sum(counts) + dropped
    for out, hidden, shift in ((72, 136, 0), (131, 77, 1)):
        run(lib, c, rows, out, hidden, torch.bfloat16, shift, form=form, counts=counts, dropped=dropped)


def test_many_strips_and_tiles(lib, c):
    run(lib, c, 5003, 1001, 333, torch.float16, 1)
    run(lib, c, 3001 + 64 + 6, 520, 712, torch.bfloat16, 0, counts=(3001, 0, 64), dropped=6)
