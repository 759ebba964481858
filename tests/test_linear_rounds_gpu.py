"""Products of linear layers in which every CTA or pair takes several tiles one after the other, on data
without zeros, against the definitions in 64 bits (GPU): the accumulators by turns, the ring's
phases from tile to tile, partial bands of the raster, ragged sums one after the other."""
import random

import pytest
import torch

import linear_reference as ref
from test_linear_gpu import make, routing_of

pytestmark = pytest.mark.gpu

UNSPLIT = [(1, 256, 1)] + [(0, tile, 1) for tile in (32, 64, 128, 256)]
SMS = 152


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def tiles(form, columns, rows):
    """Tiles of a D of so many columns and (for each group) rows; at least three for each unit."""
    m = 256 if form[0] else 128
    count = -(-columns // m) * sum(-(-r // form[1]) for r in rows)
    assert count >= 3 * (SMS // 2 if form[0] else SMS)
    return count


def group_sizes(seed, groups, least, most):
    """Sizes of every remainder by 16 and by 64, some of them zero, one past a ring of eight stages."""
    rng = random.Random(seed)
    sizes = [rng.randint(least, most) for _ in range(groups)]
    sizes[3] = sizes[4] = sizes[-2] = 0
    sizes[0], sizes[6], sizes[7], sizes[8] = 1, 64, 16, 577
    return sizes


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("form", UNSPLIT + [None])
@pytest.mark.parametrize("odd", [0, 1])
def test_dense_forward(lib, form, dtype, odd):
    rows, out, hidden = 5000 + 3 * odd, 3000 + odd, 200 + odd
    tiles(form or (1, 256, 1), out, [rows])
    m = make(rows, out, hidden, dtype, seed=51)
    got, z = lib.linear(m["x"], m["w"], m["bias"], activation="gelu", residual=m["residual"], save_preact=True, form=form)
    want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], m["residual"], "gelu")
    ref.check(got, want, err, "out")
    ref.check(z, wz, zerr, "z")


@pytest.mark.parametrize("form", UNSPLIT + [None])
@pytest.mark.parametrize("odd", [0, 1])
def test_dense_grad_x(lib, form, odd):
    rows, out, hidden = 5000 + 3 * odd, 200 + odd, 3000 + odd
    tiles(form or (1, 256, 1), hidden, [rows])
    m = make(rows, out, hidden, torch.bfloat16, seed=52)
    got = lib.linear_backward(m["grad"], None, m["w"], preact=m["z"], activation="silu", need_weight=False, form=form)[0]
    want = ref.backward(m["grad"], m["x"], m["w"], m["z"], "silu")[0]
    ref.check(got, *want, "grad_x")


@pytest.mark.parametrize("form", [f for f in UNSPLIT if f[1] != 32] + [None])
@pytest.mark.parametrize("odd", [0, 1])
def test_dense_grad_w(lib, form, odd):
    rows, out, hidden = 200 + odd, 5000 + 3 * odd, 3000 + odd
    tiles(form or (1, 256, 1), hidden, [out])
    m = make(rows, out, hidden, torch.float16, seed=53)
    got = lib.linear_backward(m["grad"], m["x"], None, preact=m["z"], activation="silu", need_x=False, need_bias=True,
                              form=form)
    want = ref.backward(m["grad"], m["x"], m["w"], m["z"], "silu")
    ref.check(got[1], *want[1], "grad_w")
    ref.check(got[2], *want[2], "grad_bias")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("form", UNSPLIT + [None])
def test_experts_forward(lib, form, dtype):
    sizes = group_sizes(1, 26, 1, 400)
    out, hidden = 3000, 200
    tiles(form or (1, 256, 1), out, sizes)
    m = make(sum(sizes) + 37, out, hidden, dtype, experts=len(sizes), seed=54)
    routing, offsets = routing_of(lib, sizes, 37)
    m["x"][offsets[-1]:] = float("nan")
    got, z = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True, form=form)
    want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], None, "silu", offsets)
    ref.check(got, want, err, "out")
    ref.check(z, wz, zerr, "z")


@pytest.mark.parametrize("form", UNSPLIT + [None])
def test_experts_grad_x(lib, form):
    sizes = group_sizes(2, 26, 1, 400)
    out, hidden = 200, 3000
    tiles(form or (1, 256, 1), hidden, sizes)
    m = make(sum(sizes) + 37, out, hidden, torch.bfloat16, experts=len(sizes), seed=55)
    routing, offsets = routing_of(lib, sizes, 37)
    for t in ("grad", "z"):
        m[t][offsets[-1]:] = float("nan")
    got = lib.moe_linear_backward(m["grad"], None, routing, m["w"], preact=m["z"], activation="gelu", need_weight=False,
                                  form=form)[0]
    want = ref.backward(m["grad"], m["x"], m["w"], m["z"], "gelu", offsets)[0]
    ref.check(got, *want, "grad_x")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("form", [f for f in UNSPLIT if f[1] != 32] + [None])
@pytest.mark.parametrize("most", [40, 300])
def test_experts_grad_w(lib, form, dtype, most):
    """Every unit has ragged sums one after the other, of one stage and of several, empty ones between them."""
    sizes = group_sizes(3, 40, 1, most)
    out, hidden = 1000, 1100
    tiles(form or (1, 256, 1), hidden, [out] * len(sizes))
    m = make(sum(sizes) + 37, out, hidden, dtype, experts=len(sizes), seed=56)
    routing, offsets = routing_of(lib, sizes, 37)
    for t in ("x", "grad", "z"):
        m[t][offsets[-1]:] = float("nan")
    got = lib.moe_linear_backward(m["grad"], m["x"], routing, None, preact=m["z"], activation="gelu", need_x=False,
                                  need_bias=True, form=form)
    want = ref.backward(m["grad"], m["x"], m["w"], m["z"], "gelu", offsets)
    ref.check(got[1], *want[1], "grad_w")
    ref.check(got[2], *want[2], "grad_bias")


@pytest.mark.parametrize("sizes,out,hidden", [([5000], 3000, 1100), (group_sizes(4, 26, 1, 400), 1000, 1100)])
def test_both_gradients_at_once(lib, sizes, out, hidden):
    """grad_x and grad_w of several tiles a unit, one taking over the other's SMs."""
    m = make(sum(sizes) + 5, out, hidden, torch.bfloat16, experts=len(sizes), seed=57)
    routing, offsets = routing_of(lib, sizes, 5)
    got = lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], preact=m["z"], activation="gelu", need_bias=True)
    for g, w, name in zip(got, ref.backward(m["grad"], m["x"], m["w"], m["z"], "gelu", offsets),
                          ("grad_x", "grad_w", "grad_bias")):
        ref.check(g, *w, name)
