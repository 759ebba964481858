"""A gradient's bits do not depend on what else the call is for, nor on the tiles it is cut into (GPU)."""
import pytest
import torch

import linear_reference as ref
from test_linear_gpu import make, routing_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


# sizes whose gradients were shared by other numbers of CTAs alone than beside each other, and some
# that were not; then experts' (rows of each, and of none)
DENSE = [(64, 2048, 2048), (27, 1157, 2900), (5, 1474, 1594), (2298, 1845, 6), (212, 904, 333), (79, 1135, 185),
         (1021, 1000, 1411), (300, 264, 520)]
EXPERTS = [([0, 1] + [0] * 15 + [1], 0, 1021, 182), ([3, 0, 5, 1, 0, 0, 1, 1, 0, 0, 0, 0], 2, 1660, 93),
           ([9, 0, 20, 31, 1, 7, 0, 9], 5, 1254, 320), ([64, 65, 300, 17], 0, 1000, 200)]


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("activation", ref.ACTIVATIONS)
def test_the_bias_s_gradient_alone_as_beside_others(lib, activation):
    """Its terms are the same numbers whether or not dz is also stored."""
    for seed in range(31, 35):
        for dtype in (torch.float16, torch.bfloat16):
            m = make(64, 2048, 64, dtype, seed=seed)
            kw = dict(preact=m["z"], activation=activation, need_bias=True)
            want = lib.linear_backward(m["grad"], m["x"], m["w"], **kw)[2]
            for x, w in ((False, False), (True, False), (False, True)):
                got = lib.linear_backward(m["grad"], m["x"], m["w"], need_x=x, need_weight=w, **kw)[2]
                assert torch.equal(bits(got), bits(want)), (seed, dtype, x, w)


@pytest.mark.parametrize("rows,out,hidden", DENSE)
def test_alone_as_beside_each_other(lib, rows, out, hidden):
    m = make(rows, out, hidden, torch.bfloat16, seed=31)
    kw = dict(preact=m["z"], activation="silu")
    want = lib.linear_backward(m["grad"], m["x"], m["w"], need_bias=True, **kw)
    for needs in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)):
        need = dict(zip(("need_x", "need_weight", "need_bias"), map(bool, needs)))
        for got, w, n in zip(lib.linear_backward(m["grad"], m["x"], m["w"], **need, **kw), want, needs):
            assert got is None if not n else torch.equal(bits(got), bits(w)), (needs, rows, out, hidden)


@pytest.mark.parametrize("counts,dropped,out,hidden", EXPERTS)
def test_experts_alone_as_beside_each_other(lib, counts, dropped, out, hidden):
    m = make(sum(counts) + dropped, out, hidden, torch.float16, experts=len(counts), seed=32)
    routing, _ = routing_of(lib, counts, dropped)
    want = lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], need_bias=True)
    for needs in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
        need = dict(zip(("need_x", "need_weight", "need_bias"), map(bool, needs)))
        for got, w, n in zip(lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], **need), want, needs):
            assert got is None if not n else torch.equal(bits(got), bits(w)), (needs, counts)


def test_tiles_change_no_bits(lib):
    """What makes that possible: forms that share sums alike sum alike."""
    m = make(333, 520, 700, torch.float16, seed=33)
    for split in (1, 2, 4):
        forms = [(0, tile, split) for tile in (64, 128, 256)] + ([(1, 256, 1)] if split == 1 else [])
        got = [lib.linear_backward(m["grad"], m["x"], m["w"], form=f) for f in forms]
        for g, f in zip(got[1:], forms[1:]):
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got[0][:2], g[:2])), f
