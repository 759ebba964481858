"""A gradient's bits do not depend on what else the call is for (GPU)."""
import pytest
import torch

import linear_reference as ref
from test_linear_gpu import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("activation", ref.ACTIVATIONS)
def test_the_bias_s_gradient_alone_as_beside_others(lib, activation):
    """Its terms are the same numbers whether or not dz is also stored (where only the sum took them, gelu's and silu's were not rounded)."""
    for seed in range(31, 35):
        for dtype in (torch.float16, torch.bfloat16):
            m = make(64, 2048, 64, dtype, seed=seed)
            kw = dict(preact=m["z"], activation=activation, need_bias=True)
            want = lib.linear_backward(m["grad"], m["x"], m["w"], **kw)[2]
            for x, w in ((False, False), (True, False), (False, True)):
                got = lib.linear_backward(m["grad"], m["x"], m["w"], need_x=x, need_weight=w, **kw)[2]
                assert torch.equal(bits(got), bits(want)), (seed, dtype, x, w)
