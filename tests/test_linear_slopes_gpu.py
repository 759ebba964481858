"""Slopes of the activations, relative to themselves over the whole range of both types (GPU)."""
import math

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def terms(z, activation):
    """The sum of the magnitudes of a slope's two terms."""
    if activation == "gelu":
        return ref.below(z) + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u, du = z, 1.0
    if activation == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    return torch.special.expit(u) + (z * du).abs() * torch.special.expit(u) * torch.special.expit(-u)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("grad", [1.0, 4096.0])
def test_slopes_keep_their_relative_accuracy(lib, activation, dtype, grad):
    """Every finite value as z; 4096 as the gradient shows twelve more bits of fp16's smallest results.

    Allowed, beside the rounding of the result: 2^-13 of the slope for its exponential (an exponent
    of up to 130 with 4 roundings and constants of 2^-24 each: 130 x 0.7 x 5 x 2^-24 is below 2^-15, and
    2^-21 for the instruction); 2^-16 of its terms for the polynomial, reciprocals and sums (8.5e-6 and
    a few 2^-23); half a step of the type's subnormal numbers, and of fp32's, which 4096 times are more.
    """
    every = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(dtype)
    every = every[torch.isfinite(every)]
    z = every[:every.numel() // 8 * 8].view(-1, 8)
    w = torch.eye(8, dtype=dtype, device="cuda")
    got = lib.linear_backward(torch.full_like(z, grad), None, w, preact=z, activation=activation, need_weight=False)[0]
    zd = z.double()
    want = ref.slope(zd, activation)
    assert torch.isfinite(want).all()
    err = grad * (2.0 ** -13 * want.abs() + 2.0 ** -16 * terms(zd, activation) + 2.0 ** -149)
    ref.check(got, grad * want, err + (2.0 ** -134 if dtype == torch.bfloat16 else 0.0), activation)


def test_far_slopes_are_not_lost(lib):
    """Slopes that bfloat16 holds, whose exponential alone is below fp32's normal numbers."""
    for activation, far in (("silu", -88.0), ("silu", -90.0), ("gelu", -13.25), ("gelu_tanh", -10.0)):
        z = torch.full((8, 8), far, dtype=torch.bfloat16, device="cuda")
        w = torch.eye(8, dtype=torch.bfloat16, device="cuda")
        got = lib.linear_backward(torch.ones_like(z), None, w, preact=z, activation=activation, need_weight=False)[0]
        want = float(ref.slope(torch.tensor(far, dtype=torch.float64), activation))
        assert abs(want) > 2.0 ** -126 and abs(float(got[0, 0]) / want - 1) <= 2.0 ** -8 + 2.0 ** -13, (activation, far)


def test_slopes_past_all_exponentials(lib):
    """Zero on the left, one on the right, also times the largest gradients."""
    for dtype in (torch.float16, torch.bfloat16):
        most = torch.finfo(dtype).max
        z = torch.tensor([-most, -1000.0, -200.0, -111.0, 111.0, 200.0, 1000.0, most], device="cuda").to(dtype).view(1, 8)
        w = torch.eye(8, dtype=dtype, device="cuda")
        for activation in ("silu", "gelu", "gelu_tanh"):
            got = lib.linear_backward(torch.full_like(z, most), None, w, preact=z, activation=activation, need_weight=False)[0]
            assert (got[0, :4] == 0).all() and (got[0, 4:] == most).all(), (activation, dtype, got)
