"""The example's edges: weights without a scale of their own, activations far from 1, and what
autograd is told (GPU)."""
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import moe_example
    return moe_example


def one_expert(layer, x):
    """Every token to expert 0 with weight 1."""
    n = x.shape[0]
    return layer(x, torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.ones(n, 1, device="cuda"))


@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -110, 2.0 ** -90, 1.0, 2.0 ** 90])
def test_weights_of_any_size(ex, form, scale):
    """All zero, so small that the least exponent has to do, and large."""
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(2, 40, 64, generator=g) * scale).bfloat16().cuda()
    x = torch.randn(5, 64, generator=g).bfloat16().cuda()
    layer = ex.ExpertProjection(w, form)
    assert -100 <= layer.weights.exponent <= 100
    got = ref.to_numpy(one_expert(layer, x))
    a = ref.values(ref.to_numpy(x), form)
    b = ref.values(ref.to_numpy(w[0]), form, layer.weights.exponent)
    want = a @ b.T
    tol = ref.product_tolerance(want, abs(a) @ abs(b).T, 64, torch.bfloat16)
    tol += ref.half_unit(abs(want) + tol, torch.bfloat16)         # rounded again by combine
    assert (abs(got - want) <= tol).all()
    assert got.any() == want.any()
    with pytest.raises(ValueError):
        ex.ExpertProjection(torch.full_like(w, float("inf")), "nvfp4")


@pytest.mark.parametrize("scale", [1e-3, 1e-7, 1e6])
def test_activations_of_any_size(ex, scale):
    """With exponent 0 blocks below 6 x 2^-10 are zero and those above 2688 cut: the layer takes the
    activations' exponent, found on a sample of them."""
    g = torch.Generator().manual_seed(2)
    w = (torch.randn(2, 40, 64, generator=g) * 0.1).bfloat16().cuda()
    x = (torch.randn(50, 64, generator=g) * scale).bfloat16().cuda()
    exponent = ex.exponent_for(x)
    layer = ex.ExpertProjection(w, activation_exponent=exponent)
    got = ref.to_numpy(one_expert(layer, x))
    a = ref.values(ref.to_numpy(x), "nvfp4", exponent)
    b = ref.values(ref.to_numpy(w[0]), "nvfp4", layer.weights.exponent)
    want = a @ b.T
    tol = ref.product_tolerance(want, abs(a) @ abs(b).T, 64, torch.bfloat16)
    tol += ref.half_unit(abs(want) + tol, torch.bfloat16)
    assert (abs(got - want) <= tol).all()
    # the largest element is 6 scales, whose rounding is 2^-4 at most: not zero, and not cut
    largest = abs(ref.to_numpy(x)).max()
    assert abs(abs(a).max() - largest) <= 2.0 ** -4 * largest


def test_second_order_is_refused(ex):
    """The gradients are not differentiable themselves, and say so instead of losing terms."""
    import multistage_smem_pipeline_gb300 as lib
    r = lib.moe_sort(torch.tensor([[0, 1], [1, -1], [0, 0]], dtype=torch.int32, device="cuda"), 2)
    x = torch.randn(3, 16, device="cuda").half().requires_grad_()
    w = torch.rand(3, 2, device="cuda").requires_grad_()
    for wrt in (x, w):
        out = ex.combine(ex.dispatch(x, r), r, w).float()
        grad, = torch.autograd.grad(out.square().sum(), wrt, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (grad.float().square().sum() + w.square().sum()).backward()
    out = ex.combine(ex.dispatch(x, r), r, w).float()
    out.square().sum().backward()                     # the first order is as it was
    assert x.grad.any() and w.grad.any()
