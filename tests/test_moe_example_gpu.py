"""The operators together: a mixture-of-experts projection, served and trained (GPU)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import moe_example
    return moe_example


@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,top_k,experts,hidden,out", [(1, 2, 8, 512, 256), (50, 3, 6, 328, 200),
                                                             (700, 4, 5, 256, 136)])
def test_served(ex, form, tokens, top_k, experts, hidden, out):
    g = torch.Generator().manual_seed(tokens)
    w = (torch.randn(experts, out, hidden, generator=g) * 0.05).half().cuda()
    x = torch.randn(tokens, hidden, generator=g).half().cuda()
    ids = torch.randint(-1, experts, (tokens, top_k), generator=g).int().cuda()   # -1: dropped
    gates = torch.rand(tokens, top_k, generator=g).cuda()
    layer = ex.ExpertProjection(w, form)
    got = ref.to_numpy(layer(x, ids, gates))
    a = ref.values(ref.to_numpy(x), form)
    b = ref.values(ref.to_numpy(w).reshape(-1, hidden), form, layer.weights.exponent)
    b = b.reshape(experts, out, hidden)
    i = ids.cpu().numpy()
    wt = np.where(i >= 0, ref.to_numpy(gates), 0.0)
    want, tol = np.zeros((tokens, out)), np.zeros((tokens, out))
    for j in range(top_k):   # a slot's product is rounded to fp16 before it is weighted
        e = np.maximum(i[:, j], 0)
        y = np.einsum("th,toh->to", a, b[e])
        mag = np.einsum("th,toh->to", np.abs(a), np.abs(b[e]))
        want += wt[:, j:j + 1] * y
        tol += wt[:, j:j + 1] * ref.product_tolerance(y, mag, hidden, torch.float16)
        tol += (top_k + 1) * 2.0 ** -24 * wt[:, j:j + 1] * mag
    tol += ref.half_unit(np.abs(want) + tol, torch.float16)
    assert (np.abs(got - want) <= tol).all()


def test_trained(ex):
    """Autograd through the package's moves against autograd through the same in plain torch."""
    import multistage_smem_pipeline_gb300 as lib
    torch.manual_seed(3)
    tokens, top_k, experts, hidden = 40, 3, 5, 72
    x = torch.randint(-3, 4, (tokens, hidden)).half().cuda()
    ids = torch.randint(0, experts, (tokens, top_k)).int().cuda()
    gates = torch.randint(1, 4, (tokens, top_k)).float().cuda()
    mix = torch.randint(-2, 3, (tokens, hidden)).half().cuda()
    r = lib.moe_sort(ids, experts)
    grads = []
    for plain in (False, True):
        xg, wg = x.clone().requires_grad_(), gates.clone().requires_grad_()
        if plain:   # small integers: exact in either order
            out = (wg[..., None] * (2 * xg.float())[:, None, :].expand(-1, top_k, -1)).sum(1)
        else:
            out = ex.combine(2 * ex.dispatch(xg, r), r, wg).float()
        (out * mix.float()).sum().backward()
        grads.append((out.detach(), xg.grad.float(), wg.grad))
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def test_command_runs(ex, capsys):
    ex.main(["--tokens", "8", "--experts", "4", "--hidden", "256", "--out", "128"])
    said = capsys.readouterr().out
    assert "same result: True" in said and "trained: loss" in said
