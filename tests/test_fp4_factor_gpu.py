"""alpha 2^(exponents) below fp32's normal numbers (GPU): the results need not be, and bfloat16 has
them.  The sums are exact here (one product a column block, small integers times powers of two), so
what separates a result from the formula in 64 bits is the rounding of the factor (2^-24), of its
product (2^-24) and of the result (2^-8, or half of bfloat16's least subnormal, 2^-134, and half
of fp32's before it, 2^-150)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def operand(rows, cols, exponent):
    """Elements of the grid with scale 448, the largest, times 2^exponent."""
    v = torch.tensor([6.0, 3.0, -2.0, 4.0, 1.0, 0.5, -1.5, 2.0], dtype=torch.float64).repeat(cols // 8)
    x = v.repeat(rows, 1) * torch.tensor([1.0, 0.5, -1.0], dtype=torch.float64)[torch.arange(rows) % 3, None]
    return (x * 448.0 * 2.0 ** exponent).to(torch.bfloat16).cuda()


# on one CTA a tile, on a tile that several share, and on pairs
@pytest.mark.parametrize("m,n,k,which", [(3, 40, 256, "single"), (5, 20, 4096, "split"),
                                         (2048, 4096, 2048, "pair")])
@pytest.mark.parametrize("ea,eb,alpha", [(-60, -60, 1.0), (-70, -70, 0.3), (-75, -76, 1.0),
                                         (-100, -60, -0.7), (-100, -75, 3.0), (0, 0, 1e-41),
                                         (-100, -100, 2.0 ** 60), (-100, -100, 1.0)])
def test_small_factors(lib, m, n, k, which, ea, eb, alpha):
    c = lib.fp4_query_config(m, n, k)
    assert which == ("pair" if c["cta_pair"] else "split" if c["split_k"] > 1 else "single")
    x, w = operand(m, k, ea), operand(n, k, eb)
    d = lib.fp4_gemm_tn(lib.fp4_quantize(x, exponent=ea), lib.fp4_quantize(w, exponent=eb), alpha=alpha,
                        dtype=torch.bfloat16)
    a = torch.from_numpy(ref.values(ref.to_numpy(x[:64]), "nvfp4", ea))
    b = torch.from_numpy(ref.values(ref.to_numpy(w[:64]), "nvfp4", eb))
    want = (float(np.float32(alpha)) * (a * 2.0 ** 60) @ b.T * 2.0 ** -60).numpy()
    got = ref.to_numpy(d[:64, :64])
    tol = np.abs(want) * (2.0 ** -8 + 4 * 2.0 ** -24) + 2.0 ** -134 + 2.0 ** -149
    assert (np.abs(got - want) <= tol).all(), (got[0, 0], want[0, 0])
    assert got.any() == (np.abs(want).max() > 2.0 ** -133)
