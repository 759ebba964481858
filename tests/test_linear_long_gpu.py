"""The longest sums that a layer of experts may have (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_sum_over_the_most_rows():
    """2^30 rows of one expert among 100 are one CTA's sum, which takes 3 s: no wait may give up meanwhile."""
    import multistage_smem_pipeline_gb300 as lib
    rows, experts = 1 << 30, 100
    assert lib.linear_query_config("grad_w", rows, 8, 8, experts)["split_k"] == 1
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    grad = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[::1 << 20] = 1
    grad[::1 << 20] = 1
    ids = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    offsets = torch.full((experts + 1,), rows, dtype=torch.int32, device="cuda")
    offsets[0] = 0
    routing = lib.Routing(offsets, ids, ids)
    grad_w = lib.moe_linear_backward(grad, x, routing, None, need_x=False)[1]
    assert lib.linear_get_device_error() == (0, 0)
    assert (grad_w[0] == rows >> 20).all() and not grad_w[1:].any()
