"""A routing stands for itself: quantising into expert order reads offsets and rows, and not the
list of experts that they were made from, which the program may have filled anew (GPU)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from test_fp4_gpu import check_stored, random_ids, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,top_k,experts,dropped", [(5, 2, 3, 0.3), (200, 4, 7, 0.1),
                                                          (64, 8, 64, 0.0), (300, 1, 1024, 0.05),
                                                          (3, 2, 1, 0.5)])
@pytest.mark.parametrize("then", ["reversed", "dropped", "beyond", "constant"])
def test_experts_may_change_after_the_sort(lib, form, tokens, top_k, experts, dropped, then):
    ids = random_ids(tokens, tokens, top_k, experts, dropped)
    before = ids.clone()
    x = rows(tokens, tokens, 272, torch.float16)
    r = lib.moe_sort(ids, experts)
    if then == "reversed":
        ids.copy_(experts - 1 - before)
    else:
        ids.fill_({"dropped": -1, "beyond": 2**31 - 1, "constant": experts - 1}[then])
    q = lib.fp4_quantize(x, format=form, routing=r)
    off, _, pairs = ref.sort(before.cpu().numpy(), experts)
    live = check_stored(q, ref.to_numpy(x)[pairs // top_k], form)
    np.testing.assert_array_equal(live, np.arange(len(pairs)) < off[-1])


def test_a_routing_of_the_programs_own(lib):
    """offsets and rows given by the program, with a list of experts that says nothing."""
    tokens, top_k, experts = 90, 3, 11
    ids = random_ids(4, tokens, top_k, experts, 0.2).cpu().numpy()
    off, order, pairs = ref.sort(ids, experts)
    r = lib.Routing(torch.from_numpy(off.astype(np.int32)).cuda(),
                    torch.from_numpy(order.astype(np.int32)).cuda(),
                    torch.full((tokens, top_k), 2**31 - 1, dtype=torch.int32, device="cuda"))
    x = rows(8, tokens, 100, torch.bfloat16)
    q = lib.fp4_quantize(x, routing=r)
    live = check_stored(q, ref.to_numpy(x)[pairs // top_k], "nvfp4")
    np.testing.assert_array_equal(live, np.arange(len(pairs)) < off[-1])
