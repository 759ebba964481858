"""Batches of products without rows (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("groups", [1, 6])
def test_no_rows_are_whole_groups(form, groups):
    import multistage_smem_pipeline_gb300 as lib
    w = lib.fp4_quantize(torch.randn(groups * 40, 96, device="cuda").half(), format=form, group_rows=40)
    x = torch.empty(0, 96, dtype=torch.float16, device="cuda")
    for group_rows in (None, 0, 16):
        q = lib.fp4_quantize(x, format=form, group_rows=group_rows)
        assert q.rows == 0 and q.scales.numel() == 0 and lib.fp4_dequantize(q).shape == (0, 96)
        assert lib.fp4_gemm_tn(q, w).shape == (0, 40)
    with pytest.raises(ValueError):
        lib.fp4_quantize(x, format=form, group_rows=-1)
    with pytest.raises(lib.GemmError):
        lib.fp4_gemm_tn(lib.fp4_quantize(x[:, :64], format=form), w)
