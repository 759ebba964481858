"""The forms that linear_query_config names, for a gradient alone and beside the other one (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import build
    build.build()
    from multistage_smem_pipeline_gb300 import experts
    return experts


SIZES = [(rows, out, hidden, experts) for rows in (1, 5, 27, 64, 200, 1021, 4000)
         for out, hidden in ((64, 64), (1000, 1411), (2048, 2048), (1157, 300), (4096, 14336), (182, 1021))
         for experts in (0, 8, 18)]


def test_both_gradients_are_cut_to_run_beside_each_other(ex):
    """Where a call for both gives each of them part of the SMs, the forms say so."""
    for rows, out, hidden in ((1021, 1000, 1411), (1021, 1000, 1000)):
        both = [ex.linear_query_config(p, rows, hidden, out, both=True) for p in ("grad_x", "grad_w")]
        assert sum(c["ctas"] for c in both) <= 152
        alone = [ex.linear_query_config(p, rows, hidden, out) for p in ("grad_x", "grad_w")]
        assert sum(c["ctas"] for c in alone) > 152
    for rows, out, hidden, experts in SIZES:
        for product in ("grad_x", "grad_w"):
            c = ex.linear_query_config(product, rows, hidden, out, experts, both=True)
            assert c["ctas"] >= 1 and c["tile"] >= (64 if product == "grad_w" else 32)
    # of the forward product there is one form
    assert ex.linear_query_config("forward", 64, 2048, 2048, both=True) == ex.linear_query_config("forward", 64, 2048, 2048)


def test_a_gradient_s_sums_are_shared_as_beside_the_other_one(ex):
    """The bits of a gradient depend on how many CTAs share its sums, and not on what else is asked for."""
    for rows, out, hidden, experts in SIZES:
        for product in ("grad_x", "grad_w"):
            alone = ex.linear_query_config(product, rows, hidden, out, experts)
            both = ex.linear_query_config(product, rows, hidden, out, experts, both=True)
            assert alone["split_k"] == both["split_k"], (product, rows, out, hidden, experts, alone, both)
