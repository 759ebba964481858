"""The form that a 4-bit product takes: what the choice is, checked without a GPU (the counts of a
GB300 are assumed) and with one, and each form by its name against exact products (GPU)."""
import pytest
import torch

FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def lib():
    from multistage_smem_pipeline_gb300 import build
    build.build()
    import multistage_smem_pipeline_gb300 as m
    return m


def form(c):
    return "pair" if c["cta_pair"] else f"split {c['split_k']}" if c["split_k"] > 1 else "single"


def choice(lib):
    # one tile a CTA at most: never pairs, however long k is, and split where tiles are few
    for k in (8192, 10496, 10497, 11008, 14336, 32768, 1 << 20):
        for m in (1, 16, 100, 128):
            assert form(lib.fp4_query_config(m, 4096, k)) == "split 4", (m, k)
            assert form(lib.fp4_query_config(m, 128, k)) == "split 8", (m, k)
            assert form(lib.fp4_query_config(m, 14336, k)) == "single"
        assert form(lib.fp4_query_config(512, 4096, k)) == "single"
    for m, n, k in [(8192, 8192, 8192), (2048, 4096, 2048), (8192, 4096, 14336)]:
        c = lib.fp4_query_config(m, n, k)
        assert form(c) == "pair" and c["tile"] == 256 and c["ctas"] == 152
    assert form(lib.fp4_query_config(8192, 4096, 256)) == "single"
    assert form(lib.fp4_query_config(32768, 2048, 4096, groups=64, by_offsets=True)) == "pair"
    assert form(lib.fp4_query_config(32, 2048, 4096, groups=64, by_offsets=True)) == "single"
    assert form(lib.fp4_query_config(4, 200, 14336, groups=3, by_offsets=True)) == "split 8"


def test_choice(lib):
    choice(lib)
    for bad in [(0, 8, 8), (8, 0, 8), (8, 8, 0), (8, 8, 2**23 + 1), (2**31, 8, 8)]:
        with pytest.raises(lib.GemmError):
            lib.fp4_query_config(*bad)
    for kw in [dict(groups=0), dict(groups=3), dict(groups=1025, by_offsets=True)]:
        with pytest.raises(lib.GemmError):
            lib.fp4_query_config(8, 8, 8, **kw)


@pytest.mark.gpu
def test_choice_on_the_device(lib):
    choice(lib)


def integers(g, rows, k):
    """Elements with scale 1 (a 6 in every block), whose products' fp32 sums are exact."""
    values = torch.tensor([0, 1, 2, 3, 4, 6, -1, -3], dtype=torch.float16, device="cuda")
    x = values[torch.randint(8, (rows, k), device="cuda", generator=g)]
    x[:, ::16] = 6
    return x


DENSE = [("single", 100, 14336, 512), ("single", 300, 700, 1000),
         ("split 2", 64, 8192, 4360), ("split 4", 33, 4000, 10500), ("split 8", 130, 260, 12000),
         ("pair", 2048, 4096, 2048), ("pair", 2065, 3900, 2080), ("pair", 1999, 3970, 2304),
         ("pair", 2300, 4000, 1100), ("pair", 2176, 4090, 1025)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("which,m,n,k", DENSE)
def test_dense(lib, fmt, which, m, n, k):
    assert form(lib.fp4_query_config(m, n, k, fmt)) == which
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x, w = integers(g, m, k), integers(g, n, k)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(x, format=fmt), lib.fp4_quantize(w, format=fmt),
                    dtype=torch.bfloat16, out=out)
    assert torch.equal(out, (x.double() @ w.double().T).to(torch.bfloat16))
    assert lib.fp4_get_device_error() == (0, 0)


UNIFORM = [("single", 6, 200, 300, 224), ("split 8", 3, 40, 200, 8200), ("split 4", 5, 200, 130, 6500),
           ("pair", 8, 300, 1000, 1056), ("pair", 30, 257, 500, 2300), ("pair", 12, 200, 1100, 2000)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("which,groups,m,n,k", UNIFORM)
def test_uniform_groups(lib, fmt, which, groups, m, n, k):
    assert form(lib.fp4_query_config(groups * m, n, k, fmt, groups=groups)) == which
    g = torch.Generator(device="cuda").manual_seed(groups)
    x, w = integers(g, groups * m, k), integers(g, groups * n, k)
    out = torch.full((groups * m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(x, format=fmt, group_rows=m),
                    lib.fp4_quantize(w, format=fmt, group_rows=n), dtype=torch.bfloat16, out=out)
    want = x.view(groups, m, k).double() @ w.view(groups, n, k).double().transpose(1, 2)
    assert torch.equal(out.view(groups, m, n), want.to(torch.bfloat16))
    assert lib.fp4_get_device_error() == (0, 0)


BY_OFFSETS = [("single", 200, 5, 300, 1040), ("split 4", 40, 3, 900, 9000),
              ("split 8", 7, 4, 130, 9000), ("pair", 5000, 4, 2048, 2048), ("pair", 9000, 20, 700, 1300)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("which,slots,experts,n,k", BY_OFFSETS)
def test_by_offsets(lib, fmt, which, slots, experts, n, k):
    c = lib.fp4_query_config(slots, n, k, fmt, groups=experts, by_offsets=True)
    assert form(c) == which
    g = torch.Generator(device="cuda").manual_seed(slots)
    x, w = integers(g, slots, k), integers(g, experts * n, k)
    ids = torch.randint(-1, experts - 1, (slots, 1), device="cuda", generator=g).int()
    ids[ids == 0] = experts - 1                     # the first expert has no rows
    r = lib.moe_sort(ids, experts)
    out = torch.full((slots, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(x, format=fmt, routing=r),
                    lib.fp4_quantize(w, format=fmt, group_rows=n), dtype=torch.bfloat16, out=out)
    off, order = r.offsets.tolist(), lib.moe_pairs(r).long()
    for e in range(experts):
        rows = slice(off[e], off[e + 1])
        want = x[order[rows]].double() @ w[e * n:(e + 1) * n].double().T
        assert torch.equal(out[rows], want.to(torch.bfloat16)), e
    assert not out[off[-1]:].any()
    assert lib.fp4_get_device_error() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("which,m,n,k", [("single", 4, 100, 256), ("split 8", 8, 300, 4096),
                                         ("split 4", 1, 4096, 14336), ("pair", 2048, 4096, 2048),
                                         ("pair", 2065, 3900, 2080)])
def test_a_wait_that_runs_out(lib, which, m, n, k):
    """Loads that never come end in the stream's error word, on every form, and the next call is
    right again."""
    assert form(lib.fp4_query_config(m, n, k)) == which
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = integers(g, m, k), integers(g, n, k)
    qx, qw = lib.fp4_quantize(x), lib.fp4_quantize(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lib.fp4_gemm_tn(qx, qw, timeout_ns=20_000_000, inject=1, stream=s)
    status, raw = lib.fp4_get_device_error(s)
    assert status == 5 and raw >> 8 in (1, 2, 3, 4, 5)
    assert lib.fp4_get_device_error(s) == (0, 0) and lib.fp4_get_device_error() == (0, 0)
    got = lib.fp4_gemm_tn(qx, qw, dtype=torch.bfloat16)
    assert torch.equal(got, (x.double() @ w.double().T).to(torch.bfloat16))
