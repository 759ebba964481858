"""4-bit quantisation and products against the 64-bit definitions (GPU)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def rows(seed, n, cols, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, cols, generator=g) * scale
    x *= torch.exp2(torch.randint(-3, 4, (1, cols), generator=g).float())
    return x.to(dtype).cuda()


def check_stored(q, x, form, exponent=0):
    """What q holds is exactly the quantisation of the float64 matrix x; NaN rows of x are skipped."""
    el, scale = ref.stored(q)
    want_el, want_scale = ref.quantise(x, form, exponent)
    live = ~np.isnan(scale).all(axis=1) if scale.shape[1] else np.ones(len(scale), bool)
    np.testing.assert_array_equal(scale[live], want_scale[live])
    np.testing.assert_array_equal(el[live], want_el[live])
    return live


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,cols", [(1, 1), (1, 16), (2, 15), (3, 33), (127, 64), (128, 256),
                                    (129, 255), (300, 1000), (5, 4099), (257, 520)])
def test_quantise_is_exact(lib, form, dtype, n, cols):
    x = rows(n + cols, n, cols, dtype)
    q = lib.fp4_quantize(x, format=form)
    live = check_stored(q, ref.to_numpy(x), form)
    assert live.all()
    want = ref.values(ref.to_numpy(x), form)
    np.testing.assert_array_equal(ref.to_numpy(lib.fp4_dequantize(q, torch.bfloat16)), want)


@pytest.mark.parametrize("exponent", [-20, -8, 3, 15])
@pytest.mark.parametrize("dtype", DTYPES)
def test_exponent(lib, exponent, dtype):
    x = rows(exponent + 50, 40, 320, dtype, scale=2.0 ** (exponent / 2))
    q = lib.fp4_quantize(x, exponent=exponent)
    assert check_stored(q, ref.to_numpy(x), "nvfp4", exponent).all()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_every_16_bit_value(lib, form, dtype):
    """Each finite value of the type in a block with each of many maxima (all significands)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    vals = bits[torch.isfinite(bits.float())]
    size = ref.BLOCK[form]
    vals = torch.cat([vals, vals[:-len(vals) % (size - 1)]]) if len(vals) % (size - 1) else vals
    body = vals.view(-1, size - 1)
    top = body.float().abs().amax(dim=1, keepdim=True)
    blocks = []
    for m in [1.0, 1.07, 1.2, 1.33, 1.5, 1.61, 1.75, 1.9, 3.0, 7.3]:
        blocks.append(torch.cat([body, (top * m).clamp(max=float(torch.finfo(dtype).max)).to(dtype)],
                                dim=1))
    x = torch.cat(blocks).reshape(-1, 16 * size).contiguous() if (len(body) * 10) % 16 == 0 else \
        torch.cat(blocks)
    x = x.cuda()
    q = lib.fp4_quantize(x, format=form)
    el, scale = ref.stored(q)
    want_el, want_scale = ref.quantise(ref.to_numpy(x), form)
    np.testing.assert_array_equal(scale, want_scale)
    np.testing.assert_array_equal(el, want_el)


@pytest.mark.parametrize("form", FORMATS)
def test_special_blocks(lib, form):
    """Zeros, negative zeros, subnormals, the largest values, and blocks with NaN or infinity."""
    x = torch.zeros(8, 64, dtype=torch.float16)
    x[1] = -0.0
    x[2] = 6e-8
    x[3, ::3] = 65504.0
    x[4] = 1.0
    x[4, 5] = float("nan")
    x[5] = 1.0
    x[5, 40] = float("-inf")
    x[6] = -2.5
    x[7, 63] = -0.001
    q = lib.fp4_quantize(x.cuda(), format=form)
    el, scale = ref.stored(q)
    want_el, want_scale = ref.quantise(ref.to_numpy(x), form)
    np.testing.assert_array_equal(scale, want_scale)
    np.testing.assert_array_equal(el, want_el)
    got = ref.to_numpy(lib.fp4_dequantize(q, torch.bfloat16))
    size = ref.BLOCK[form]
    assert np.isnan(got[4, :size]).all() and not np.isnan(got[4, size:]).any()
    bad = 40 // size * size
    assert np.isnan(got[5, bad:bad + size]).all() and np.isnan(got[5]).sum() == size


def test_strided_and_misaligned_rows(lib):
    base = rows(3, 70, 600, torch.float16)
    for x in (base[:, 8:408], base[:, 1:300], base[::2, :512], base[3:4, 7:]):
        q = lib.fp4_quantize(x)
        assert check_stored(q, ref.to_numpy(x), "nvfp4").all()


def test_groups_start_tiles_of_their_own(lib):
    x = rows(4, 5 * 130, 96, torch.bfloat16)
    q = lib.fp4_quantize(x, format="mxfp4", group_rows=130)
    assert q.groups == 5 and q.scales.shape[0] == 10
    assert check_stored(q, ref.to_numpy(x), "mxfp4").all()
    np.testing.assert_array_equal(ref.to_numpy(lib.fp4_dequantize(q, torch.bfloat16)),
                                  ref.values(ref.to_numpy(x), "mxfp4"))


def random_ids(seed, tokens, top_k, experts, dropped=0.0, only=None):
    rng = np.random.RandomState(seed)
    ids = rng.randint(0, experts, (tokens, top_k)) if only is None else \
        np.array(only)[rng.randint(0, len(only), (tokens, top_k))]
    ids[rng.rand(tokens, top_k) < dropped] = rng.choice([-1, experts, -(2**31), 2**31 - 1])
    return torch.from_numpy(ids.astype(np.int32)).cuda()


ROUTED = [(1, 1, 1, 0.0, None), (1, 8, 64, 0.0, None), (7, 3, 5, 0.3, None),
          (300, 2, 3, 0.1, None), (513, 4, 40, 0.0, [0, 39]), (64, 2, 16, 1.0, None),
          (2000, 1, 7, 0.5, [3])]


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("tokens,top_k,experts,dropped,only", ROUTED)
@pytest.mark.parametrize("cols", [48, 1003])
def test_quantise_into_expert_order(lib, form, tokens, top_k, experts, dropped, only, cols):
    ids = random_ids(tokens, tokens, top_k, experts, dropped, only)
    x = rows(cols, tokens, cols, torch.float16)
    r = lib.moe_sort(ids, experts)
    q = lib.fp4_quantize(x, format=form, routing=r)
    q.scales  # a row per slot, tiles by offsets
    pairs, off = lib.moe_pairs(r).cpu().numpy(), r.offsets.cpu().numpy()
    want = ref.to_numpy(x)[pairs // top_k]
    live = check_stored(q, want, form)
    np.testing.assert_array_equal(live, np.arange(len(pairs)) < off[-1])
    back = ref.to_numpy(lib.fp4_dequantize(q, torch.bfloat16))
    np.testing.assert_array_equal(back[:off[-1]], ref.values(want, form)[:off[-1]])
    assert not back[off[-1]:].any()


# ------------------------------------------------------------------ products
def product_case(lib, seed, m, n, k, form, dtype, groups=1, w_exponent=-4):
    x = rows(seed, m, k, dtype)
    w = (rows(seed + 1, groups * n, k, torch.float16) * 0.05).half()
    qw = lib.fp4_quantize(w, format=form, exponent=w_exponent if form == "nvfp4" else 0,
                          group_rows=n)
    a = ref.values(ref.to_numpy(x), form)
    b = ref.values(ref.to_numpy(w), form, qw.exponent).reshape(groups, n, k)
    return x, qw, a, b


def check_product(got, a, b, k, dtype, alpha=1.0):
    """a: rows x k, b: n x k (float64)."""
    want = alpha * (a @ b.T)
    mag = abs(alpha) * (np.abs(a) @ np.abs(b).T)
    tol = ref.product_tolerance(want, mag, k, dtype)
    err = np.abs(ref.to_numpy(got) - want)
    assert (err <= tol).all(), (err.max(), np.argmax(err - tol), np.count_nonzero(err > tol))


PRODUCTS = [(1, 1, 1), (1, 128, 256), (1, 130, 32), (2, 7, 100), (16, 256, 512), (17, 129, 257),
            (31, 64, 64), (33, 300, 1024), (100, 1000, 768), (128, 128, 2048), (129, 257, 1056),
            (256, 512, 256), (257, 384, 4096), (300, 1337, 96), (700, 520, 640), (1, 4096, 4096),
            (5, 33, 8200), (520, 1030, 1300), (1024, 1024, 512), (64, 2048, 2880)]


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(lib, form, m, n, k):
    dtype = DTYPES[(m + n) % 2]
    x, qw, a, b = product_case(lib, m * 7 + n, m, n, k, form, dtype)
    got = lib.fp4_gemm_tn(lib.fp4_quantize(x, format=form), qw, dtype=dtype)
    check_product(got, a, b[0], k, dtype)
    assert lib.fp4_get_device_error() == (0, 0)


# Few tiles and a long k: several CTAs share a tile.
@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 4096), (33, 130, 5000), (100, 300, 9000),
                                   (128, 128, 16384), (127, 257, 2049), (260, 100, 6000),
                                   (16, 2500, 4100), (96, 20, 1024)])
def test_product_with_k_shared(lib, form, m, n, k):
    dtype = DTYPES[m % 2]
    x, qw, a, b = product_case(lib, m * 5 + n, m, n, k, form, dtype)
    q = lib.fp4_quantize(x, format=form)
    got = lib.fp4_gemm_tn(q, qw, dtype=dtype)
    check_product(got, a, b[0], k, dtype)
    assert torch.equal(got, lib.fp4_gemm_tn(q, qw, dtype=dtype))
    assert lib.fp4_get_device_error() == (0, 0)


@pytest.mark.parametrize("tokens,top_k,experts,dropped", [(1, 2, 4, 0.0), (3, 2, 5, 0.4),
                                                          (90, 1, 3, 0.1), (5, 3, 2, 1.0)])
def test_products_by_expert_with_k_shared(lib, tokens, top_k, experts, dropped):
    n, k = 200, 4360
    ids = random_ids(tokens, tokens, top_k, experts, dropped)
    x, qw, a, b = product_case(lib, tokens, tokens, n, k, "nvfp4", torch.float16, groups=experts)
    r = lib.moe_sort(ids, experts)
    out = lib.fp4_gemm_tn(lib.fp4_quantize(x, routing=r), qw)
    off, pairs = r.offsets.cpu().numpy(), lib.moe_pairs(r).cpu().numpy()
    for e in range(experts):
        if off[e] < off[e + 1]:
            seg = slice(off[e], off[e + 1])
            check_product(out[seg], a[pairs[seg] // top_k], b[e], k, torch.float16)
    assert not out[off[-1]:].any()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m,n,k", [(3, 40, 256), (130, 260, 512), (513, 390, 960)])
def test_product_of_small_integers_is_exact(lib, form, m, n, k):
    """Elements +-{0, 1, 2, 3, 4, 6} with scale 1 (a 6 in every block, or one of 4 for the power of
    two): every partial sum is an integer that fp32 holds, so only the last rounding is left."""
    rng = np.random.RandomState(m)
    a = rng.choice([0, 1, 2, 3, 4, 6, -1, -3], (m, k)).astype(np.float64)
    b = rng.choice([0, 1, 0, 2, -1, -2, 0, 4], (n, k)).astype(np.float64)
    a[:, ::16] = 6
    b[:, ::16] = 6
    qa = lib.fp4_quantize(torch.from_numpy(a).half().cuda(), format=form)
    qb = lib.fp4_quantize(torch.from_numpy(b).half().cuda(), format=form)
    _, scale = ref.stored(qa)
    assert (scale == 1).all()
    want = torch.from_numpy(a @ b.T).half()
    assert torch.equal(lib.fp4_gemm_tn(qa, qb).cpu(), want)


def test_alpha_and_exponents(lib):
    x, qw, a, b = product_case(lib, 9, 40, 100, 300, "nvfp4", torch.float16)
    q = lib.fp4_quantize(x, exponent=-3)
    av = ref.values(ref.to_numpy(x), "nvfp4", -3)
    for alpha in (0.0, -0.37, 3.5):
        check_product(lib.fp4_gemm_tn(q, qw, alpha=alpha), av, b[0], 300, torch.float16, alpha)


def test_output_beyond_fp16_is_infinite(lib):
    x = torch.full((2, 64), 1000.0, dtype=torch.float16, device="cuda")
    q = lib.fp4_quantize(x)
    assert torch.isposinf(lib.fp4_gemm_tn(q, q)).all()
    d = lib.fp4_gemm_tn(q, q, dtype=torch.bfloat16)
    assert torch.isfinite(d).all()


def test_nan_stays_in_its_row_and_column(lib):
    x, qw, a, b = product_case(lib, 11, 140, 150, 520, "nvfp4", torch.float16)
    x[131, 517] = float("nan")
    x[7, 3] = float("inf")
    w = rows(12, 150, 520, torch.float16)
    w[149, 0] = float("nan")
    got = ref.to_numpy(lib.fp4_gemm_tn(lib.fp4_quantize(x), lib.fp4_quantize(w)))
    want = np.zeros_like(got, dtype=bool)
    want[[131, 7]] = True
    want[:, 149] = True
    np.testing.assert_array_equal(np.isnan(got), want)


def test_empty_extents(lib):
    x0 = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    w = lib.fp4_quantize(rows(1, 48, 64, torch.float16))
    assert lib.fp4_gemm_tn(lib.fp4_quantize(x0), w).shape == (0, 48)
    k0 = torch.empty(5, 0, dtype=torch.float16, device="cuda")
    d = torch.full((5, 7), 3.0, dtype=torch.float16, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(k0), lib.fp4_quantize(k0.new_empty(7, 0)), out=d)
    assert not d.any()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("tokens,top_k,experts,dropped,only",
                         ROUTED + [(40, 4, 64, 0.0, None), (1500, 4, 9, 0.02, None),
                                   (900, 1, 2, 0.0, None)])
@pytest.mark.parametrize("n,k", [(72, 160), (300, 1040)])
def test_products_by_expert(lib, form, tokens, top_k, experts, dropped, only, n, k):
    dtype = DTYPES[tokens % 2]
    ids = random_ids(tokens + 1, tokens, top_k, experts, dropped, only)
    x, qw, a, b = product_case(lib, tokens, tokens, n, k, form, dtype, groups=experts)
    r = lib.moe_sort(ids, experts)
    out = torch.full((r.slots, n), float("nan"), dtype=dtype, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(x, format=form, routing=r), qw, dtype=dtype, out=out)
    off, pairs = r.offsets.cpu().numpy(), lib.moe_pairs(r).cpu().numpy()
    for e in range(experts):
        if off[e] < off[e + 1]:
            seg = slice(off[e], off[e + 1])
            check_product(out[seg], a[pairs[seg] // top_k], b[e], k, dtype)
    assert not out[off[-1]:].any()
    assert lib.fp4_get_device_error() == (0, 0)


# Enough rows an expert that CTA pairs share a tile; with 600 experts what a CTA keeps of the
# groups leaves its ring a stage less.
@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("slots,experts,n,k", [(6000, 5, 1500, 2048), (153600, 600, 512, 2048)])
def test_large_products_by_expert_are_exact(lib, form, slots, experts, n, k):
    """Small integers with scale 1, as above: the fp32 sums are exact in any order."""
    g = torch.Generator(device="cuda").manual_seed(slots)
    values = torch.tensor([0, 1, 2, 3, 4, 6, -1, -3], dtype=torch.float16, device="cuda")
    x = values[torch.randint(8, (slots, k), device="cuda", generator=g)]
    w = values[torch.randint(8, (experts * n, k), device="cuda", generator=g)]
    x[:, ::16] = 6
    w[:, ::16] = 6
    # uneven, one expert without rows, some slots dropped
    weight = torch.rand(experts, device="cuda", generator=g) + 0.5
    weight[1] = 0
    ids = torch.multinomial(weight, slots, replacement=True, generator=g).int()
    ids[torch.rand(slots, device="cuda", generator=g) < 0.02] = -1
    r = lib.moe_sort(ids.view(-1, 1), experts)
    qw = lib.fp4_quantize(w, format=form, group_rows=n)
    out = torch.full((slots, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.fp4_gemm_tn(lib.fp4_quantize(x, format=form, routing=r), qw, dtype=torch.bfloat16, out=out)
    off, order = r.offsets.tolist(), lib.moe_pairs(r).long()
    for e in range(experts):
        seg = slice(off[e], off[e + 1])
        want = x[order[seg]].double() @ w[e * n:(e + 1) * n].double().T
        assert torch.equal(out[seg], want.to(torch.bfloat16)), e
    assert not out[off[-1]:].any()
    assert lib.fp4_get_device_error() == (0, 0)


@pytest.mark.parametrize("m,n", [(3, 50), (200, 70)])
def test_uniform_groups(lib, m, n):
    """A batch of products: the same number of rows for every weight."""
    g, k = 6, 224
    x, qw, a, b = product_case(lib, 21, g * m, n, k, "mxfp4", torch.bfloat16, groups=g)
    q = lib.fp4_quantize(x, format="mxfp4", group_rows=m)
    got = lib.fp4_gemm_tn(q, qw, dtype=torch.bfloat16).view(g, m, n)
    for i in range(g):
        check_product(got[i], a[i * m:(i + 1) * m], b[i], k, torch.bfloat16)


def test_other_stream_and_repeats(lib):
    """The same bits on a side stream, again and again, without waiting in between."""
    x, qw, a, b = product_case(lib, 31, 390, 520, 1024, "nvfp4", torch.float16)
    first = lib.fp4_gemm_tn(lib.fp4_quantize(x), qw).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [lib.fp4_gemm_tn(lib.fp4_quantize(x), qw) for _ in range(5)]
    s.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    q = lib.fp4_quantize(x, stream=s)
    d = lib.fp4_gemm_tn(q, qw, stream=s)
    s.synchronize()
    assert torch.equal(first, d)


@pytest.mark.parametrize("m,n,k", [(4, 100, 256), (8, 300, 4096), (600, 4096, 512)])
def test_a_wait_that_runs_out_is_reported(lib, m, n, k):
    """On one CTA a tile, on a tile shared by several, and on pairs: loads that never come end in
    an error word of that stream, and the next call is right again."""
    x, qw, a, b = product_case(lib, m, m, n, k, "nvfp4", torch.float16)
    q = lib.fp4_quantize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lib.fp4_gemm_tn(q, qw, timeout_ns=20_000_000, inject=1, stream=s)
    assert lib.fp4_get_device_error() == (0, 0)
    status, raw = lib.fp4_get_device_error(s)
    assert status == 5 and raw >> 8 in (1, 2, 3, 4, 5)
    assert lib.fp4_get_device_error(s) == (0, 0)
    check_product(lib.fp4_gemm_tn(q, qw), a, b[0], k, torch.float16)


def test_outputs_belong_to_the_stream_of_the_call(lib):
    """Memory that work queued on the current stream still reads is not handed to a call that runs
    on another stream at once."""
    x, qw, a, b = product_case(lib, 33, 64, 512, 256, "nvfp4", torch.float16)
    q = lib.fp4_quantize(x)
    want = lib.fp4_gemm_tn(q, qw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = torch.full((64, 512), 7.0, dtype=torch.float16, device="cuda")
    address = kept.data_ptr()
    torch.cuda._sleep(20_000_000)                 # about 10 ms of the current stream
    copy = kept.clone()                           # reads `kept` after that
    del kept                                      # ... which the allocator may now reuse
    got = lib.fp4_gemm_tn(q, qw, stream=s)
    assert got.data_ptr() != address
    torch.cuda.synchronize()
    assert (copy == 7).all() and torch.equal(got, want)


def test_captured_into_a_graph(lib):
    x, qw, a, b = product_case(lib, 41, 24, 520, 1024, "nvfp4", torch.float16, groups=4)
    ids = random_ids(5, 24, 2, 4)
    def call():
        r = lib.moe_sort(ids, 4)
        return lib.fp4_gemm_tn(lib.fp4_quantize(x, routing=r), qw)
    want = call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    got.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got)


def test_offsets_past_32_bits(lib):
    """D of more than 2^32 bytes, and elements past 2^31: the last rows are right."""
    m, n, k = 70000, 32000, 32
    x = rows(51, m, k, torch.float16)
    w = rows(52, n, k, torch.float16)
    qw = lib.fp4_quantize(w)
    d = lib.fp4_gemm_tn(lib.fp4_quantize(x), qw)
    pick = torch.tensor([0, 1, 33000, 67107, 67108, 67109, m - 2, m - 1])
    a = ref.values(ref.to_numpy(x[pick.cuda()]), "nvfp4")
    check_product(d[pick.cuda()], a, ref.values(ref.to_numpy(w), "nvfp4"), k, torch.float16)


def test_refusals(lib):
    x = rows(1, 8, 64, torch.float16)
    q = lib.fp4_quantize(x)
    with pytest.raises(TypeError):
        lib.fp4_quantize(x.float())
    with pytest.raises(ValueError):
        lib.fp4_quantize(x.t())
    with pytest.raises(ValueError):
        lib.fp4_quantize(x, format="int4")
    with pytest.raises(ValueError):
        lib.fp4_quantize(x, group_rows=3)
    with pytest.raises(TypeError):
        lib.fp4_gemm_tn(q, q, dtype=torch.float32)
    with pytest.raises(lib.GemmError):
        lib.fp4_gemm_tn(q, lib.fp4_quantize(x, format="mxfp4"))
    with pytest.raises(lib.GemmError):
        lib.fp4_gemm_tn(q, lib.fp4_quantize(rows(2, 8, 96, torch.float16)))
    with pytest.raises(lib.GemmError):
        lib.fp4_gemm_tn(q, lib.fp4_quantize(x, group_rows=4))
    with pytest.raises(ValueError):
        lib.fp4_gemm_tn(q, q, out=torch.empty(8, 9, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        lib.Fp4Matrix(q.codes, q.scales[:, :1], cols=64)
    with pytest.raises(ValueError):
        lib.Fp4Matrix(q.codes, q.scales, cols=65)
    r = lib.moe_sort(torch.zeros(9, 1, dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(ValueError):
        lib.fp4_quantize(x, routing=r)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,cols", [(3, 1), (33, 7), (17, 9), (130, 255), (16, 257), (40, 264),
                                    (129, 1000), (21, 1411)])
def test_values_at_any_alignment(lib, form, dtype, n, cols):
    """Outputs that start at any 2-byte address, and nothing around them is written."""
    x = rows(n + cols, n, cols, torch.float16)
    q = lib.fp4_quantize(x, format=form)
    want = torch.from_numpy(ref.values(ref.to_numpy(x), form)).to(dtype)   # exact in either type
    for first in range(8):
        flat = torch.full((n * cols + 16,), 7.25, dtype=dtype, device="cuda")
        lib.fp4_dequantize(q, dtype=dtype, out=flat[first:first + n * cols].view(n, cols))
        got = flat.cpu()
        assert torch.equal(got[first:first + n * cols].view(n, cols), want)
        assert (got[:first] == 7.25).all() and (got[first + n * cols:] == 7.25).all()
