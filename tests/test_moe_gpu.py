"""The routing of tokens to experts, the way back, and both gradients (GPU).

Tolerances.  Sums of k terms (or of H products, for the weights' gradient) in fp32 differ from the
exact ones by at most (terms + 1) 2^-24 of the sum of magnitudes, and outputs are then rounded to
their type once (half a unit).  Rows that are only moved are equal bit for bit."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]

SHAPES = [  # tokens, top_k, experts, hidden, dropped
    (1, 1, 1, 8, 0.0), (1, 8, 64, 2048, 0.0), (3, 2, 5, 1, 0.0), (16, 4, 64, 1411, 0.2),
    (77, 6, 60, 136, 0.0), (130, 3, 7, 7, 0.5), (500, 2, 1024, 64, 0.0), (1021, 6, 60, 250, 0.05),
    (40, 64, 100, 40, 0.1), (2048, 8, 128, 32, 0.0), (50, 4, 8, 96, 1.0), (4099, 8, 256, 16, 0.02),
    (3000, 4, 16, 45, 0.03), (1300, 8, 5, 2051, 0.1)]


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def make(seed, tokens, top_k, experts, dropped):
    rng = np.random.RandomState(seed)
    popular = rng.rand(experts) ** 3 + 1e-3
    ids = rng.choice(experts, (tokens, top_k), p=popular / popular.sum())
    lost = rng.rand(tokens, top_k) < dropped
    ids = np.where(lost, rng.choice([-1, experts, 2**31 - 1, -(2**31)], (tokens, top_k)), ids)
    return ids


def to_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def check_sort(lib, ids, experts):
    r = lib.moe_sort(to_gpu(ids, torch.int32), experts)
    off, rows, pairs = ref.sort(ids, experts)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(r.rows.cpu().numpy(), rows)
    np.testing.assert_array_equal(lib.moe_pairs(r).cpu().numpy(), pairs)
    return r


@pytest.mark.parametrize("tokens,top_k,experts,hidden,dropped", SHAPES)
def test_sort(lib, tokens, top_k, experts, hidden, dropped):
    check_sort(lib, make(tokens, tokens, top_k, experts, dropped), experts)


@pytest.mark.parametrize("tokens,top_k,experts", [(8192, 8, 128), (33333, 3, 17), (200001, 2, 1024),
                                                  (1 << 20, 1, 2), (70000, 64, 300)])
def test_sort_of_many(lib, tokens, top_k, experts):
    check_sort(lib, make(1, tokens, top_k, experts, 0.03), experts)


@pytest.mark.parametrize("tokens", [1, 31, 32, 33, 1023, 1024, 1025, 4095, 4096, 4097, 8191, 8193,
                                    16384, 16385, 32769])
def test_sort_around_the_block_sizes(lib, tokens):
    check_sort(lib, make(tokens, tokens, 1, 9, 0.1), 9)
    check_sort(lib, np.zeros((tokens, 1), dtype=np.int64), 3)          # all to the first
    check_sort(lib, np.full((tokens, 1), 2, dtype=np.int64), 3)        # ... the last
    check_sort(lib, np.full((tokens, 1), -1, dtype=np.int64), 3)       # ... to none


def test_sort_of_nothing(lib):
    r = lib.moe_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert r.offsets.tolist() == [0] * 6 and r.slots == 0
    x = torch.empty(0, 16, dtype=torch.float16, device="cuda")
    assert lib.moe_dispatch(x, r).shape == (0, 16)
    assert lib.moe_combine(x, r, torch.empty(0, 4, device="cuda")).shape == (0, 16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top_k,experts,hidden,dropped", SHAPES)
def test_rows_out_and_back(lib, dtype, tokens, top_k, experts, hidden, dropped):
    ids = make(tokens + 9, tokens, top_k, experts, dropped)
    rng = np.random.RandomState(tokens)
    kept = (ids >= 0) & (ids < experts)
    r = lib.moe_sort(to_gpu(ids, torch.int32), experts)
    off, rows, pairs = ref.sort(ids, experts)
    live = np.arange(tokens * top_k) < off[-1]
    x = to_gpu(rng.randn(tokens, hidden), dtype)
    xd = ref.to_numpy(x)

    got = lib.moe_dispatch(x, r)
    np.testing.assert_array_equal(ref.to_numpy(got), np.where(live[:, None], xd[pairs // top_k], 0))

    # what dropped slots hold must not be looked at
    y = to_gpu(rng.randn(tokens * top_k, hidden), dtype)
    w = to_gpu(rng.rand(tokens, top_k), torch.float32)
    y[~torch.from_numpy(live).cuda()] = float("nan")
    w[~torch.from_numpy(kept).cuda()] = float("inf")
    yd = np.where(live[:, None], ref.to_numpy(y), 0)[rows]
    wd = np.where(kept, ref.to_numpy(w), 0)
    out = lib.moe_combine(y, r, w)
    check_sum(out, (wd[..., None] * yd).sum(1), np.abs(wd[..., None] * yd).sum(1), top_k, dtype)
    back = lib.moe_dispatch_backward(y, r)
    check_sum(back, yd.sum(1), np.abs(yd).sum(1), top_k, dtype)

    grad = to_gpu(rng.randn(tokens, hidden), dtype)
    gd = ref.to_numpy(grad)
    grad_y, grad_w = lib.moe_combine_backward(grad, y, r, w)
    want = np.where(live[:, None], wd.reshape(-1)[pairs][:, None] * gd[pairs // top_k], 0)
    check_sum(grad_y, want, np.abs(want), 1, dtype)
    prod = np.where(kept[..., None], gd[:, None, :] * yd, 0)
    err = np.abs(ref.to_numpy(grad_w) - prod.sum(2))
    assert (err <= (hidden + 1) * 2.0 ** -24 * np.abs(prod).sum(2)).all()


def check_sum(got, want, magnitude, terms, dtype):
    acc = (terms + 1) * 2.0 ** -24 * magnitude
    err = np.abs(ref.to_numpy(got) - want)
    assert (err <= acc + ref.half_unit(np.abs(want) + acc, dtype)).all(), err.max()


def test_gradients_are_differences(lib):
    """combine is linear in y and in the weights, and dispatch in x: with small integers all of it
    is exact, so a unit step in one input changes the loss by exactly its gradient."""
    tokens, top_k, experts, hidden = 9, 3, 4, 40
    rng = np.random.RandomState(0)
    ids = make(3, tokens, top_k, experts, 0.2)
    r = lib.moe_sort(to_gpu(ids, torch.int32), experts)
    x = to_gpu(rng.randint(-3, 4, (tokens, hidden)), torch.float16)
    w = to_gpu(rng.randint(-2, 3, (tokens, top_k)), torch.float32)
    grad = to_gpu(rng.randint(-2, 3, (tokens, hidden)), torch.float16)

    def loss(x, w, dy=None):
        y = lib.moe_dispatch(x, r)
        if dy is not None:
            y = y + dy
        return (lib.moe_combine(y, r, w).double() * grad.double()).sum().item()

    y = lib.moe_dispatch(x, r)
    grad_y, grad_w = lib.moe_combine_backward(grad, y, r, w)
    grad_x = lib.moe_dispatch_backward(grad_y, r)
    base = loss(x, w)
    for t in range(tokens):
        for j in range(top_k):
            w2 = w.clone()
            w2[t, j] += 1
            assert loss(x, w2) - base == grad_w[t, j].item()
    for _ in range(40):
        t, h = rng.randint(tokens), rng.randint(hidden)
        x2 = x.clone()
        x2[t, h] += 1
        assert loss(x2, w) - base == grad_x[t, h].item()
        row = rng.randint(tokens * top_k)
        dy = torch.zeros_like(y)
        dy[row, h] = 1
        assert loss(x, w, dy) - base == grad_y[row, h].item()


def test_strided_and_misaligned_rows(lib):
    base = torch.randn(50, 530, device="cuda").half()
    ids = make(1, 50, 2, 6, 0.1)
    r = lib.moe_sort(to_gpu(ids, torch.int32), 6)
    off, rows, pairs = ref.sort(ids, 6)
    live = np.arange(100) < off[-1]
    for x in (base[:, 16:528], base[:, 1:512], base[:, 3:4]):
        want = np.where(live[:, None], ref.to_numpy(x)[pairs // 2], 0)
        np.testing.assert_array_equal(ref.to_numpy(lib.moe_dispatch(x, r)), want)
    # outputs that start off a 16-byte boundary
    flat = torch.empty(100 * 64 + 1, dtype=torch.float16, device="cuda")
    out = flat[1:].view(100, 64)
    x = base[:, :64]
    lib.moe_dispatch(x, r, out=out)
    np.testing.assert_array_equal(ref.to_numpy(out),
                                  np.where(live[:, None], ref.to_numpy(x)[pairs // 2], 0))


def test_rows_past_32_bits(lib):
    """A gathered matrix of more than 2^31 elements."""
    tokens, top_k, hidden = 40000, 8, 7168
    ids = torch.arange(tokens * top_k, dtype=torch.int32, device="cuda").view(tokens, top_k) % 11
    r = lib.moe_sort(ids, 11)
    x = torch.randn(tokens, hidden, device="cuda").half()
    y = lib.moe_dispatch(x, r)
    last = torch.arange(tokens * top_k - 5, tokens * top_k, device="cuda")
    assert torch.equal(y[last], x[(lib.moe_pairs(r)[last] // top_k).long()])
    w = torch.full((tokens, top_k), 0.125, device="cuda")
    assert torch.equal(lib.moe_combine(y, r, w)[-5:], x[-5:])


def test_same_bits_every_time(lib):
    ids = make(2, 700, 6, 20, 0.05)
    r = lib.moe_sort(to_gpu(ids, torch.int32), 20)
    y = torch.randn(4200, 1000, device="cuda").bfloat16()
    g = torch.randn(700, 1000, device="cuda").bfloat16()
    w = torch.rand(700, 6, device="cuda")
    first = lib.moe_combine(y, r, w), *lib.moe_combine_backward(g, y, r, w)
    for _ in range(3):
        again = lib.moe_combine(y, r, w), *lib.moe_combine_backward(g, y, r, w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("make_in", [False, True])
@pytest.mark.parametrize("read_in", [False, True])
def test_arrays_inside_and_outside_inference_mode(lib, make_in, read_in):
    """A routing's and a matrix's tensors are parts of one buffer, whichever mode asks for them."""
    ids = torch.tensor([[2, 0], [1, 2], [-1, 2]], dtype=torch.int32, device="cuda")
    x = torch.arange(3 * 40, device="cuda").view(3, 40).half()
    with torch.inference_mode(make_in):
        r = lib.moe_sort(ids, 3)
        q = lib.fp4_quantize(x, format="mxfp4", routing=r)
    with torch.inference_mode(read_in):
        offsets, rows, codes, scales = r.offsets, r.rows, q.codes, q.scales
        same = lib.Routing(offsets, rows, ids)
        again = lib.Fp4Matrix(codes, scales, cols=40, format="mxfp4", routing=same)
        assert torch.equal(lib.fp4_dequantize(again), lib.fp4_dequantize(q))
    assert offsets.tolist() == [0, 1, 2, 5]
    assert rows.tolist() == [[2, 0], [1, 3], [5, 4]]
    assert codes.shape == (6, 32) and scales.shape == (6 // 128 + 3, 2, 512)
    assert offsets.untyped_storage().data_ptr() == rows.untyped_storage().data_ptr()
    del r, q, same, again
    assert offsets.tolist() == [0, 1, 2, 5]


def test_refusals(lib):
    ids = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    r = lib.moe_sort(ids, 3)
    y = torch.zeros(10, 16, dtype=torch.float16, device="cuda")
    w = torch.zeros(5, 2, device="cuda")
    with pytest.raises(TypeError):
        lib.moe_sort(ids.long(), 3)
    with pytest.raises(ValueError):
        lib.moe_sort(ids.t(), 3)
    with pytest.raises(ValueError):
        lib.moe_sort(ids, 1025)
    with pytest.raises(ValueError):
        lib.moe_dispatch(y, r)
    with pytest.raises(TypeError):
        lib.moe_combine(y.float(), r, w)
    with pytest.raises(TypeError):
        lib.moe_combine(y, r, w.half())
    with pytest.raises(ValueError):
        lib.moe_combine(y, r, w[:, :1])
    with pytest.raises(ValueError):
        lib.moe_combine(y[:9], r, w)
    with pytest.raises(ValueError):
        lib.moe_combine_backward(y[:5, :8], y, r, w)
    with pytest.raises(ValueError):
        lib.moe_combine(y, r, w, out=y[:4])
