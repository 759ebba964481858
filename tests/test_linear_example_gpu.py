"""The example's 16-bit layers: gradients through autograd against autograd in 64 bits, and what
autograd is told (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from multistage_smem_pipeline_gb300 import moe_example
    return moe_example


def leaf(seed, *sizes, scale=1.0, dtype=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*sizes, device="cuda", generator=g) * scale).to(dtype).requires_grad_()


def plain(z, activation):
    return {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: torch.nn.functional.gelu(z),
            "gelu_tanh": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[activation]()


def close(got, want, roundings, dtype):
    """Roundings to the type, each by half a unit of terms of either sign: a norm adds them in squares,
    so that the sum of their bounds holds with room to spare."""
    unit = torch.finfo(dtype).eps / 2
    assert got.dtype == dtype or got.dtype == torch.float32
    assert (got.double() - want).norm() <= roundings * unit * want.norm()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("activation", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_s_gradients(ex, activation, dtype):
    x, w, b, r = leaf(1, 50, 72, dtype=dtype), leaf(2, 40, 72, scale=0.2, dtype=dtype), leaf(3, 40, dtype=dtype), \
        leaf(4, 50, 40, dtype=dtype)
    mix = leaf(5, 50, 40, dtype=dtype).detach()
    out = ex.linear(x, w, b, r, activation)
    (out.float() * mix.float()).sum().backward()
    d = [t.detach().double().requires_grad_() for t in (x, w, b, r)]
    want = plain(d[0] @ d[1].t() + d[2], activation) + d[3]
    (want * mix.double()).sum().backward()
    close(out.detach(), want.detach(), 1, dtype)
    assert torch.equal(r.grad, mix)
    # z, dz and the result are rounded; a slope changes by 1.2 times what z does, and relu's by 1 where z's
    # sign does, which a rounding never changes
    for got, exact in zip((x, w, b), d):
        close(got.grad, exact.grad, 4, dtype)


def test_only_what_is_needed(ex):
    for needs in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)):
        x, w, b = leaf(1, 20, 16), leaf(2, 24, 16), leaf(3, 24)
        for t, n in zip((x, w, b), needs):
            t.requires_grad_(bool(n))
        r = leaf(4, 20, 24)
        ex.linear(x, w, b, r, "gelu").float().sum().backward()      # an expanded gradient
        assert [t.grad is not None for t in (x, w, b)] == [bool(n) for n in needs]
        assert torch.equal(r.grad, torch.ones_like(r))


def test_a_layer_of_experts(ex):
    import multistage_smem_pipeline_gb300 as lib
    tokens, top_k, experts, hidden, inner = 40, 3, 5, 72, 56
    g = torch.Generator(device="cuda").manual_seed(7)
    ids = torch.randint(-1, experts, (tokens, top_k), device="cuda", generator=g).int()
    gates = torch.rand(tokens, top_k, device="cuda", generator=g).requires_grad_()
    leaves = [leaf(1, tokens, hidden), leaf(2, experts, inner, hidden, scale=0.1), leaf(3, experts, inner),
              leaf(4, experts, hidden, inner, scale=0.1), leaf(5, experts, hidden), gates]
    x, up, up_b, down, down_b, _ = leaves
    mix = leaf(6, tokens, hidden).detach()
    r = lib.moe_sort(ids, experts)
    rows = ex.expert_linear(ex.dispatch(x, r), r, up, up_b, "gelu_tanh")
    out = ex.combine(ex.expert_linear(rows, r, down, down_b), r, gates)
    (out.float() * mix.float()).sum().backward()

    xd, upd, upb, downd, downb, gd = d = [t.detach().double().requires_grad_() for t in leaves]
    e = ids.long().clamp(min=0)
    h = plain(torch.einsum("tkoh,th->tko", upd[e], xd) + upb[e], "gelu_tanh")
    y = torch.einsum("tkho,tko->tkh", downd[e], h) + downb[e]
    want = torch.where((ids >= 0)[..., None], gd[..., None] * y, 0.0).sum(1)
    (want * mix.double()).sum().backward()
    for got, exact in zip([out.detach()] + [t.grad for t in leaves], [want.detach()] + [t.grad for t in d]):
        close(got, exact, 8, torch.float16)       # rows, h, y and out; their four gradients


def test_no_second_derivatives(ex):
    x, w = leaf(1, 8, 16), leaf(2, 24, 16)
    gx, = torch.autograd.grad(ex.linear(x, w).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|differentiate"):
        gx.float().sum().backward()


def test_command_runs(ex, capsys):
    ex.main(["--tokens", "9", "--experts", "4", "--hidden", "256", "--out", "120", "--format", "mxfp4"])
    said = capsys.readouterr().out
    assert "same result: True" in said and "dense layer" in said
