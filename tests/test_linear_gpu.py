"""Linear layers with bias, activation and residual, dense and by expert, and their gradients (GPU),
against the definitions in 64 bits (linear_reference.py, which derives the tolerances)."""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]
# every way of cutting a product: (cta_pair, tile, split_k)
FORMS = [(1, 256, 1)] + [(0, tile, split) for tile in (32, 64, 128, 256) for split in (1, 2, 4, 8)]
FEW = [(0, rows, split) for rows in (1, 2, 4, 8) for split in (1, 2, 4, 8)]   # forward alone

# rows, out, in
SHAPES = [(1, 8, 8), (1, 1, 1), (1, 300, 64), (2, 64, 72), (31, 33, 63), (32, 256, 64), (33, 40, 65),
          (64, 16, 128), (65, 250, 200), (127, 129, 130), (128, 128, 64), (129, 257, 192),
          (200, 328, 264), (256, 256, 256), (257, 513, 96), (300, 1000, 77), (517, 1001, 141),
          (700, 520, 1000)]


@pytest.fixture(scope="module")
def lib():
    import multistage_smem_pipeline_gb300 as m
    return m


def values(seed, *sizes, dtype=torch.float16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*sizes, device="cuda", generator=g) * scale).to(dtype)


def make(rows, out, hidden, dtype, experts=None, seed=0):
    lead = () if experts is None else (experts,)
    return {"x": values(seed, rows, hidden, dtype=dtype),
            "w": values(seed + 1, *lead, out, hidden, dtype=dtype, scale=2 * max(hidden, 1) ** -0.5),
            "bias": values(seed + 2, *lead, out, dtype=dtype),
            "residual": values(seed + 3, rows, out, dtype=dtype),
            "grad": values(seed + 4, rows, out, dtype=dtype),
            "z": values(seed + 5, rows, out, dtype=dtype, scale=2.0)}


def routing_of(lib, counts, dropped=0, top_k=1):
    """A routing with so many rows for each expert, then those of dropped slots."""
    ends = torch.tensor([0] + list(counts)).cumsum(0)
    slots = int(ends[-1]) + dropped
    assert slots % top_k == 0
    ids = torch.zeros(slots // top_k, top_k, dtype=torch.int32, device="cuda")
    rows = torch.arange(slots, dtype=torch.int32, device="cuda").view(ids.shape)
    return lib.Routing(ends.int().cuda(), rows, ids), ends.tolist()


def check_forward(lib, m, activation, bias=True, residual=True, form=None):
    b, r = (m["bias"] if bias else None), (m["residual"] if residual else None)
    out, z = lib.linear(m["x"], m["w"], b, activation=activation, residual=r, save_preact=True, form=form)
    want, err, wz, zerr = ref.forward(m["x"], m["w"], b, r, activation)
    ref.check(out, want, err, f"out {activation} {form}")
    ref.check(z, wz, zerr, f"z {form}")
    again = lib.linear(m["x"], m["w"], b, activation=activation, residual=r, form=form)
    assert torch.equal(again, out)


def check_backward(lib, m, activation, routing=None, offsets=None, form=None):
    z = None if activation == "none" else m["z"]
    weight = form is None or form[1] != 32       # grad_w has no such tiles
    kw = dict(preact=z, activation=activation, need_weight=weight, need_bias=True, form=form)
    if routing is None:
        got = lib.linear_backward(m["grad"], m["x"], m["w"], **kw)
    else:
        got = lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], **kw)
    want = ref.backward(m["grad"], m["x"], m["w"], z, activation, offsets)
    for g, (v, e), name in zip(got, want, ("grad_x", "grad_w", "grad_bias")):
        if g is not None:
            ref.check(g, v, e, f"{name} {activation} {form}")
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,out,hidden", SHAPES)
def test_forward(lib, dtype, rows, out, hidden):
    m = make(rows, out, hidden, dtype)
    for i, activation in enumerate(ref.ACTIVATIONS):
        check_forward(lib, m, activation, bias=i % 2 == 0, residual=i % 3 != 0)
    check_forward(lib, m, "gelu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,out,hidden", SHAPES)
def test_backward(lib, dtype, rows, out, hidden):
    m = make(rows, out, hidden, dtype)
    for activation in ref.ACTIVATIONS:
        check_backward(lib, m, activation)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,out,hidden", [(1, 8, 8), (40, 72, 1000), (130, 264, 200), (300, 520, 648),
                                             (129, 257, 66)])
def test_every_form(lib, form, rows, out, hidden):
    dtype = DTYPES[(rows + form[1]) % 2]
    m = make(rows, out, hidden, dtype, seed=7)
    check_forward(lib, m, "silu", form=form)
    check_backward(lib, m, "silu", form=form)


@pytest.mark.parametrize("form", FEW)
@pytest.mark.parametrize("rows,out,hidden", [(1, 8, 8), (1, 1, 1), (3, 257, 1000), (8, 72, 2056), (9, 30, 4097),
                                             (21, 3, 513), (5, 1003, 24)])
def test_few_rows(lib, form, rows, out, hidden):
    for dtype in DTYPES:
        m = make(rows, out, hidden, dtype, seed=17)
        check_forward(lib, m, "gelu", form=form)
        counts = (2, 0, rows, 1)
        m = make(rows + 5, out, hidden, dtype, experts=4, seed=19)
        routing, offsets = routing_of(lib, counts, 2)
        m["x"][offsets[-1]:] = float("nan")
        got, z = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True, form=form)
        want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], None, "silu", offsets)
        ref.check(got, want, err, "out")
        ref.check(z, wz, zerr, "z")


@pytest.mark.parametrize("form", [None] + FORMS)
@pytest.mark.parametrize("counts,dropped", [((5,), 0), ((0, 3, 0, 0, 1), 4), ((16, 33, 130, 0, 65, 257), 6),
                                            ((128, 64, 256, 16), 0), ((1, 1, 1, 1, 1, 1, 1, 1), 8),
                                            ((0, 0, 0), 3), ((301, 95), 100)])
def test_experts(lib, form, counts, dropped):
    dtype = DTYPES[len(counts) % 2]
    for out, hidden in ((72, 136), (257, 100), (24, 77)):
        rows = sum(counts) + dropped
        m = make(rows, out, hidden, dtype, experts=len(counts), seed=3)
        routing, offsets = routing_of(lib, counts, dropped)
        for t in ("x", "grad", "z"):      # rows of nobody must not be looked at
            m[t][offsets[-1]:] = float("nan")
        got, z = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="gelu", save_preact=True, form=form)
        want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], None, "gelu", offsets)
        ref.check(got, want, err, "out")
        ref.check(z, wz, zerr, "z")
        check_backward(lib, m, "gelu", routing, offsets, form)
        check_backward(lib, m, "none", routing, offsets, form)


@pytest.mark.parametrize("form", [None] + FORMS)
def test_a_neighbour_s_nan_stays_its_own(lib, form):
    """Rows and weights of one expert that are NaN or infinite change nothing of another's."""
    counts = (13, 70, 1, 130)
    for out, hidden in ((40, 72), (33, 50)):
        m = make(sum(counts), out, hidden, torch.float16, experts=4, seed=11)
        routing, offsets = routing_of(lib, counts)
        clean = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="relu", form=form)
        grads = check_backward(lib, m, "relu", routing, offsets, form)
        for e in range(4):
            d = {k: v.clone() for k, v in m.items()}
            a, b = offsets[e], offsets[e + 1]
            for t, v in (("x", "nan"), ("grad", "inf"), ("z", "nan")):
                d[t][a:b] = float(v)
            d["w"][e] = float("inf")
            d["bias"][e] = float("nan")
            out2 = lib.moe_linear(d["x"], routing, d["w"], d["bias"], activation="relu", form=form)
            others = [i for i in range(4) if i != e]
            for i in others:
                s = slice(offsets[i], offsets[i + 1])
                assert torch.equal(out2[s], clean[s])
            gx, gw, gb = lib.moe_linear_backward(d["grad"], d["x"], routing, d["w"], preact=d["z"], activation="relu",
                                                 need_weight=grads[1] is not None, need_bias=True, form=form)
            for i in others:
                s = slice(offsets[i], offsets[i + 1])
                assert torch.equal(gx[s], grads[0][s])
                assert gw is None or torch.equal(gw[i], grads[1][i])
                assert torch.equal(gb[i], grads[2][i])


@pytest.mark.parametrize("form", [None, (1, 256, 1), (0, 128, 1), (0, 256, 8)])
def test_small_integers_are_exact(lib, form):
    """Sums that fp32 and the type hold exactly come out bit for bit, whatever the form."""
    for dtype in DTYPES:
        g = torch.Generator(device="cuda").manual_seed(5)
        x = torch.randint(-1, 2, (300, 200), device="cuda", generator=g).to(dtype)
        w = torch.randint(-1, 2, (264, 200), device="cuda", generator=g).to(dtype)
        b = torch.randint(-3, 4, (264,), device="cuda", generator=g).to(dtype)
        grad = (torch.randint(0, 12, (300, 264), device="cuda", generator=g) == 0).to(dtype)
        assert torch.equal(lib.linear(x, w, b, form=form).double(), x.double() @ w.double().t() + b.double())
        gx, gw, gb = lib.linear_backward(grad, x, w, need_bias=True, form=form)
        assert torch.equal(gx.double(), grad.double() @ w.double())
        assert torch.equal(gw.double(), grad.double().t() @ x.double())
        assert torch.equal(gb.double(), grad.double().sum(0))


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_and_misaligned_rows(lib, dtype):
    rows, out, hidden = 70, 136, 200

    def cut(t, first, gap):
        wide = torch.full((t.shape[0], t.shape[1] + first + gap), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, first:first + t.shape[1]] = t
        return wide[:, first:first + t.shape[1]]

    m = make(rows, out, hidden, dtype, seed=21)
    for first, gap in ((0, 8), (8, 16), (1, 0), (3, 4), (0, 1)):
        d = dict(m)
        for t in ("x", "w", "residual", "grad"):
            d[t] = cut(m[t], first, gap)
        check_forward(lib, d, "gelu_tanh")
        check_backward(lib, d, "gelu_tanh")
        check_backward(lib, d, "none")
    # outputs, biases and kept sums off a 16-byte boundary
    flat = torch.empty(rows * out + 1, dtype=dtype, device="cuda")
    got = flat[1:].view(rows, out)
    bias = torch.empty(out + 1, dtype=dtype, device="cuda")[1:].copy_(m["bias"])
    want = lib.linear(m["x"], m["w"], m["bias"], residual=m["residual"])
    assert lib.linear(m["x"], m["w"], bias, residual=m["residual"], out=got) is not None
    assert torch.equal(got, want)
    z = torch.empty(rows * out + 3, dtype=dtype, device="cuda")[3:].view(rows, out).copy_(m["z"])
    for a, b in zip(lib.linear_backward(m["grad"], m["x"], m["w"], preact=z, activation="silu", need_bias=True),
                    lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="silu", need_bias=True)):
        assert torch.equal(a, b)


def test_empty_sizes(lib):
    for dtype in DTYPES:
        for rows, out, hidden in ((0, 8, 16), (5, 0, 16), (5, 8, 0), (0, 0, 0), (5, 7, 0), (0, 7, 5), (300, 300, 0)):
            m = make(rows, out, hidden, dtype)
            check_forward(lib, m, "gelu")
            check_backward(lib, m, "silu")
            check_backward(lib, m, "none")
    routing, offsets = routing_of(lib, (0, 0))
    m = make(0, 24, 16, torch.float16, experts=2)
    assert lib.moe_linear(m["x"], routing, m["w"], m["bias"]).shape == (0, 24)
    for g in lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], need_bias=True):
        assert not g.any()


def test_each_gradient_alone(lib):
    m = make(90, 72, 136, torch.bfloat16, seed=2)
    both = lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True)
    kw = dict(preact=m["z"], activation="gelu")
    gx, none1, none2 = lib.linear_backward(m["grad"], None, m["w"], need_weight=False, **kw)
    assert none1 is None and none2 is None and torch.equal(gx, both[0])
    none1, gw, none2 = lib.linear_backward(m["grad"], m["x"], None, need_x=False, **kw)
    assert none1 is None and none2 is None and torch.equal(gw, both[1])
    none1, none2, gb = lib.linear_backward(m["grad"], None, None, need_x=False, need_weight=False, need_bias=True, **kw)
    assert none1 is None and none2 is None and torch.equal(gb, both[2])
    assert lib.linear_backward(m["grad"], m["x"], m["w"], need_x=False, need_weight=False, **kw) == (None,) * 3


@pytest.mark.parametrize("activation", ref.ACTIVATIONS)
def test_gradients_are_differences(lib, activation):
    """The gradients against central differences of the forward pass in 64 bits."""
    rows, out, hidden = 9, 16, 24
    m = make(rows, out, hidden, torch.float16, seed=9)
    x, w, b, g = (m[k].double() for k in ("x", "w", "bias", "grad"))
    z = x @ w.t() + b
    z16 = z.half()
    gx, gw, gb = lib.linear_backward(m["grad"], m["x"], m["w"], preact=z16, activation=activation, need_bias=True)

    def loss(x, w, b):
        return (ref.act(x @ w.t() + b, activation) * g).sum().item()

    # z is rounded to fp16 (2^-11 of up to 8) before the slope, whose own slope is below 1.1; dz is
    # rounded to fp16: together 2^-8 of grad for each term of a sum
    h = 1e-6
    for t, got, terms in ((x, gx, w.abs().sum(0)[None, :].expand(rows, -1)), (w, gw, x.abs().sum(0)[None, :].expand(out, -1)),
                          (b, gb, torch.full((out,), float(rows), device="cuda"))):
        for i in range(0, t.numel(), 7):
            at = torch.unravel_index(torch.tensor(i), t.shape)
            keep = t[at].item()
            if activation == "relu" and z.abs().min() < 1e-4:
                pytest.skip("a kink in the way")
            t[at] = keep + h
            up = loss(x, w, b)
            t[at] = keep - h
            down = loss(x, w, b)
            t[at] = keep
            allowed = 2.0 ** -8 * float(terms[at]) * float(g.abs().max()) + 1e-4
            assert abs((up - down) / (2 * h) - float(got[at])) <= allowed


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("activation", ref.ACTIVATIONS)
def test_activations_over_their_whole_range(lib, dtype, activation):
    """Every finite value of the type as z, by the identity (in >= 1 of one input), and as preact."""
    every = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(dtype)
    every = every[torch.isfinite(every)]
    n = every.numel() // 8 * 8
    x = every[:n].view(-1, 8)
    w = torch.eye(8, dtype=dtype, device="cuda")
    got = lib.linear(x, w, activation=activation)
    want = ref.act(x.double(), activation)
    err = 2.0 ** -14 * want.abs() + 2.0 ** -126
    big = want.abs() > torch.finfo(dtype).max
    ref.check(torch.where(big, 0.0, got.double()).to(dtype), torch.where(big, 0.0, want), err, activation)
    if activation != "none":
        one = torch.ones_like(x)
        gx = lib.linear_backward(one, None, w, preact=x, activation=activation, need_weight=False)[0]
        s = ref.slope(x.double().clamp(-100, 100), activation)
        ref.check(gx, s, 2.0 ** -13 * torch.minimum(s.abs() + 2.0 ** -4, torch.ones_like(s)), "slope " + activation)


def test_nan_and_infinity_come_through(lib):
    x = torch.tensor([[float("nan")] * 8, [float("inf")] + [0.0] * 7, [1.0] * 8], device="cuda").half()
    w = torch.eye(8, device="cuda").half()
    for activation in ref.ACTIVATIONS:
        out = lib.linear(x, w, activation=activation)
        assert out[0].isnan().all() and torch.isfinite(out[2]).all()
        g = lib.linear_backward(torch.ones_like(x), None, w, preact=x, activation=activation, need_weight=False)[0]
        assert torch.isfinite(g[2]).all()
    s = lib.linear_backward(torch.ones_like(x), None, w, preact=torch.full_like(x, float("inf")), activation="silu",
                            need_weight=False)[0]
    assert (s == 1).all()


def test_same_bits_every_time(lib):
    m = make(700, 264, 520, torch.bfloat16, seed=4)
    first = lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True)
    for _ in range(3):
        again = lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed(lib):
    m = make(200, 264, 136, torch.float16, experts=3, seed=6)
    routing, offsets = routing_of(lib, (70, 0, 125), 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, z = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True)
        grads = lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], preact=z, activation="silu", need_bias=True)
    for seed in (1, 2):
        n = make(200, 264, 136, torch.float16, experts=3, seed=100 * seed)
        for k in ("x", "w", "bias", "grad"):
            m[k].copy_(n[k])
        graph.replay()
        got, gz = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True)
        assert torch.equal(out, got) and torch.equal(z, gz)
        for a, b in zip(grads, lib.moe_linear_backward(m["grad"], m["x"], routing, m["w"], preact=gz, activation="silu",
                                                       need_bias=True)):
            assert torch.equal(a, b)


def test_on_other_streams_at_once(lib):
    sets = [make(150, 200, 333, torch.float16, seed=40 + i) for i in range(3)]
    want = [lib.linear(m["x"], m["w"], m["bias"], activation="gelu") for m in sets]
    grads = [lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True) for m in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        for s, m in zip(streams, sets):
            got.append((lib.linear(m["x"], m["w"], m["bias"], activation="gelu", stream=s),
                        lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True,
                                            stream=s)))
    torch.cuda.synchronize()
    for i, (o, g) in enumerate(got):
        assert torch.equal(o, want[i % 3])
        assert all(torch.equal(a, b) for a, b in zip(g, grads[i % 3]))
    assert all(lib.linear_get_device_error(s) == (0, 0) for s in streams)


@pytest.mark.parametrize("form", [None, (1, 256, 1), (0, 64, 1), (0, 128, 8), (0, 256, 2)])
def test_the_most_experts(lib, form):
    """1024 experts, most of them without a row, one with many."""
    counts = [0] * 1024
    for e, rows in ((0, 1), (1, 17), (500, 300), (501, 2), (1023, 33)):
        counts[e] = rows
    m = make(sum(counts) + 5, 40, 72, torch.bfloat16, experts=1024, seed=21)
    routing, offsets = routing_of(lib, counts, 5)
    for t in ("x", "grad", "z"):
        m[t][offsets[-1]:] = float("nan")
    got, z = lib.moe_linear(m["x"], routing, m["w"], m["bias"], activation="silu", save_preact=True, form=form)
    want, err, wz, zerr = ref.forward(m["x"], m["w"], m["bias"], None, "silu", offsets)
    ref.check(got, want, err, "out")
    ref.check(z, wz, zerr, "z")
    check_backward(lib, m, "silu", routing, offsets, form)


def test_two_graphs_replayed_at_once(lib):
    """Each has workspaces of its own (unaligned rows are copied to them, dz and strips are there)."""
    sets = [make(230, 201, 335, torch.float16, seed=60 + i) for i in range(2)]
    calls = [lambda m=m: (lib.linear(m["x"], m["w"], m["bias"], activation="gelu"),
                          *lib.linear_backward(m["grad"], m["x"], m["w"], preact=m["z"], activation="gelu", need_bias=True))
             for m in sets]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(c())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,out,hidden", [(300, 264, 520), (2000, 1000, 1411)])
def test_what_follows_a_backward_pass_follows_all_of_it(lib, rows, out, hidden):
    """grad_w may run beside grad_x: the next kernels still come after both, and what came before, before."""
    m = make(rows, out, hidden, torch.bfloat16, seed=70)
    w2 = values(71, 64, hidden, dtype=torch.bfloat16, scale=0.05)
    kw = dict(preact=m["z"], activation="silu", need_bias=True)
    want = [t.clone() for t in lib.linear_backward(m["grad"], m["x"], m["w"], **kw)]
    then = lib.linear(want[0], w2)
    torch.cuda.synchronize()
    d = {k: torch.empty_like(m[k]) for k in ("x", "w", "grad", "z")}
    kw["preact"] = d["z"]
    results = []
    for _ in range(10):
        for k in d:
            d[k].copy_(m[k])
        g = lib.linear_backward(d["grad"], d["x"], d["w"], **kw)
        results.append((*g, lib.linear(g[0], w2)))
        for k in d:
            d[k].fill_(float("nan"))
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, (*want, then)))


@pytest.mark.parametrize("form", [(1, 256, 1), (0, 128, 1), (0, 256, 4)])
def test_a_wait_that_runs_out_is_reported(lib, form):
    m = make(300, 264, 400, torch.float16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert lib.linear_get_device_error(s) == (0, 0)
    lib.linear(m["x"], m["w"], form=form, timeout_ns=20_000_000, inject=1, stream=s)
    status, raw = lib.linear_get_device_error(s)
    assert status == 5 and raw & 0xff == 5 and raw >> 8
    assert lib.linear_get_device_error(s) == (0, 0)
    got = lib.linear(m["x"], m["w"], form=form, stream=s)
    s.synchronize()
    ref.check(got, *ref.forward(m["x"], m["w"])[:2], "after")


def test_matrices_past_32_bits(lib):
    """More than 2^31 elements in x, in out and in w."""
    rows, hidden = 1 << 19, 4160
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    x[-3:] = values(1, 3, hidden, dtype=torch.bfloat16)
    w = values(2, 64, hidden, dtype=torch.bfloat16, scale=0.05)
    out = lib.linear(x, w)
    ref.check(out[-3:], *ref.forward(x[-3:], w)[:2], "long x")
    assert not out[:-3].any()
    grad = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    grad[-3:] = values(3, 3, 64, dtype=torch.bfloat16)
    gx, gw, gb = lib.linear_backward(grad, x, w, need_bias=True)
    want = ref.backward(grad[-3:], x[-3:], w, None)
    ref.check(gx[-3:], *want[0], "grad_x")
    ref.check(gw, want[1][0], want[1][1] + 2 * rows * 2.0 ** -23 * want[1][0].abs(), "grad_w")
    ref.check(gb, want[2][0], want[2][1], "grad_bias")
    assert not gx[:-3].any()
    del x, gx, out
    experts = 8
    w = torch.zeros(experts, 1 << 16, hidden, dtype=torch.bfloat16, device="cuda")
    w[-1, -16:] = values(4, 16, hidden, dtype=torch.bfloat16, scale=0.05)
    routing, offsets = routing_of(lib, [0] * 7 + [5])
    x = values(5, 5, hidden, dtype=torch.bfloat16)
    out = lib.moe_linear(x, routing, w)
    ref.check(out[:, -16:], *ref.forward(x, w[-1, -16:])[:2], "long w")
    assert not out[:, :-16].any()


def test_together_with_the_routing(lib):
    """Sort, dispatch, two layers of experts, combine, and all the way back, against 64-bit autograd."""
    tokens, top_k, experts, hidden, inner = 60, 3, 5, 72, 136
    g = torch.Generator(device="cuda").manual_seed(12)
    ids = torch.randint(-1, experts, (tokens, top_k), device="cuda", generator=g).int()
    gates = torch.rand(tokens, top_k, device="cuda", generator=g)
    x = values(1, tokens, hidden, dtype=torch.float16)
    w1 = values(2, experts, inner, hidden, dtype=torch.float16, scale=0.1)
    w2 = values(3, experts, hidden, inner, dtype=torch.float16, scale=0.1)
    b1, b2 = values(4, experts, inner, dtype=torch.float16), values(5, experts, hidden, dtype=torch.float16)
    mix = values(6, tokens, hidden, dtype=torch.float16)

    r = lib.moe_sort(ids, experts)
    rows = lib.moe_dispatch(x, r)
    h, z = lib.moe_linear(rows, r, w1, b1, activation="silu", save_preact=True)
    y = lib.moe_linear(h, r, w2, b2)
    out = lib.moe_combine(y, r, gates)
    gy, ggates = lib.moe_combine_backward(mix, y, r, gates)
    gh, gw2, gb2 = lib.moe_linear_backward(gy, h, r, w2, need_bias=True)
    grows, gw1, gb1 = lib.moe_linear_backward(gh, rows, r, w1, preact=z, activation="silu", need_bias=True)
    gx = lib.moe_dispatch_backward(grows, r)

    leaves = [t.double().requires_grad_() for t in (x, gates, w1, b1, w2, b2)]
    xd, gd, w1d, b1d, w2d, b2d = leaves
    e = ids.long().clamp(min=0)
    hd = torch.einsum("tkoh,th->tko", w1d[e], xd) + b1d[e]
    hd = hd * torch.sigmoid(hd)
    yd = torch.einsum("tkho,tko->tkh", w2d[e], hd) + b2d[e]
    outd = torch.where((ids >= 0)[..., None], gd[..., None] * yd, 0.0).sum(1)
    (outd * mix.double()).sum().backward()
    # a chain of roundings to fp16 (rows, h, y, out; and five on the way back) of terms with random
    # signs: each leaves 2^-11 of its size, and a norm adds them in squares: 8 x 2^-11 bounds them all
    for got, want in ((out, outd), (gx, xd.grad), (ggates, gd.grad), (gw1, w1d.grad), (gb1, b1d.grad),
                      (gw2, w2d.grad), (gb2, b2d.grad)):
        assert (got.double() - want).norm() <= 8 * 2.0 ** -11 * want.norm()
