"""Timed cases of the 4-bit products and of the routing of tokens to experts.

Five kinds of case, each one pass of what a program does:

  route     tokens sorted by expert, and their rows gathered in that order
  step      the same in training: sorted, gathered, put back with weights, and both gradients
  quantise  a matrix into 4-bit blocks and back (what a calibration or a fake-quantised layer runs)
  linear    a 4-bit linear layer: the activations quantised, then the product with kept 4-bit weights
  experts   one projection of a mixture-of-experts layer: sort, quantise into expert order, the
            experts' products, and the weighted sum back into token order

`own` chooses between the package's kernels and the same mathematics in elementary torch operations.

Formats.  A block of 16 (nvfp4) or 32 (mxfp4) neighbours along a row shares a scale; an element is
E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  nvfp4: the scale is E4M3, amax / 6 / 2^e to
the nearest, with one exponent e for the whole matrix.  mxfp4: the scale is the power of two
2^(floor(log2 amax) - 2), held as E8M0, and e is 0.  Elements are x / (scale 2^e) to the nearest, ties to
even, at most 6 in magnitude.

Weights are kept packed as the package's layout has them: two elements a byte, the even one in the low
half, rows padded to 32 elements; scales in tiles of 128 rows by 4 blocks, 512 bytes each, row r's four
at 16 (r % 32) + 4 (r / 32), columns padded to 256 elements.
"""
import math

import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}
DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WEIGHT_EXPONENT = -8     # of nvfp4 weights N(0, 0.02): block maxima / 6 land well inside E4M3


def listed():
    return [
        # a few sequences being decoded: the call is all latency
        {"name": "route 16 tokens", "kind": "route", "tokens": 16, "top_k": 4, "experts": 64, "hidden": 2048, "dtype": "fp16", "dropped": 0.0},
        # a prompt batch whose length is no round number
        {"name": "route 4099 tokens", "kind": "route", "tokens": 4099, "top_k": 8, "experts": 128, "hidden": 4096, "dtype": "bf16", "dropped": 0.0},
        # a small training step with an odd row width (rows start at any 2-byte address) and dropped slots
        {"name": "step 1021 x 1411", "kind": "step", "tokens": 1021, "top_k": 6, "experts": 60, "hidden": 1411, "dtype": "fp16", "dropped": 0.05},
        # a training step of ordinary size
        {"name": "step 8192 x 4096", "kind": "step", "tokens": 8192, "top_k": 8, "experts": 128, "hidden": 4096, "dtype": "bf16", "dropped": 0.02},
        # calibrating one layer's activations, ragged in both directions
        {"name": "quantise 777 x 1000 mx", "kind": "quantise", "rows": 777, "cols": 1000, "format": "mxfp4", "dtype": "fp16"},
        # a weight matrix of the headline size
        {"name": "quantise 8192 x 8192 nv", "kind": "quantise", "rows": 8192, "cols": 8192, "format": "nvfp4", "dtype": "bf16"},
        # one token through the skinny configuration's layer
        {"name": "linear 1 x 14336 x 4096", "kind": "linear", "rows": 1, "out": 14336, "hidden": 4096, "format": "nvfp4", "dtype": "fp16"},
        # the skinny configuration itself
        {"name": "linear 128 x 14336 x 4096", "kind": "linear", "rows": 128, "out": 14336, "hidden": 4096, "format": "mxfp4", "dtype": "fp16"},
        # the headline configuration's size
        {"name": "linear 8192 cubed", "kind": "linear", "rows": 8192, "out": 8192, "hidden": 8192, "format": "nvfp4", "dtype": "fp16"},
        # decoding: each expert sees a token or two, and its weights are what costs
        {"name": "experts 8 tokens", "kind": "experts", "tokens": 8, "top_k": 4, "experts": 64, "hidden": 4096, "out": 2048, "format": "nvfp4", "dtype": "bf16", "dropped": 0.0},
        # a short prompt with ragged sizes in everything, some slots dropped
        {"name": "experts 517 tokens mx", "kind": "experts", "tokens": 517, "top_k": 2, "experts": 20, "hidden": 1440, "out": 1000, "format": "mxfp4", "dtype": "fp16", "dropped": 0.05},
        # a prompt batch
        {"name": "experts 4096 tokens", "kind": "experts", "tokens": 4096, "top_k": 8, "experts": 64, "hidden": 4096, "out": 2048, "format": "nvfp4", "dtype": "bf16", "dropped": 0.0},
    ]


def _log_size(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm; half of them a multiple of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = (n + 7) // 8 * 8
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["route", "step", "quantise", "linear", "experts"])
    dtype = rng.choice(["fp16", "bf16"])
    form = rng.choice(["nvfp4", "mxfp4"])
    if kind in ("route", "step"):
        c = {"kind": kind, "tokens": _log_size(rng, 1, 8192), "top_k": rng.randint(1, 8), "experts": _log_size(rng, 8, 256),
             "hidden": _log_size(rng, 256, 4096), "dtype": dtype, "dropped": rng.choice([0.0, 0.05])}
    elif kind == "quantise":
        c = {"kind": kind, "rows": _log_size(rng, 1, 8192), "cols": _log_size(rng, 64, 8192), "format": form, "dtype": dtype}
    elif kind == "linear":
        c = {"kind": kind, "rows": _log_size(rng, 1, 8192), "out": _log_size(rng, 128, 8192), "hidden": _log_size(rng, 128, 8192), "format": form, "dtype": dtype}
    else:
        c = {"kind": kind, "tokens": _log_size(rng, 1, 4096), "top_k": rng.randint(1, 8), "experts": _log_size(rng, 8, 64),
             "hidden": _log_size(rng, 256, 4096), "out": _log_size(rng, 256, 2048), "format": form, "dtype": dtype, "dropped": rng.choice([0.0, 0.05])}
    return c


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, cols, dtype):
    """Activations: normal values, some columns ten times the others, as residual streams have them."""
    x = torch.randn(n, cols, device="cuda", generator=g)
    loud = torch.rand(cols, device="cuda", generator=g) < 0.01
    return (x * torch.where(loud, 10.0, 1.0)).to(DTYPE[dtype])


def _routing(g, case):
    """The top_k experts of each token under uneven popularity, their softmax weights, and -1 in dropped slots."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    score = torch.randn(t, e, device="cuda", generator=g) + 0.5 * torch.randn(e, device="cuda", generator=g)
    top, ids = torch.topk(score, k, dim=1)
    weights = torch.softmax(top, dim=1)
    lost = torch.rand(t, k, device="cuda", generator=g) < case["dropped"]
    return torch.where(lost, -1, ids).to(torch.int32), weights


def _weights(g, groups, n, cols, form):
    """groups x n x cols weights N(0, 0.02) as packed codes, tiled scales and the matrix's exponent."""
    exponent = WEIGHT_EXPONENT if form == "nvfp4" else 0
    w = torch.randn(groups * n, cols, device="cuda", generator=g) * 0.02
    codes, scales = _encode(w.half().float(), form, exponent)
    return {"codes": _pack(codes), "scales": _tile(scales.view(groups, n, -1), form), "exponent": exponent}


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind in ("route", "step", "experts"):
        s["x"] = _rows(g, case["tokens"], case["hidden"], case["dtype"])
        s["ids"], s["weights"] = _routing(g, case)
    if kind == "step":
        s["grad"] = torch.randn(case["tokens"], case["hidden"], device="cuda", generator=g).to(DTYPE[case["dtype"]])
    if kind == "quantise":
        s["x"] = _rows(g, case["rows"], case["cols"], case["dtype"])
    if kind == "linear":
        s["x"] = _rows(g, case["rows"], case["hidden"], case["dtype"])
        s["w"] = _weights(g, 1, case["out"], case["hidden"], case["format"])
    if kind == "experts":
        s["w"] = _weights(g, case["experts"], case["out"], case["hidden"], case["format"])
        # the rows an expert's buffer holds in a program that pads experts to one capacity
        s["capacity"] = max(1, int(torch.bincount(s["ids"].flatten().long() + 1, minlength=2)[1:].max()))
    return s


# ------------------------------------------------------------------ the plain forms
def _blocks(x, form):
    """fp32 rows padded with zeros to whole blocks: rows x blocks x block."""
    size = BLOCK[form]
    pad = -x.shape[1] % size
    return torch.nn.functional.pad(x, (0, pad)).view(x.shape[0], -1, size)


def _encode(x, form, exponent):
    """(codes 0..15, rows x cols; scale bytes, rows x blocks) of fp32 rows."""
    b = _blocks(x, form)
    top = b.abs().amax(dim=2)
    if form == "nvfp4":
        six = torch.tensor(6.0, device=x.device)     # on the device: divided by, not multiplied by its inverse
        scale = (top / six * 2.0 ** -exponent).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = scale.view(torch.uint8)
        value = scale.float()
    else:
        # the exponent field of amax is floor(log2 amax) + 127
        byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0).to(torch.uint8)
        value = _power_of_two(byte)
    step = (value * 2.0 ** exponent)[..., None]
    y = torch.where(step > 0, b / step, torch.zeros_like(b))
    a = y.abs()
    # how many midpoints of the grid lie below: from odd codes a tie goes up, from even ones it stays
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(b)
    return code.view(x.shape[0], -1)[:, :x.shape[1]].to(torch.uint8), byte


def _power_of_two(byte):
    """2^(byte - 127), put together from its bits: the byte is the exponent field, 2^-127 a subnormal."""
    return torch.where(byte > 0, byte.int() << 23, 1 << 22).view(torch.float32)


def _pack(codes):
    codes = torch.nn.functional.pad(codes, (0, -codes.shape[1] % 32))
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _tile(scales, form):
    """groups x rows x blocks scale bytes as (groups tiles) x chunks x 512."""
    groups, rows, blocks = scales.shape
    scales = torch.nn.functional.pad(scales, (0, -blocks % (256 // BLOCK[form]), 0, -rows % 128))
    tiles, chunks = scales.shape[1] // 128, scales.shape[2] // 4
    t = scales.view(groups, tiles, 4, 32, chunks, 4).permute(0, 1, 4, 3, 2, 5)
    return t.reshape(groups * tiles, chunks, 512).contiguous()


def _untile(scales, groups, rows, blocks):
    chunks = scales.shape[1]
    t = scales.view(groups, -1, chunks, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    return t.reshape(groups, -1, 4 * chunks)[:, :rows, :blocks]


def _decode(codes, scales, form, exponent):
    """fp32 rows x cols from codes 0..15 and scale bytes rows x blocks."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    value = scales.contiguous().view(torch.float8_e4m3fn).float() if form == "nvfp4" else _power_of_two(scales)
    value = value * 2.0 ** exponent
    size = BLOCK[form]
    return grid[codes.int()] * value.repeat_interleave(size, dim=-1)[..., :codes.shape[-1]]


def _plain_weights(w, groups, n, cols, form):
    """groups x n x cols fp32 from the kept weights."""
    codes = torch.stack((w["codes"] & 15, w["codes"] >> 4), dim=2).view(groups, n, -1)[..., :cols]
    scales = _untile(w["scales"], groups, n, -(-cols // BLOCK[form]))
    return _decode(codes, scales, form, w["exponent"])


def _plain_sort(ids, experts):
    """offsets (experts + 1), the row of each slot, and the slot of each row; dropped slots come last."""
    key = torch.where((ids < 0) | (ids >= experts), experts, ids).flatten()
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=ids.device)
    offsets = (key[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(dim=1)
    return offsets, rows.view(ids.shape), slots, key.view(ids.shape)


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    x = s["x"].float()
    dtype = s["x"].dtype
    if kind == "quantise":
        codes, scales = _encode(x, case["format"], 0)
        return {"values": _decode(codes, scales, case["format"], 0).to(dtype)}
    if kind == "linear":
        codes, scales = _encode(x, case["format"], 0)
        a = _decode(codes, scales, case["format"], 0)
        b = _plain_weights(s["w"], 1, case["out"], case["hidden"], case["format"])[0]
        return {"out": (a @ b.t()).to(dtype)}
    experts, k = case["experts"], case["top_k"]
    offsets, rows, slots, key = _plain_sort(s["ids"], experts)
    kept = key < experts
    if kind in ("route", "step"):
        live = kept.flatten()[slots][:, None]
        y = torch.where(live, x[slots // k], 0.0)
        if kind == "route":
            return {"offsets": offsets.int(), "rows": rows.int(), "gathered": y.to(dtype)}
        w = torch.where(kept, s["weights"], 0.0)
        out = (w[..., None] * y[rows]).sum(dim=1)
        grad = s["grad"].float()
        grad_y = w.flatten()[slots][:, None] * grad[slots // k]
        grad_w = torch.where(kept, (grad[:, None, :] * y[rows]).sum(dim=2), 0.0)
        grad_x = torch.where(kept[..., None], grad_y.to(dtype).float()[rows], 0.0).sum(dim=1)
        return {"out": out.to(dtype), "grad_rows": grad_y.to(dtype), "grad_weights": grad_w, "grad_x": grad_x.to(dtype)}
    # experts: rows of expert e go to e's part of a buffer of `capacity` rows each
    cap, n, hidden = s["capacity"], case["out"], case["hidden"]
    codes, scales = _encode(x, case["format"], 0)
    a = _decode(codes, scales, case["format"], 0)
    b = _plain_weights(s["w"], experts, n, hidden, case["format"])
    place = torch.where(kept, key * cap + rows - offsets[key], experts * cap).long()
    source = torch.zeros(experts * cap + 1, dtype=torch.int64, device=x.device)
    source[place.flatten()] = torch.arange(key.numel(), device=x.device) // k
    y = torch.bmm(a[source[:-1]].view(experts, cap, hidden), b.transpose(1, 2)).view(-1, n)
    y = torch.where(kept[..., None], y[place.clamp(max=experts * cap - 1)], 0.0)
    return {"out": (s["weights"][..., None] * y).sum(dim=1).to(dtype)}


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import multistage_smem_pipeline_gb300 as lib
    case, kind = s["case"], s["case"]["kind"]
    if kind == "quantise":
        q = lib.fp4_quantize(s["x"], format=case["format"])
        return {"values": lib.fp4_dequantize(q, dtype=s["x"].dtype)}
    if kind in ("linear", "experts"):
        w = lib.Fp4Matrix(s["w"]["codes"], s["w"]["scales"], cols=case["hidden"], format=case["format"],
                          exponent=s["w"]["exponent"], group_rows=case["out"])
    if kind == "linear":
        return {"out": lib.fp4_gemm_tn(lib.fp4_quantize(s["x"], format=case["format"]), w, dtype=s["x"].dtype)}
    routing = lib.moe_sort(s["ids"], case["experts"])
    if kind == "experts":
        q = lib.fp4_quantize(s["x"], format=case["format"], routing=routing)
        y = lib.fp4_gemm_tn(q, w, dtype=s["x"].dtype)
        return {"out": lib.moe_combine(y, routing, s["weights"])}
    y = lib.moe_dispatch(s["x"], routing)
    if kind == "route":
        return {"offsets": routing.offsets, "rows": routing.rows, "gathered": y}
    out = lib.moe_combine(y, routing, s["weights"])
    grad_y, grad_w = lib.moe_combine_backward(s["grad"], y, routing, s["weights"])
    grad_x = lib.moe_dispatch_backward(grad_y, routing)
    return {"out": out, "grad_rows": grad_y, "grad_weights": grad_w, "grad_x": grad_x}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the exact values
def work(case):
    kind = case["kind"]
    if kind == "quantise":
        return {"bytes": 4.0 * case["rows"] * case["cols"], "flops": 3.0 * case["rows"] * case["cols"]}
    if kind == "linear":
        m, n, k = case["rows"], case["out"], case["hidden"]
        return {"bytes": 2.0 * m * k + n * k * (0.5 + 1.0 / BLOCK[case["format"]]) + 2.0 * m * n, "flops": 2.0 * m * n * k}
    t, k, h, e = case["tokens"], case["top_k"], case["hidden"], case["experts"]
    slots = t * k
    kept = slots * (1 - case["dropped"])
    if kind == "route":
        return {"bytes": 2.0 * (t + slots) * h + 4 * slots * 2 + 4 * (e + 1), "flops": float(slots)}
    if kind == "step":
        # ids, weights and x in, out; the output's gradient in; the gradients of the rows, weights and x out
        return {"bytes": 2.0 * (4 * t + slots) * h + 12.0 * slots, "flops": 2.0 * kept * h * 3}
    n = case["out"]
    met = e * (1 - (1 - 1 / e) ** kept)     # experts that are expected to have a row at all
    return {"bytes": 2.0 * t * h + met * n * h * (0.5 + 1.0 / BLOCK[case["format"]]) + 2.0 * t * n + 8.0 * slots,
            "flops": 2.0 * kept * n * h}


def _round_to(a, bits, least):
    """Non-negative fp64 to the nearest number of `bits` significant bits whose exponent is at least `least`, ties to even."""
    _, e = torch.frexp(a)
    unit = _two_to((e - 1).clamp(min=least) - (bits - 1))
    return torch.round(a / unit) * unit


def _two_to(e):
    """2^e in fp64, from its bits: pow() on the GPU need not be exact."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _exact_quantised(x, form, exponent):
    x = x.double()
    size = BLOCK[form]
    wide = torch.zeros(x.shape[0], -(-x.shape[1] // size) * size, dtype=torch.float64, device=x.device)
    wide[:, :x.shape[1]] = x
    top = wide.view(x.shape[0], -1, size).abs().max(dim=2).values
    if form == "nvfp4":
        scale = torch.clamp(_round_to(top / torch.full_like(top, 6.0 * 2.0 ** exponent), 4, -6), max=448.0) * 2.0 ** exponent
    else:
        _, e = torch.frexp(top)
        scale = torch.where(top > 0, _two_to((e - 3).clamp(min=-127)), torch.zeros_like(top))
    scale = scale.repeat_interleave(size, dim=1)
    unit = torch.where(scale > 0, wide / torch.where(scale > 0, scale, 1.0), 0.0)
    q = torch.clamp(_round_to(unit.abs(), 2, 0), max=6.0) * torch.sign(unit) * scale
    return q[:, :x.shape[1]]


def _exact_weights(w, groups, n, cols, form):
    code = torch.empty(groups * n, 2 * w["codes"].shape[1], dtype=torch.int64, device=w["codes"].device)
    code[:, 0::2] = w["codes"] % 16
    code[:, 1::2] = w["codes"] // 16
    m = code % 8
    value = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * _two_to(m // 2 - 1))
    value = torch.where(code >= 8, -value, value)[:, :cols].double()
    r = torch.arange(groups * n, device=code.device)
    tile = (r // n) * -(-n // 128) + (r % n) // 128
    block = torch.arange(cols, device=code.device) // BLOCK[form]
    at = 16 * (r % n % 32) + 4 * (r % n % 128 // 32)
    byte = w["scales"].flatten()[((tile[:, None] * w["scales"].shape[1] + block // 4) * 512 + at[:, None] + block % 4)].long()
    if form == "nvfp4":
        e, f = byte // 8, byte % 8
        scale = torch.where(e > 0, (8 + f) * _two_to(e - 10), f * 2.0 ** -9)
    else:
        scale = _two_to(byte - 127)
    return (value * scale * 2.0 ** w["exponent"]).view(groups, n, cols)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    x = s["x"].double()
    if kind == "quantise":
        return {"values": _exact_quantised(x, case["format"], 0)}
    if kind == "linear":
        a = _exact_quantised(x, case["format"], 0)
        return {"out": a @ _exact_weights(s["w"], 1, case["out"], case["hidden"], case["format"])[0].t()}
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    ids, w = s["ids"].long(), s["weights"].double()
    ids = torch.where((ids >= 0) & (ids < e), ids, e)
    if kind == "experts":
        a = _exact_quantised(x, case["format"], 0)
        b = _exact_weights(s["w"], e, case["out"], case["hidden"], case["format"])
        out = torch.zeros(t, case["out"], dtype=torch.float64, device=x.device)
        for i in range(e):
            tok, j = torch.nonzero(ids == i, as_tuple=True)
            out.index_add_(0, tok, w[tok, j][:, None] * (a[tok] @ b[i].t()))
        return {"out": out}
    order = sorted(range(t * k), key=ids.flatten().tolist().__getitem__)
    slot = torch.tensor(order, device=x.device)
    kept = (ids.flatten()[slot] < e).double()[:, None]
    y = x[slot // k] * kept
    if kind == "route":
        return {"offsets": None, "rows": None, "gathered": y}
    row = torch.argsort(slot)
    flat = torch.where(ids.flatten() < e, w.flatten(), 0.0)
    grad = s["grad"].double()
    out = (flat[:, None] * y[row]).view(t, k, -1).sum(dim=1)
    grad_w = ((grad.repeat_interleave(k, dim=0) * y[row]).sum(dim=1) * (ids.flatten() < e)).view(t, k)
    grad_y = flat[slot][:, None] * grad[slot // k]
    grad_x = flat.view(t, k).sum(dim=1)[:, None] * grad
    return {"out": out, "grad_rows": grad_y, "grad_weights": grad_w, "grad_x": grad_x}
