"""Timed cases of linear layers in 16 bits: dense ones and the experts of a mixture, forward and back.

Four kinds of case, each one pass of what a program does:

  linear            out = act(x w^T + bias) + residual; in training also the sums z before the activation
  linear backward   the gradients of x, w and bias from the output's gradient, the kept z, x and w
  experts           the rows of every expert through its own weights: out[r] = act(x[r] w[e]^T + bias[e]) for
                    the rows r of expert e
  experts backward  its gradients; an expert's gradient of w and bias is the sum over its own rows

`own` chooses between the package's kernels and the same mathematics in elementary torch operations.

Activations: none; relu max(z, 0); gelu z P(Z <= z) of a standard normal Z; gelu_tanh, its usual form with a
tanh; silu z / (1 + e^-z).  Matrices are fp16 or bf16, row by row; sums are in 32 bits or more.

Rows of experts are in expert order, as the package's moe_sort and moe_dispatch leave them: expert e has the
rows offsets[e] to offsets[e + 1] - 1, and the rows of dropped slots come last.  Those give zeros, and count
in no gradient.
"""
import math

import torch

own = False

DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
CUBIC = 0.044715     # of gelu_tanh: z sigmoid(2 sqrt(2 / pi) (z + CUBIC z^3))


def listed():
    return [
        # one token through the skinny configuration's layer: its weights are what costs
        {"name": "linear 1 x 14336 x 4096", "kind": "linear", "rows": 1, "out": 14336, "hidden": 4096, "dtype": "bf16",
         "activation": "silu", "residual": False, "save": False},
        # the skinny configuration itself
        {"name": "linear 128 x 14336 x 4096", "kind": "linear", "rows": 128, "out": 14336, "hidden": 4096, "dtype": "fp16",
         "activation": "gelu", "residual": False, "save": False},
        # a short prompt, odd in every direction: rows start at any 2-byte address
        {"name": "linear 517 x 1001 x 1411", "kind": "linear", "rows": 517, "out": 1001, "hidden": 1411, "dtype": "fp16",
         "activation": "relu", "residual": True, "save": False},
        # the way back to the residual stream, for a prompt batch
        {"name": "linear 4096 x 4096 x 14336", "kind": "linear", "rows": 4096, "out": 4096, "hidden": 14336, "dtype": "bf16",
         "activation": "none", "residual": True, "save": False},
        # the headline configuration's size, in training
        {"name": "linear 8192 cubed", "kind": "linear", "rows": 8192, "out": 8192, "hidden": 8192, "dtype": "bf16",
         "activation": "gelu_tanh", "residual": False, "save": True},
        # a small training step with odd widths
        {"name": "linear backward 1021 x 1000 x 1411", "kind": "linear backward", "rows": 1021, "out": 1000, "hidden": 1411,
         "dtype": "fp16", "activation": "relu"},
        # a training step of ordinary size
        {"name": "linear backward 8192 x 4096 x 4096", "kind": "linear backward", "rows": 8192, "out": 4096, "hidden": 4096,
         "dtype": "bf16", "activation": "gelu"},
        # decoding: each expert sees a token or two
        {"name": "experts 8 tokens", "kind": "experts", "tokens": 8, "top_k": 4, "experts": 64, "hidden": 4096, "out": 2048,
         "dtype": "bf16", "activation": "silu", "save": False, "dropped": 0.0},
        # a short prompt with ragged sizes in everything, some slots dropped
        {"name": "experts 517 tokens", "kind": "experts", "tokens": 517, "top_k": 2, "experts": 20, "hidden": 1440, "out": 1000,
         "dtype": "fp16", "activation": "gelu", "save": False, "dropped": 0.05},
        # a prompt batch in training
        {"name": "experts 4096 tokens", "kind": "experts", "tokens": 4096, "top_k": 8, "experts": 64, "hidden": 4096, "out": 2048,
         "dtype": "bf16", "activation": "silu", "save": True, "dropped": 0.0},
        # the ragged prompt's step back
        {"name": "experts backward 517 tokens", "kind": "experts backward", "tokens": 517, "top_k": 2, "experts": 20, "hidden": 1440,
         "out": 1000, "dtype": "fp16", "activation": "gelu", "dropped": 0.05},
        # the prompt batch's step back
        {"name": "experts backward 4096 tokens", "kind": "experts backward", "tokens": 4096, "top_k": 8, "experts": 64,
         "hidden": 4096, "out": 2048, "dtype": "bf16", "activation": "silu", "dropped": 0.0},
    ]


def _log_size(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm; half of them a multiple of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = (n + 7) // 8 * 8
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["linear", "linear backward", "experts", "experts backward"])
    c = {"kind": kind, "dtype": rng.choice(["fp16", "bf16"]), "activation": rng.choice(ACTIVATIONS)}
    if kind == "linear":
        c.update(rows=_log_size(rng, 1, 8192), out=_log_size(rng, 64, 8192), hidden=_log_size(rng, 64, 8192),
                 residual=rng.random() < 0.5, save=rng.random() < 0.5)
    elif kind == "linear backward":
        c.update(rows=_log_size(rng, 1, 8192), out=_log_size(rng, 64, 4096), hidden=_log_size(rng, 64, 4096))
    else:
        c.update(tokens=_log_size(rng, 1, 4096), top_k=rng.randint(1, 8), experts=_log_size(rng, 8, 64),
                 hidden=_log_size(rng, 64, 4096), out=_log_size(rng, 64, 2048), dropped=rng.choice([0.0, 0.05]))
        if kind == "experts":
            c["save"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _rows(g, n, cols, dtype):
    """Activations: normal values, some columns ten times the others, as residual streams have them."""
    x = torch.randn(n, cols, device="cuda", generator=g)
    loud = torch.rand(cols, device="cuda", generator=g) < 0.01
    return (x * torch.where(loud, 10.0, 1.0)).to(DTYPE[dtype])


def _normal(g, *sizes, scale, dtype):
    return torch.randn(*sizes, device="cuda", dtype=torch.float32, generator=g).mul_(scale).to(DTYPE[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, dtype, n, hidden = case["kind"], case["dtype"], case["out"], case["hidden"]
    s = {"case": case}
    if kind.startswith("linear"):
        rows, experts = case["rows"], None
        s["x"] = _rows(g, rows, hidden, dtype)
        s["w"] = _normal(g, n, hidden, scale=0.02, dtype=dtype)
        s["bias"] = _normal(g, n, scale=0.1, dtype=dtype)
        if case.get("residual"):
            s["residual"] = _rows(g, rows, n, dtype)
    else:
        # the experts of each token under uneven popularity, -1 in dropped slots, and where the slots go
        experts, k = case["experts"], case["top_k"]
        score = torch.randn(case["tokens"], experts, device="cuda", generator=g) + 0.5 * torch.randn(experts, device="cuda", generator=g)
        ids = torch.topk(score, k, dim=1).indices
        ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < case["dropped"], -1, ids)
        key = torch.where(ids < 0, experts, ids).flatten()
        slots = torch.sort(key, stable=True).indices
        place = torch.empty_like(slots)
        place[slots] = torch.arange(slots.numel(), device="cuda")
        ends = torch.cumsum(torch.bincount(key, minlength=experts + 1), 0)[:experts]
        s["ids"] = ids.int()
        s["rows"] = place.view(ids.shape).int()
        s["offsets"] = torch.nn.functional.pad(ends, (1, 0)).int()
        s["bounds"] = s["offsets"].tolist()      # for a program that calls one product per expert
        rows = slots.numel()
        live = torch.arange(rows, device="cuda") < ends[-1]
        tokens = _rows(g, case["tokens"], hidden, dtype)
        s["x"] = torch.where(live[:, None], tokens[slots // k], 0.0).to(DTYPE[dtype])
        s["w"] = _normal(g, experts, n, hidden, scale=0.02, dtype=dtype)
        s["bias"] = _normal(g, experts, n, scale=0.1, dtype=dtype)
    if kind.endswith("backward"):
        s["grad"] = _normal(g, rows, n, scale=0.05, dtype=dtype)
        if case["activation"] != "none":         # what the forward pass kept
            s["z"] = torch.zeros(rows, n, device="cuda", dtype=DTYPE[dtype])
            for a, b, w, bias in _spans(s):
                s["z"][a:b] = s["x"][a:b] @ w.t() + bias
    return s


def _spans(s):
    """(first row, end, weights, bias) of each matrix that a row may meet."""
    if s["w"].dim() == 2:
        return [(0, s["x"].shape[0], s["w"], s["bias"])]
    b = s["bounds"]
    return [(b[e], b[e + 1], s["w"][e], s["bias"][e]) for e in range(len(b) - 1)]


# ------------------------------------------------------------------ the plain forms
def _act(z, name):
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -(0.5 ** 0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + CUBIC * z * z * z)))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def _slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(z * -(0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name in ("gelu_tanh", "silu"):
        u, du = z, 1.0
        if name == "gelu_tanh":
            u = 2 * math.sqrt(2 / math.pi) * (z + CUBIC * z * z * z)
            du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * CUBIC * z * z)
        up = 1 / (1 + torch.exp(-u))
        return up + z * du * up * (1 / (1 + torch.exp(u)))
    return torch.ones_like(z)


def _plain(s):
    case, act = s["case"], s["case"]["activation"]
    dtype, x = s["x"].dtype, s["x"]
    if case["kind"].endswith("backward"):
        grad_x = torch.zeros_like(x, dtype=torch.float32)
        grad_w = torch.zeros_like(s["w"])
        grad_b = torch.zeros_like(s["bias"])
        for i, (a, b, w, _) in enumerate(_spans(s)):
            dz = s["grad"][a:b].float()
            if act != "none":
                dz = dz * _slope(s["z"][a:b].float(), act)
            grad_x[a:b] = dz @ w.float()
            to_w, to_b = (grad_w, grad_b) if w is s["w"] else (grad_w[i], grad_b[i])
            to_w.copy_(dz.t() @ x[a:b].float())
            to_b.copy_(dz.sum(dim=0))
        return {"grad_x": grad_x.to(dtype), "grad_w": grad_w, "grad_bias": grad_b}
    z = torch.zeros(x.shape[0], case["out"], device=x.device)
    out = torch.zeros_like(z)
    for a, b, w, bias in _spans(s):
        z[a:b] = x[a:b].float() @ w.float().t() + bias.float()
        out[a:b] = _act(z[a:b], act)
    if "residual" in s:
        out = out + s["residual"].float()
    return {"out": out.to(dtype), "z": z.to(dtype)} if case["save"] else {"out": out.to(dtype)}


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import multistage_smem_pipeline_gb300 as lib
    case, act = s["case"], s["case"]["activation"]
    if case["kind"] == "linear":
        got = lib.linear(s["x"], s["w"], s["bias"], activation=act, residual=s.get("residual"), save_preact=case["save"])
    elif case["kind"] == "linear backward":
        got = lib.linear_backward(s["grad"], s["x"], s["w"], activation=act, preact=s.get("z"), need_bias=True)
    else:
        routing = lib.Routing(s["offsets"], s["rows"], s["ids"])
        if case["kind"] == "experts":
            got = lib.moe_linear(s["x"], routing, s["w"], s["bias"], activation=act, save_preact=case["save"])
        else:
            got = lib.moe_linear_backward(s["grad"], s["x"], routing, s["w"], activation=act, preact=s.get("z"), need_bias=True)
    if case["kind"].endswith("backward"):
        return dict(zip(("grad_x", "grad_w", "grad_bias"), got))
    return dict(zip(("out", "z"), got)) if case["save"] else {"out": got}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the exact values
def work(case):
    n, h = case["out"], case["hidden"]
    if case["kind"].startswith("linear"):
        rows = kept = case["rows"]
        met = 1.0
    else:
        e = case["experts"]
        rows = case["tokens"] * case["top_k"]
        kept = rows * (1 - case["dropped"])
        met = e * (1 - (1 - 1 / e) ** kept)     # experts that are expected to have a row at all
    if case["kind"].endswith("backward"):
        kept_z = 0 if case["activation"] == "none" else kept * n
        whole = case.get("experts", 1)          # a gradient is written for every expert, zero or not
        return {"bytes": 2.0 * (kept * (n + h) + kept_z + met * n * h + rows * h + whole * (n * h + n)),
                "flops": 4.0 * kept * n * h}
    outs = rows * n * (2 if case["save"] else 1) + (rows * n if case.get("residual") else 0)
    return {"bytes": 2.0 * (kept * h + met * (n * h + n) + outs), "flops": 2.0 * kept * n * h}


def _exact_act(z, name):
    """(the activation, its derivative) in fp64."""
    zero, one = torch.zeros_like(z), torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "relu":
        return torch.maximum(z, zero), torch.where(z > 0, one, zero)
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p * (1 + z * torch.special.expit(-z))
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + CUBIC * z ** 3))
    # (1 + t) / 2 without the cancellation where t is near -1
    p = torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + CUBIC * z ** 3))
    return z * p, p + z / 2 * (1 - t) * (1 + t) * math.sqrt(2 / math.pi) * (1 + 3 * CUBIC * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    act, x, w = case["activation"], s["x"].double(), s["w"]
    if w.dim() == 2:
        groups = [(torch.arange(x.shape[0], device=x.device), w.double(), s["bias"].double())]
    else:
        owner = torch.bucketize(torch.arange(x.shape[0], device=x.device), s["offsets"][1:].long(), right=True)
        groups = [(torch.nonzero(owner == e)[:, 0], w[e].double(), s["bias"][e].double()) for e in range(w.shape[0])]
    if case["kind"].endswith("backward"):
        grad_x, grad_w, grad_b = torch.zeros_like(x), [], []
        for rows, we, _ in groups:
            dz = s["grad"][rows].double()
            if act != "none":
                dz = dz * _exact_act(s["z"][rows].double(), act)[1]
            grad_x.index_copy_(0, rows, torch.einsum("rn,nh->rh", dz, we))
            grad_w.append(torch.einsum("rn,rh->nh", dz, x[rows]))
            grad_b.append(torch.einsum("rn->n", dz))
        grad_w, grad_b = (torch.stack(t).view(like.shape) for t, like in ((grad_w, w), (grad_b, s["bias"])))
        return {"grad_x": grad_x, "grad_w": grad_w, "grad_bias": grad_b}
    z = torch.zeros(x.shape[0], case["out"], dtype=torch.float64, device=x.device)
    out = torch.zeros_like(z)
    for rows, we, bias in groups:
        ze = torch.addmm(bias, x[rows], we.t())
        z.index_copy_(0, rows, ze)
        out.index_copy_(0, rows, _exact_act(ze, act)[0])
    if "residual" in s:
        out += s["residual"].double()
    return {"out": out, "z": z} if case["save"] else {"out": out}
