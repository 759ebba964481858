"""Plain 64-bit forms of linear layers and their gradients, written from the definitions, with the
error that each result may have.

Errors.  Operands are exact in the reference.  (1) Sums on the tensor cores: as for the 4-bit
products, at most 2 K_pad errors of 2^-23 of the sum of magnitudes S, K_pad being K rounded up to 64.
(2) bias and residual: an fp32 addition each, 2^-24.  (3) Activations: every slope is below 1.13, so
the error before one grows at most by that.  Their own evaluation has the relative error of an
exponential e^t with |t| <= 90 and of a few operations: (2 + 1.173 |t|) 2^-23 for the intrinsic, as
much again for a rounded t, which is below 2^-14; erfc(x) has 2 x^2 times the relative error of its
argument (2^-22) and a few units, the same for x^2 <= 90.  Slopes are sums of two such terms, of
magnitude below 1.2: 2^-13 at most absolutely, and far less where they matter.  (4) dz is rounded to 16
bits for the products.  (5) Results are rounded once, by half a unit.
"""
import math

import torch

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def half_unit(ref, dtype):
    a = ref.abs()
    if dtype == torch.float16:
        return torch.clamp(a * 2.0 ** -11, min=2.0 ** -25)
    return a * 2.0 ** -8


def below(z):
    """P(Z <= z) of a standard normal Z, with its relative accuracy in the tail (torch.special.ndtr on
    the GPU has none: -7.75 gives 4.607e-15, which is 4.595e-15)."""
    return 0.5 * torch.erfc(-z / math.sqrt(2))


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * below(z)
    if name == "gelu_tanh":
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.special.expit(z)


def slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return below(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u, du = z, 1.0
    if name == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    return torch.special.expit(u) + z * du * torch.special.expit(u) * torch.special.expit(-u)


def spans(offsets, rows):
    """(first row, end) of each group; one group without offsets."""
    if offsets is None:
        return [(0, rows)]
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def pad64(k):
    return max(-(-k // 64) * 64, 64)


def forward(x, w, bias=None, residual=None, activation="none", offsets=None):
    """(out, its error, z, its error) in fp64, errors without the last rounding."""
    ws = w[None] if w.dim() == 2 else w
    bs = None if bias is None else (bias[None] if bias.dim() == 1 else bias).double()
    z = torch.zeros(x.shape[0], ws.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(z)
    for g, (a, b) in enumerate(spans(offsets, x.shape[0])):
        xd, wd = x[a:b].double(), ws[g].double()
        z[a:b] = xd @ wd.t()
        mag[a:b] = xd.abs() @ wd.abs().t()
        if bs is not None:
            z[a:b] += bs[g]
    zerr = 2 * pad64(x.shape[1]) * 2.0 ** -23 * mag + 2.0 ** -24 * z.abs()
    out = act(z, activation)
    err = 1.13 * zerr
    if activation not in ("none", "relu"):
        err = err + 2.0 ** -14 * out.abs()
    if residual is not None:
        out = out + residual.double()
        err = err + 2.0 ** -24 * out.abs()
    return out, err, z, zerr


def backward(grad, x, w, preact, activation="none", offsets=None):
    """((grad_x, error), (grad_w, error), (grad_bias, error))."""
    dtype = grad.dtype
    ws = w[None] if w.dim() == 2 else w
    gx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    gxe = torch.zeros_like(gx)
    gw = torch.zeros(ws.shape, dtype=torch.float64, device=x.device)
    gwe = torch.zeros_like(gw)
    gb = torch.zeros(ws.shape[:2], dtype=torch.float64, device=x.device)
    gbe = torch.zeros_like(gb)
    for g, (a, b) in enumerate(spans(offsets, x.shape[0])):
        xd, wd, dz = x[a:b].double(), ws[g].double(), grad[a:b].double()
        err = torch.zeros_like(dz)
        if activation != "none":
            if activation != "relu":
                err = dz.abs() * 2.0 ** -13
            dz = dz * slope(preact[a:b].double(), activation)
            err = err + 2.0 ** -24 * dz.abs()
        gb[g] = dz.sum(0)
        gbe[g] = err.sum(0) + (b - a + 1) * 2.0 ** -24 * dz.abs().sum(0)
        if activation not in ("none", "relu"):
            err = err + half_unit(dz.abs() + err, dtype)
        gx[a:b] = dz @ wd
        gxe[a:b] = err @ wd.abs() + 2 * pad64(dz.shape[1]) * 2.0 ** -23 * (dz.abs() @ wd.abs())
        gw[g] = dz.t() @ xd
        gwe[g] = err.t() @ xd.abs() + 2 * pad64(b - a) * 2.0 ** -23 * (dz.abs().t() @ xd.abs())
    return (gx, gxe), (gw.view(w.shape), gwe.view(w.shape)), \
        tuple(t[0] if w.dim() == 2 else t for t in (gb, gbe))


def check(got, want, err, what=""):
    """got is the reference, rounded once, but for err."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    off = (got.double() - want).abs()
    allowed = err + half_unit(want.abs() + err, got.dtype)
    bad = ~(off <= allowed)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} off, first at {i}: "
                             f"{float(got[i])} for {float(want[i])}, allowed {float(allowed[i])}")
