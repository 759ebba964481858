"""One projection of a mixture-of-experts layer, served and trained, on the package's kernels.

    python -m multistage_smem_pipeline_gb300.moe_example [--tokens T] [--experts E] [--top-k K]
        [--hidden H] [--out N] [--format nvfp4|mxfp4]

Serving: `ExpertProjection` keeps the experts' weights in 4 bits; a forward sorts the tokens'
slots by expert, quantises each token once into the rows of its slots, multiplies each row with
its expert's weights and sums the slots back into token order with the router's weights.  The
forward is also captured into a CUDA graph, as a decoding loop would run it.

Training: `dispatch` and `combine` are the same moves as autograd functions around experts that
the program computes itself (here a 16-bit scale per expert, to keep the example short).
"""
from __future__ import annotations

import argparse
import math

import torch
from torch.autograd.function import once_differentiable

from . import (Fp4Matrix, Routing, fp4_gemm_tn, fp4_quantize, moe_combine, moe_combine_backward,
               moe_dispatch, moe_dispatch_backward, moe_sort)


def exponent_for(x: torch.Tensor) -> int:
    """The exponent of an nvfp4 matrix: the largest block maximum / 6 just within E4M3's 448."""
    top = float(x.abs().amax()) if x.numel() else 0.0
    if not math.isfinite(top):
        raise ValueError("values must be finite")
    return min(max(math.ceil(math.log2(top / (6 * 448))), -100), 100) if top > 0 else 0


class ExpertProjection:
    """experts x out x hidden weights (float16 or bfloat16) kept in 4 bits.

    activation_exponent: of the activations in nvfp4 (exponent_for a sample of them).  With 0,
    blocks of 16 whose largest element is below 6 * 2^-10 are zero, and values above 2688 are cut.
    """

    def __init__(self, weights: torch.Tensor, format: str = "nvfp4", activation_exponent: int = 0):
        experts, out, hidden = weights.shape
        self.experts, self.out = experts, out
        exponent = exponent_for(weights) if format == "nvfp4" else 0
        self.format, self.activation_exponent = format, activation_exponent
        self.weights: Fp4Matrix = fp4_quantize(weights.reshape(experts * out, hidden), format=format,
                                               exponent=exponent, group_rows=out)

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor) -> torch.Tensor:
        """x: tokens x hidden; ids, gates: tokens x top_k experts (int32) and weights (float32)."""
        routing = moe_sort(ids, self.experts)
        rows = fp4_quantize(x, format=self.format, exponent=self.activation_exponent, routing=routing)
        y = fp4_gemm_tn(rows, self.weights, dtype=x.dtype)
        return moe_combine(y, routing, gates)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, routing):
        ctx.routing = routing
        return moe_dispatch(x, routing)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        return moe_dispatch_backward(grad_y.contiguous(), ctx.routing), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, routing):
        ctx.routing = routing
        ctx.save_for_backward(y, weights)
        return moe_combine(y, routing, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        y, weights = ctx.saved_tensors
        grad_y, grad_w = moe_combine_backward(grad_out.contiguous(), y, ctx.routing, weights)
        return grad_y, grad_w, None


def dispatch(x: torch.Tensor, routing: Routing) -> torch.Tensor:
    """moe_dispatch with its gradient (of first order)."""
    return _Dispatch.apply(x, routing)


def combine(y: torch.Tensor, routing: Routing, weights: torch.Tensor) -> torch.Tensor:
    """moe_combine with its gradients (of first order)."""
    return _Combine.apply(y, weights, routing)


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=4)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--out", type=int, default=1024)
    p.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    a = p.parse_args(argv)
    torch.manual_seed(0)
    dev = torch.device("cuda")
    w = (torch.randn(a.experts, a.out, a.hidden, device=dev) * a.hidden ** -0.5).bfloat16()
    x = torch.randn(a.tokens, a.hidden, device=dev).bfloat16()
    top, ids = torch.topk(torch.randn(a.tokens, a.experts, device=dev), a.top_k, dim=1)
    ids, gates = ids.int(), torch.softmax(top, dim=1)

    layer = ExpertProjection(w, a.format)
    y = layer(x, ids, gates)
    full = torch.einsum("tkoh,th->tko", w[ids.long()].float(), x.float())
    want = (gates[..., None] * full).sum(1)
    rel = float((y.float() - want).norm() / want.norm())
    print(f"served: {a.tokens} tokens x {a.top_k} of {a.experts} experts, {a.hidden} -> {a.out}, "
          f"{a.format}: {rel:.3f} of the 16-bit layer's norm off (4-bit weights and activations)")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(x, ids, gates)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    same = torch.equal(captured, y)
    print(f"as a graph: {start.elapsed_time(end) * 10:.1f} us a forward, same result: {same}")

    x16 = x.clone().requires_grad_()
    g16 = gates.clone().requires_grad_()
    scale = torch.randn(a.experts, 1, device=dev).bfloat16().requires_grad_()
    routing = moe_sort(ids, a.experts)
    rows = dispatch(x16, routing)
    counts = routing.offsets.diff()
    rows = rows * scale.repeat_interleave(counts, dim=0, output_size=rows.shape[0])
    loss = combine(rows, routing, g16).float().square().mean()
    loss.backward()
    print(f"trained: loss {loss.item():.4f}, gradient norms: x {x16.grad.float().norm():.4f}, "
          f"router weights {g16.grad.norm():.4f}, experts {scale.grad.float().norm():.4f}")


if __name__ == "__main__":
    main()
