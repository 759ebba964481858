"""4-bit matrices, their product, the routing of tokens to experts, and linear
layers in 16 bits: the binding of include/moe_fp4.h and include/linear.h.  Checks and marshalling only (compiled, in
csrc/experts_binding.cpp): every step runs in the library's CUDA kernels, on
the current stream or the one given, and nothing falls back.

    routing = moe_sort(ids, experts)                    # ids: tokens x top_k
    q = fp4_quantize(x, routing=routing)                # x's rows in expert order
    y = fp4_gemm_tn(q, weights)                         # weights: an Fp4Matrix of experts
    out = moe_combine(y, routing, gates)                # back in token order

In 16 bits, with gradients:

    h = moe_linear(moe_dispatch(x, routing), routing, w, bias, activation="gelu")
    y = linear(x, w, bias, residual=x)                  # dense

Tensors given as `out` are written in place; without it one is allocated.  The calls record no
gradients, whatever their inputs require: the package's moe_example has them as autograd functions.
"""
from __future__ import annotations

import os

from . import build as _build
from . import binding  # noqa: F401  (loads the library)

if not os.path.exists(_build.BINDING):
    raise ImportError(f"{_build.BINDING} is missing: build it with "
                      "`python -m multistage_smem_pipeline_gb300.build`")

from .lib._experts import (  # noqa: E402,F401
    Fp4Matrix, Routing, fp4_dequantize, fp4_gemm_tn, fp4_get_device_error, fp4_quantize,
    fp4_query_config, fp4_scale_bytes, linear, linear_backward, linear_get_device_error,
    linear_query_config, moe_combine, moe_combine_backward, moe_dispatch, moe_dispatch_backward,
    moe_linear, moe_linear_backward, moe_pairs, moe_sort)

# The C functions of moe_fp4.h.
EXPORTED = ("fp4_code_bytes", "fp4_scale_bytes", "fp4_quantize", "fp4_dequantize", "fp4_gemm_tn",
            "fp4_gemm_tn_ex", "fp4_query_config", "fp4_get_device_error", "moe_sort", "moe_pairs",
            "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward")

# Those of linear.h.
EXPORTED_LINEAR = ("linear_forward", "linear_backward", "linear_forward_workspace",
                   "linear_backward_workspace", "linear_query_config", "linear_get_device_error")
