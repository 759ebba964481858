"""GB300-native multi-stage pipelined fp16 TN GEMM (D = A * B^T).

The compute path is the C-ABI library built from ``csrc/`` (TMA + mbarrier
stage ring + tcgen05/TMEM kernels for sm_103a).  ``binding`` marshals torch
tensors into that library; it has no fallback of any kind.  ``experts`` is
the same for 4-bit matrices, their product and the routing of tokens to
experts.
"""
_EXPORTS = ("gemm_tn_f16", "gemm_tn_f16_ex", "gemm_f16_scaled", "gemm_tn_f16_from_host",
            "get_device_error",
            "minimum_stages", "query_config", "probe_latencies", "library_path", "status_string",
            "GemmError")
_EXPERTS = ("Fp4Matrix", "Routing", "fp4_quantize", "fp4_dequantize", "fp4_gemm_tn",
            "fp4_query_config", "fp4_scale_bytes", "fp4_get_device_error", "moe_sort", "moe_pairs",
            "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward")
__all__ = list(_EXPORTS + _EXPERTS)


def __getattr__(name):
    # the CUDA library is loaded on first use, so that importing the package
    # (e.g. for ``synthetic``) works on machines without it
    if name in _EXPORTS:
        from . import binding as module
    elif name in _EXPERTS:
        from . import experts as module
    else:
        raise AttributeError(name)
    globals()[name] = value = getattr(module, name)  # the next look-up finds it here
    return value
