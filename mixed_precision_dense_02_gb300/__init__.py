"""GB300-native dense multiply-accumulate D = A*B + C.

FP16/BF16 inputs accumulate in FP32, INT8 in INT32, FP64 in FP64, plus a
batched small-tile form in which one A block is broadcast across a group of
neighbouring batch entries, and the operators that bring large language
models onto it: 8-bit floating-point operands with block scales (made by a
fused norm or a quantiser), products grouped by expert and their router, layer
norm, and products with low-rank adapters of many requests, each with its
gradients.  The arithmetic runs in hand-written sm_103a CUDA kernels behind a C
ABI (``include/mma_gb300.h``); this package is the thin Python binding over it (argument marshalling only) plus the seeded input
generator.  The CUDA library is loaded on first use; if it is missing, every
compute call raises -- there is no CPU fallback.
"""
from .binding import (gemm, gemm_ex, gemm_batched, gemm_i8_ex, library_path, load,  # noqa: F401
                      rmsnorm_f8, rmsnorm_backward, layernorm, layernorm_f8,
                      layernorm_backward, quantize_f8, gemm_f8, gemm_grouped,
                      gemm_grouped_wgrad, gemm_grouped_f8, gemm_lora, gemm_lora_wgrad, Routing,
                      route, route_backward, MMAError)

__all__ = ["gemm", "gemm_ex", "gemm_batched", "gemm_i8_ex", "rmsnorm_f8",
           "rmsnorm_backward", "layernorm", "layernorm_f8", "layernorm_backward",
           "quantize_f8", "gemm_f8", "gemm_grouped", "gemm_grouped_wgrad",
           "gemm_grouped_f8", "gemm_lora", "gemm_lora_wgrad", "Routing", "route",
           "route_backward", "load", "library_path", "MMAError"]
