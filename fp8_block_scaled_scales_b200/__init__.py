"""FP8 (E4M3) 128x128 block-scaled GEMM for B200 (sm_100a).

The compute lives in libdg.so (hand-written CUDA kernels behind a C ABI,
include/dg.h); this package is its Python binding plus the seeded input
generators used by the tests and the benchmark.
"""
from .binding import (DGError, dgrad_blockscaled, gemm_1x128, gemm_blockscaled,  # noqa: F401
                      gemm_blockscaled_bf16a, grouped_dgrad_contiguous, grouped_gemm_contiguous,
                      grouped_gemm_masked, grouped_wgrad_contiguous, last_device_status, moe_capacity, moe_combine,
                      moe_combine_backward, moe_dispatch_quantize, moe_dispatch_quantize_masked, moe_sort,
                      moe_sort_masked, quantize_blockwise, quantize_1x128, set_kernel_control, swiglu_quantize,
                      swiglu_quantize_backward, swiglu_quantize_masked, version, wgrad_blockscaled)
