"""Fine-grained-scaled FP8 GEMM for MI355X (gfx950).

The entry points mirror the C ABI of libfg8.so (include/fg8.h).  Importing
the package does not load the library; the first call does, and raises if it
has not been built.
"""
from ._lib import (  # noqa: F401
    Fg8Error,
    bf16_tile_choice,
    fp8_quantize,
    gemm_bf16_epilogue,
    gemm_bf16_epilogue_backward,
    gemm_fp8_blockscaled,
    gemm_fp8_blockscaled_noalloc,
    gemm_mxfp8,
    gemm_workspace_bytes,
    grouped_gemm_bf16,
    grouped_gemm_bf16_dgrad,
    grouped_gemm_bf16_wgrad,
    grouped_gemm_fp8_contiguous,
    grouped_gemm_fp8_contiguous_swiglu,
    grouped_gemm_fp8_kgrouped,
    grouped_gemm_fp8_masked,
    grouped_gemm_mxfp8_contiguous,
    layer_norm,
    layer_norm_backward,
    moe_capacity,
    moe_combine,
    moe_combine_backward,
    moe_contiguous_layout_fp8,
    tile_choice,
    version,
)
