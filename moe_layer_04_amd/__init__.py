"""Fused Mixture-of-Experts layer for one AMD MI355X (gfx950).

The layer -- top-k softmax router, expert-sorted token permutation, grouped
expert GEMMs with a fused SiLU*up epilogue, weighted un-permute combine --
runs in hand-written HIP kernels behind the C ABI of include/moe.h
(libmoe.so), as one call or in pieces with their gradients, the router's balance
loss and gradients and activations kept in 8 bits; this package is its thin
ctypes binding plus the seeded input generator used by tests and benchmarks.
"""
from ._binding import (MOE_BF16, FusedForwardGraph, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED,
                       MOE_ERR_WORKSPACE, MOE_FP8_E4M3, MOE_FP8_E4M3_ROWWISE, MOE_MXFP4_E2M1, MOE_OK, MOE_REGIME_AUTO,
                       MOE_REGIME_DECODE, MOE_REGIME_PREFILL, MoEError, NOALLOC_SCRATCH_BYTES, Plan, fused_plan, fused_routing, load_library,
                       moe_align, moe_align_ex, moe_fused_forward, moe_fused_forward_noalloc,
                       moe_quant_rows_e4m3, moe_topk,
                       status_string, workspace_size)
from ._operators import (MOE_PRODUCT_DW, MOE_PRODUCT_DX, MOE_PRODUCT_FWD, MOE_PRODUCT_STREAM,
                         MOE_PRODUCT_TILES_64, MOE_PRODUCT_TILES_128, MOE_PRODUCT_TILES_256,
                         ProductPlan, grouped_plan, moe_block_norm, moe_block_norm_bwd,
                         moe_grouped_gemm, moe_grouped_gemm_dw, moe_grouped_gemm_dx, moe_silu_mul,
                         moe_silu_mul_bwd)
from ._checkpoint import (moe_ckpt_restore, moe_ckpt_rows, moe_grouped_gemm_dw_ckpt,
                          moe_silu_mul_bwd_ckpt, moe_silu_mul_ckpt)
from ._router_grad import moe_balance, moe_balance_bwd, moe_topk_bwd

__all__ = [
    "MOE_BF16", "MOE_FP8_E4M3", "MOE_FP8_E4M3_ROWWISE", "MOE_MXFP4_E2M1", "MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED",
    "MOE_ERR_WORKSPACE", "MOE_ERR_HIP", "MOE_REGIME_AUTO", "MOE_REGIME_DECODE",
    "MOE_REGIME_PREFILL", "MoEError", "load_library", "moe_topk", "moe_align", "moe_align_ex",
    "moe_quant_rows_e4m3", "moe_fused_forward", "status_string", "workspace_size",
    "FusedForwardGraph", "Plan", "fused_plan", "fused_routing", "moe_fused_forward_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw", "moe_silu_mul",
    "moe_silu_mul_bwd", "moe_block_norm", "moe_block_norm_bwd", "ProductPlan", "grouped_plan",
    "MOE_PRODUCT_FWD", "MOE_PRODUCT_DX", "MOE_PRODUCT_DW", "MOE_PRODUCT_STREAM",
    "MOE_PRODUCT_TILES_64", "MOE_PRODUCT_TILES_128", "MOE_PRODUCT_TILES_256",
    "moe_ckpt_rows", "moe_ckpt_restore", "moe_silu_mul_ckpt", "moe_silu_mul_bwd_ckpt",
    "moe_grouped_gemm_dw_ckpt", "moe_balance", "moe_balance_bwd", "moe_topk_bwd",
]
