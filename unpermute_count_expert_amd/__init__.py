"""MI355X (gfx950) fused MoE expert pipeline: count -> permute -> fp8 grouped
GEMM (w13) -> SiLU-and-mul + fp8 requant -> fp8 grouped GEMM (w2) -> unpermute
with topk weight and reduce, chunked over tokens.

The compute lives in libmoe_hip.so (C ABI in include/moe.h); this package is
its ctypes binding plus small device-resident layer wrappers: MoeLayer (fp8
weights, forward) and MoeTrainLayer (bf16 weights, forward and backward, with
the gradients' global norm and clipping; with a checkpoint on fused kernels
and less memory, in bf16 or 8 bits).
"""
from ._lib import (MOE_ACT_IDENTITY, MOE_ACT_SILU_MUL, MoeError, MoeProblem, load,  # noqa: F401
                   moe_act_quant, moe_count, moe_forward_chunked, moe_forward_workspace_size, moe_forward_workspace_slices,
                   moe_grouped_gemm_fp8, moe_grouped_gemm_tile_rows, moe_max_rows, moe_permute, moe_permute_workspace_size,
                   moe_quant_permute, moe_grouped_gemm_fp8_small, moe_act_quant_partials, moe_unpermute_partials,
                   moe_forward_plan_info, moe_unpermute_weight_reduce, problem, MOE_DTYPE_BF16, MOE_DTYPE_F32,
                   moe_permute_bf16, moe_grouped_gemm_bf16, moe_grouped_gemm_bf16_dgrad, moe_grouped_gemm_bf16_wgrad,
                   moe_silu_mul, moe_silu_mul_bwd, moe_unpermute_weight_reduce_bwd, moe_grad_workspace_size,
                   moe_grad_sumsq, moe_grad_clip, moe_checkpoint, moe_checkpoint_restore, moe_permute_rows,
                   moe_grouped_gemm_bf16_silu_mul, moe_grouped_gemm_bf16_dgrad_silu_mul, moe_topk_weights_bwd,
                   moe_grouped_gemm_bf16_plan_info, MOE_GEMM_BF16_FORWARD, MOE_GEMM_BF16_DGRAD, MOE_GEMM_BF16_WGRAD,
                   MOE_GEMM_BF16_SILU_MUL, MOE_GEMM_BF16_DGRAD_SILU_MUL)
from .layer import MoeLayer, MoeTrainLayer  # noqa: F401
