"""One expert-parallel rank's share of an MoE layer on AMD Instinct MI355X.

Route (router logits, top-k, combine weights) -> dispatch (rows grouped by
local expert) -> grouped SwiGLU expert MLPs -> combine (weighted sum in the
original token order), all in hand-written gfx950 HIP kernels behind the
C-ABI of ``include/moe.h``; this package is its Python binding. Beside them:
the whole share for a few tokens in two kernels, the expert MLPs in 8-bit
integers, the norms before and after the block, routing by scores and groups,
bf16 products with an epilogue, and the layer with a shared expert.
"""
from ._binding import (  # noqa: F401
    LIB_PATH, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_OK, FEW_TOKENS,
    MAX_GROUPS, NOALLOC_SCRATCH_BYTES, SIGNATURES,
    MoEError, block_workspace_size, check, expert_ffn_i8_workspace_size, few_workspace_size,
    forward_i8_workspace_size, forward_workspace_layout, forward_workspace_size, gemm_workspace_size,
    layer_workspace_size, lib, moe_block_forward, moe_combine, moe_combine_f32, moe_dispatch, moe_expert_ffn,
    moe_expert_ffn_i8, moe_forward, moe_forward_f32, moe_forward_few, moe_forward_few_f32, moe_forward_fused,
    moe_forward_i8, moe_forward_noalloc, moe_forward_profiled, moe_gemm, moe_gemm_i8, moe_layer_forward,
    moe_norm_post, moe_norm_pre, moe_quantize_rows, moe_quantize_weights, moe_route, moe_route_scored, moe_select,
    status_string,
)
