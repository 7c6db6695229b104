"""MI355X (gfx950) MoE expert layer: HIP kernels behind a C ABI, with a thin ctypes binding.

The layer runs route -> permute -> FC1 + (OAI-)SwiGLU + 1x128 requant -> FC2 -> combine
on one GPU's share of the experts.  Beside it stand its parts for callers with a router or
experts of their own: tokens sorted by expert and back, with gradients,
MXFP4 quantisation and products, the router's balance loss with its gradient, and 4-bit weights
with group scales.  ``binding`` holds the entry points (same names as
the C ABI); ``synth`` makes seeded synthetic inputs; ``build`` compiles the library.
"""
from .binding import (  # noqa: F401
    MoeBalanceDesc, MoeDispatchDesc, MoeError, MoeInt4Desc, MoeLayerDesc, MoeMxfp4Desc, MoeMxfp4GemmDesc, MoeW4GemmDesc,
    alloc_balance_workspace, alloc_sort_workspace, alloc_workspace, desc_from_workload, lib, make_balance_desc, make_desc,
    make_dispatch_desc, make_int4_desc, make_mxfp4_desc, make_mxfp4_gemm_desc, make_w4_gemm_desc, moe_balance_loss,
    moe_balance_loss_backward, moe_balance_workspace_size, moe_combine, moe_combine_backward, moe_dequantize_int4,
    moe_dequantize_mxfp4, moe_dispatch, moe_dispatch_backward, moe_grouped_fc1_swiglu, moe_grouped_fc2_combine, moe_layer,
    moe_mxfp4_gemm, moe_quantize_int4, moe_quantize_mxfp4, moe_route_permute, moe_sort_tokens, moe_sort_workspace_size,
    moe_w4_gemm, moe_workspace_size,
)
