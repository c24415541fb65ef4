"""MI355X (gfx950) MoE routing, dispatch and combine.

The compute lives in the HIP library ``libmoe_dc.so`` (C ABI in
``include/moe_dc.h``); this package is its PyTorch binding.  Importing it
without the built library raises ImportError -- there is no CPU fallback.
"""
from .api import (BalanceLoss, DispatchResult, MoeError, default_sort_cutoff, moe_abi_version, moe_balance_loss,
                  moe_balance_loss_backward, moe_balance_loss_workspace_bytes, moe_combine,
                  moe_dequant_int4, moe_gather_gemm_int4, moe_gather_gemm_int4_workspace_bytes, moe_quantize_int4,
                  moe_combine_backward, moe_dequant_mxfp4, moe_dequant_rows,
                  moe_dispatch, moe_dispatch_backward, moe_dispatch_workspace_bytes, moe_gather_gemm_mxfp4,
                  moe_gather_gemm_mxfp4_workspace_bytes, moe_gather_rows,
                  moe_gather_swiglu, moe_gather_swiglu_combine,
                  moe_gather_swiglu_workspace_bytes,
                  moe_grouped_gemm_fp8, moe_grouped_gemm_mxfp4, moe_grouped_swiglu,
                  moe_grouped_swiglu_workspace_bytes, moe_quantize_mxfp4, moe_resolve_sorted, moe_route_dispatch,
                  moe_route_dispatch_noalloc, moe_route_dispatch_workspace_bytes, moe_route_topk,
                  moe_route_topk_backward,
                  moe_scatter_rows)
from ._lib import LIB_PATH, MOE_NOALLOC_SCRATCH_BYTES, MOE_SORT_AUTO, MOE_SORT_OFF, MOE_SORT_ON

__all__ = ["BalanceLoss", "moe_balance_loss", "moe_balance_loss_backward", "moe_balance_loss_workspace_bytes",
           "moe_quantize_int4", "moe_dequant_int4", "moe_gather_gemm_int4", "moe_gather_gemm_int4_workspace_bytes",
           "DispatchResult", "MoeError", "default_sort_cutoff", "moe_abi_version", "moe_combine",
           "moe_combine_backward", "moe_dispatch_backward", "moe_route_topk_backward",
           "moe_dequant_rows",
           "moe_dispatch", "moe_dispatch_workspace_bytes", "moe_gather_rows",
           "moe_gather_swiglu", "moe_gather_swiglu_combine",
           "moe_gather_swiglu_workspace_bytes",
           "moe_grouped_gemm_fp8", "moe_grouped_swiglu",
           "moe_grouped_swiglu_workspace_bytes", "moe_resolve_sorted", "moe_route_topk",
           "moe_scatter_rows", "moe_route_dispatch", "moe_route_dispatch_noalloc",
           "moe_route_dispatch_workspace_bytes",
           "moe_quantize_mxfp4", "moe_dequant_mxfp4", "moe_grouped_gemm_mxfp4", "moe_gather_gemm_mxfp4",
           "moe_gather_gemm_mxfp4_workspace_bytes",
           "LIB_PATH", "MOE_NOALLOC_SCRATCH_BYTES", "MOE_SORT_AUTO", "MOE_SORT_OFF", "MOE_SORT_ON"]
