"""B200-native (sm_100a) sparse mixture-of-experts feed-forward layer.

The CUDA library ``libmoe.so`` (C-ABI in ``include/moe.h``) does all the work; this package is its thin
Python binding (``_native``) plus a layer object that owns buffers and calls the entry points in order
(``layer.MoEFFN``). Importing the package loads the library and fails if it has not been built.
"""
from . import _native
from ._native import (MoEError, ROUTE_MODES, block_norm_backward_workspace_size, block_norm_in, block_norm_in_backward,
                      block_norm_out, block_norm_out_backward, few_tokens, few_tokens_workspace_size, fp8_block_quantize,
                      fp8_row_quantize, get_device_error, grouped_gemm_down, grouped_gemm_down_fp8, grouped_gemm_gateup,
                      grouped_gemm_gateup_fp8, permute, permute_workspace_size, route_topk, topk_from_logits,
                      unpermute_combine)
from .layer import MoEBlock, MoEFFN

__all__ = ["MoEFFN", "MoEBlock", "MoEError", "ROUTE_MODES", "route_topk", "topk_from_logits", "permute",
           "permute_workspace_size", "grouped_gemm_gateup", "grouped_gemm_down", "unpermute_combine",
           "few_tokens", "few_tokens_workspace_size", "fp8_block_quantize", "fp8_row_quantize",
           "grouped_gemm_gateup_fp8", "grouped_gemm_down_fp8", "block_norm_in", "block_norm_out",
           "block_norm_in_backward", "block_norm_out_backward", "block_norm_backward_workspace_size",
           "get_device_error"]
