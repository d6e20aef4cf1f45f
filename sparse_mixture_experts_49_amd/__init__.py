"""MI355X-native (gfx950) sparsely-gated Mixture-of-Experts layer, with a scored router, its
gradients and MXFP4 experts beside it, layer norm, balance loss by sequence and low-rank adapters.

The layer runs in hand-written HIP kernels behind the C ABI of
libmoe_mi355x.so (header: include/moe_mi355x.h); this package is its ctypes
binding.  Build the library with ``python -m sparse_mixture_experts_49_amd.build``.
"""
from .binding import (ENTRY_POINTS, MOE_CAPACITY_DROP, MOE_CAPACITY_REROUTE, MOE_FFN_AUTO, MOE_FFN_STREAM, MOE_FFN_TILED, MOE_H_AUTO,
                      MOE_H_BF16, MOE_H_SPLIT, Desc, MoeError, MxDesc, MxWeights, Routing, ScoreDesc, ScoreGrads,
                      ScoreRouting, Weights, alloc_h, alloc_mx, alloc_mx_workspace, alloc_score_workspace,
                      alloc_workspace, forward, load_library, moe_combine, moe_ffn_down,
                      moe_ffn_up, moe_ffn_up_gather, moe_forward, moe_forward_noalloc, moe_read_probe, moe_grouped_ffn, moe_mx_dequantize, moe_mx_dispatch,
                      moe_mx_ffn_down, moe_mx_ffn_up, moe_mx_forward, moe_mx_quantize, moe_mx_workspace_size, moe_permute, moe_query_plan,
                      moe_route, moe_score_backward, moe_score_route, moe_score_workspace_size,
                      moe_shared_ffn, moe_workspace_size)
from .binding import (BalanceDesc, BalanceOut, NormDesc, alloc_balance_workspace, alloc_norm_workspace, moe_balance_backward,
                      moe_balance_loss, moe_balance_workspace_size, moe_layer_norm, moe_layer_norm_backward,
                      moe_norm_workspace_size, moe_score_backward_add)
from .binding import (MxBlock, alloc_mx_block_workspace, moe_mx_block_forward, moe_mx_block_workspace_size)
from .binding import (LoraDesc, LoraWeights, alloc_lora_shared_workspace, alloc_lora_workspace, moe_lora_linear,
                      moe_lora_shared_ffn, moe_lora_shared_workspace_size, moe_lora_workspace_size)

__all__ = ["ENTRY_POINTS", "MOE_CAPACITY_DROP", "MOE_CAPACITY_REROUTE", "MOE_FFN_AUTO", "MOE_FFN_STREAM", "MOE_FFN_TILED", "MOE_H_AUTO",
           "MOE_H_BF16", "MOE_H_SPLIT", "Desc", "MoeError", "MxDesc", "MxWeights", "Routing", "ScoreDesc", "ScoreGrads",
           "ScoreRouting", "Weights", "alloc_h", "alloc_mx", "alloc_mx_workspace", "alloc_score_workspace",
           "alloc_workspace", "forward", "load_library", "moe_combine", "moe_ffn_down",
           "moe_ffn_up", "moe_ffn_up_gather", "moe_forward", "moe_forward_noalloc", "moe_read_probe", "moe_grouped_ffn", "moe_mx_dequantize", "moe_mx_dispatch",
           "moe_mx_ffn_down", "moe_mx_ffn_up", "moe_mx_forward", "moe_mx_quantize", "moe_mx_workspace_size", "moe_permute", "moe_query_plan",
           "moe_route", "moe_score_backward", "moe_score_route", "moe_score_workspace_size",
           "moe_shared_ffn", "moe_workspace_size",
           "BalanceDesc", "BalanceOut", "NormDesc", "alloc_balance_workspace", "alloc_norm_workspace", "moe_balance_backward",
           "moe_balance_loss", "moe_balance_workspace_size", "moe_layer_norm", "moe_layer_norm_backward",
           "moe_norm_workspace_size", "moe_score_backward_add",
           "MxBlock", "alloc_mx_block_workspace", "moe_mx_block_forward", "moe_mx_block_workspace_size",
           "LoraDesc", "LoraWeights", "alloc_lora_shared_workspace", "alloc_lora_workspace", "moe_lora_linear",
           "moe_lora_shared_ffn", "moe_lora_shared_workspace_size", "moe_lora_workspace_size"]
