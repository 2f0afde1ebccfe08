"""GB300-native (sm_103a) post-router MoE layer: forward and backward behind a C ABI.

The compute lives in ``csrc/`` (CUDA kernels, built into ``_lib/libmoe.so``);
``binding`` is a thin ctypes marshalling layer with the C entry points' names.
"""
from .binding import (HostPipe, MoEDecoder, MoELayer, MoENorm, MoERouter, MoeError, load, main_grads_from_combined, moe_backward, moe_config, moe_create,
                      moe_handle_config, moe_host_pipe_create, moe_host_pipe_destroy, moe_host_pipe_size, moe_host_pipe_sync,
                      moe_host_step,
                      moe_destroy, moe_device_status, moe_export_routing, moe_forward, moe_forward_topk, moe_kernel_name, moe_launch_count,
                      moe_profile_enable, moe_profile_read, moe_profile_select, moe_route_noalloc,
                      moe_prepare_weights, moe_quantize_mxfp8, moe_selftest_timeout, mxfp8_weight, mxfp8_view,
                      moe_main_grads, moe_saved_create, moe_saved_destroy, moe_saved_size, moe_weights,
                      moe_workspace_size, set_expert_tables, set_main_grad_tables, set_mx_expert_tables, weights_from_combined, wview,
                      moe_decode, moe_decode_create, moe_decode_destroy, moe_decode_size, moe_decode_status,
                      moe_norm_backward, moe_norm_backward_size, moe_norm_config, moe_norm_forward,
                      moe_router_backward, moe_router_config, moe_router_forward, moe_router_size,
                      MOE_B_COL, MOE_B_ROW, MOE_B_SQUARE, FeedForwardWeights, MoEFeedForward, MoEFp8Linear, fp8_dequantize, fp8_quantize,
                      fp8_scales_shape, moe_ffn_config, moe_ffn_size, moe_fp8_selftest_timeout, moe_fp8_status, moe_linear_config, moe_linear_size,
                      weights_from_combined_mxfp8)
from .block import BlockParams, DenseBlock, DenseParams, MoEBlock

__all__ = ["BlockParams", "DenseBlock", "DenseParams", "HostPipe", "MoEBlock", "MoEDecoder", "MoELayer", "MoENorm", "MoERouter", "MoeError", "load", "main_grads_from_combined", "moe_backward", "moe_config", "moe_create",
           "moe_handle_config", "moe_host_pipe_create", "moe_host_pipe_destroy", "moe_host_pipe_size", "moe_host_pipe_sync",
           "moe_host_step",
           "moe_destroy", "moe_device_status", "moe_export_routing", "moe_forward", "moe_forward_topk", "moe_kernel_name",
           "moe_launch_count", "moe_profile_enable", "moe_profile_read", "moe_profile_select", "moe_route_noalloc",
           "moe_prepare_weights", "moe_quantize_mxfp8", "moe_selftest_timeout", "mxfp8_weight", "mxfp8_view",
           "moe_main_grads", "moe_saved_create", "moe_saved_destroy", "moe_saved_size", "moe_weights",
           "moe_workspace_size", "set_expert_tables", "set_main_grad_tables", "set_mx_expert_tables", "weights_from_combined", "wview",
           "moe_decode", "moe_decode_create", "moe_decode_destroy", "moe_decode_size", "moe_decode_status",
           "moe_norm_backward", "moe_norm_backward_size", "moe_norm_config", "moe_norm_forward",
           "moe_router_backward", "moe_router_config", "moe_router_forward", "moe_router_size",
           "MOE_B_COL", "MOE_B_ROW", "MOE_B_SQUARE", "FeedForwardWeights", "MoEFeedForward", "MoEFp8Linear", "fp8_dequantize", "fp8_quantize",
           "fp8_scales_shape", "moe_ffn_config", "moe_ffn_size", "moe_fp8_selftest_timeout", "moe_fp8_status", "moe_linear_config", "moe_linear_size",
           "weights_from_combined_mxfp8"]
