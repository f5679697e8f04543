"""MI355X-native forward pass of one Mixture-of-Experts layer.

gate (float32 logits, top-k, renormalised weights) -> dispatch (histogram,
scan, stable permutation, optional per-token affine FP8 rows) -> grouped
SwiGLU expert FFN (bf16 matrix cores) -> combine (weighted un-permute), and
the backward of these. Beside them: linear layers per expert or dense, forward
and backward (moe_grouped_linear, moe_linear), and activation checkpoints in 8
bits (moe_pack_rows8, moe_grouped_ffn_save8).
The work runs in the HIP kernels of libmoe_mi355x.so behind the C ABI in
include/moe.h; this package is its ctypes binding. Build the library with
``python mixture_experts_routing_gemm_amd/build.py``.
"""

from ._binding import (  # noqa: F401
    EXPORTS, MOE_BF16, MOE_ERR_BAD_INDEX, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED,
    MOE_ERR_WORKSPACE, MOE_F32, MOE_FP8_E4M3, MOE_OK, MOE_OVERFLOW_DROP, MOE_OVERFLOW_REASSIGN,
    MOE_QUANT_EXPERT, MOE_QUANT_GLOBAL, MOE_QUANT_TOKEN, MOE_QUANT_TOKEN_ABSMAX,
    FP8W_KERNELS, STAGE_COMBINE, STAGE_DISPATCH, STAGE_FFN, STAGE_FFN_BACKWARD, STAGE_FORWARD_FP8W,
    STAGE_GATE_BACKWARD,
    STAGE_FORWARD, STAGE_GATE, MoEError, alloc_workspace, make_shape, moe_combine, moe_combine_backward,
    moe_dispatch, moe_dispatch_backward, moe_dispatch_noalloc, moe_gate_backward,
    moe_forward, moe_forward_fp8w, moe_forward_kernel_count, moe_fp8_weight_scale_floats,
    moe_quantize_weights, moe_forward_kernel_name, moe_forward_traced,
    moe_gate_topk, moe_get_device_error, moe_grouped_ffn, moe_grouped_ffn_backward, moe_shape,
    moe_ffn_saved_bytes, alloc_saved, moe_grouped_ffn_save, moe_grouped_ffn_backward_saved,
    MOE_FN_GELU, MOE_FN_NONE, MOE_FN_RELU, MOE_FN_SILU, MOE_SAVE_ACT, MOE_SAVE_INT8, MOE_SAVE_NONE,
    STAGE_LINEAR, STAGE_LINEAR_BACKWARD, STAGE_FFN_BACKWARD8, alloc_linear_saved, alloc_linear_workspace, alloc_rows8,
    make_linear_shape, moe_grouped_linear, moe_grouped_linear_backward, moe_linear, moe_linear_backward,
    moe_linear_saved_bytes, moe_linear_shape, moe_linear_workspace_bytes, moe_pack_rows8, moe_rows8_bytes,
    moe_unpack_rows8, moe_ffn_saved8_bytes, alloc_saved8, moe_grouped_ffn_save8,
    moe_grouped_ffn_backward_saved8, moe_workspace_bytes,
    moe_workspace_init, shape_of, status_string)
from .buffers import ForwardBuffers  # noqa: F401
