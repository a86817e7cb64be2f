"""GB300-native fused data-parallel step: gradient accumulation, ring-order reduce-scatter, averaging with
loss-scale unscaling and a global non-finite skip, ZeRO-partitioned mixed-precision Adam, and the bf16
parameter all-gather -- all n replicas' buffers in one GPU's memory.

Beside the step, the training-pass operators that fill its gradient buffers: embedding lookup and gradient, the norms around
a block, 8-bit activation checkpoints with the gated activation and the weight gradient that use them.

The computation lives in libdpstep.so (CUDA, sm_103a; C ABI in include/dpstep.h and include/dpops.h).  This package is its
binding; importing it without the built library raises ImportError.
"""
from ._lib import (  # noqa: F401
    DP_ERR_ALIGNMENT, DP_ERR_CUDA, DP_ERR_INVALID_ARG, DP_ERR_IO, DP_ERR_TIMEOUT, DP_MAX_N, DP_MAX_NA, DP_MAX_SEG,
    DP_DEFER_COMMIT, DP_DEVICE_SCALE, DP_KERNEL_SEG, DP_OK, DP_ORDER_RING, DP_ORDER_TREE, DP_SUM_COMPENSATED, DP_SUM_PLAIN, LIB, LIB_PATH, STATE_BYTES, DPError,
    Layout, adam, dp_accumulate, dp_adam_shard, dp_allgather_params, dp_checkpoint_info, dp_checkpoint_load,
    dp_checkpoint_save, dp_commit_single_pass, dp_commit_step, dp_get_wait_timeout_ns, dp_global_batch, dp_kernel_launches, dp_memory_model,
    dp_read_status, dp_reduce_scatter_avg, dp_reduce_scatter_micro, dp_scaler_init, dp_selftest_wait_timeout, dp_set_wait_timeout_ns,
    dp_state_init, dp_step, dp_step_from_host, dp_step_reduce, dp_step_scaled, dp_step_single_pass,
    dp_step_single_pass_from_host, dp_step_static, dp_step_update,
    dp_traffic_model, new_state, read_state, scaler)
from .ops import (  # noqa: F401
    DP_ACT_GELU, DP_ACT_SILU, DP_BF16, DP_CKPT8_GROUP, DP_F32, DP_GATE_CHANNEL, DP_GATE_NONE, DP_GATE_TOKEN, DP_MAX_NORM_DIM,
    DP_NORM_LAYER, DP_NORM_POST, DP_NORM_PRE, DP_NORM_RMS, dp_act_ckpt8, dp_act_ckpt8_grad, dp_block_norm,
    dp_block_norm_grad, dp_block_norm_t, dp_block_norm_workspace_size, dp_ckpt8_decode, dp_ckpt8_encode, dp_ckpt8_pitch,
    dp_embedding, dp_embedding_grad, dp_embedding_workspace_size, dp_wgrad8, dp_wgrad8_workspace_size, new_ckpt8)
