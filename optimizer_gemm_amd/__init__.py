"""MI355X (gfx950) fused weight-gradient + optimizer step (FORGE) behind a C ABI.

The kernels live in libforge.so (optimizer_gemm_amd/csrc, declared in
include/forge.h); this package only builds and binds them.
"""
from .forge import (  # noqa: F401
    OPTIMIZERS, SLOTS, ForgeError, default_hyper, dgrad, describe, lib, make_hyper, new_states,
    optimizer_step, rand16, sr_bf16, status_str, step_scalars, version, wgrad, wgrad_step, wgrad_unfused,
    wgrad_unfused_noalloc, wgrad_step_group, MAX_GROUP,
    dyn_value, dyn_encode, mfma_peak,
    ACTS, linear, linear_act_backward, gated, gated_backward, gated_dgrad, dgrad_group, linear_cross_entropy,
    linear_cross_entropy_backward, linear_cross_entropy_step,
    MAX_EXPERTS, expert_plan, expert_dispatch, expert_combine, expert_combine_backward, expert_linear, expert_gated,
    expert_gated_dgrad, expert_dgrad_group, expert_wgrad, expert_wgrad_step,
    quantize_rows, linear_q8, gated_q8, expert_linear_q8, expert_gated_q8,
)
