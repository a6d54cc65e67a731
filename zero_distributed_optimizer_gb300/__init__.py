"""GB300-native ZeRO-1 distributed-optimizer step (Megatron-style, flat buffer).

The work runs in libdopt.so (hand-written sm_103a CUDA kernels behind the C
ABI declared in include/dopt.h); this package is its thin Python binding.
The library is loaded on first use and every call raises if it is missing.
"""
from .binding import (  # noqa: F401
    DOPT_BF16,
    DOPT_CHECK_ALIGN,
    DOPT_CHECK_INDEX,
    DOPT_CLIP_WORKSPACE_BYTES,
    DOPT_COUNTER_BAD_STEP,
    DOPT_E_ALIGN,
    DOPT_E_ARG,
    DOPT_E_CUDA,
    DOPT_E_LAYOUT,
    DOPT_E_NOMEM,
    DOPT_E_STATE,
    DOPT_FP16,
    DOPT_FP32,
    DOPT_MAX_D,
    DOPT_OK,
    DOPT_STEP_COUNTER_BYTES,
    DOPT_STEP_GATHER,
    DOPT_STEP_HOST_GRADS,
    DOPT_STEP_HOST_PARAMS,
    DOPT_STEP_PARAMS_FP16,
    DOPT_STEP_ROUND_GRAD,
    DOPT_STEP_SKIP_NONFINITE,
    DOPT_STEP_STAGE,
    AdamConfig,
    DoptError,
    HostStepper,
    Layout,
    StepPlan,
    device_checks,
    dopt_allreduce,
    dopt_build_range_map,
    dopt_gather,
    dopt_step,
    dopt_step_allreduce,
    dopt_step_buckets,
    dopt_step_clipped,
    dopt_step_clipped_counted,
    dopt_step_clipped_noalloc,
    dopt_step_counted,
    clip_report,
    clip_workspace,
    counter_diagnostics,
    counter_scalars,
    counter_state,
    dopt_stream_probe,
    read_clip_report,
    stage_timeouts,
    stage_wait_test,
    step_counter,
    step_from_host,
    version,
)

# The layer operators' binding imports torch, so it is loaded on first use.
_LAYER_OPS = (
    "DOPT_ACT_GELU",
    "DOPT_ACT_SILU",
    "DOPT_ACT_SWIGLU",
    "DOPT_CKPT_BLOCK",
    "DOPT_CKPT_PITCH",
    "DOPT_MAX_COLS",
    "DOPT_MAX_EXPERTS",
    "DOPT_MAX_GROUPS",
    "DOPT_MAX_TOPK",
    "DOPT_WGRAD_ACCUMULATE",
    "DOPT_WGRAD_MAX_ROWS",
    "Checkpoint",
    "checkpoint",
    "ckpt_bytes",
    "dopt_ckpt_act_grad",
    "dopt_ckpt_load",
    "dopt_ckpt_save",
    "dopt_ckpt_wgrad",
    "dopt_route_combine",
    "dopt_route_combine_grad",
    "dopt_route_dispatch",
    "dopt_route_sort",
    "route_workspace",
    "WgradPlan",
    "wgrad_plan",
    "wgrad_timeouts",
    "wgrad_wait_test",
    "wgrad_workspace",
)

# The same for the operators of a language model's ends and residual stream.
_MODEL_OPS = (
    "DOPT_EMBED_ACCUMULATE",
    "DOPT_EMBED_MAX_TOKENS",
    "DOPT_HEAD_ACCUMULATE",
    "DOPT_HEAD_MAX_ROWS",
    "DOPT_HEAD_MAX_VOCAB",
    "DOPT_NORM_ACCUMULATE",
    "DOPT_NORM_LAYER",
    "DOPT_NORM_MAX_COLS",
    "DOPT_NORM_RMS",
    "dopt_embed",
    "dopt_embed_grad",
    "dopt_head_loss",
    "dopt_head_loss_grad",
    "dopt_norm",
    "dopt_norm_grad",
    "embed_workspace",
    "head_loss_grad_workspace",
    "head_loss_workspace",
    "head_timeouts",
    "head_wait_test",
    "norm_workspace",
)


def __getattr__(name):
    if name in _LAYER_OPS:
        from . import layer_ops as module
    elif name in _MODEL_OPS:
        from . import model_ops as module
    else:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    value = globals()[name] = getattr(module, name)
    return value


def __dir__():
    return sorted(set(globals()) | set(_LAYER_OPS) | set(_MODEL_OPS))
