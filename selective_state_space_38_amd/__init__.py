"""MI355X (gfx950) selective-scan (Mamba S6) library: a C-ABI shared library
with hand-written HIP kernels, and a thin PyTorch binding."""

from .api import (  # noqa: F401
    selective_scan_fwd,
    selective_scan_fwd_aggregate,
    selective_scan_carry_combine,
    selective_scan_bwd,
    ckpt_buffer,
    record_buffer,
    selective_state_update,
    causal_conv1d_fwd,
    causal_conv1d_update,
    mamba_block_fwd,
    check_device_errors,
    fwd_plan,
)
from .layer import (  # noqa: F401
    gated_scan_fwd,
    gated_scan_bwd,
    gated_ckpt_buffer,
    gated_state_update,
    rms_norm_fwd,
    rms_norm_fp8,
    rms_norm_bwd,
    fp8_quantize,
    fp8_quantize_weight,
    fp8_linear,
)
from .feed_forward import (  # noqa: F401
    expert_route_fwd,
    expert_route_bwd,
    expert_sort,
    expert_gather,
    expert_combine_fwd,
    expert_combine_bwd,
    expert_linear_fwd,
    expert_linear_bwd,
    linear_fwd,
    linear_bwd,
)
