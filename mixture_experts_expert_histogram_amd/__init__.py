"""Routed mixture-of-experts expert computation on AMD Instinct MI355X (gfx950).

The computation runs in hand-written HIP kernels behind the C ABI declared in
``include/moe.h``; this package is its thin Python binding.  ``build`` compiles
the library in-tree.
"""
from ._lib import (  # noqa: F401
    EXPORTED, LIB_PATH, MOE_ERR_BAD_EXPERT_ID, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_OK,
    FEW_MAX_TOKENS, NEWTON_SCHULZ, NOALLOC_SCRATCH_BYTES, MoeDesc, MoeError, ResidualGrads, bwd, bwd_sep,
    check_device_status, empty_workspace, few_workspace_size, ffn_bwd, ffn_fwd, ffn_workspace_size, fwd, fwd_few,
    fwd_few_logits, fwd_logits, fwd_noalloc, fwd_sep, library, make_desc, muon_step, mx_dequantize, mx_fwd, mx_fwd_logits,
    mx_quantize, mx_workspace_size, norm_bwd, norm_fwd, norm_workspace_size, ortho_workspace_size, orthogonalize,
    residual_bwd, residual_fwd, route, route_workspace_size, router, router_bwd, status_str, timing_disable, timing_enable,
    timing_read, workspace_size,
)
