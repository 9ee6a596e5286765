"""Routed mixture-of-experts expert computation on AMD Instinct MI355X (gfx950).

The computation runs in hand-written HIP kernels behind the C ABI declared in
``include/moe.h``; this package is its thin Python binding.  ``build`` compiles
the library in-tree.
"""
from ._lib import (  # noqa: F401
    EXPORTED, LIB_PATH, MOE_ERR_BAD_EXPERT_ID, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_OK,
    FEW_MAX_TOKENS, NOALLOC_SCRATCH_BYTES, MoeDesc, MoeError, bwd, bwd_sep, check_device_status, empty_workspace,
    few_workspace_size, fwd, fwd_few, fwd_few_logits, fwd_logits, fwd_noalloc, fwd_sep, library,
    make_desc, mx_dequantize, mx_fwd, mx_fwd_logits, mx_quantize, mx_workspace_size, route, route_workspace_size, router, router_bwd, status_str, timing_disable, timing_enable,
    timing_read, workspace_size,
)
