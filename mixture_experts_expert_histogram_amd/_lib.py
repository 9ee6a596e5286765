"""ctypes binding of the C ABI in include/moe.h (argument marshalling only).

Every step of the computation runs in the HIP library; torch supplies device
memory and the current stream.  Loading fails loudly if the library is not
built: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_mi355x.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP, MOE_ERR_BAD_EXPERT_ID = range(6)
MOE_BF16, MOE_F32 = 0, 1
MOE_SWIGLU, MOE_CLAMPED_GLU = 0, 1
MOE_GU_CONCAT, MOE_GU_INTERLEAVED = 0, 1

EXPORTED = ["moe_workspace_size", "moe_route_workspace_size", "moe_route", "moe_router", "moe_fwd",
            "moe_fwd_logits", "moe_fwd_sep", "moe_bwd", "moe_bwd_sep", "moe_router_bwd", "moe_check_device_status",
            "moe_status_str", "moe_timing_enable", "moe_timing_disable", "moe_timing_read", "moe_fwd_noalloc",
            "moe_few_workspace_size", "moe_fwd_few", "moe_fwd_few_logits", "moe_mx_quantize", "moe_mx_dequantize",
            "moe_mx_workspace_size", "moe_mx_fwd", "moe_mx_fwd_logits", "moe_ffn_workspace_size", "moe_ffn_fwd",
            "moe_ffn_bwd", "moe_norm_workspace_size", "moe_norm_fwd", "moe_norm_bwd", "moe_residual_fwd",
            "moe_residual_bwd", "moe_ortho_workspace_size", "moe_orthogonalize", "moe_muon_step"]

# Most tokens of fwd_few (moe.h).
FEW_MAX_TOKENS = 128

# Size of the library's per-GPU scratch array behind moe_fwd_noalloc (moe.h).
NOALLOC_SCRATCH_BYTES = 64 << 20


class MoeDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("gu_layout", ctypes.c_int32),
                ("clamp_limit", ctypes.c_float), ("glu_alpha", ctypes.c_float),
                ("grad_dtype", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class OrthoDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float)]


class Muon(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("decay", ctypes.c_float), ("nesterov", ctypes.c_int32)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_double)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


_lib = None


def library() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"MoE HIP library not built: {LIB_PATH} is missing "
                          "(run `python -m mixture_experts_expert_histogram_amd.build`)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    pd = ctypes.POINTER(MoeDesc)
    psz = ctypes.POINTER(ctypes.c_size_t)
    lib.moe_workspace_size.argtypes = [pd, psz, psz, psz]
    lib.moe_route_workspace_size.argtypes = [pd, psz]
    lib.moe_route.argtypes = [pd, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_router.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.moe_fwd_logits.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.moe_router_bwd.argtypes = [pd, vp, vp, vp, vp, vp]
    lib.moe_fwd_sep.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.moe_bwd_sep.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_bwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_fwd_noalloc.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.moe_few_workspace_size.argtypes = [pd, psz]
    lib.moe_fwd_few.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_fwd_few_logits.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_mx_quantize.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    lib.moe_mx_dequantize.argtypes = [vp, vp, i32, i64, i64, vp, vp]
    lib.moe_mx_workspace_size.argtypes = [pd, psz]
    lib.moe_mx_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_mx_fwd_logits.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    pn, po, pm = ctypes.POINTER(NormDesc), ctypes.POINTER(OrthoDesc), ctypes.POINTER(Muon)
    lib.moe_ffn_workspace_size.argtypes = [pd, psz, psz, psz]
    lib.moe_ffn_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.moe_ffn_bwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_norm_workspace_size.argtypes = [pn, psz]
    lib.moe_norm_fwd.argtypes = [pn, vp, vp, vp, vp]
    lib.moe_norm_bwd.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_residual_fwd.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_residual_bwd.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_ortho_workspace_size.argtypes = [po, psz]
    lib.moe_orthogonalize.argtypes = [po, vp, vp, vp, sz, vp]
    lib.moe_muon_step.argtypes = [po, pm, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_check_device_status.argtypes = [vp, vp]
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_timing_enable.argtypes = [ctypes.c_int32]
    lib.moe_timing_disable.argtypes = []
    lib.moe_timing_read.argtypes = [ctypes.POINTER(KernelTime), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
    for name in EXPORTED:
        if name != "moe_status_str":
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return library().moe_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _dt(name) -> int:
    if name in ("bf16", "bfloat16"):
        return MOE_BF16
    if name in ("fp32", "float32"):
        return MOE_F32
    raise ValueError(f"unsupported dtype {name}")


def make_desc(T, H, I, E, K, dtype="bf16", act="swiglu", layout="concat", limit=7.0, alpha=1.702,
              grad_dtype=None) -> MoeDesc:
    return MoeDesc(int(T), int(H), int(I), int(E), int(K), _dt(dtype),
                   MOE_CLAMPED_GLU if act == "clamped" else MOE_SWIGLU,
                   MOE_GU_INTERLEAVED if layout == "interleaved" else MOE_GU_CONCAT,
                   float(limit), float(alpha), _dt(grad_dtype or dtype))


def workspace_size(desc: MoeDesc) -> Tuple[int, int, int]:
    f, b, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().moe_workspace_size(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b), ctypes.byref(s)),
           "moe_workspace_size")
    return f.value, b.value, s.value


def route_workspace_size(desc: MoeDesc) -> int:
    r = ctypes.c_size_t()
    _check(library().moe_route_workspace_size(ctypes.byref(desc), ctypes.byref(r)), "moe_route_workspace_size")
    return r.value


# ---------------------------------------------------------------- torch layer
def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ids32(topk_ids):
    import torch
    return topk_ids if topk_ids.dtype == torch.int32 and topk_ids.is_contiguous() else \
        topk_ids.to(torch.int32).contiguous()


def _f32(x):
    import torch
    return x if x.dtype == torch.float32 and x.is_contiguous() else x.to(torch.float32).contiguous()


def _desc_for(hidden, topk_ids, w_gate_up, w_down, act, layout, limit, alpha, grad_dtype=None) -> MoeDesc:
    import torch
    T, H = hidden.shape
    E, I2, H2 = w_gate_up.shape
    if H2 != H or tuple(w_down.shape) != (E, H, I2 // 2) or topk_ids.shape[0] != T:
        raise ValueError("inconsistent MoE shapes")
    for t in (hidden, w_gate_up, w_down):
        if t.dtype != hidden.dtype or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("hidden and weights must be contiguous device tensors of one dtype")
    dt = "bf16" if hidden.dtype == torch.bfloat16 else ("fp32" if hidden.dtype == torch.float32 else None)
    if dt is None:
        raise ValueError(f"unsupported dtype {hidden.dtype}")
    return make_desc(T, H, I2 // 2, E, topk_ids.shape[1], dt, act, layout, limit, alpha, grad_dtype)


def empty_workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def route(topk_ids, E: int, ws=None):
    """counts [E], offsets [E+1], sorted_slot [S], inv_pos [S] (int32 device tensors)."""
    import torch
    ids = _ids32(topk_ids)
    T, K = ids.shape
    d = make_desc(T, 8, 8, E, K)
    dev = ids.device
    nbytes = route_workspace_size(d)
    ws = empty_workspace(nbytes, dev) if ws is None else ws
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ss = torch.empty(T * K, dtype=torch.int32, device=dev)
    ip = torch.empty(T * K, dtype=torch.int32, device=dev)
    _check(library().moe_route(ctypes.byref(d), _ptr(ids), _ptr(counts), _ptr(offsets), _ptr(ss), _ptr(ip),
                               _ptr(ws), ws.numel(), _stream()), "moe_route")
    return counts, offsets, ss, ip, ws


def router(logits, K: int, ws=None, out=None):
    """Top-K of router logits [T,E] (fp32) and their softmax, with the routing.

    Returns (topk_ids int32 [T,K], topk_weights fp32 [T,K], counts [E],
    offsets [E+1], sorted_slot [S], inv_pos [S], ws)."""
    import torch
    lg = _f32(logits)
    if not lg.is_cuda or lg.dim() != 2:
        raise ValueError("router takes device logits [T, E]")
    T, E = lg.shape
    d = make_desc(T, 8, 8, E, K)
    dev = lg.device
    ws = empty_workspace(route_workspace_size(d), dev) if ws is None else ws
    if out is None:
        out = (torch.empty((T, K), dtype=torch.int32, device=dev), torch.empty((T, K), dtype=torch.float32, device=dev))
    ids, w = out
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ss = torch.empty(T * K, dtype=torch.int32, device=dev)
    ip = torch.empty(T * K, dtype=torch.int32, device=dev)
    _check(library().moe_router(ctypes.byref(d), _ptr(lg), _ptr(ids), _ptr(w), _ptr(counts), _ptr(offsets),
                                _ptr(ss), _ptr(ip), _ptr(ws), ws.numel(), _stream()), "moe_router")
    return ids, w, counts, offsets, ss, ip, ws


def router_bwd(topk_ids, topk_weights, d_topk_weights, E: int, out=None):
    """d_logits fp32 [T,E] from the routing-weight gradient."""
    import torch
    ids, w, g = _ids32(topk_ids), _f32(topk_weights), _f32(d_topk_weights)
    T, K = ids.shape
    if tuple(w.shape) != (T, K) or tuple(g.shape) != (T, K):
        raise ValueError("topk_ids, topk_weights and d_topk_weights must all be [T, K]")
    if not (ids.is_cuda and w.is_cuda and g.is_cuda):
        raise ValueError("router_bwd takes device tensors")
    d = make_desc(T, 8, 8, E, K)
    out = torch.empty((T, E), dtype=torch.float32, device=ids.device) if out is None else out
    _check(library().moe_router_bwd(ctypes.byref(d), _ptr(ids), _ptr(w), _ptr(g), _ptr(out), _stream()),
           "moe_router_bwd")
    return out


def fwd_logits(hidden, logits, K: int, w_gate_up, w_down, act="swiglu", layout="concat", limit=7.0, alpha=1.702,
               save=False, ws=None, out=None, saved=None, routing=None):
    """Forward from router logits [T,E]; returns (out, topk_ids, topk_weights, saved-or-None, ws)."""
    import torch
    lg = _f32(logits)
    T, E = lg.shape
    if T != hidden.shape[0] or E != w_gate_up.shape[0]:
        raise ValueError("logits must be [T, E] for hidden [T, H] and w_gate_up [E, 2I, H]")
    dev = hidden.device
    if routing is None:
        routing = (torch.empty((T, K), dtype=torch.int32, device=dev),
                   torch.empty((T, K), dtype=torch.float32, device=dev))
    ids, w = routing
    d = _desc_for(hidden, ids, w_gate_up, w_down, act, layout, limit, alpha)
    fws, _, sbytes = workspace_size(d)
    ws = empty_workspace(fws, dev) if ws is None else ws
    out = torch.empty_like(hidden) if out is None else out
    if save and saved is None:
        saved = empty_workspace(sbytes, dev)
    _check(library().moe_fwd_logits(ctypes.byref(d), _ptr(hidden), _ptr(lg), _ptr(w_gate_up), _ptr(w_down),
                                    _ptr(out), _ptr(ids), _ptr(w), _ptr(saved) if save else None,
                                    _nbytes(saved) if save else 0, _ptr(ws), ws.numel(), _stream()),
           "moe_fwd_logits")
    return out, ids, w, (saved if save else None), ws


def fwd(hidden, topk_ids, topk_weights, w_gate_up, w_down, act="swiglu", layout="concat", limit=7.0,
        alpha=1.702, save=False, ws=None, out=None, saved=None):
    """Forward pass; returns (out, saved-or-None, ws)."""
    import torch
    d = _desc_for(hidden, topk_ids, w_gate_up, w_down, act, layout, limit, alpha)
    ids, w = _ids32(topk_ids), _f32(topk_weights)
    fws, _, sbytes = workspace_size(d)
    ws = empty_workspace(fws, hidden.device) if ws is None else ws
    out = torch.empty_like(hidden) if out is None else out
    if save and saved is None:
        saved = empty_workspace(sbytes, hidden.device)
    _check(library().moe_fwd(ctypes.byref(d), _ptr(hidden), _ptr(ids), _ptr(w), _ptr(w_gate_up), _ptr(w_down),
                             _ptr(out), _ptr(saved) if save else None, _nbytes(saved) if save else 0, _ptr(ws),
                             ws.numel(), _stream()), "moe_fwd")
    return out, (saved if save else None), ws


def fwd_noalloc(hidden, topk_ids, topk_weights, w_gate_up, w_down, act="swiglu", layout="concat", limit=7.0,
                alpha=1.702, out=None, saved=None, bad_ids=None):
    """Forward with the library's own per-GPU scratch as workspace (moe_fwd_noalloc);
    returns out.  `saved` (optional) receives Z as for fwd(save=True); `bad_ids`
    (optional int32 device tensor of one element) the number of bad-id slots."""
    import torch
    d = _desc_for(hidden, topk_ids, w_gate_up, w_down, act, layout, limit, alpha)
    ids, w = _ids32(topk_ids), _f32(topk_weights)
    out = torch.empty_like(hidden) if out is None else out
    _check(library().moe_fwd_noalloc(ctypes.byref(d), _ptr(hidden), _ptr(ids), _ptr(w), _ptr(w_gate_up),
                                     _ptr(w_down), _ptr(out), _ptr(saved), _nbytes(saved), _ptr(bad_ids),
                                     _stream()), "moe_fwd_noalloc")
    return out


def bwd(hidden, topk_ids, topk_weights, w_gate_up, w_down, d_out, saved=None, act="swiglu", layout="concat",
        limit=7.0, alpha=1.702, ws=None, grads=None, grad_dtype=None):
    """Backward pass; returns (d_hidden, d_topk_weights, d_w_gate_up, d_w_down, ws).

    grad_dtype: "bf16" or "fp32" storage of the weight gradients (default: the
    activation dtype)."""
    import torch
    d = _desc_for(hidden, topk_ids, w_gate_up, w_down, act, layout, limit, alpha, grad_dtype)
    ids, w = _ids32(topk_ids), _f32(topk_weights)
    _, bws, _ = workspace_size(d)
    ws = empty_workspace(bws, hidden.device) if ws is None else ws
    if grads is None:
        gdt = torch.float32 if d.grad_dtype == MOE_F32 else torch.bfloat16
        grads = (torch.empty_like(hidden), torch.empty(ids.shape, dtype=torch.float32, device=hidden.device),
                 torch.empty(w_gate_up.shape, dtype=gdt, device=hidden.device),
                 torch.empty(w_down.shape, dtype=gdt, device=hidden.device))
    dh, dw, dgu, dd = grads
    _check(library().moe_bwd(ctypes.byref(d), _ptr(hidden), _ptr(ids), _ptr(w), _ptr(w_gate_up), _ptr(w_down),
                             _ptr(d_out.contiguous()), _ptr(saved), _nbytes(saved), _ptr(dh), _ptr(dw), _ptr(dgu),
                             _ptr(dd), _ptr(ws), ws.numel(), _stream()), "moe_bwd")
    return dh, dw, dgu, dd, ws


def _sep_desc(hidden, topk_ids, w_gate, w_up, w_down, act, limit, alpha, grad_dtype=None) -> MoeDesc:
    import torch
    T, H = hidden.shape
    E, I, H2 = w_gate.shape
    if (H2 != H or tuple(w_up.shape) != (E, I, H) or tuple(w_down.shape) != (E, H, I)
            or topk_ids.shape[0] != T):
        raise ValueError("inconsistent MoE shapes")
    for t in (hidden, w_gate, w_up, w_down):
        if t.dtype != hidden.dtype or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("hidden and weights must be contiguous device tensors of one dtype")
    dt = "bf16" if hidden.dtype == torch.bfloat16 else ("fp32" if hidden.dtype == torch.float32 else None)
    if dt is None:
        raise ValueError(f"unsupported dtype {hidden.dtype}")
    return make_desc(T, H, I, E, topk_ids.shape[1], dt, act, "concat", limit, alpha, grad_dtype)


def fwd_sep(hidden, topk_ids, topk_weights, w_gate, w_up, w_down, act="swiglu", limit=7.0, alpha=1.702, save=False,
            ws=None, out=None, saved=None):
    """Forward with separate gate and up weights [E, I, H]; returns (out, saved-or-None, ws)."""
    import torch
    d = _sep_desc(hidden, topk_ids, w_gate, w_up, w_down, act, limit, alpha)
    ids, w = _ids32(topk_ids), _f32(topk_weights)
    fws, _, sbytes = workspace_size(d)
    ws = empty_workspace(fws, hidden.device) if ws is None else ws
    out = torch.empty_like(hidden) if out is None else out
    if save and saved is None:
        saved = empty_workspace(sbytes, hidden.device)
    _check(library().moe_fwd_sep(ctypes.byref(d), _ptr(hidden), _ptr(ids), _ptr(w), _ptr(w_gate), _ptr(w_up),
                                 _ptr(w_down), _ptr(out), _ptr(saved) if save else None,
                                 _nbytes(saved) if save else 0, _ptr(ws), ws.numel(), _stream()), "moe_fwd_sep")
    return out, (saved if save else None), ws


def bwd_sep(hidden, topk_ids, topk_weights, w_gate, w_up, w_down, d_out, saved=None, act="swiglu", limit=7.0,
            alpha=1.702, ws=None, grads=None, grad_dtype=None):
    """Backward with separate gate and up weights; returns
    (d_hidden, d_topk_weights, d_w_gate, d_w_up, d_w_down, ws)."""
    import torch
    d = _sep_desc(hidden, topk_ids, w_gate, w_up, w_down, act, limit, alpha, grad_dtype)
    ids, w = _ids32(topk_ids), _f32(topk_weights)
    _, bws, _ = workspace_size(d)
    ws = empty_workspace(bws, hidden.device) if ws is None else ws
    if grads is None:
        gdt = torch.float32 if d.grad_dtype == MOE_F32 else torch.bfloat16
        grads = (torch.empty_like(hidden), torch.empty(ids.shape, dtype=torch.float32, device=hidden.device),
                 torch.empty(w_gate.shape, dtype=gdt, device=hidden.device),
                 torch.empty(w_up.shape, dtype=gdt, device=hidden.device),
                 torch.empty(w_down.shape, dtype=gdt, device=hidden.device))
    dh, dw, dg, du, dd = grads
    _check(library().moe_bwd_sep(ctypes.byref(d), _ptr(hidden), _ptr(ids), _ptr(w), _ptr(w_gate), _ptr(w_up),
                                 _ptr(w_down), _ptr(d_out.contiguous()), _ptr(saved), _nbytes(saved), _ptr(dh),
                                 _ptr(dw), _ptr(dg), _ptr(du), _ptr(dd), _ptr(ws), ws.numel(), _stream()),
           "moe_bwd_sep")
    return dh, dw, dg, du, dd, ws


# ---------------------------------------------------------------- few tokens, 4-bit weights
# A decode step's calls take a few microseconds on the GPU, so their host side is kept short: the binding's functions are
# looked up once, sizes of a descriptor are kept, and checks run on what the caller passed only.
def _raw_stream(index: int) -> int:
    """The current stream of a device as an integer, by torch's direct query where it has one (0.1 us against 3)."""
    import torch
    q = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return q(index) if q is not None else torch.cuda.current_stream(index).cuda_stream


def _on_device(device, f, *args) -> int:
    """f(*args, stream) with the tensors' device current and its current stream; returns the status."""
    import torch
    if device.index == torch.cuda.current_device():
        return f(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        return f(*args, _raw_stream(device.index))


def _launch(device, where: str, f, *args):
    """Call f(*args, stream) on the current stream of the tensors' device."""
    status = _on_device(device, f, *args)
    if status != MOE_OK:
        raise MoeError(status, where)


def _need(t, name: str, shape, dtype, device):
    """t must be a contiguous tensor of this shape and type on the device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _size_of(f, desc: MoeDesc, where: str) -> int:
    n = ctypes.c_size_t()
    _check(f(ctypes.byref(desc), ctypes.byref(n)), where)
    return n.value


def few_workspace_size(desc: MoeDesc) -> int:
    return _size_of(library().moe_few_workspace_size, desc, "moe_few_workspace_size")


def mx_workspace_size(desc: MoeDesc) -> int:
    return _size_of(library().moe_mx_workspace_size, desc, "moe_mx_workspace_size")


_served_sizes = {}


def _served_desc(size_of, *key):
    """(descriptor, workspace bytes) of a serving call, kept by the descriptor's values (at most 4096 of them)."""
    got = _served_sizes.get((size_of, key))
    if got is None:
        d = make_desc(*key)
        if len(_served_sizes) >= 4096:
            _served_sizes.clear()
        got = _served_sizes[(size_of, key)] = (ctypes.byref(d), size_of(d))
    return got


def _served(where, size_of, hidden, routing, K, weights, E, I, act, layout, limit, alpha, ws, out):
    """Shared call of the serving forwards.  routing: (topk_ids, topk_weights), or the logits [T,E] when K is given."""
    import torch
    if not hidden.is_cuda or hidden.dim() != 2:
        raise ValueError("hidden must be a device tensor [T, H]")
    if act not in ("swiglu", "clamped") or layout not in ("concat", "interleaved"):
        raise ValueError(f"unknown act {act!r} or layout {layout!r}")
    dev = hidden.device
    T, H = hidden.shape
    dt = "bf16" if hidden.dtype == torch.bfloat16 else ("fp32" if hidden.dtype == torch.float32 else None)
    if dt is None:
        raise ValueError(f"unsupported dtype {hidden.dtype}")
    _need(hidden, "hidden", (T, H), hidden.dtype, dev)
    logits = None
    if K is not None:
        logits = _f32(routing)
        _need(logits, "logits", (T, E), torch.float32, dev)
        ids = torch.empty((T, int(K)), dtype=torch.int32, device=dev)
        w = torch.empty((T, int(K)), dtype=torch.float32, device=dev)
    else:
        ids, w = _ids32(routing[0]), _f32(routing[1])
        if ids.dim() != 2:
            raise ValueError("topk_ids must be [T, K]")
        _need(ids, "topk_ids", (T, ids.shape[1]), torch.int32, dev)
        _need(w, "topk_weights", ids.shape, torch.float32, dev)
    d, nbytes = _served_desc(size_of, T, H, I, E, ids.shape[1], dt, act, layout, float(limit), float(alpha))
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, on {dev}")
    if out is None:
        out = torch.empty_like(hidden)
    else:
        _need(out, "out", (T, H), hidden.dtype, dev)
    f = getattr(library(), where)
    wp = [t.data_ptr() for t in weights]
    if logits is None:
        _launch(dev, where, f, d, hidden.data_ptr(), ids.data_ptr(), w.data_ptr(), *wp, out.data_ptr(), ws.data_ptr(),
                _nbytes(ws))
    else:
        _launch(dev, where, f, d, hidden.data_ptr(), logits.data_ptr(), *wp, out.data_ptr(), ids.data_ptr(), w.data_ptr(),
                ws.data_ptr(), _nbytes(ws))
    return out, ids, w, ws


def _dense_experts(hidden, w_gate_up, w_down):
    """(E, I) of plain expert weights [E,2I,H], [E,H,I] of hidden's type."""
    if w_gate_up.dim() != 3 or w_gate_up.shape[1] % 2:
        raise ValueError("w_gate_up must be [E, 2I, H]")
    E, I = w_gate_up.shape[0], w_gate_up.shape[1] // 2
    H = hidden.shape[-1]
    _need(w_gate_up, "w_gate_up", (E, 2 * I, H), hidden.dtype, hidden.device)
    _need(w_down, "w_down", (E, H, I), hidden.dtype, hidden.device)
    return E, I


def fwd_few(hidden, topk_ids, topk_weights, w_gate_up, w_down, act="swiglu", layout="concat", limit=7.0, alpha=1.702,
            ws=None, out=None):
    """Forward for at most FEW_MAX_TOKENS tokens (decoding); returns (out, ws).  No backward."""
    E, I = _dense_experts(hidden, w_gate_up, w_down)
    out, _, _, ws = _served("moe_fwd_few", few_workspace_size, hidden, (topk_ids, topk_weights), None,
                            (w_gate_up, w_down), E, I, act, layout, limit, alpha, ws, out)
    return out, ws


def fwd_few_logits(hidden, logits, K: int, w_gate_up, w_down, act="swiglu", layout="concat", limit=7.0, alpha=1.702,
                   ws=None, out=None):
    """fwd_few from router logits [T,E]; returns (out, topk_ids, topk_weights, ws)."""
    E, I = _dense_experts(hidden, w_gate_up, w_down)
    return _served("moe_fwd_few_logits", few_workspace_size, hidden, logits, K, (w_gate_up, w_down), E, I, act, layout,
                   limit, alpha, ws, out)


def mx_quantize(w, out=None):
    """Rows of w [..., C] (bf16 or fp32, C a multiple of 32) in 4-bit microscaled floating point; returns
    (codes uint8 [..., C/2], scales uint8 [..., C/32])."""
    import torch
    if not w.is_cuda or w.dim() < 1 or not w.is_contiguous():
        raise ValueError("mx_quantize takes a contiguous device tensor [..., C]")
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported dtype {w.dtype}")
    C = w.shape[-1]
    if C < 1 or C % 32:
        raise ValueError(f"the last dimension must be a multiple of 32, got {C}")
    lead = tuple(w.shape[:-1])
    if out is None:
        out = (torch.empty(lead + (C // 2,), dtype=torch.uint8, device=w.device),
               torch.empty(lead + (C // 32,), dtype=torch.uint8, device=w.device))
        codes, scales = out
    else:
        codes, scales = out
        _need(codes, "codes", lead + (C // 2,), torch.uint8, w.device)
        _need(scales, "scales", lead + (C // 32,), torch.uint8, w.device)
    _launch(w.device, "moe_mx_quantize", library().moe_mx_quantize, _ptr(w),
            MOE_BF16 if w.dtype == torch.bfloat16 else MOE_F32, w.numel() // C, C, _ptr(codes), _ptr(scales))
    return codes, scales


def mx_dequantize(codes, scales, dtype="bf16", out=None):
    """The values that codes [..., C/2] and scales [..., C/32] stand for, as bf16 or fp32 [..., C]: exact,
    but infinite from 2^128 on (scale bytes 253 and 254, which mx_quantize does not write)."""
    import torch
    if not codes.is_cuda or codes.dim() < 1:
        raise ValueError("mx_dequantize takes device tensors")
    lead, C = tuple(codes.shape[:-1]), 2 * codes.shape[-1]
    if C < 1 or C % 32:
        raise ValueError(f"codes must hold whole blocks of 32 columns, got {C} columns")
    _need(codes, "codes", lead + (C // 2,), torch.uint8, codes.device)
    _need(scales, "scales", lead + (C // 32,), torch.uint8, codes.device)
    kind = _dt(dtype)
    tdt = torch.bfloat16 if kind == MOE_BF16 else torch.float32
    if out is None:
        out = torch.empty(lead + (C,), dtype=tdt, device=codes.device)
    else:
        _need(out, "out", lead + (C,), tdt, codes.device)
    _launch(codes.device, "moe_mx_dequantize", library().moe_mx_dequantize, _ptr(codes), _ptr(scales), kind,
            out.numel() // C, C, _ptr(out))
    return out


def _mx_experts(hidden, gate_up, down):
    """(E, I) of expert weights as (codes, scales) pairs."""
    import torch
    (gc, gs), (dc, ds) = gate_up, down
    if gc.dim() != 3 or gc.shape[1] % 2:
        raise ValueError("gate_up codes must be [E, 2I, H/2]")
    E, I = gc.shape[0], gc.shape[1] // 2
    H, dev = hidden.shape[-1], hidden.device
    if hidden.dtype != torch.bfloat16 or H % 32 or I % 32:
        raise ValueError("4-bit experts take bf16 hidden states, H and I multiples of 32")
    _need(gc, "gate_up codes", (E, 2 * I, H // 2), torch.uint8, dev)
    _need(gs, "gate_up scales", (E, 2 * I, H // 32), torch.uint8, dev)
    _need(dc, "down codes", (E, H, I // 2), torch.uint8, dev)
    _need(ds, "down scales", (E, H, I // 32), torch.uint8, dev)
    return E, I


def mx_fwd(hidden, topk_ids, topk_weights, gate_up, down, act="swiglu", layout="concat", limit=7.0, alpha=1.702, ws=None,
           out=None):
    """Forward on 4-bit expert weights: gate_up and down are the (codes, scales) of mx_quantize(w_gate_up [E,2I,H])
    and mx_quantize(w_down [E,H,I]); hidden is bf16.  Returns (out, ws).  No backward."""
    E, I = _mx_experts(hidden, gate_up, down)
    out, _, _, ws = _served("moe_mx_fwd", mx_workspace_size, hidden, (topk_ids, topk_weights), None,
                            (*gate_up, *down), E, I, act, layout, limit, alpha, ws, out)
    return out, ws


def mx_fwd_logits(hidden, logits, K: int, gate_up, down, act="swiglu", layout="concat", limit=7.0, alpha=1.702, ws=None,
                  out=None):
    """mx_fwd from router logits [T,E]; returns (out, topk_ids, topk_weights, ws)."""
    E, I = _mx_experts(hidden, gate_up, down)
    return _served("moe_mx_fwd_logits", mx_workspace_size, hidden, logits, K, (*gate_up, *down), E, I, act, layout, limit,
                   alpha, ws, out)


# ---------------------------------------------------------------- around the routed experts
def _kind(t, name: str) -> int:
    """MOE_BF16 or MOE_F32 of a tensor."""
    import torch
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return MOE_BF16 if t.dtype == torch.bfloat16 else MOE_F32


def _workspace(ws, nbytes: int, device):
    import torch
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, on {device}")
    return ws


def _result(t, name: str, shape, dtype, device):
    """The given output tensor, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, shape, dtype, device)
    return t


_native = None


def _block():
    """The native half of the binding of these operators (csrc/binding.cpp): checks, outputs and the call."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries, which the module is linked to)
        library()
        from . import _block as native
        native.init(_check, _raw_stream)
        _native = native
    return _native


_ACTS, _LAYOUTS = {"swiglu": MOE_SWIGLU, "clamped": MOE_CLAMPED_GLU}, {"concat": MOE_GU_CONCAT, "interleaved": MOE_GU_INTERLEAVED}


def _codes(act, layout):
    try:
        return _ACTS[act], _LAYOUTS[layout]
    except KeyError:
        raise ValueError(f"unknown act {act!r} or layout {layout!r}") from None


def ffn_workspace_size(desc: MoeDesc) -> Tuple[int, int, int]:
    """(forward, backward, saved) bytes of the feed-forward block; desc with E = K = 1."""
    f, b, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().moe_ffn_workspace_size(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b), ctypes.byref(s)),
           "moe_ffn_workspace_size")
    return f.value, b.value, s.value


def ffn_fwd(x, w_gate_up, w_down, gate=None, add=None, act="swiglu", layout="concat", limit=7.0, alpha=1.702, save=False,
            ws=None, out=None, saved=None):
    """Gated feed-forward block of every token (a shared expert, a dense layer):
    add + sigmoid(gate) Wd phi(Wgu x) for x [T,H], w_gate_up [2I,H], w_down [H,I], gate fp32 [T], add [T,H].
    save: keep the gate and up values for ffn_bwd, in `saved` if given (which is refused without save).
    Returns (out, saved-or-None, ws); `out` may be `add`."""
    return (_native or _block()).ffn_fwd(x, w_gate_up, w_down, gate, *_codes(act, layout), limit, alpha, add, save, ws, out,
                                         saved)


def ffn_bwd(x, w_gate_up, w_down, d_out, saved=None, gate=None, act="swiglu", layout="concat", limit=7.0, alpha=1.702,
            ws=None, grads=None, grad_dtype=None):
    """Backward pass of ffn_fwd; returns (d_x, d_gate-or-None, d_w_gate_up, d_w_down, ws).  The gradient of `add` is
    d_out.  grad_dtype: "bf16" or "fp32" storage of the weight gradients (default: the activation dtype)."""
    return (_native or _block()).ffn_bwd(x, w_gate_up, w_down, gate, *_codes(act, layout), limit, alpha, d_out, saved,
                                         -1 if grad_dtype is None else _dt(grad_dtype), ws, *(grads or (None,) * 4))


GATE_NONE, GATE_ROW, GATE_COLUMN, GATE_FULL = range(4)   # moe_gate_t


def norm_workspace_size(desc: NormDesc) -> int:
    return _size_of(library().moe_norm_workspace_size, desc, "moe_norm_workspace_size")


def norm_fwd(x, w, eps=1e-5, out=None):
    """w x / rms(x) of each row of x [T,H]; w [H] of x's type."""
    return (_native or _block()).norm_fwd(x, w, eps, out)


def norm_bwd(x, w, d_y, d_add=None, eps=1e-5, ws=None, grads=None):
    """Backward pass of norm_fwd; d_add [T,H], the gradient that reaches x beside the norm, is added to d_x.
    Returns (d_x, d_w fp32 [H], ws); d_x may be d_add."""
    return (_native or _block()).norm_bwd(x, w, d_y, d_add, eps, ws, *(grads or (None, None)))


def residual_fwd(x, h, w_post=None, gate=None, scale=1.0, w_next=None, eps=1e-5, x_new=None, y=None):
    """The step after a block: x_new = x + scale gate n with n = w_post h / rms(h) (h without w_post), and the next
    block's norm y = w_next x_new / rms(x_new) (None without w_next).  x, h [T,H]; w_post, w_next [H]; gate [T,1] (one
    for each token), [H] (one for each channel) or [T,H]; all of one type.  A gate of one dimension is always the
    channels', also where T = H: ffn_fwd's logits [T] go in as [T,1].  Returns (x_new, y); x_new may be x."""
    return (_native or _block()).residual_fwd(x, h, w_post, gate, scale, w_next, eps, x_new, y)


class ResidualGrads(NamedTuple):
    """Gradients of residual_fwd; None for what it did not have.  d_w_post, d_w_next and the gradients of gates [T,1] and
    [H] are fp32 sums, the others have x's type."""
    d_x: object
    d_h: object
    d_gate: object
    d_w_post: object
    d_w_next: object
    ws: object


def residual_bwd(x_new, h, d_x_new=None, d_y=None, w_post=None, gate=None, scale=1.0, w_next=None, eps=1e-5, ws=None,
                 grads: Optional[ResidualGrads] = None) -> ResidualGrads:
    """Backward pass of residual_fwd, given its x_new and the gradients of x_new (None: zero) and, with w_next, of y.
    grads: where to put the results (its ws is not used)."""
    return ResidualGrads._make((_native or _block()).residual_bwd(x_new, h, d_x_new, d_y, w_post, gate, scale, w_next, eps, ws,
                                                                  *(grads[:5] if grads else (None,) * 5)))


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)   # the usual coefficients


def ortho_workspace_size(desc: OrthoDesc) -> int:
    return _size_of(library().moe_ortho_workspace_size, desc, "moe_ortho_workspace_size")


def _ortho(g, name, out_dtype, steps, coef, eps):
    if not g.is_cuda or g.dim() < 2:
        raise ValueError(f"{name} must be a device tensor [.., M, N]")
    _need(g, name, g.shape, g.dtype, g.device)
    M, N = g.shape[-2:]
    E = 1
    for n in g.shape[:-2]:
        E *= n
    a, b, c = (float(v) for v in coef)
    d = OrthoDesc(E, M, N, _kind(g, name), out_dtype, int(steps), a, b, c, float(eps))
    return d, ortho_workspace_size(d)


def orthogonalize(g, steps=5, coef=NEWTON_SCHULZ, eps=1e-7, dtype="bf16", ws=None, out=None):
    """Newton-Schulz orthogonalisation of each matrix of g [.., M, N] (bf16 or fp32): X = g / (|g| + eps), then `steps`
    times X <- a X + b (X X^T) X + c (X X^T)^2 X with coef = (a, b, c).  Returns (X of `dtype`, ws)."""
    import torch
    kind = _dt(dtype)
    d, nbytes = _ortho(g, "g", kind, steps, coef, eps)
    out = _result(out, "out", g.shape, torch.bfloat16 if kind == MOE_BF16 else torch.float32, g.device)
    ws = _workspace(ws, nbytes, g.device)
    _launch(g.device, "moe_orthogonalize", library().moe_orthogonalize, ctypes.byref(d), _ptr(g), _ptr(out), _ptr(ws),
            _nbytes(ws))
    return out, ws


def muon_step(w, g, m, lr, momentum=0.95, nesterov=True, decay=0.0, steps=5, coef=NEWTON_SCHULZ, eps=1e-7, ws=None, out=None):
    """One optimiser step with orthogonalised updates, for each matrix of w [.., M, N] (bf16 or fp32), its gradient g
    (bf16 or fp32) and its momentum m (fp32):  m <- momentum m + g,  u = g + momentum m (nesterov) or m,
    w <- (1 - decay) w - lr orthogonalize(u).  In place, or into out = (w, m).  Returns (w, m, ws)."""
    import torch
    d, nbytes = _ortho(g, "g", _kind(w, "w"), steps, coef, eps)
    _need(w, "w", g.shape, w.dtype, g.device)
    _need(m, "m", g.shape, torch.float32, g.device)
    w_out, m_out = out if out is not None else (w, m)
    if out is not None:
        _need(w_out, "out[0]", w.shape, w.dtype, w.device)
        _need(m_out, "out[1]", m.shape, m.dtype, m.device)
    ws = _workspace(ws, nbytes, g.device)
    opt = Muon(float(lr), float(momentum), float(decay), 1 if nesterov else 0)
    _launch(g.device, "moe_muon_step", library().moe_muon_step, ctypes.byref(d), ctypes.byref(opt), _ptr(w), _ptr(g), _ptr(m),
            _ptr(w_out), _ptr(m_out), _ptr(ws), _nbytes(ws))
    return w_out, m_out, ws


def check_device_status(ws) -> int:
    """Synchronises the current stream of ws's device; returns the status code of the last routing in ws."""
    return _on_device(ws.device, library().moe_check_device_status, _ptr(ws))


def timing_enable(max_launches: int = 4096):
    _check(library().moe_timing_enable(int(max_launches)), "moe_timing_enable")


def timing_disable():
    _check(library().moe_timing_disable(), "moe_timing_disable")


def timing_read():
    """{kernel name: (launches, total_ms)} of the launches timed since the last read."""
    n = ctypes.c_int32()
    buf = (KernelTime * 64)()
    _check(library().moe_timing_read(buf, 64, ctypes.byref(n)), "moe_timing_read")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(min(n.value, 64))}
