// C ABI of the operators around the routed experts: argument checks, workspace
// layouts and launches of the feed-forward block, the norms and the
// orthogonalisation.
#include <math.h>

#include <initializer_list>

#include "../../include/moe.h"
#include "ffn.h"
#include "norm.h"
#include "ortho.h"

using namespace moe;

namespace {

constexpr int64_t kMaxSide = int64_t(1) << 20;   // 32-bit offsets within a tile's rows

// Tiles of the largest kind that a product of m x n results may run on, 256 x 256 unless told.
inline int64_t tiles(int64_t m, int64_t n, int64_t side = 256) { return ((m + side - 1) / side) * ((n + side - 1) / side); }

inline size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }

// Every pointer present (where `need`) and 16-byte aligned.
bool aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if ((uintptr_t)p & 15u) return false;
  return true;
}
bool present(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return false;
  return true;
}
bool dtype_ok(int32_t d) { return d == MOE_BF16 || d == MOE_F32; }

moe_status_t launched(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  (void)hipGetLastError();
  return MOE_ERR_HIP;
}

// ------------------------------------------------------------ feed-forward block
struct FfnLayout {
  size_t a, f_end;                          // forward
  size_t z, dz, aw, part, b_end;            // backward
  size_t ids, w, f_route, dw, b_route;      // fp32: the block as one expert; offsets of moe_fwd's and moe_bwd's workspaces
  size_t saved;
  bool one_expert;                          // fp32
};

moe_status_t ffn_check(const moe_desc_t* d, FfnLayout* L) {
  size_t fws = 0, bws = 0, saved = 0;
  const moe_status_t st = moe_workspace_size(d, &fws, &bws, &saved);
  if (st != MOE_OK) return st;
  if (d->E != 1 || d->K != 1) return MOE_ERR_INVALID_ARG;
  if (d->H > kMaxSide || d->I > kMaxSide || d->H * d->I > (int64_t(1) << 28)) return MOE_ERR_UNSUPPORTED;
  if (d->T > (int64_t(1) << 30) || tiles(d->T, 2 * d->I > d->H ? 2 * d->I : d->H) > MAX_TILES) return MOE_ERR_UNSUPPORTED;
  const size_t esz = d->dtype == MOE_BF16 ? 2 : 4, T = (size_t)d->T, I = (size_t)d->I;
  *L = {};
  L->one_expert = d->dtype == MOE_F32;
  L->a = 0;
  // fp32: a of the few-token kernels, or the products' result before add
  L->f_end = align_up(T * (size_t)(L->one_expert && d->H > d->I ? d->H : d->I) * esz);
  if (L->one_expert) {
    L->ids = L->f_end;
    L->w = L->ids + align_up(T * 4);
    L->f_route = L->w + align_up(T * 4);
    L->f_end = L->f_route + fws;
    L->dw = L->f_route;
    L->b_route = L->dw + align_up(T * 4);
    L->b_end = L->b_route + bws;
    L->saved = saved;
  } else {
    L->saved = ffn_z_floats(d->T, d->I) * sizeof(float);
    L->z = 0;
    L->dz = align_up(L->saved);
    L->aw = L->dz + align_up(T * 2 * I * 2);
    L->part = L->aw + align_up(T * I * 2);
    L->b_end = L->part + align_up(T * (size_t)ffn_parts(d->I) * sizeof(float));
  }
  if (L->f_end == 0) L->f_end = 256;
  if (L->b_end == 0) L->b_end = 256;
  return MOE_OK;
}

FfnArgs ffn_args(const moe_desc_t* d, const void* x, const void* w_gate_up, const void* w_down, const float* gate) {
  FfnArgs p = {};
  const size_t esz = d->dtype == MOE_BF16 ? 2 : 4;
  const bool inter = d->gu_layout == MOE_GU_INTERLEAVED;
  p.x = x;
  p.gu = p.gu_g = w_gate_up;
  p.gu_u = (const char*)w_gate_up + (inter ? 1 : d->I) * d->H * esz;
  p.gu_rs = inter ? 2 * d->H : d->H;
  p.wd = w_down;
  p.gate = gate;
  p.T = (int)d->T; p.H = (int)d->H; p.I = (int)d->I;
  p.act = d->act == MOE_CLAMPED_GLU; p.layout = inter; p.grad_f32 = d->grad_dtype == MOE_F32;
  p.limit = d->clamp_limit; p.alpha = d->glu_alpha;
  return p;
}

#define TRY(x)                                \
  do {                                        \
    const moe_status_t st_ = (x);             \
    if (st_ != MOE_OK) return st_;            \
  } while (0)

// ------------------------------------------------------------ norms
moe_status_t norm_check(const moe_norm_desc_t* d) {
  if (!d || d->T < 0 || d->H < 1 || !dtype_ok(d->dtype) || d->gate_kind < MOE_GATE_NONE || d->gate_kind > MOE_GATE_FULL ||
      !(d->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (d->H % 8 != 0 || d->H > NORM_MAX_H || d->T > NORM_MAX_T) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
size_t norm_ws(const moe_norm_desc_t* d) {
  const int64_t rows = d->T < 1 ? 1 : d->T < NORM_GRID ? d->T : NORM_GRID;
  return (size_t)rows * 3 * d->H * sizeof(float);
}
NormArgs norm_args(const moe_norm_desc_t* d) {
  NormArgs p = {};
  p.T = (int)d->T; p.H = (int)d->H; p.gate_kind = d->gate_kind; p.scale = d->scale; p.eps = d->eps;
  return p;
}

// ------------------------------------------------------------ orthogonalisation
struct OrthoLayout {
  size_t part, x0, x1, l0, l1, p, q, pd, qd, end;
};

// Largest sizes of the iterates' singular values s, and of b x + c x^2 and a + b
// x + c x^2 over their squares x, must leave the fp16 iterates room.  Singular
// values start at most 1; the largest |s (a + b x + c x^2)| over the present
// interval is the next one's end.  Extremes of a polynomial over [0, top]: at
// the end or where the derivative, here at most quadratic in x, is zero.
bool coefficients_ok(const moe_ortho_desc_t* d) {
  const double a = d->a, b = d->b, c = d->c;
  const double disc = 9 * b * b - 20 * a * c, root = disc >= 0 ? sqrt(disc) : 0;
  const double places[] = {(-3 * b + root) / (10 * c), (-3 * b - root) / (10 * c), -a / (3 * b), -b / (2 * c)};
  double top = 1.001;
  for (int i = 0; i < d->steps; ++i) {
    const double end = top * top;
    double next = 0, q = 0;
    const auto at = [&](double x) {
      const double r = x * (b + x * c);
      next = fmax(next, sqrt(x) * fabs(a + r));
      q = fmax(q, fmax(fabs(r), fabs(a + r)));
    };
    at(0);
    at(end);
    for (double x : places)
      if (x > 0 && x < end) at(x);   // not where a coefficient is zero (infinite or NaN)
    if (!isfinite(a) || !isfinite(b) || !isfinite(c) || !(top <= 3.0) || !(q <= 14.6)) return false;
    top = 1.001 * next;
  }
  return true;
}

moe_status_t ortho_check(const moe_ortho_desc_t* d, OrthoLayout* L) {
  if (!d || d->E < 0 || d->M < 1 || d->N < 1 || !dtype_ok(d->dtype) || !dtype_ok(d->out_dtype) || !(d->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (d->M % 8 != 0 || d->N % 8 != 0 || d->M > kMaxSide || d->N > kMaxSide || d->E > 65535 || d->steps < 1 || d->steps > 64)
    return MOE_ERR_UNSUPPORTED;
  if (d->E * tiles(d->M, d->N, d->M < ORTHO_NARROW || d->N < ORTHO_NARROW ? 128 : 256) > MAX_TILES) return MOE_ERR_UNSUPPORTED;
  if (!coefficients_ok(d)) return MOE_ERR_UNSUPPORTED;
  const size_t S = (size_t)(d->M < d->N ? d->M : d->N), E = (size_t)d->E;
  L->part = 0;
  L->x0 = align_up(E * ORTHO_PARTS * sizeof(double));
  const size_t x = align_up(E * d->M * d->N * 2);
  L->x1 = L->x0 + x;
  L->l0 = L->x1 + x;
  L->l1 = L->l0 + x;
  L->p = L->l1 + x;
  L->q = L->p + align_up(E * S * S * 2);
  L->pd = L->q + align_up(E * S * S * 2);
  L->qd = L->pd + align_up(E * S * sizeof(float));
  L->end = L->qd + align_up(E * S * sizeof(float));
  return MOE_OK;
}

OrthoArgs ortho_args(const moe_ortho_desc_t* d, const OrthoLayout& L, void* ws) {
  OrthoArgs p = {};
  char* b = (char*)ws;
  p.part = (double*)(b + L.part);
  p.x0 = b + L.x0; p.x1 = b + L.x1; p.l0 = b + L.l0; p.l1 = b + L.l1; p.p = b + L.p; p.q = b + L.q;
  p.pd = (float*)(b + L.pd); p.qd = (float*)(b + L.qd);
  p.E = (int)d->E; p.M = (int)d->M; p.N = (int)d->N; p.S = (int)(d->M < d->N ? d->M : d->N);
  p.steps = d->steps; p.a = d->a; p.b = d->b; p.c = d->c; p.eps = d->eps;
  p.g_f32 = d->dtype == MOE_F32; p.out_f32 = d->out_dtype == MOE_F32;
  return p;
}

}  // namespace

extern "C" {

moe_status_t moe_ffn_workspace_size(const moe_desc_t* desc, size_t* fwd_ws, size_t* bwd_ws, size_t* saved_bytes) {
  FfnLayout L;
  TRY(ffn_check(desc, &L));
  if (fwd_ws) *fwd_ws = L.f_end;
  if (bwd_ws) *bwd_ws = L.b_end;
  if (saved_bytes) *saved_bytes = L.saved;
  return MOE_OK;
}

moe_status_t moe_ffn_fwd(const moe_desc_t* desc, const void* x, const void* w_gate_up, const void* w_down,
                         const float* gate, const void* add, void* out, void* saved, size_t saved_bytes, void* ws,
                         size_t ws_bytes, hipStream_t stream) {
  FfnLayout L;
  TRY(ffn_check(desc, &L));
  if (!present({w_gate_up, w_down, ws}) || (desc->T > 0 && !present({x, out}))) return MOE_ERR_INVALID_ARG;
  if (!aligned({x, w_gate_up, w_down, gate, add, out, saved, ws})) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.f_end || (saved && saved_bytes < L.saved)) return MOE_ERR_WORKSPACE;
  if (desc->T == 0) return MOE_OK;
  FfnArgs p = ffn_args(desc, x, w_gate_up, w_down, gate);
  char* b = (char*)ws;
  p.a = b + L.a;
  p.add = add;
  p.out = out;
  if (desc->T <= (L.one_expert ? FFN_FEW_F32 : FFN_FEW_BF16) && !saved)
    return launched(launch_ffn_few(L.one_expert ? 1 : 0, p, stream));
  if (!L.one_expert) {
    p.z = (float*)saved;
    TRY(launched(launch_ffn_gate_up(p, stream)));
    return launched(launch_ffn_down(p, stream));
  }
  // fp32: the products of one expert that takes every token
  int32_t* ids = (int32_t*)(b + L.ids);
  float* w = (float*)(b + L.w);
  void* y = add ? b + L.a : out;   // out may be add
  TRY(launched(launch_ffn_one_expert(gate, p.T, ids, w, stream)));
  TRY(moe_fwd(desc, x, ids, w, w_gate_up, w_down, y, saved, saved_bytes, b + L.f_route, ws_bytes - L.f_route, stream));
  return add ? launched(launch_ffn_add((const float*)add, (const float*)y, (long)(desc->T * desc->H), (float*)out, stream))
             : MOE_OK;
}

moe_status_t moe_ffn_bwd(const moe_desc_t* desc, const void* x, const void* w_gate_up, const void* w_down,
                         const float* gate, const void* d_out, const void* saved, size_t saved_bytes, void* d_x,
                         float* d_gate, void* d_w_gate_up, void* d_w_down, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  FfnLayout L;
  TRY(ffn_check(desc, &L));
  if (!present({w_gate_up, w_down, d_w_gate_up, d_w_down, ws})) return MOE_ERR_INVALID_ARG;
  if (desc->T > 0 && (!present({x, d_out, d_x}) || (gate && !d_gate))) return MOE_ERR_INVALID_ARG;
  if (!aligned({x, w_gate_up, w_down, gate, d_out, saved, d_x, d_gate, d_w_gate_up, d_w_down, ws})) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.b_end || (saved && saved_bytes < L.saved)) return MOE_ERR_WORKSPACE;
  const size_t wbytes = (size_t)desc->H * desc->I * (desc->grad_dtype == MOE_F32 ? 4 : 2);
  if (desc->T == 0) {
    TRY(launched(launch_fill_zero(d_w_gate_up, 2 * wbytes, stream)));
    return launched(launch_fill_zero(d_w_down, wbytes, stream));
  }
  char* b = (char*)ws;
  if (L.one_expert) {
    int32_t* ids = (int32_t*)(b + L.ids);
    float *w = (float*)(b + L.w), *dw = (float*)(b + L.dw);
    TRY(launched(launch_ffn_one_expert(gate, (int)desc->T, ids, w, stream)));
    TRY(moe_bwd(desc, x, ids, w, w_gate_up, w_down, d_out, saved, saved_bytes, d_x, dw, d_w_gate_up, d_w_down,
                b + L.b_route, ws_bytes - L.b_route, stream));
    return gate ? launched(launch_ffn_dgate(gate, dw, (int)desc->T, d_gate, stream)) : MOE_OK;
  }
  FfnArgs p = ffn_args(desc, x, w_gate_up, w_down, gate);
  p.dout = d_out;
  p.dz = b + L.dz; p.aw = b + L.aw; p.part = (float*)(b + L.part);
  p.dx = d_x;
  p.dgate = gate ? d_gate : nullptr;
  p.dgu = d_w_gate_up; p.dwd = d_w_down;
  p.z = (float*)saved;
  if (!saved) {
    p.z = (float*)(b + L.z);
    TRY(launched(launch_ffn_gate_up(p, stream)));
  }
  TRY(launched(launch_ffn_down_dgrad(p, stream)));
  TRY(launched(launch_ffn_gate_up_dgrad(p, stream)));
  return launched(launch_ffn_wgrads(p, stream));
}

moe_status_t moe_norm_workspace_size(const moe_norm_desc_t* desc, size_t* bwd_ws) {
  TRY(norm_check(desc));
  if (!bwd_ws) return MOE_ERR_INVALID_ARG;
  *bwd_ws = norm_ws(desc);
  return MOE_OK;
}

moe_status_t moe_norm_fwd(const moe_norm_desc_t* desc, const void* x, const void* w, void* y, hipStream_t stream) {
  TRY(norm_check(desc));
  if (desc->gate_kind != MOE_GATE_NONE || !w || (desc->T > 0 && !present({x, y})) || !aligned({x, w, y}))
    return MOE_ERR_INVALID_ARG;
  if (desc->T == 0) return MOE_OK;
  NormArgs p = norm_args(desc);
  p.x = x; p.w_next = w; p.y = y;
  return launched(launch_norm_fwd(desc->dtype, p, stream));
}

moe_status_t moe_norm_bwd(const moe_norm_desc_t* desc, const void* x, const void* w, const void* d_y, const void* d_add,
                          void* d_x, float* d_w, void* ws, size_t ws_bytes, hipStream_t stream) {
  TRY(norm_check(desc));
  if (desc->gate_kind != MOE_GATE_NONE || !present({w, d_w, ws}) || (desc->T > 0 && !present({x, d_y, d_x})) ||
      !aligned({x, w, d_y, d_add, d_x, d_w, ws}))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < norm_ws(desc)) return MOE_ERR_WORKSPACE;
  NormArgs p = norm_args(desc);
  p.x = x; p.w_next = w; p.d_y = d_y; p.d_new = d_add; p.d_x = d_x; p.d_w_next = d_w; p.part = (float*)ws;
  return launched(launch_norm_bwd(desc->dtype, p, stream));
}

moe_status_t moe_residual_fwd(const moe_norm_desc_t* desc, const void* x, const void* h, const void* w_post,
                              const void* gate, const void* w_next, void* x_new, void* y, hipStream_t stream) {
  TRY(norm_check(desc));
  if ((desc->gate_kind == MOE_GATE_NONE) != !gate) return MOE_ERR_INVALID_ARG;
  if (desc->T > 0 && (!present({x, h, x_new}) || (w_next && !y))) return MOE_ERR_INVALID_ARG;
  if (!aligned({x, h, w_post, gate, w_next, x_new, y})) return MOE_ERR_INVALID_ARG;
  if (desc->T == 0) return MOE_OK;
  NormArgs p = norm_args(desc);
  p.x = x; p.h = h; p.w_post = w_post; p.gate = gate; p.w_next = w_next; p.x_new = x_new; p.y = y;
  return launched(launch_norm_fwd(desc->dtype, p, stream));
}

moe_status_t moe_residual_bwd(const moe_norm_desc_t* desc, const void* x_new, const void* h, const void* w_post,
                              const void* gate, const void* w_next, const void* d_x_new, const void* d_y, void* d_x,
                              void* d_h, void* d_gate, float* d_w_post, float* d_w_next, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  TRY(norm_check(desc));
  if ((desc->gate_kind == MOE_GATE_NONE) != !gate) return MOE_ERR_INVALID_ARG;
  if (!ws || (gate && !d_gate) || (w_post && !d_w_post) || (w_next && !d_w_next)) return MOE_ERR_INVALID_ARG;
  if (desc->T > 0 && (!present({h, d_x, d_h}) || (w_next && !present({x_new, d_y})))) return MOE_ERR_INVALID_ARG;
  if (!aligned({x_new, h, w_post, gate, w_next, d_x_new, d_y, d_x, d_h, d_gate, d_w_post, d_w_next, ws}))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < norm_ws(desc)) return MOE_ERR_WORKSPACE;
  NormArgs p = norm_args(desc);
  p.x = x_new; p.h = h; p.w_post = w_post; p.gate = gate; p.w_next = w_next; p.d_new = d_x_new; p.d_y = d_y;
  p.d_x = d_x; p.d_h = d_h; p.d_gate = d_gate; p.d_w_post = d_w_post; p.d_w_next = d_w_next; p.part = (float*)ws;
  if (desc->T == 0) p.h = ws;   // only its presence counts: the sums over no rows
  return launched(launch_norm_bwd(desc->dtype, p, stream));
}

moe_status_t moe_ortho_workspace_size(const moe_ortho_desc_t* desc, size_t* ws_bytes) {
  OrthoLayout L;
  TRY(ortho_check(desc, &L));
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  *ws_bytes = L.end;
  return MOE_OK;
}

moe_status_t moe_orthogonalize(const moe_ortho_desc_t* desc, const void* g, void* out, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  OrthoLayout L;
  TRY(ortho_check(desc, &L));
  if (!aligned({g, out, ws})) return MOE_ERR_INVALID_ARG;
  if (desc->E == 0) return MOE_OK;
  if (!present({g, out, ws})) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.end) return MOE_ERR_WORKSPACE;
  OrthoArgs p = ortho_args(desc, L, ws);
  p.g = g;
  p.out = out;
  return launched(launch_ortho(p, stream));
}

moe_status_t moe_muon_step(const moe_ortho_desc_t* desc, const moe_muon_t* opt, const void* w, const void* g,
                           const float* m, void* w_out, float* m_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  OrthoLayout L;
  TRY(ortho_check(desc, &L));
  if (!opt || (opt->nesterov != 0 && opt->nesterov != 1) || !aligned({w, g, m, w_out, m_out, ws})) return MOE_ERR_INVALID_ARG;
  if (desc->E == 0) return MOE_OK;
  if (!present({w, g, m, w_out, m_out, ws})) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.end) return MOE_ERR_WORKSPACE;
  OrthoArgs p = ortho_args(desc, L, ws);
  p.g = g; p.m = m; p.m_out = m_out; p.w = w; p.out = w_out;
  p.momentum = opt->momentum; p.nesterov = opt->nesterov; p.lr = opt->lr; p.keep = 1.f - opt->decay;
  return launched(launch_ortho(p, stream));
}

}  // extern "C"
