// The norms around a block and the step between them, each one pass over its
// rows:
//
//   n = w_post h / rms(h)  (n = h without w_post),  x' = x + scale gate n,
//   y = w_next x' / rms(x'),   rms(v)^2 = mean(v^2) + eps
//
// and, given the gradients of x' and y, with v^ = v / rms(v):
//
//   norm's gradient   N(v, w, g) = (w g - v^ mean(w g v^)) / rms(v)
//   t = d_x' + N(x', w_next, d_y),    d_x = t,       d_w_next = sum d_y x'^
//   d_n = scale gate t,               d_h = N(h, w_post, d_n),
//   d_w_post = sum d_n h^,            d_gate = scale t n, summed to gate's shape
//
// The norm before a block is the same without h (t = d_add + ..).  Bound by HBM:
// a row is read once, kept in registers as it came (16 elements a thread, a
// workgroup a row) and its sums meet through LDS, twice a row; workgroups of a
// backward pass stay and add the weights' gradients of their rows up in
// registers, the next row's loads issued before the present one's sums.  All
// arithmetic is fp32; nothing is saved between the passes, as the rows that the
// statistics need are read anyway.  The step after a block, bf16, 32768 rows of
// 4096: forward 185 us (5.8 TB/s), backward 291 us (5.6 TB/s), reduction 5; the
// norm before one, 4096 rows of 2880: 8.8, 18.7 and 4.0 us.  Workgroups that stay
// were slower forward (198 to 209 us), two rows ahead no faster backward.  Short
// rows share backward workgroups (32768 rows of 512, column gate, 137 -> 61 us, of
// 1048 176 -> 119).
#include "gemm_common.h"
#include "norm.h"

namespace moe {
namespace {

enum { GATE_NONE = 0, GATE_ROW = 1, GATE_COLUMN = 2, GATE_FULL = 3 };
constexpr int V = 2;   // groups of 8 elements a thread

// 8 consecutive elements as they lie in memory.  Stores are non-temporal: rows
// are written once and L2 keeps what is read (the backward pass of 32768 rows of
// 4096 308 -> 291 us, of 4096 rows of 2880 20.9 -> 19.6).
typedef uint32_t u32x4_nt __attribute__((ext_vector_type(4)));
typedef float f32x4_nt __attribute__((ext_vector_type(4)));
template <typename T> struct Raw;
template <> struct Raw<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *(const uint4*)p; }
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* f) {
    const u32x4_nt v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    __builtin_nontemporal_store(v, (u32x4_nt*)p);
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) { a = *(const float4*)p; b = *(const float4*)(p + 4); }
  __device__ __forceinline__ void clear() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    __builtin_nontemporal_store(f32x4_nt{f[0], f[1], f[2], f[3]}, (f32x4_nt*)p);
    __builtin_nontemporal_store(f32x4_nt{f[4], f[5], f[6], f[7]}, (f32x4_nt*)(p + 4));
  }
};
__device__ __forceinline__ float one_value(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
__device__ __forceinline__ float one_value(const float* p) { return *p; }

// Sums of N values over the threads of a row (blockDim.x, whole waves; MANY: a
// workgroup holds blockDim.y rows), in each of them; wave sums meet in
// red[waves][4].  Alternate calls use different halves of red, so one barrier a
// call is enough: a half is written again only after the next call's barrier,
// which every thread reaches after its reads of this one.
template <bool MANY = false, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int& half) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d);
  if (nw == 1) return;
  float* r = red + half * 64 + (MANY ? threadIdx.y * nw * 4 : 0);
  half ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[wave * 4 + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += r[w * 4 + i];
}

// A thread's columns: 8 from each of V groups, threads side by side.
__device__ __forceinline__ int column(int j) { return (j * blockDim.x + threadIdx.x) * 8; }

template <typename T>
__device__ __forceinline__ void load_row(Raw<T> (&r)[V], const T* p, size_t row, int H) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = column(j);
    if (p && c < H) r[j].load(p + row * H + c);
    else r[j].clear();
  }
}

// ------------------------------------------------------------------ forward
template <typename T, bool H_IN>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormArgs p) {
  __shared__ float red[128];
  int half = 0;
  const size_t row = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= (size_t)p.T) return;
  const int H = p.H;
  Raw<T> x[V], h[V], wp[V], wn[V], gt[V];
  load_row(x, (const T*)p.x, row, H);
  if (H_IN) {
    load_row(h, (const T*)p.h, row, H);
    load_row(wp, (const T*)p.w_post, 0, H);
    if (p.gate_kind >= GATE_COLUMN) load_row(gt, (const T*)p.gate, p.gate_kind == GATE_FULL ? row : 0, H);
  }
  load_row(wn, (const T*)p.w_next, 0, H);
  float xv[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) x[j].get(xv[j]);
  if (H_IN) {
    float f = p.scale;
    if (p.gate_kind == GATE_ROW) f *= one_value((const T*)p.gate + row);
    float r = 1.f;
    if (p.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v[8];
        h[j].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e] * v[e];
      }
      block_sum(s, red, half);
      r = rsqrtf(s[0] / H + p.eps);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8], w[8], g[8];
      h[j].get(v);
      wp[j].get(w);
      if (p.gate_kind >= GATE_COLUMN) gt[j].get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float n = p.w_post ? v[e] * r * w[e] : v[e];
        if (p.gate_kind >= GATE_COLUMN) n *= g[e];
        xv[j][e] += f * n;
      }
      const int c = column(j);
      if (c < H) Raw<T>::store((T*)p.x_new + row * H + c, xv[j]);
    }
    if (!p.w_next) return;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += xv[j][e] * xv[j][e];
  block_sum(s, red, half);
  const float r = rsqrtf(s[0] / H + p.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float w[8];
    wn[j].get(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) xv[j][e] *= r * w[e];
    const int c = column(j);
    if (c < H) Raw<T>::store((T*)p.y + row * H + c, xv[j]);
  }
}

// ------------------------------------------------------------------ backward
// kind: the gate's; MAXT: most threads.  With more than 512 the registers do not
// hold a second row, so the next one is loaded after the present one.  With
// NORM_SHORT a workgroup works on blockDim.y rows at a time (all of them reach
// every barrier) and adds their sums up at its end: short rows would leave the
// card to 512 workgroups of one or two waves each.  Two waves a SIMD have to fit
// (launch bounds of 512).
template <typename T, bool H_IN, int kind, int MAXT>
__global__ __launch_bounds__(MAXT < 512 ? 512 : MAXT) void norm_bwd_kernel(NormArgs p) {
  constexpr bool AHEAD = MAXT <= 512, MANY = MAXT == NORM_SHORT;
  __shared__ float red[128];
  int half = 0;
  const int H = p.H;
  const bool next = p.w_next != nullptr, post = H_IN && p.w_post != nullptr;
  Raw<T> wn[V], wp[V], gc[V];
  load_row(wn, (const T*)p.w_next, 0, H);
  if (H_IN) {
    load_row(wp, (const T*)p.w_post, 0, H);
    load_row(gc, kind == GATE_COLUMN ? (const T*)p.gate : nullptr, 0, H);
  }
  float an[V][8], ap[V][8], ag[V][8];   // sums over this workgroup's rows
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) an[j][e] = ap[j][e] = ag[j][e] = 0.f;

  struct Row { Raw<T> x[V], dy[V], dn[V], h[V]; } c, r;
  const auto fetch = [&](size_t row, Row& r) {
    load_row(r.x, next ? (const T*)p.x : nullptr, row, H);
    load_row(r.dy, next ? (const T*)p.d_y : nullptr, row, H);
    load_row(r.dn, (const T*)p.d_new, row, H);
    if (H_IN) load_row(r.h, (const T*)p.h, row, H);
  };
  const int R = MANY ? blockDim.y : 1, group = MANY ? threadIdx.y : 0, stride = gridDim.x * R;
  const auto row_of = [&](int first) { return MANY ? min(first + group, p.T - 1) : first; };
  if (AHEAD) fetch(row_of(blockIdx.x * R), r);
  for (int first = blockIdx.x * R; first < p.T; first += stride) {
    const bool live = !MANY || first + group < p.T;   // past the last row: the last one again, and nothing comes of it
    const int row = row_of(first);
    if (AHEAD) c = r;
    else fetch(row, c);
    float f = p.scale;
    if (kind == GATE_ROW) f *= one_value((const T*)p.gate + row);
    Raw<T> gf[V];
    if (kind == GATE_FULL) load_row(gf, (const T*)p.gate, row, H);
    if (AHEAD && first + stride < p.T) fetch(row_of(first + stride), r);
    float s[3] = {0.f, 0.f, 0.f};   // x'^2, w_next d_y x', h^2
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float x[8], dy[8], w[8], h[8];
      c.x[j].get(x); c.dy[j].get(dy); wn[j].get(w);
      if (H_IN) c.h[j].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] += x[e] * x[e];
        s[1] += w[e] * dy[e] * x[e];
        if (H_IN) s[2] += h[e] * h[e];
      }
    }
    block_sum<MANY>(s, red, half);
    const float rx = rsqrtf(s[0] / H + p.eps), mx = s[1] / H * rx * rx * rx;
    const float rh = post ? rsqrtf(s[2] / H + p.eps) : 1.f;
    float t[V][8];
    float q[2] = {0.f, 0.f};   // w_post d_n h, t n
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float x[8], dy[8], w[8], h[8], g[8], u[8];
      c.x[j].get(x); c.dy[j].get(dy); wn[j].get(w); c.dn[j].get(t[j]);
      if (H_IN) { c.h[j].get(h); wp[j].get(u); }
      if (kind == GATE_COLUMN) gc[j].get(g);
      if (kind == GATE_FULL) gf[j].get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (next) {
          if (live) an[j][e] += dy[e] * x[e] * rx;
          t[j][e] += rx * w[e] * dy[e] - mx * x[e];
        }
        if (H_IN) {
          const float n = post ? h[e] * rh * u[e] : h[e];
          const float d = f * (kind >= GATE_COLUMN ? g[e] : 1.f) * t[j][e];
          if (post) {
            q[0] += u[e] * d * h[e];
            if (live) ap[j][e] += d * h[e] * rh;
          }
          q[1] += t[j][e] * n;
          if (kind == GATE_COLUMN && live) ag[j][e] += p.scale * t[j][e] * n;
        }
      }
      const int col = column(j);
      if (live && col < H) Raw<T>::store((T*)p.d_x + (size_t)row * H + col, t[j]);
    }
    if (!H_IN) continue;
    if (post || kind == GATE_ROW) block_sum<MANY>(q, red, half);
    if (kind == GATE_ROW && live && threadIdx.x == 0) ((float*)p.d_gate)[row] = p.scale * q[1];
    const float mh = q[0] / H * rh * rh * rh;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float h[8], u[8], g[8], dh[8], dg[8];
      c.h[j].get(h); wp[j].get(u);
      if (kind == GATE_COLUMN) gc[j].get(g);
      if (kind == GATE_FULL) gf[j].get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = f * (kind >= GATE_COLUMN ? g[e] : 1.f) * t[j][e];
        dh[e] = post ? rh * u[e] * d - mh * h[e] : d;
        dg[e] = p.scale * t[j][e] * (post ? h[e] * rh * u[e] : h[e]);
      }
      const int col = column(j);
      if (live && col < H) {
        Raw<T>::store((T*)p.d_h + (size_t)row * H + col, dh);
        if (kind == GATE_FULL) Raw<T>::store((T*)p.d_gate + (size_t)row * H + col, dg);
      }
    }
  }
  if constexpr (MANY) {   // at most NORM_SHORT threads, 16 columns each
    __shared__ float sums[16 * NORM_SHORT];
    const auto join = [&](float (&a)[V][8]) {
      __syncthreads();
      float* own = sums + (group * blockDim.x + threadIdx.x) * 16;   // read only by the same column's threads
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) own[(j * 8 + e) ^ (threadIdx.x & 15)] = a[j][e];
      __syncthreads();
      if (group > 0) return;
      for (int g = 1; g < R; ++g)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) a[j][e] += own[g * blockDim.x * 16 + ((j * 8 + e) ^ (threadIdx.x & 15))];
    };
    if (next) join(an);
    if (post) join(ap);
    if (kind == GATE_COLUMN) join(ag);
    if (group > 0) return;
  }
  float* part = p.part + (size_t)blockIdx.x * 3 * H;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = column(j);
    if (col >= H) continue;
    const auto put = [&](float* to, const float* f) {   // read back at once
      *(float4*)to = make_float4(f[0], f[1], f[2], f[3]);
      *(float4*)(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
    };
    if (next) put(part + col, an[j]);
    if (post) put(part + H + col, ap[j]);
    if (kind == GATE_COLUMN) put(part + 2 * (size_t)H + col, ag[j]);
  }
}

// Column sums of the workgroups' partial sums, in a fixed order: 64 columns of
// one of the three a workgroup, 16 threads a column.
struct ReduceArgs {
  const float* part;
  float* out[3];
  int rows, H;
};
__global__ __launch_bounds__(1024) void norm_reduce_kernel(ReduceArgs p) {
  __shared__ float red[16][64];
  float* out = p.out[blockIdx.y];
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  float v = 0.f;
  if (c < p.H && p.rows > 0) {   // all loads in flight; rows past the last read the last one
    const float* a = p.part + (size_t)blockIdx.y * p.H + c;
    float t[NORM_GRID / 16];
#pragma unroll
    for (int i = 0; i < NORM_GRID / 16; ++i) t[i] = a[(size_t)min(g + 16 * i, p.rows - 1) * 3 * p.H];
#pragma unroll
    for (int i = 0; i < NORM_GRID / 16; ++i) v += g + 16 * i < p.rows ? t[i] : 0.f;
  }
  red[g][threadIdx.x & 63] = v;
  __syncthreads();
  if (g == 0 && c < p.H) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
    out[c] = s;
  }
}

// Threads of a workgroup: whole waves with V groups of 8 elements each.
int norm_threads(int H) { return (H / 8 + 64 * V - 1) / (64 * V) * 64; }

template <typename T>
hipError_t fwd(const NormArgs& p, hipStream_t s) {
  const int nt = norm_threads(p.H);
  // a launch holds fewer than 2^32 threads along x
  const dim3 grid(p.T < NORM_ROWS ? p.T : NORM_ROWS, (p.T + NORM_ROWS - 1) / NORM_ROWS);
  return run_kernel("norm_fwd", s, [&] {
    if (p.h) norm_fwd_kernel<T, true><<<grid, nt, 0, s>>>(p);
    else norm_fwd_kernel<T, false><<<grid, nt, 0, s>>>(p);
  });
}

template <typename T, int MAXT>
void run_bwd(const NormArgs& p, int grid, dim3 nt, hipStream_t s) {
  if (!p.h) norm_bwd_kernel<T, false, GATE_NONE, MAXT><<<grid, nt, 0, s>>>(p);
  else if (p.gate_kind == GATE_NONE) norm_bwd_kernel<T, true, GATE_NONE, MAXT><<<grid, nt, 0, s>>>(p);
  else if (p.gate_kind == GATE_ROW) norm_bwd_kernel<T, true, GATE_ROW, MAXT><<<grid, nt, 0, s>>>(p);
  else if (p.gate_kind == GATE_COLUMN) norm_bwd_kernel<T, true, GATE_COLUMN, MAXT><<<grid, nt, 0, s>>>(p);
  else norm_bwd_kernel<T, true, GATE_FULL, MAXT><<<grid, nt, 0, s>>>(p);
}

template <typename T>
hipError_t bwd(const NormArgs& p, hipStream_t s) {
  // rows of a workgroup: as many as fit NORM_SHORT threads and leave every workgroup some
  const int nt = norm_threads(p.H), fit = nt < NORM_SHORT ? NORM_SHORT / nt : 1, want = (int)(((long)p.T + NORM_GRID - 1) / NORM_GRID);
  const int R = want < 1 ? 1 : fit < want ? fit : want, all = (p.T + R - 1) / R, grid = all < NORM_GRID ? all : NORM_GRID;
  if (grid > 0) {
    const hipError_t e = run_kernel("norm_bwd", s, [&] {
      if (R > 1) run_bwd<T, NORM_SHORT>(p, grid, dim3(nt, R), s);
      else if (nt <= 512) run_bwd<T, 512>(p, grid, nt, s);
      else run_bwd<T, 1024>(p, grid, nt, s);
    });
    if (e != hipSuccess) return e;
  }
  const ReduceArgs r = {p.part, {p.w_next ? p.d_w_next : nullptr, p.h && p.w_post ? p.d_w_post : nullptr,
                                 p.h && p.gate_kind == GATE_COLUMN ? (float*)p.d_gate : nullptr}, grid, p.H};
  if (!r.out[0] && !r.out[1] && !r.out[2]) return hipSuccess;
  return run_kernel("norm_reduce", s, [&] { norm_reduce_kernel<<<dim3((p.H + 63) / 64, 3), 1024, 0, s>>>(r); });
}

}  // namespace

hipError_t launch_norm_fwd(int dtype, const NormArgs& p, hipStream_t s) {
  return dtype == 0 ? fwd<uint16_t>(p, s) : fwd<float>(p, s);
}
hipError_t launch_norm_bwd(int dtype, const NormArgs& p, hipStream_t s) {
  return dtype == 0 ? bwd<uint16_t>(p, s) : bwd<float>(p, s);
}

}  // namespace moe
