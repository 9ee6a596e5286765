// Newton-Schulz orthogonalisation of stacked matrices, and the optimiser step
// around it:
//
//   m' = mu m + g,  u = g + mu m' (Nesterov) or m'   (a step; otherwise u = g)
//   X = u / (|u| + eps)                                (2-norm of all elements)
//   `steps` times:  P = X X^T,  Q = a I + b P + c P P,  X <- Q X
//                   (matrices with more rows than columns: P = X^T X, X <- X Q)
//   w' = (1 - decay) w - lr X                          (a step; otherwise out = X)
//
// The products are bound by the matrix cores.  P and Q are symmetric, so only
// their tiles on and above the diagonal are computed and the others are their
// mirrors: 3 S^2 L + S^3 of 4 S^2 L + 2 S^3 operations a step (S the smaller, L
// the larger side).  No operand is ever transposed in memory: the products
// that contract over rows read their operands with transposing LDS reads.
//
// P, Q and the products' X are fp16, which the singular values' known range
// allows (at most 1.21 with the usual coefficients; the host checks others): 11
// significant bits where bf16 has 8, at the same matrix rate.  X itself is a pair
// of fp16 values, 22 bits: the rounding of a matrix of low rank (the gradient of an
// expert with few slots) lies outside of its range for the most part, where each
// step multiplies it by a.  With one value a 512 x 512 matrix of rank 1 was 0.15
// off, of rank 64 0.021; now 2.4e-4 and 7.6e-4.  The low half takes part in no
// product:
//
//   X <- Q X = D X + (Q - D) X_high,   D a diagonal
//
// costs reads and writes, not matrix work.  What X_high's rounding, r, does is (Q -
// D) r: nothing outside of X's range with D = a I, and least within it with D =
// diag(Q).  What is left outside grows by a with every later step, so D is a I,
// and diag(Q) in the last two steps.  D is kept in fp32 and takes up what the
// rounding of the rest of Q's diagonal leaves out; what P's diagonal's rounding
// takes away goes into Q's.  From the iteration in 64 bits, in the 2-norm: 1.5e-3
// at most from 64 x 64 on, at any rank, 5e-4 to 8e-4 mostly; up to 4e-3 where a few
// roundings are all of it (8 rows, or elements in a few rows or columns only); a
// bf16 result's own rounding, 1.66e-3, comes on top.  (With all of Q's products on the pair: 1e-4 to 1.1e-3,
// for another 2 S^2 L operations a step.)
// Factors 2^6 on X and 2^12 on P and Q keep small elements out of the subnormal
// range.  Sums and the polynomial's terms are fp32, the norm is summed in 64 bits
// (no overflow or underflow of fp32 gradients' squares).
//
// 16 matrices of 2880 x 2880, five steps: 8.85 ms, a step 419 us for P (65 % of the
// matrix cores busy at 1.65 GHz), 460 for Q (57 %) and 888 for X (53 %; 712 and 75
// % without the pair, whose reads and writes at the tiles' ends have no matrix work
// beside them), before them 51 us for the norm and 127 for the first X (5.2 and 6.3
// TB/s).  The sides are 11.25 tiles of 256, which count as 12, and diagonal tiles
// are whole: P and Q compute 23 % more than half a square, X 14 % more than it
// needs.
#include "dense_tiles.h"
#include "ortho.h"

namespace moe {
namespace dense {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f16x2_t v = {(_Float16)lo, (_Float16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
// As pack_pair, to fp16.
__device__ __forceinline__ u32x4 pack_pair_f16(const float* lo, const float* hi) {
  const auto a = __builtin_amdgcn_permlane32_swap(pack_f16(lo[0], lo[1]), pack_f16(hi[0], hi[1]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(pack_f16(lo[2], lo[3]), pack_f16(hi[2], hi[3]), false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}

// ------------------------------------------------------------------ norm and first iterate
// x (times ORTHO_X) as its fp16 value, and what that leaves.
__device__ __forceinline__ float low_half(float x) { return (x - (float)(_Float16)x) * ORTHO_LOW; }
// The two groups of four that pack_pair_f16 joined.
__device__ __forceinline__ void unpack_pair_f16(u32x4 w, float* lo, float* hi) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const f16x2_t l0 = __builtin_bit_cast(f16x2_t, (uint32_t)a[0]), l1 = __builtin_bit_cast(f16x2_t, (uint32_t)b[0]);
  const f16x2_t h0 = __builtin_bit_cast(f16x2_t, (uint32_t)a[1]), h1 = __builtin_bit_cast(f16x2_t, (uint32_t)b[1]);
  lo[0] = (float)l0[0]; lo[1] = (float)l0[1]; lo[2] = (float)l1[0]; lo[3] = (float)l1[1];
  hi[0] = (float)h0[0]; hi[1] = (float)h0[1]; hi[2] = (float)h1[0]; hi[3] = (float)h1[1];
}

// 8 gradients (or updates) from element i on.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float* v) {
  if constexpr (F32) {
    const float4 a = *(const float4*)((const float*)p + i), b = *(const float4*)((const float*)p + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *(const uint4*)((const uint16_t*)p + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(float, e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
}

// The sum of every thread's value, in a fixed order, in every thread.
__device__ __forceinline__ double sum_256(double v, double (&red)[4]) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// The update's squares, summed by workgroup, and a step's new momentum: one
// pass over g (and m), bound by HBM (a step of 8 matrices of 5760 x 2880 with
// fp32 gradients: 288 us, 5.5 TB/s).
template <bool F32>
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoArgs p) {
  __shared__ double red[4];
  const size_t n = (size_t)p.M * p.N, at = n * blockIdx.y;
  double sum = 0.0;
  for (size_t i = (blockIdx.x * 256ul + threadIdx.x) * 8; i < n; i += gridDim.x * 2048ul) {
    float u[8];
    load8<F32>(p.g, at + i, u);
    if (p.m) {
      float m[8];
      load8<true>(p.m, at + i, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = p.momentum * m[e] + u[e];
        u[e] = p.nesterov ? u[e] + p.momentum * m[e] : m[e];
      }
      *(float4*)(p.m_out + at + i) = make_float4(m[0], m[1], m[2], m[3]);
      *(float4*)(p.m_out + at + i + 4) = make_float4(m[4], m[5], m[6], m[7]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)u[e] * u[e];
  }
  sum = sum_256(sum, red);
  if (threadIdx.x == 0) p.part[blockIdx.y * ORTHO_PARTS + blockIdx.x] = sum;
}

// X = u / (|u| + eps), times ORTHO_X, in two halves; a step's u again from g and m'
// (the same step: 300 us, 5.3 TB/s).
template <bool F32>
__global__ __launch_bounds__(256) void ortho_scale_kernel(OrthoArgs p, int parts) {
  static_assert(ORTHO_PARTS <= 256, "a partial sum a thread");
  __shared__ double red[4];
  const size_t n = (size_t)p.M * p.N, at = n * blockIdx.y;
  const double sum = sum_256((int)threadIdx.x < parts ? p.part[blockIdx.y * ORTHO_PARTS + threadIdx.x] : 0.0, red);
  // in two factors, whose product may be past fp32's range (eps of 0 and subnormal updates; huge ones, an infinite eps)
  const double whole = ORTHO_X / (sqrt(sum) + (double)p.eps), part = fmin(fmax(whole, 0x1p-100), 0x1p100);
  const float f = (float)part, f2 = sum == 0.0 ? 0.f : (float)(whole / part + 0.0 * sum);   // NaN with an infinity or NaN in u
  for (size_t i = (blockIdx.x * 256ul + threadIdx.x) * 8; i < n; i += gridDim.x * 2048ul) {
    float u[8];
    load8<F32>(p.g, at + i, u);
    if (p.m) {
      float m[8];
      load8<true>(p.m_out, at + i, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = p.nesterov ? u[e] + p.momentum * m[e] : m[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= f, u[e] *= f2;
    *(uint4*)((uint16_t*)p.x0 + at + i) = make_uint4(pack_f16(u[0], u[1]), pack_f16(u[2], u[3]), pack_f16(u[4], u[5]),
                                                    pack_f16(u[6], u[7]));
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = low_half(u[e]);
    *(uint4*)((uint16_t*)p.l0 + at + i) = make_uint4(pack_f16(u[0], u[1]), pack_f16(u[2], u[3]), pack_f16(u[4], u[5]),
                                                    pack_f16(u[6], u[7]));
  }
}

// ------------------------------------------------------------------ symmetric products
struct SymArgs {
  const uint16_t* a;   // [E] matrices: rows of K (ROWS), or K rows of S
  const uint16_t* p;   // QUAD: [E,S,S], P
  uint16_t* out;       // [E,S,S]
  const float* pd;     // QUAD: [E,S], P's diagonal less its fp16 value
  float* diag;         // [E,S]: what the stored diagonal leaves out
  size_t a_step;       // elements of a matrix of a
  int E, S, K, tiles;  // tiles: of a side
  float a_diag, b, c;  // QUAD: a_diag I + b P + c A A^T, a_diag never stored
  int keep_diag;       // QUAD: b P + c A A^T has its diagonal stored, else zeros there
};

// out = A A^T (QUAD: b P + c A A^T) for square tiles on and above the
// diagonal, each stored where it belongs and, mirrored, below.  The mirror goes through
// LDS: the tile is written there as it lies in the registers and read back with
// the transposing reads.  COLS: A is held as its transpose (K rows of S).
template <class C, bool COLS, bool QUAD>
__global__ __launch_bounds__(256, 1) void ortho_sym_kernel(SymArgs p) {
  static_assert(C::FM == C::FN && C::LDS >= 2 * C::BM * C::BN, "square tiles, held in the ring's LDS");
  __shared__ __align__(1024) char lds[C::LDS];
  const int per = p.tiles * (p.tiles + 1) / 2;
  const int t = deal(blockIdx.x, per * p.E);
  if (t < 0) return;
  const int e = t / per;
  int nt = t - e * per, mt = 0;   // row mt has tiles - mt tiles, from the diagonal on
  while (nt >= p.tiles - mt) nt -= p.tiles - mt++;
  nt += mt;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, m0 = mt * C::BM, n0 = nt * C::BN, S = p.S, K = p.K;
  f32x16 acc[C::FM][C::FN];
  const uint16_t* A = p.a + p.a_step * e;
  if constexpr (COLS) {
    CSrc<C::NBA> as;
    CSrc<C::NBB> bs;
    as.init(A, S, m0, S, wave, lane);
    bs.init(A, S, n0, S, wave, lane);
    mainloop<C, f16x8_t>(as, bs, K, lds, acc, wave, lane);
  } else {
    KSrc<C::NBA> as;
    KSrc<C::NBB> bs;
    as.init(A + (size_t)m0 * K, nullptr, [&](int r) { return (uint32_t)(min(r, S - 1 - m0) * K * 2); }, wave, lane);
    bs.init(A + (size_t)n0 * K, nullptr, [&](int r) { return (uint32_t)(min(r, S - 1 - n0) * K * 2); }, wave, lane);
    mainloop<C, f16x8_t>(as, bs, K, lds, acc, wave, lane);
  }
  const uint16_t* P = p.p + (size_t)S * S * e;
  float* diag = p.diag + (size_t)S * e;
  uint16_t* out = p.out + (size_t)S * S * e;
  // panels [BM rows][64 columns] of LDS, 16-byte chunks permuted as in FragSrc
  const int r32 = lane & 31, x = (((r32 >> 1) & 1) << 2) | (((r32 >> 3) & 1) << 1);
  struct Held { f16x4_t v[4]; };
  const int c4 = 4 * (lane >> 5);
  float dr[C::FM] = {};
  if (QUAD && mt == nt) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) dr[i] = p.pd[(size_t)S * e + min(m0 + wm * 32 * C::FM + 32 * i + r32, S - 1)];
  }
  each_fragment<C, Held, 4>(
      [&](int i, int j, Held& h) __attribute__((always_inline)) {   // rows and columns past the last read the last one
        if (!QUAD) return;
        const uint16_t* row = P + (size_t)min(m0 + wm * 32 * C::FM + 32 * i + r32, S - 1) * S;
#pragma unroll
        for (int v = 0; v < 4; ++v) h.v[v] = *(const f16x4_t*)(row + min(n0 + (wn * C::FN + j) * 32 + 8 * v, S - 8) + c4);
      },
      [&](int i, int j, const Held& held) __attribute__((always_inline)) {
        const int tr = wm * 32 * C::FM + 32 * i + r32, row = m0 + tr;
        float mine = 0.f;
        const bool on_diag = mt == nt && wm * C::FM + i == wn * C::FN + j;   // the diagonal passes through this fragment
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int tc = (wn * C::FN + j) * 32 + 16 * q;
          float v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float s = acc[i][j][8 * q + 4 * h + k];
              v[h][k] = QUAD ? p.b * (float)held.v[2 * q + h][k] + p.c * s : s;
            }
            if (on_diag) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool on = r32 == 16 * q + 8 * h + c4 + k;
                // with P's element as it was before its rounding
                if (QUAD) v[h][k] += on ? (p.b + 2.f * p.c * (float)held.v[2 * q + h][k]) * dr[i] : 0.f;
                mine = on ? v[h][k] : mine;
                if (QUAD && on && !p.keep_diag) v[h][k] = 0.f;
              }
            }
            if (mt != nt) {
              const int ct = tc + 8 * h;
              *(uint2*)(lds + (ct >> 6) * (C::BM * 128) + tr * 128 + ((((ct >> 3) & 7) ^ x) << 4) + 2 * c4) =
                  make_uint2(pack_f16(v[h][0], v[h][1]), pack_f16(v[h][2], v[h][3]));
            }
          }
          const u32x4 o = pack_pair_f16(v[0], v[1]);
          const int cc = n0 + tc + 2 * c4;
          if (row < S && cc < S) *(u32x4*)(out + (size_t)row * S + cc) = o;
        }
        if (on_diag && (r32 & 4) == c4 && row < S) {   // the lane that holds the row's diagonal element
          const float r = QUAD && !p.keep_diag ? 0.f : (float)(_Float16)mine;
          diag[row] = QUAD ? p.a_diag + (mine - r) : mine - r;
        }
      });
  if (mt == nt) return;
  __syncthreads();
  // 32 columns x 16 rows a read: lane -> column lane % 32, rows 8 (lane / 32) .. + 7
  const int g = lane >> 4, s4 = lane & 15, kr = ((g >> 1) << 3) + (s4 >> 2);
  const int kx = (((kr >> 1) & 1) << 2) | (((kr >> 3) & 1) << 1);
#pragma unroll 1
  for (int cb = wave; cb < C::BN / 32; cb += 4) {
    const int chunk = ((cb & 1) << 2) + ((g & 1) << 1) + ((s4 & 3) >> 1);
    const lds_char* base = (const lds_char*)lds + (cb >> 1) * (C::BM * 128) + kr * 128 + ((chunk ^ kx) << 4) + (s4 & 1) * 8;
    const int c = n0 + cb * 32 + r32;
#pragma unroll
    for (int k = 0; k < C::BM / 16; ++k) {
      struct { s16x4_t h[2]; } v;
      v.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + k * 2048));
      v.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + k * 2048 + 512));
      const int r = m0 + k * 16 + 8 * (lane >> 5);
      if (c < S && r < S) *(u32x4*)(out + (size_t)c * S + r) = __builtin_bit_cast(u32x4, v);
    }
  }
}

// ------------------------------------------------------------------ X <- Q X (or X Q)
enum { TO_X = 0, TO_BF16 = 1, TO_F32 = 2 };
struct UpdateArgs {
  const uint16_t *x, *low, *q;
  const float* qd;   // [E,S]: for each row (of Q X) or column (of X Q) the multiple of X that q's products leave out
  void* out;
  uint16_t* out_low; // TO_X
  const void* w;   // the weights that a step updates, or null
  int E, M, N, S, mt, nt;
  float lr, keep;
};
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const uint2 w = *(const uint2*)p;
  v[0] = __builtin_bit_cast(float, w.x << 16); v[1] = __builtin_bit_cast(float, w.x & 0xffff0000u);
  v[2] = __builtin_bit_cast(float, w.y << 16); v[3] = __builtin_bit_cast(float, w.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 w = *(const float4*)p;
  v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

template <class C, bool WIDE, int TO>
__global__ __launch_bounds__(256, 1) void ortho_update_kernel(UpdateArgs p) {
  using T = std::conditional_t<TO == TO_F32, float, uint16_t>;
  __shared__ __align__(1024) char lds[C::LDS];
  const int per = p.mt * p.nt, t = deal(blockIdx.x, per * p.E);
  if (t < 0) return;
  const int e = t / per;
  int mt, nt;
  tile_at(t - e * per, p.mt, p.nt, mt, nt);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, m0 = mt * C::BM, n0 = nt * C::BN, M = p.M, N = p.N, S = p.S;
  f32x16 acc[C::FM][C::FN];
  const size_t at = (size_t)M * N * e;
  const int r0 = m0 + wm * 32 * C::FM + (lane & 31), c00 = n0 + wn * 32 * C::FN, c4 = 4 * (lane >> 5);
  const bool step = TO != TO_X && p.w != nullptr;
  const uint16_t *X = p.x + (size_t)M * N * e, *Q = p.q + (size_t)S * S * e;
  const float qd = p.qd[(size_t)S * e + min((WIDE ? m0 : n0) + (int)threadIdx.x, S - 1)];   // of tile row or column threadIdx.x
  const auto rows = [&](auto& src, const uint16_t* b, int r0, int n) {   // rows of S
    src.init(b + (size_t)r0 * S, nullptr, [&](int r) { return (uint32_t)(min(r, n - 1 - r0) * S * 2); }, wave, lane);
  };
  KSrc<C::NBA> as;
  if constexpr (WIDE) {
    CSrc<C::NBB> bs;
    rows(as, Q, m0, S);
    bs.init(X, N, n0, N, wave, lane);
    mainloop<C, f16x8_t>(as, bs, S, lds, acc, wave, lane);
  } else {
    KSrc<C::NBB> bs;
    rows(as, X, m0, M);
    rows(bs, Q, n0, S);
    mainloop<C, f16x8_t>(as, bs, S, lds, acc, wave, lane);
  }
  const float f = TO == TO_X ? 1.f / ORTHO_P : 1.f / (ORTHO_X * ORTHO_P);   // the products carry ORTHO_X ORTHO_P
  lds_float* fac = (lds_float*)lds;
  if ((int)threadIdx.x < (WIDE ? C::BM : C::BN)) fac[threadIdx.x] = f * qd;
  __syncthreads();
  struct Held { float w[4][4]; u32x4 x[2], low[2]; };
  each_fragment<C, Held, TO == TO_X ? 4 : 2>(
      [&](int i, int j, Held& h) __attribute__((always_inline)) {   // rows and columns past the last read the last one
        const size_t row = at + (size_t)min(r0 + 32 * i, M - 1) * N;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const size_t el = row + min(c00 + 32 * j + 16 * q + 2 * c4, N - 8);
          h.x[q] = *(const u32x4*)(p.x + el);
          h.low[q] = *(const u32x4*)(p.low + el);
        }
        if (!step) return;
#pragma unroll
        for (int v = 0; v < 4; ++v) load4((const T*)p.w + row + min(c00 + 32 * j + 8 * v, N - 8) + c4, h.w[v]);
      },
      [&](int i, int j, const Held& held) __attribute__((always_inline)) {
        const int row = r0 + 32 * i;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c = c00 + 32 * j + 16 * q;
          float v[2][4], x[2][4], low[2][4];
          unpack_pair_f16(held.x[q], x[0], x[1]);
          unpack_pair_f16(held.low[q], low[0], low[1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4 d;
            if constexpr (WIDE) d = f32x4{1.f, 1.f, 1.f, 1.f} * fac[row - m0];
            else d = *(lds_f32x4*)(fac + (c - n0) + 8 * h + c4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float r = acc[i][j][8 * q + 4 * h + k];
              const float o = f * r + d[k] * (x[h][k] + low[h][k] * (1.f / ORTHO_LOW));
              v[h][k] = step ? p.keep * held.w[2 * q + h][k] - p.lr * o : o;
            }
          }
          if constexpr (TO == TO_F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (row < M && c + 8 * h < N)
                store4<float>((float*)p.out + at + (size_t)row * N + c + 8 * h + c4, v[h][0], v[h][1], v[h][2], v[h][3]);
          } else {
            const u32x4 o = TO == TO_X ? pack_pair_f16(v[0], v[1]) : pack_pair(v[0], v[1]);
            const int cc = c + 2 * c4;
            const size_t el = at + (size_t)row * N + cc;
            if (row < M && cc < N) *(u32x4*)((uint16_t*)p.out + el) = o;
            if constexpr (TO == TO_X) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[h][k] = low_half(v[h][k]);
              const u32x4 l = pack_pair_f16(v[0], v[1]);
              if (row < M && cc < N) *(u32x4*)(p.out_low + el) = l;
            }
          }
        }
      });
}

// ------------------------------------------------------------------ host
template <class C, bool COLS, bool QUAD>
hipError_t run_sym(const SymArgs& p, hipStream_t s) {
  const auto k = ortho_sym_kernel<C, COLS, QUAD>;
  const long tiles = (long)p.E * p.tiles * (p.tiles + 1) / 2;
  return run_kernel(QUAD ? "ortho_quad" : "ortho_gram", s, [&] { k<<<deal_grid(tiles), C::NT, 0, s>>>(p); });
}
// Square tiles only.
hipError_t sym(SymArgs p, bool cols, bool quad, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_square_tile(square_tile_kind(p.S, p.K, p.E), [&](auto c) {
    using C = decltype(c);
    p.tiles = (p.S + C::BM - 1) / C::BM;
    e = quad ? run_sym<C, false, true>(p, s) : cols ? run_sym<C, true, false>(p, s) : run_sym<C, false, false>(p, s);
  });
  return e;
}

template <class C, bool WIDE, int TO>
hipError_t run_update(const UpdateArgs& p, hipStream_t s) {
  const auto k = ortho_update_kernel<C, WIDE, TO>;
  return run_kernel("ortho_update", s, [&] { k<<<deal_grid((long)p.E * p.mt * p.nt), C::NT, 0, s>>>(p); });
}
hipError_t update(UpdateArgs p, int to, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.M, p.N, p.S, p.E, p.S < ORTHO_NARROW ? 3 : 0), [&](auto c) {   // 3: tiles of at most 128 x 128
    using C = decltype(c);
    p.mt = (p.M + C::BM - 1) / C::BM;
    p.nt = (p.N + C::BN - 1) / C::BN;
    const auto run = [&](auto wide) {
      constexpr bool W = decltype(wide)::value;
      return to == TO_X ? run_update<C, W, TO_X>(p, s) : to == TO_BF16 ? run_update<C, W, TO_BF16>(p, s) : run_update<C, W, TO_F32>(p, s);
    };
    e = p.M <= p.N ? run(std::true_type{}) : run(std::false_type{});
  });
  return e;
}

}  // namespace dense

using namespace dense;

hipError_t launch_ortho(const OrthoArgs& p, hipStream_t s) {
  const size_t n = (size_t)p.M * p.N;
  // workgroups of a matrix: 4 groups of 8 elements a thread, or more where that makes over 4096 in all
  const size_t want = (n + 8191) / 8192, most = 4096 / p.E < 16 ? 16 : 4096 / p.E < ORTHO_PARTS ? 4096 / p.E : ORTHO_PARTS;
  const int parts = (int)(want < most ? want : most);
  hipError_t e = run_kernel("ortho_norm", s, [&] {
    if (p.g_f32) ortho_norm_kernel<true><<<dim3(parts, p.E), 256, 0, s>>>(p);
    else ortho_norm_kernel<false><<<dim3(parts, p.E), 256, 0, s>>>(p);
  });
  if (e != hipSuccess) return e;
  e = run_kernel("ortho_scale", s, [&] {
    if (p.g_f32) ortho_scale_kernel<true><<<dim3(parts, p.E), 256, 0, s>>>(p, parts);
    else ortho_scale_kernel<false><<<dim3(parts, p.E), 256, 0, s>>>(p, parts);
  });
  const bool wide = p.M <= p.N;
  uint16_t *x = (uint16_t*)p.x0, *y = (uint16_t*)p.x1, *xl = (uint16_t*)p.l0, *yl = (uint16_t*)p.l1, *P = (uint16_t*)p.p, *Q = (uint16_t*)p.q;
  const size_t ss = (size_t)p.S * p.S;
  for (int i = 0; i < p.steps && e == hipSuccess; ++i) {
    const bool last = i + 1 == p.steps;
    // X X^T carries ORTHO_X^2 = ORTHO_P; P P carries ORTHO_P^2
    e = sym({x, nullptr, P, nullptr, p.pd, n, p.E, p.S, wide ? p.N : p.M, 0, 0.f, 0.f, 1.f, 1}, !wide, false, s);
    if (e == hipSuccess)
      e = sym({P, P, Q, p.pd, p.qd, ss, p.E, p.S, p.S, 0, ORTHO_P * p.a, p.b, p.c / ORTHO_P, i + 2 < p.steps}, false, true, s);
    if (e == hipSuccess)
      e = update({x, xl, Q, p.qd, last ? p.out : y, yl, last ? p.w : nullptr, p.E, p.M, p.N, p.S, 0, 0, p.lr, p.keep},
                 !last ? TO_X : p.out_f32 ? TO_F32 : TO_BF16, s);
    std::swap(x, y);
    std::swap(xl, yl);
  }
  return e;
}

}  // namespace moe
