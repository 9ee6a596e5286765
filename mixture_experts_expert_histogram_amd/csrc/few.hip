// The whole layer for a few tokens (decoding): one kernel for the gate_up
// projection with its activation, one for the down projection, one for the
// sum over a token's experts (one token: two kernels, below).
//
//   a[s]   = phi(Wgu[e_s] x_t)        s = t K + k, e_s = ids[s]
//   y[s]   = w_s Wd[e_s] a[s]
//   out[t] = sum_k y[t K + k]
//
// a is rounded to the activations' type, as the matrix cores take it (bf16
// layers: 2.4e-3 from 64 bits in the 2-norm, 1.7e-3 with a in fp32); y and
// every sum are fp32.
//
// With a few tokens an expert holds one or two slots, and the time is that of
// reading the active experts' weights once (again for each 64 of an expert's
// slots, 32 on 4-bit weights): 2 flops a weight byte against the
// 300 where the matrix cores would bound it.  So nothing here is staged for
// reuse: a wave reads its weight rows (32 of plain weights, 64 of 4-bit ones)
// straight into matrix-core fragments (16 rows by k, every lane 16 bytes of one
// row) and multiplies them with 16 to 64 token columns, whose fragments come
// from L1/L2.  The lanes' share of k follows from the 16-byte loads (lane group
// g of 4 holds the g-th 16 bytes of a row's 64), and the token fragments are
// read in the same k order, so no operand is ever shuffled.  The waves of a
// workgroup take k units in turn and their partial sums meet in LDS in wave
// order.
//
// No routing pass precedes it: a workgroup finds its expert's slots by a scan
// over the ids (at most T K of them), in slot order.  Nothing depends on the
// order in which workgroups run, and no atomics are used.
//
// Loads are buffer loads whose offset is put past the buffer's end where a
// row, a token or a k chunk does not exist: they return zero without memory
// traffic and without a branch.
#include <type_traits>

#include "few.h"
#include "mx.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

enum { W_BF16 = 0, W_F32 = 1, W_MX = 2 };

constexpr uint32_t kPast = 0x80000000u;   // byte offset past every buffer

// A unit of a weight row's k: WQ times 64 bytes, of which a lane holds 16.
// XQ: 16-byte loads of a token row for the same k; XSZ: bytes a token element.
// Plain weights go by whole cache lines (16 tokens' gpt-oss-shaped layer: 420 us;
// in units of 64 bytes, a line's halves to two waves, 473, and 478 with twice
// the units in flight).
template <int KIND> struct Unit;
template <> struct Unit<W_BF16> { static constexpr int K = 64, WQ = 2, XQ = 2, XSZ = 2; };
template <> struct Unit<W_F32> { static constexpr int K = 32, WQ = 2, XQ = 2, XSZ = 4; };
template <> struct Unit<W_MX> { static constexpr int K = 128, WQ = 1, XQ = 4, XSZ = 2; };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), 0, (int)kPast, 0x00027000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Weight rows of one wave: G groups of 16 rows.  off is this lane's row (lane
// % 16) in bytes from the group's base, soff the row's scales in bytes from
// the start of the workgroup's scales in LDS (sc).
template <int G>
struct Rows {
  __amdgpu_buffer_rsrc_t w[G];
  uint32_t off[G], soff[G];
  const uint8_t* sc;
};

// The scales of a workgroup's rows in LDS: up to two runs of consecutive rows
// (the gate and the up rows where they are apart), each of `bytes` bytes, a
// multiple of 16.  Read in whole runs: a byte load for each lane's block
// touches a cache line a row for 4 bytes of it, and took a fifth of the time
// of a 32-token gpt-oss-shaped layer.  fetch() issues the loads of all but very
// long rows, store() writes them to LDS.
template <int NTHREADS>
struct Scales {
  __amdgpu_buffer_rsrc_t at[2];
  uint32_t bytes[2];
  u32x4_t v[2];
  // byte o of the runs, one after the other
  __device__ __forceinline__ u32x4_t get(uint32_t o) const {
    return o < bytes[0] ? load16(at[0], o) : load16(at[1], o - bytes[0] < bytes[1] ? o - bytes[0] : kPast);
  }
  __device__ __forceinline__ void fetch(int tid) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = get((i * NTHREADS + tid) * 16);
  }
  __device__ __forceinline__ void store(uint8_t* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t o = (i * NTHREADS + tid) * 16;
      if (o < bytes[0] + bytes[1]) *(u32x4_t*)(lds + o) = v[i];
    }
    for (uint32_t o = (2 * NTHREADS + tid) * 16; o < bytes[0] + bytes[1]; o += NTHREADS * 16) *(u32x4_t*)(lds + o) = get(o);
  }
};

// One unit of a wave: its weight rows, and the same k of the token columns.
template <int KIND, int G, int NT>
struct UnitRegs {
  u32x4_t w[G][Unit<KIND>::WQ], x[NT][Unit<KIND>::XQ];
  uint32_t s[G];
};

// k of a lane's chunk q of unit u (q of the WQ weight chunks; a mx chunk is a block)
template <int KIND>
__device__ __forceinline__ int chunk_k(int u, int q, int lane) {
  using UN = Unit<KIND>;
  return u * UN::K + q * (UN::K / UN::WQ) + (lane >> 4) * (UN::K / UN::WQ / 4);
}

template <int KIND, int G, int NT>
__device__ __forceinline__ void load_w(const Rows<G>& r, int u, int K, int lane, UnitRegs<KIND, G, NT>& t) {
  using UN = Unit<KIND>;
#pragma unroll
  for (int q = 0; q < UN::WQ; ++q) {
    const bool ok = chunk_k<KIND>(u, q, lane) < K;   // K is a multiple of a lane's share
#pragma unroll
    for (int h = 0; h < G; ++h) t.w[h][q] = load16(r.w[h], ok ? r.off[h] + (u * UN::WQ + q) * 64 + (lane >> 4) * 16 : kPast);
  }
}
// The unit's scales (they are in LDS by now) and token rows; xoff[n]: byte
// offset of this lane's token row of column tile n (kPast: no token).
template <int KIND, int G, int NT>
__device__ __forceinline__ void load_x(const Rows<G>& r, __amdgpu_buffer_rsrc_t xr, const uint32_t (&xoff)[NT], int u, int K,
                                       int lane, UnitRegs<KIND, G, NT>& t) {
  using UN = Unit<KIND>;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < UN::XQ; ++q) {
      const int k = KIND == W_MX ? chunk_k<KIND>(u, 0, lane) + q * 8 : chunk_k<KIND>(u, q, lane);
      t.x[n][q] = load16(xr, k < K && xoff[n] != kPast ? xoff[n] + k * UN::XSZ : kPast);
    }
  if constexpr (KIND == W_MX) {
    const int b = u * 4 + (lane >> 4);
#pragma unroll
    for (int h = 0; h < G; ++h) t.s[h] = r.sc[r.soff[h] + (b * 32 < K ? b : 0)];
  }
}

// Accumulator element v of a lane is weight row 4 (lane / 16) + v of the
// group, token column lane % 16.
template <int KIND, int G, int NT>
__device__ __forceinline__ void mma(const UnitRegs<KIND, G, NT>& t, f32x4 (&acc)[G][NT]) {
  using UN = Unit<KIND>;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    if constexpr (KIND == W_BF16) {
#pragma unroll
      for (int q = 0; q < UN::WQ; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[h][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, t.w[h][q]),
                                                              __builtin_bit_cast(bf16x8_t, t.x[n][q]), acc[h][n], 0, 0, 0);
    } else if constexpr (KIND == W_F32) {
#pragma unroll
      for (int q = 0; q < UN::WQ; ++q) {
        const f32x4 wf = __builtin_bit_cast(f32x4, t.w[h][q]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const f32x4 xf = __builtin_bit_cast(f32x4, t.x[n][q]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[h][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[i], xf[i], acc[h][n], 0, 0, 0);
        }
      }
    } else {
      const float sc = mx_scale(t.s[h]);
      const u32x4_t w = t.w[h][0];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bf16x8_t wq = mx_expand(w[q], sc);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[h][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wq, __builtin_bit_cast(bf16x8_t, t.x[n][q]), acc[h][n], 0, 0, 0);
      }
    }
  }
}

// The dot products of a wave's weight rows over its k units u0, u0 + du, ...:
// a ring of D units in registers, each loaded D units ahead.  start() issues
// the weights' first loads, before the token rows are known; run() the rest.
template <int KIND, int G, int NT, int D>
struct Dot {
  UnitRegs<KIND, G, NT> ring[D];
  __device__ __forceinline__ void start(const Rows<G>& r, int u0, int du, int K, int lane) {
#pragma unroll
    for (int d = 0; d < D; ++d) load_w<KIND, G, NT>(r, u0 + d * du, K, lane, ring[d]);
  }
  __device__ __forceinline__ void run(const Rows<G>& r, __amdgpu_buffer_rsrc_t xr, const uint32_t (&xoff)[NT], int u0,
                                      int du, int K, int lane, f32x4 (&acc)[G][NT]) {
#pragma unroll
    for (int d = 0; d < D; ++d) load_x<KIND, G, NT>(r, xr, xoff, u0 + d * du, K, lane, ring[d]);
    const int nu = (K + Unit<KIND>::K - 1) / Unit<KIND>::K;
    for (int u = u0; u < nu; u += D * du) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        mma<KIND, G, NT>(ring[d], acc);
        load_w<KIND, G, NT>(r, u + (d + D) * du, K, lane, ring[d]);
        load_x<KIND, G, NT>(r, xr, xoff, u + (d + D) * du, K, lane, ring[d]);
        __builtin_amdgcn_sched_barrier(0);   // or every product of the ring moves before its reloads
      }
    }
  }
};

template <int G, int NT>
__device__ __forceinline__ void zero(f32x4 (&acc)[G][NT]) {
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// A workgroup barrier that orders LDS accesses only: loads in flight stay so.
__device__ __forceinline__ void lds_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The slots of expert e, ascending, in LDS; returns their number.  Every
// thread of the workgroup calls it.
template <int NW>
__device__ __forceinline__ int find_slots(const FewArgs& p, int e, uint16_t* list, int* cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint64_t lower = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  int c = 0;
  for (int s0 = 0; s0 < p.S; s0 += NW * 64) {
    const int s = s0 + tid;
    const bool hit = s < p.S && p.ids[s] == e;
    const uint64_t m = __ballot(hit);
    if (lane == 0) cnt[wave] = __popcll(m);
    lds_sync();
    int at = c + __popcll(m & lower);
    for (int v = 0; v < NW; ++v) {
      at += v < wave ? cnt[v] : 0;
      c += cnt[v];
    }
    if (hit) list[at] = (uint16_t)s;
    lds_sync();
  }
  return c;
}

// The waves' partial sums of RT column tiles from n0 in LDS: [wave][group]
// [column tile][column 16][row 16], read back summed in wave order.
template <int G, int NT, int RT>
__device__ __forceinline__ void put_partial(float* red, int wave, int lane, const f32x4 (&acc)[G][NT], int n0) {
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int n = 0; n < RT; ++n)
      *(f32x4*)(red + (((wave * G + h) * RT + n) * 16 + (lane & 15)) * 16 + 4 * (lane >> 4)) = acc[h][n0 + n];
}
// element (row j, token column c) of group h
template <int G, int NT, int NW>
__device__ __forceinline__ float get_sum(const float* red, int h, int j, int c) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += red[(((w * G + h) * NT + (c >> 4)) * 16 + (c & 15)) * 16 + j];
  return v;
}

template <int KIND> struct Elem { using T = uint16_t; };
template <> struct Elem<W_F32> { using T = float; };

// Per weight kind: row groups of a wave, units in flight with one column tile
// and with more, waves of a workgroup, waves a SIMD that the registers allow
// for, and the most column tiles of a pass.  Up to 64 tokens of an expert are
// one pass over its weights: with passes of 32, 8 experts of 2880 x 2880 took
// 156 us at 64 tokens, top-4, and take 132 (4-bit weights, whose fragments of
// 64 rows leave no registers for it, stay at 32).  4 row groups for plain
// weights read each token row half as often and were faster above 30 tokens an
// expert (125 us there), but slower below (16 tokens, 128 experts: 484 us
// against 428) and in small layers.
template <int KIND> struct Tune;
template <> struct Tune<W_BF16> { static constexpr int G = 2, D1 = 2, D2 = 1, NW = 4, OCC = 4, NT = 4; };
template <> struct Tune<W_F32> { static constexpr int G = 2, D1 = 2, D2 = 1, NW = 4, OCC = 4, NT = 4; };
template <> struct Tune<W_MX> { static constexpr int G = 4, D1 = 1, D2 = 1, NW = 4, OCC = 3, NT = 2; };
constexpr int RED_NT = 2;   // column tiles whose partial sums are in LDS at once

// Rows of G/2 gate and up groups: groups 2i and 2i+1 are the gate and up rows
// of activation columns j0 + 16 i .. +15.
template <int KIND, int G, int NTH>
__device__ __forceinline__ void gate_up_rows(const FewArgs& p, int e, int j0, int lane, uint8_t* sc, Rows<G>& r,
                                             Scales<NTH>& runs) {
  const long at = p.gu_es * e + p.gu_rs * j0;
  const uint32_t sb = p.H / 32;   // bytes of a row's scales
  const int nj = min(8 * G, p.I - j0);
  const bool inter = p.gu_rs != p.H / 2;   // gate and up rows in turn: one run
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const int j = min((h >> 1) * 16 + (lane & 15), nj - 1);
    r.w[h] = rsrc((const char*)(h & 1 ? p.gu_u : p.gu_g) + at);
    r.off[h] = (uint32_t)(p.gu_rs * j);
    r.soff[h] = inter ? (2 * j + (h & 1)) * sb : (h & 1 ? nj + j : j) * sb;
  }
  r.sc = sc;
  runs.at[0] = rsrc((const char*)p.gus_g + at / 16);
  runs.at[1] = rsrc((const char*)p.gus_u + at / 16);
  runs.bytes[0] = (inter ? 2 : 1) * nj * sb;
  runs.bytes[1] = inter ? 0 : nj * sb;
}
template <int KIND, int G, int NTH>
__device__ __forceinline__ void down_rows(const FewArgs& p, int e, int h0, int lane, uint8_t* sc, Rows<G>& r,
                                          Scales<NTH>& runs) {
  const long at = p.d_rs * ((long)p.H * e + h0);
  const uint32_t sb = p.I / 32;
  const int nh = min(16 * G, p.H - h0);
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const int j = min(h * 16 + (lane & 15), nh - 1);
    r.w[h] = rsrc((const char*)p.Wd + at);
    r.off[h] = (uint32_t)(p.d_rs * j);
    r.soff[h] = j * sb;
  }
  r.sc = sc;
  runs.at[0] = runs.at[1] = rsrc((const char*)p.sd + at / 16);
  runs.bytes[0] = nh * sb;
  runs.bytes[1] = 0;
}

// Grid row y stands for expert y when there are at least E slots, otherwise
// for the expert of slot y.
__device__ __forceinline__ int expert_of(const FewArgs& p) {
  return p.S < p.E ? __builtin_amdgcn_readfirstlane(p.ids[blockIdx.y]) : (int)blockIdx.y;
}
// Whether another grid row has this expert: its first slot's row works.
__device__ __forceinline__ bool not_mine(const FewArgs& p, int c, const uint16_t* list) {
  return c == 0 || (p.S < p.E && list[0] != blockIdx.y);
}

// ---------------------------------------------------------------- gate_up
// One workgroup: 8 G activation columns of one expert for all its tokens, 16
// of them at a time, or 32 or 64 where it has more.
// 128 experts of 2880 x 2880, top-4: 16 tokens bf16 279 us, 1.69 GB read at 5.9
// TB/s, bound by HBM (a large copy moves 4.8, the best pass here 6.9).  32
// tokens on 4-bit weights 134 us, 0.70 GB at 4.9 TB/s, bound by the loads'
// path (busy 88 % of the time): a load covers 64 bytes a row, and as many bytes
// of tokens as of codes are loaded.  256 experts of 4096 x 2048, 48 tokens,
// top-8: 960 us bf16.
template <int KIND, int G, int NT, int D, int NW>
__device__ __forceinline__ void gate_up_pass(const FewArgs& p, const Rows<G>& r, Dot<KIND, G, NT, D>& dot, int j0, int c0,
                                             int c, const uint16_t* list, float* red, int wave, int lane) {
  using T = typename Elem<KIND>::T;
  uint32_t xoff[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = c0 + n * 16 + (lane & 15);
    xoff[n] = i < c ? (uint32_t)(list[i] / p.K) * (uint32_t)(p.H * Unit<KIND>::XSZ) : kPast;
  }
  f32x4 acc[G][NT];
  zero<G, NT>(acc);
  dot.run(r, rsrc(p.X), xoff, wave, NW, p.H, lane, acc);
  T* a = (T*)p.a;
  constexpr int RT = NT < RED_NT ? NT : RED_NT;
#pragma unroll
  for (int n0 = 0; n0 < NT; n0 += RT) {
    put_partial<G, NT, RT>(red, wave, lane, acc, n0);
    lds_sync();
    for (int o = threadIdx.x; o < 8 * G * 16 * RT; o += NW * 64) {
      const int j = o % (8 * G), t = o / (8 * G), i = c0 + n0 * 16 + t;
      if (i < c && j0 + j < p.I) {
        const float gv = get_sum<G, RT, NW>(red, 2 * (j >> 4), j & 15, t), uv = get_sum<G, RT, NW>(red, 2 * (j >> 4) + 1, j & 15, t);
        store_val<T>(a + (size_t)list[i] * p.I + j0 + j, glu_fwd(gv, uv, p.act, p.limit, p.alpha));
      }
    }
    lds_sync();
  }
}

template <int KIND>
__global__ __launch_bounds__(Tune<KIND>::NW * 64, Tune<KIND>::OCC) void few_gate_up_kernel(FewArgs p) {
  using TU = Tune<KIND>;
  constexpr int G = TU::G, NW = TU::NW;
  extern __shared__ char few_lds[];
  __shared__ int cnt[NW];
  __shared__ __align__(16) float red[NW * G * RED_NT * 256];
  uint16_t* list = (uint16_t*)few_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {   // slots with an id outside [0,E)
    int bad = 0;
    for (int s = lane; s < p.S; s += 64) bad += (unsigned)p.ids[s] >= (unsigned)p.E;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) bad += __shfl_xor(bad, d);
    if (lane == 0) p.status[0] = bad;
  }
  const int e = expert_of(p);
  if ((unsigned)e >= (unsigned)p.E) return;
  const int j0 = blockIdx.x * 8 * G;
  const int c = find_slots<NW>(p, e, list, cnt);
  if (not_mine(p, c, list)) return;
  Rows<G> r;
  Scales<NW * 64> scales;
  uint8_t* sc = (uint8_t*)few_lds + ((2 * p.S + 15) & ~15);
  gate_up_rows<KIND, G>(p, e, j0, lane, sc, r, scales);
  if constexpr (KIND == W_MX) scales.fetch(threadIdx.x);
  if (c <= 16) {
    Dot<KIND, G, 1, TU::D1> dot;
    dot.start(r, wave, NW, p.H, lane);
    if constexpr (KIND == W_MX) {
      scales.store(sc, threadIdx.x);
      lds_sync();
    }
    gate_up_pass<KIND, G, 1, TU::D1, NW>(p, r, dot, j0, 0, c, list, red, wave, lane);
  } else {
    if constexpr (KIND == W_MX) {
      scales.store(sc, threadIdx.x);
      lds_sync();
    }
    const auto pass = [&](auto n, int c0) {
      constexpr int NT = decltype(n)::value;
      Dot<KIND, G, NT, TU::D2> dot;
      dot.start(r, wave, NW, p.H, lane);
      gate_up_pass<KIND, G, NT, TU::D2, NW>(p, r, dot, j0, c0, c, list, red, wave, lane);
    };
    int c0 = 0;
    if constexpr (TU::NT > 2)
      for (; c - c0 > 32; c0 += 16 * TU::NT) pass(std::integral_constant<int, TU::NT>{}, c0);
    for (; c0 < c; c0 += 32) pass(std::integral_constant<int, 2>{}, c0);
  }
}

// ---------------------------------------------------------------- down
// One workgroup: 16 G output columns of one expert's slots, as gate_up: 145
// us, 71 us and 490 us for the calls above, at the same rates.
template <int KIND, int G, int NT, int D, int NW>
__device__ __forceinline__ void down_pass(const FewArgs& p, const Rows<G>& r, Dot<KIND, G, NT, D>& dot, int h0, int c0, int c,
                                          const uint16_t* list, float* red, int wave, int lane) {
  uint32_t xoff[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = c0 + n * 16 + (lane & 15);
    xoff[n] = i < c ? (uint32_t)list[i] * (uint32_t)(p.I * Unit<KIND>::XSZ) : kPast;
  }
  f32x4 acc[G][NT];
  zero<G, NT>(acc);
  dot.run(r, rsrc(p.a), xoff, wave, NW, p.I, lane, acc);
  constexpr int RT = NT < RED_NT ? NT : RED_NT;
#pragma unroll
  for (int n0 = 0; n0 < NT; n0 += RT) {
    put_partial<G, NT, RT>(red, wave, lane, acc, n0);
    lds_sync();
    for (int o = threadIdx.x; o < 16 * G * 16 * RT; o += NW * 64) {
      const int j = o % (16 * G), t = o / (16 * G), i = c0 + n0 * 16 + t;
      if (i < c && h0 + j < p.H) {
        const int s = list[i];
        p.y[(size_t)s * p.H + h0 + j] = p.w[s] * get_sum<G, RT, NW>(red, j >> 4, j & 15, t);
      }
    }
    lds_sync();
  }
}

template <int KIND>
__global__ __launch_bounds__(Tune<KIND>::NW * 64, Tune<KIND>::OCC) void few_down_kernel(FewArgs p) {
  using TU = Tune<KIND>;
  constexpr int G = TU::G, NW = TU::NW;
  extern __shared__ char few_lds[];
  __shared__ int cnt[NW];
  __shared__ __align__(16) float red[NW * G * RED_NT * 256];
  uint16_t* list = (uint16_t*)few_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = expert_of(p);
  if ((unsigned)e >= (unsigned)p.E) return;
  const int h0 = blockIdx.x * 16 * G;
  const int c = find_slots<NW>(p, e, list, cnt);
  if (not_mine(p, c, list)) return;
  Rows<G> r;
  Scales<NW * 64> scales;
  uint8_t* sc = (uint8_t*)few_lds + ((2 * p.S + 15) & ~15);
  down_rows<KIND, G>(p, e, h0, lane, sc, r, scales);
  if constexpr (KIND == W_MX) scales.fetch(threadIdx.x);
  if (c <= 16) {
    Dot<KIND, G, 1, TU::D1> dot;
    dot.start(r, wave, NW, p.I, lane);
    if constexpr (KIND == W_MX) {
      scales.store(sc, threadIdx.x);
      lds_sync();
    }
    down_pass<KIND, G, 1, TU::D1, NW>(p, r, dot, h0, 0, c, list, red, wave, lane);
  } else {
    if constexpr (KIND == W_MX) {
      scales.store(sc, threadIdx.x);
      lds_sync();
    }
    const auto pass = [&](auto n, int c0) {
      constexpr int NT = decltype(n)::value;
      Dot<KIND, G, NT, TU::D2> dot;
      dot.start(r, wave, NW, p.I, lane);
      down_pass<KIND, G, NT, TU::D2, NW>(p, r, dot, h0, c0, c, list, red, wave, lane);
    };
    int c0 = 0;
    if constexpr (TU::NT > 2)
      for (; c - c0 > 32; c0 += 16 * TU::NT) pass(std::integral_constant<int, TU::NT>{}, c0);
    for (; c0 < c; c0 += 32) pass(std::integral_constant<int, 2>{}, c0);
  }
}

// ---------------------------------------------------------------- sum over k
// out[t] = the sum over k, in k order, of the valid slots' rows (fp32): a launch
// and a trip to L2, 5 us at 16 tokens of 2880 (0.8 MB).
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void few_combine_kernel(FewArgs p) {
  const int chunks = p.H / 4;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T * chunks) return;
  const int t = i / chunks, c = i - t * chunks;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < p.K; ++k) {
    const int s = t * p.K + k;
    if ((unsigned)p.ids[s] < (unsigned)p.E) v += *(const f32x4*)(p.y + (size_t)s * p.H + 4 * c);
  }
  if (OUT_BF16)
    store4<uint16_t>((uint16_t*)p.out + (size_t)t * p.H + 4 * c, v[0], v[1], v[2], v[3]);
  else
    store4<float>((float*)p.out + (size_t)t * p.H + 4 * c, v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------- one token
// One token's slots are K experts' rows with one column, so no list is
// needed; its two kernels are the whole layer.  128 experts of 2880 x 2880,
// top-4, from logits: bf16 29 us for 133 MB (4.6 TB/s) and 17 us for 66 MB (3.9
// TB/s), 4-bit 13 and 9 us.  Neither rate is the memory's.  A wave of 4-bit
// weights has one unit in flight and waits for it 6 times in the gate_up kernel
// and 12 times in the down kernel (K of 2880), and the down kernel's 180
// workgroups leave 76 of the 256 CUs idle; how much of the time is those waits
// and how much the launches' start and end has not been measured.
//
// The choice from logits: an expert's rank is the number of better ones (a
// larger logit, or an equal one with a lower id; NaN is never chosen), counted
// by every workgroup for itself from LDS, which costs less than a launch.
// The weights follow the router's arithmetic: exp(l_k - l_0) summed in k order.
template <int NT_>
__device__ __forceinline__ void choose_one(const FewArgs& p, float* lg, int* ids, float* top) {
  for (int e = threadIdx.x; e < p.E; e += NT_) lg[e] = p.logits[e];
  for (int e = p.E + threadIdx.x; e < ((p.E + 3) & ~3); e += NT_) lg[e] = -__builtin_inff();
  for (int k = threadIdx.x; k < p.K; k += NT_) ids[k] = -1;
  lds_sync();
  for (int e = threadIdx.x; e < p.E; e += NT_) {
    const float v = lg[e];
    int rank = 0;
    for (int o = 0; o < p.E; o += 4) {
      const f32x4 q = *(const f32x4*)(lg + o);
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += (int)(q[i] > v) | ((int)(q[i] == v) & (int)(o + i < e));
    }
    if (v == v && rank < p.K) {
      ids[rank] = e;
      top[rank] = v;
    }
  }
  lds_sync();
}

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64, 4) void few_one_gate_up_kernel(FewArgs p) {
  using T = typename Elem<KIND>::T;
  constexpr int G = 2;
  constexpr int D = KIND == W_MX ? 1 : 2;
  extern __shared__ char few_lds[];
  __shared__ __align__(16) float red[NW * G * 16];
  __shared__ int ids[64];
  __shared__ float top[64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  int e;
  if (p.logits) {
    choose_one<NW * 64>(p, (float*)few_lds, ids, top);
    e = __builtin_amdgcn_readfirstlane(ids[blockIdx.y]);
    if (first && (int)threadIdx.x < p.K) {
      const int k = threadIdx.x;
      float denom = 0.f, z = 0.f;
      for (int q = 0; q < p.K; ++q) {
        const float zq = ids[q] >= 0 ? expf(top[q] - top[0]) : 0.f;
        denom += zq;
        if (q == k) z = zq;
      }
      p.ids_out[k] = ids[k];
      p.w_out[k] = ids[k] >= 0 ? z / denom : 0.f;
    }
  } else {
    e = __builtin_amdgcn_readfirstlane(p.ids[blockIdx.y]);
  }
  if (first && wave == 0) {
    const int id = lane < p.K ? (p.logits ? ids[lane] : p.ids[lane]) : 0;
    const uint64_t bad = __ballot((unsigned)id >= (unsigned)p.E);
    if (lane == 0) p.status[0] = __popcll(bad);
  }
  if ((unsigned)e >= (unsigned)p.E) return;
  const int j0 = blockIdx.x * 16;
  Rows<G> r;
  Scales<NW * 64> scales;
  uint8_t* sc = (uint8_t*)few_lds;
  gate_up_rows<KIND, G>(p, e, j0, lane, sc, r, scales);
  if constexpr (KIND == W_MX) scales.fetch(threadIdx.x);
  Dot<KIND, G, 1, D> dot;
  dot.start(r, wave, NW, p.H, lane);
  if constexpr (KIND == W_MX) {
    if (p.logits) lds_sync();   // every thread is past the logits there
    scales.store(sc, threadIdx.x);
    lds_sync();
  }
  const uint32_t xoff[1] = {(lane & 15) == 0 ? 0u : kPast};
  f32x4 acc[G][1];
  zero<G, 1>(acc);
  dot.run(r, rsrc(p.X), xoff, wave, NW, p.H, lane, acc);
  if ((lane & 15) == 0) {
#pragma unroll
    for (int h = 0; h < G; ++h) *(f32x4*)(red + (wave * G + h) * 16 + 4 * (lane >> 4)) = acc[h][0];
  }
  lds_sync();
  if (threadIdx.x < 16 && j0 + (int)threadIdx.x < p.I) {
    float gv = 0.f, uv = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      gv += red[(w * G) * 16 + threadIdx.x];
      uv += red[(w * G + 1) * 16 + threadIdx.x];
    }
    store_val<T>((T*)p.a + (size_t)blockIdx.y * p.I + j0 + threadIdx.x, glu_fwd(gv, uv, p.act, p.limit, p.alpha));
  }
}

// One workgroup: 16 output columns over all K slots.  The waves are split
// over the slots, and over k where there are more waves than slots.
template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64, 4) void few_one_down_kernel(FewArgs p) {
  using T = typename Elem<KIND>::T;
  constexpr int D = KIND == W_MX ? 1 : 2;
  extern __shared__ char few_lds[];
  __shared__ __align__(16) float red[NW * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = p.K < NW ? NW / p.K : 1, groups = NW / split;
  const int h0 = blockIdx.x * 16;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < p.K; s0 += groups) {
    const int s = s0 + wave / split;
    const int e = s < p.K && wave < split * groups ? __builtin_amdgcn_readfirstlane(p.ids[s]) : -1;
    const bool ok = (unsigned)e < (unsigned)p.E;
    Rows<1> r;
    Scales<64> scales;   // each slot's scales by the waves that share it
    uint8_t* sc = (uint8_t*)few_lds + (wave / split) * 16 * (p.I / 32);
    Dot<KIND, 1, 1, D> dot;
    if (ok) {
      down_rows<KIND, 1>(p, e, h0, lane, sc, r, scales);
      if constexpr (KIND == W_MX)
        if (wave % split == 0) scales.fetch(lane);
      dot.start(r, wave % split, split, p.I, lane);
    }
    if constexpr (KIND == W_MX) {
      if (s0) lds_sync();
      if (ok && wave % split == 0) scales.store(sc, lane);
      lds_sync();
    }
    if (!ok) continue;
    const float w = p.w[s];
    const uint32_t xoff[1] = {(lane & 15) == 0 ? (uint32_t)s * (uint32_t)(p.I * Unit<KIND>::XSZ) : kPast};
    f32x4 acc[1][1];
    zero<1, 1>(acc);
    dot.run(r, rsrc(p.a), xoff, wave % split, split, p.I, lane, acc);
    sum += w * acc[0][0];
  }
  if ((lane & 15) == 0) *(f32x4*)(red + wave * 16 + 4 * (lane >> 4)) = sum;
  lds_sync();
  if (threadIdx.x < 16 && h0 + (int)threadIdx.x < p.H) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w * 16 + threadIdx.x];
    store_val<T>((T*)p.out + h0 + threadIdx.x, v);
  }
}

template <int KIND>
hipError_t launch_one(const FewArgs& p, hipStream_t stream) {
  constexpr int NW = 4, NWD = KIND == W_MX ? 8 : 16;
  const size_t lg = p.logits ? (size_t)((p.E + 3) & ~3) * sizeof(float) : 0;
  const size_t gs = KIND == W_MX ? (size_t)32 * (p.H / 32) : 0;
  const size_t lds = lg > gs ? lg : gs;
  const size_t dsc = KIND == W_MX ? (size_t)16 * (p.K < NWD ? p.K : NWD) * (p.I / 32) : 0;
  const hipError_t err = run_kernel(KIND == W_MX ? "few_mx_gate_up" : "few_gate_up", stream, [&] {
    few_one_gate_up_kernel<KIND, NW><<<dim3((p.I + 15) / 16, p.K), NW * 64, lds, stream>>>(p);
  });
  if (err != hipSuccess) return err;
  return run_kernel(KIND == W_MX ? "few_mx_down" : "few_down", stream, [&] {
    few_one_down_kernel<KIND, NWD><<<(p.H + 15) / 16, NWD * 64, dsc, stream>>>(p);
  });
}

template <int KIND>
hipError_t launch(const FewArgs& p, hipStream_t stream) {
  using TU = Tune<KIND>;
  hipError_t err;
  if (p.T == 1) return launch_one<KIND>(p, stream);
  if (p.logits) {
    err = launch_topk(p.logits, p.T, p.K, p.E, p.ids_out, p.w_out, stream);
    if (err != hipSuccess) return err;
  }
  const size_t list = ((size_t)p.S * sizeof(uint16_t) + 15) & ~15;
  const auto lds = [&](int K) { return list + (KIND == W_MX ? (size_t)16 * TU::G * (K / 32) : 0); };
  const int gy = p.S < p.E ? p.S : p.E;
  err = run_kernel(KIND == W_MX ? "few_mx_gate_up" : "few_gate_up", stream, [&] {
    few_gate_up_kernel<KIND><<<dim3((p.I + 8 * TU::G - 1) / (8 * TU::G), gy), TU::NW * 64, lds(p.H), stream>>>(p);
  });
  if (err != hipSuccess) return err;
  err = run_kernel(KIND == W_MX ? "few_mx_down" : "few_down", stream, [&] {
    few_down_kernel<KIND><<<dim3((p.H + 16 * TU::G - 1) / (16 * TU::G), gy), TU::NW * 64, lds(p.I), stream>>>(p);
  });
  if (err != hipSuccess) return err;
  return run_kernel("few_combine", stream, [&] {
    const int grid = (p.T * (p.H / 4) + 255) / 256;
    if (KIND == W_F32) few_combine_kernel<false><<<grid, 256, 0, stream>>>(p);
    else few_combine_kernel<true><<<grid, 256, 0, stream>>>(p);
  });
}

}  // namespace

hipError_t launch_few(int kind, const FewArgs& p, hipStream_t stream) {
  switch (kind) {
    case W_BF16: return launch<W_BF16>(p, stream);
    case W_F32: return launch<W_F32>(p, stream);
    default: return launch<W_MX>(p, stream);
  }
}

}  // namespace moe
