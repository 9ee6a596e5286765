// Grouped products on microscaled 4-bit expert weights, for the calls that the
// few-token kernels do not take (more than 128 tokens, many slots an expert,
// long rows; the rule is in api.cpp): the gate_up projection with its activation
// and the down projection with the routing weight, over the routed positions.
//
// The activation is rounded to bf16, the second product's operand type; every
// sum and the down product's rows are fp32.
//
// One workgroup (4 waves) computes BM = 32 or 64 positions x 256 weight
// rows of one expert on v_mfma_f32_16x16x32_bf16, BM x 64 a wave, fp32
// accumulators.
//
// * The weights go from global memory straight to registers as codes, one or
//   two cache lines (256 or 512 k, a "line" below) of each of a wave's 64 rows
//   at a time and one such line ahead.  A load covers 16 rows x 64 bytes: lane
//   group g = lane / 16 holds block g of its row's 4 (32 x 32 tiles would take
//   32 rows x 32 bytes a load, which cost the loads' path twice the cache
//   lines).  Each 8 codes become a bf16 fragment by four conversions that apply
//   the scale (exact).  No two waves share weight rows, so LDS would only add a
//   copy.  Rows that do not start on a cache line (H = 2880: 1440 bytes) share
//   their end lines between successive loads, and a tile's lines are evicted
//   from L2 before the next load comes: 1.5 times the weights' bytes at 256 k,
//   1.27 at 512, which the 32-position tiles have the registers for (512
//   tokens 442 -> 430 us).
// * The scales of the tile's rows go to LDS before the loop, in whole runs of
//   rows: loaded from global memory a lane a block, they touch as many cache
//   lines as the codes do.
// * The activations (4 times the weights' bytes per element) are shared by the
//   4 waves through LDS, two stages of 128 k moved by buffer loads to LDS.
//   Lane group g takes k 32 g + 8 q of a stage in step q, where its codes are.
// * Rows past an expert's positions, weight rows past the matrix and k past
//   its end are loads past their buffer's end, which give zeros.
// * A tile's 16-row blocks without a position are skipped (the count is the
//   same for all waves), so a tile of few rows costs few products.
// * Two workgroups a CU cover each other's waits.
//
// Measured (gate_up, down; us and what the memory system did):
//   512 tokens, top-4, 128 experts of 2880 x 2880: 254, 140; HBM 5.8 and 4.8
//     TB/s, the loads' path busy 87 and 77 %, matrix cores 18 and 16 %
//   2048, top-8, 256 of 4096 x 2048: 647, 395; 4.2 and 3.3 TB/s, 89 and 87 %,
//     41 and 33 %
//   4096, top-4, 128 of 2880 x 2880: 581, 333; 2.9 and 2.6 TB/s, 84 and 81 %,
//     46 and 41 %
// Copies that left a part out showed the conversions to be hidden (4096 tokens
// 980 us of 985) and the weights' loads to cost most (784 without those after
// the first line, 836 without those of activations), so what bounds it is the
// loads' latency and path.  Loading the next line at once in one stage
// instead of over the line's stages (1010 us), or between the products instead
// of before them (989 to 1003), was slower, as were 8 waves of 32 rows (1001).
#include <atomic>
#include <type_traits>

#include "gemm_mx.h"
#include "mx.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_vp;

constexpr uint32_t kPast = 0x80000000u;   // byte offset past every buffer

template <int BM_>
struct MxCfg {
  static constexpr int BM = BM_, BN = 256, BK = 128, NW = 4, NT = NW * 64;
  static constexpr int FM = BM / 16, FN = 4;   // 16 x 16 blocks of a wave: positions, weight rows
  static constexpr int HALF = BM * 64;     // elements of a stage's 64-k half
  static constexpr int NB = BM / 8 / NW;   // 1 KB loads of a wave per half (8 rows of 128 bytes)
  static constexpr int LS = BM == 32 ? 4 : 2;   // stages whose codes of a row are loaded together
  // Waves a SIMD that the registers allow for: 231 of 256 with 32 positions, 254
  // (down) and 256 (gate_up) with 64, where two values are spilled around one of
  // the loops and none inside a loop.
  static constexpr int OCC = 2;
};

// A raw buffer of 2^31 bytes at p (wave-uniform) as its four descriptor words.
__device__ __forceinline__ u32x4_t buffer_words(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) & 0xffffu, kPast, 0x00027000u};
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), 0, (int)kPast, 0x00027000);
}

// 16 bytes a lane from the buffer at off to LDS at dst + 16 lane; zeros where
// off lies past the buffer.  One asm block, untracked by the compiler: the
// stage loop waits for it (vmcnt) before its barrier.
__device__ __forceinline__ void dma16(u32x4_t rs, uint32_t off, uint16_t* dst) {
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_vp)dst;
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(off), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(lds))
      : "memory", "m0");
}

// A 64-k half is [row][64] with 16-byte chunk c of row r at slot
// c ^ ((r / 2) % 8): 16 lanes that read one chunk of 16 consecutive rows hit
// 16 bank groups.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// The activation rows of a tile: load j of wave w covers rows 8 (w NB + j) ..
// +8; off[j] is this lane's row in bytes (kPast: no such row).
template <class C>
struct ActRows {
  u32x4_t rs;
  uint32_t off[C::NB];
  int kc[C::NB];   // first k of this lane's chunk within a half
  __device__ __forceinline__ void issue(int s, int K, uint16_t* stage, int wave) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) {
        const int k = s * C::BK + h * 64 + kc[j];
        dma16(rs, k < K && off[j] != kPast ? off[j] + 2 * k : kPast, stage + h * C::HALF + (wave * C::NB + j) * 512);
      }
  }
};

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The weight rows of a wave, 4 groups of 16 (gate_up: gate, gate, up, up):
// row lane % 16 of group f, off in bytes from the tile's first gate (up) row or
// output row, sc its scales in bytes from the start of the tile's in LDS.
struct WRows {
  __amdgpu_buffer_rsrc_t w[2];
  uint32_t off[4], sc[4];
};
// LS stages' codes of each row: c[f][j] is the lane's block 4 j + g of them.
template <int LS>
struct WLine {
  u32x4_t c[4][LS];
};
// Part J of line t: 4 / LS of the groups.
template <bool GATE_UP, int LS>
__device__ __forceinline__ void load_line(const WRows& r, int part, int t, int nb, int lane, WLine<LS>& w) {
#pragma unroll
  for (int f = 4 / LS * part; f < 4 / LS * (part + 1); ++f)
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      const int b = t * 4 * LS + 4 * j + (lane >> 4);
      w.c[f][j] = load16(r.w[GATE_UP ? f >> 1 : 0], b < nb ? r.off[f] + b * 16 : kPast);
    }
}

// Place of scale byte a in LDS: 4 bytes stay free after each 128, or the 16
// rows of a read would hit one bank where a row has 128 scales.
__device__ __forceinline__ uint32_t scale_at(uint32_t a) { return a + (a >> 7) * 4; }
__device__ __forceinline__ void put_scales(uint8_t* lds, uint32_t a, u32x4_t v) {
  uint32_t* d = (uint32_t*)(lds + scale_at(a));   // a is a multiple of 16
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = v[i];
}

// The scale bytes of stage s for the wave's 4 groups.
__device__ __forceinline__ void read_scales(const uint8_t* scales, const WRows& r, int s, int nb, int lane, uint32_t (&sb)[4]) {
  const int b = min(4 * s + (lane >> 4), nb - 1);
#pragma unroll
  for (int f = 0; f < 4; ++f) sb[f] = scales[scale_at(r.sc[f] + b)];
}

// acc += a stage (128 k), for the tile's first NF blocks of 16 positions, in
// steps of 32 k: a step's activations are read from LDS one step ahead, and
// issue() (the next stage's loads) runs behind the first read.  sb holds the
// stage's scale bytes and, afterwards, the next stage's.
template <class C, int NF, class Issue>
__device__ __forceinline__ void stage_products(const uint16_t* stage, const uint8_t* scales, const WRows& r,
                                               const WLine<C::LS>& w, int j, int s, int nb, uint32_t (&sb)[4],
                                               f32x4 (&acc)[C::FM][C::FN], int lane, Issue issue) {
  const int r16 = lane & 15, g = lane >> 4;
  const uint16_t* half = stage + (g >> 1) * C::HALF;
  bf16x8_t a[2][NF];
  auto read = [&](int q, bf16x8_t (&to)[NF]) {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int row = i * 16 + r16;
      to[i] = *(const bf16x8_t*)(half + row * 64 + (((4 * (g & 1) + q) ^ swz(row)) << 3));
    }
  };
  read(0, a[0]);
  issue();
  float sc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) sc[f] = mx_scale(sb[f]);
  read_scales(scales, r, s + 1, nb, lane, sb);
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q < 3) read(q + 1, a[(q + 1) & 1]);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const bf16x8_t bw = mx_expand(w.c[f][j][q], sc[f]);
#pragma unroll
      for (int i = 0; i < NF; ++i)
        acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw, a[q & 1][i], acc[i][f], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_setprio(0);
}

constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }   // vmcnt <= n, lgkmcnt 0

// Stage s = LS t + J: the stage's activations have landed (they were issued one
// stage ago, before that stage's 4 weight loads: of those the first stage of a
// line needs the last ones itself, the others leave them in flight; at the
// loop's end, where some have no use and are not issued, nothing is counted on)
// and every wave is past its reads of the stage before, whose buffer the next
// stage's loads then fill (zeros, past the last stage).
template <class C, bool GATE_UP, int NF, int J, bool TAIL = false>
__device__ __forceinline__ void one_stage(const ActRows<C>& ar, const WRows& wr, const uint8_t* scales, int t, int nb,
                                          int K, uint16_t* lds, const WLine<C::LS>& cur, WLine<C::LS>& next,
                                          uint32_t (&sb)[4], f32x4 (&acc)[C::FM][C::FN], int wave, int lane) {
  const int s = C::LS * t + J;
  __builtin_amdgcn_s_waitcnt(wait_vm(J == 0 || TAIL ? 0 : 4));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  stage_products<C, NF>(lds + (J & 1) * 2 * C::HALF, scales, wr, cur, J, s, nb, sb, acc, lane, [&] {
    ar.issue(s + 1, K, lds + (~J & 1) * 2 * C::HALF, wave);
    load_line<GATE_UP>(wr, J, t + 1, nb, lane, next);
    asm volatile("" ::: "memory");   // the loads stay here: the next stage's wait counts them
    __builtin_amdgcn_sched_barrier(0);
  });
}

// The loop's body is two lines, without a branch: with a stage skipped on some
// path, the compiler has to take loads into a line's registers for still in
// flight wherever they are loaded again, and waits there for everything,
// the activations just issued among it.
template <class C, bool GATE_UP, int NF>
__device__ __forceinline__ void mainloop(const ActRows<C>& ar, const WRows& wr, const uint8_t* scales, int K, uint16_t* lds,
                                         WLine<C::LS>& l0, f32x4 (&acc)[C::FM][C::FN], int wave, int lane) {
  const int nb = K >> 5, ns = (nb + 3) >> 2;
  WLine<C::LS> l1;
  uint32_t sb[4];
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();   // every wave's scales are in LDS
  asm volatile("" ::: "memory");
  read_scales(scales, wr, 0, nb, lane, sb);
  const auto stage = [&](auto j, auto tail, int t, const WLine<C::LS>& cur, WLine<C::LS>& next) {
    one_stage<C, GATE_UP, NF, decltype(j)::value, decltype(tail)::value>(ar, wr, scales, t, nb, K, lds, cur, next, sb, acc, wave,
                                                                          lane);
  };
  using std::integral_constant;
  using no = std::false_type;
  using yes = std::true_type;
  int t = 0;
  for (; C::LS * (t + 2) <= ns; t += 2) {
    stage(integral_constant<int, 0>{}, no{}, t, l0, l1);
    stage(integral_constant<int, 1>{}, no{}, t, l0, l1);
    if constexpr (C::LS == 4) {
      stage(integral_constant<int, 2>{}, no{}, t, l0, l1);
      stage(integral_constant<int, 3>{}, no{}, t, l0, l1);
    }
    stage(integral_constant<int, 0>{}, no{}, t + 1, l1, l0);
    stage(integral_constant<int, 1>{}, no{}, t + 1, l1, l0);
    if constexpr (C::LS == 4) {
      stage(integral_constant<int, 2>{}, no{}, t + 1, l1, l0);
      stage(integral_constant<int, 3>{}, no{}, t + 1, l1, l0);
    }
  }
  // what is left: less than two lines, each stage behind the question whether it exists
  const int left = ns - C::LS * t;
  [&] {
    if (left < 1) return;
    stage(integral_constant<int, 0>{}, yes{}, t, l0, l1);
    if (left < 2) return;
    stage(integral_constant<int, 1>{}, yes{}, t, l0, l1);
    if constexpr (C::LS == 4) {
      if (left < 3) return;
      stage(integral_constant<int, 2>{}, yes{}, t, l0, l1);
      if (left < 4) return;
      stage(integral_constant<int, 3>{}, yes{}, t, l0, l1);
    }
    if (left <= C::LS) return;
    stage(integral_constant<int, 0>{}, yes{}, t + 1, l1, l0);
    if constexpr (C::LS == 4) {
      if (left < 6) return;
      stage(integral_constant<int, 1>{}, yes{}, t + 1, l1, l0);
      if (left < 7) return;
      stage(integral_constant<int, 2>{}, yes{}, t + 1, l1, l0);
    }
  }();
  __builtin_amdgcn_s_waitcnt(wait_vm(0));   // no load into LDS outlives the tile
}

// `bytes` bytes (a multiple of 16) of scales at p to LDS, from scale byte `to`.
template <int NTHREADS>
__device__ __forceinline__ void scales_to_lds(const char* p, uint32_t bytes, uint8_t* lds, uint32_t to) {
  const __amdgpu_buffer_rsrc_t b = buffer_of(p);
  uint32_t o = threadIdx.x * 16;
  for (; o + 3 * NTHREADS * 16 < bytes; o += 4 * NTHREADS * 16) {
    u32x4_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load16(b, o + i * NTHREADS * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) put_scales(lds, to + o + i * NTHREADS * 16, v[i]);
  }
  for (; o < bytes; o += NTHREADS * 16) put_scales(lds, to + o, load16(b, o));
}

template <class C, bool GATE_UP>
__global__ __launch_bounds__(C::NT, C::OCC) void mx_gemm_kernel(MxArgs p) {
  extern __shared__ __align__(1024) char mx_dyn[];   // two stages, then the scales
  uint16_t* lds = (uint16_t*)mx_dyn;
  uint8_t* scales = (uint8_t*)(lds + 4 * C::HALF);
  const GArgs& g = p.g;
  int e, m0, rows, nt;
  if (!row_tile<C::BM>(g, e, m0, rows, nt)) return;
  {   // an expert's tiles share its positions evenly, in blocks of 16: 72 on tiles of 64 are 48 and 24, not 64 and 8
    const int off = g.offsets[e], n = g.offsets[e + 1] - off, tiles = (n + C::BM - 1) / C::BM;
    const int share = ((n + tiles - 1) / tiles + 15) & ~15, mt = (m0 - off) / C::BM;
    m0 = off + mt * share;
    rows = min(share, n - mt * share);
    if (rows <= 0) return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = GATE_UP ? g.H : g.I, nb = K >> 5;
  WRows wr;
  WLine<C::LS> l0;
  // the tile's first column, its columns, and the wave's own
  constexpr int BC = GATE_UP ? C::BN / 2 : C::BN, WC = BC / C::NW;
  const int c0 = nt * BC, ncol = min(BC, (GATE_UP ? g.I : g.H) - c0);
  const size_t at = GATE_UP ? (size_t)p.gu_es * e + (size_t)p.gu_rs * c0 : ((size_t)g.H * e + c0) * (size_t)(g.I / 2);
  const uint32_t rs = GATE_UP ? (uint32_t)p.gu_rs : (uint32_t)(g.I / 2);   // bytes between columns' rows
  const bool inter = GATE_UP && p.gu_rs != K / 2;   // gate and up rows in turn: one run of scales
  wr.w[0] = buffer_of((const char*)(GATE_UP ? p.gu_g : p.Wd) + at);
  wr.w[1] = buffer_of((const char*)(GATE_UP ? p.gu_u : p.Wd) + at);
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int j = min(wave * WC + (GATE_UP ? f & 1 : f) * 16 + (lane & 15), ncol - 1);
    wr.off[f] = rs * (uint32_t)j;
    wr.sc[f] = nb * (GATE_UP ? (inter ? 2 * j + (f >> 1) : (f >> 1) * ncol + j) : j);
  }
#pragma unroll
  for (int part = 0; part < C::LS; ++part) load_line<GATE_UP>(wr, part, 0, nb, lane, l0);
  ActRows<C> ar;
  ar.rs = buffer_words(GATE_UP ? g.A : (const void*)((const uint16_t*)g.A + (size_t)m0 * g.I));
#pragma unroll
  for (int j = 0; j < C::NB; ++j) {
    const int row = (wave * C::NB + j) * 8 + (lane >> 3);
    ar.kc[j] = ((lane & 7) ^ swz(row)) * 8;
    const uint32_t r = row < rows ? (GATE_UP ? (uint32_t)g.tok_of_pos[m0 + row] : (uint32_t)row) : 0u;
    ar.off[j] = row < rows ? r * (uint32_t)(K * 2) : kPast;
  }
  const uint32_t run = (uint32_t)(ncol * nb);
  if (GATE_UP) {
    scales_to_lds<C::NT>((const char*)p.gus_g + at / 16, inter ? 2 * run : run, scales, 0);
    if (!inter) scales_to_lds<C::NT>((const char*)p.gus_u + at / 16, run, scales, run);
  } else {
    scales_to_lds<C::NT>((const char*)p.sd + at / 16, run, scales, 0);
  }
  ar.issue(0, K, lds, wave);
  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int f = 0; f < C::FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nf = (rows + 15) >> 4;
  auto loop = [&](auto n) { mainloop<C, GATE_UP, decltype(n)::value>(ar, wr, scales, K, lds, l0, acc, wave, lane); };
  using std::integral_constant;
  if constexpr (C::FM == 4) {
    if (nf == 4) loop(integral_constant<int, 4>{});
    else if (nf == 3) loop(integral_constant<int, 3>{});
    else if (nf == 2) loop(integral_constant<int, 2>{});
    else loop(integral_constant<int, 1>{});
  } else {
    if (nf == 2) loop(integral_constant<int, 2>{});
    else loop(integral_constant<int, 1>{});
  }
  // Accumulator element v of a lane: position 16 i + lane % 16, weight row 4
  // (lane / 16) + v of group f.
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = i * 16 + (lane & 15);
    if (row >= rows) continue;
    const size_t pos = (size_t)(m0 + row);
    if constexpr (GATE_UP) {
      uint32_t d[2][2];   // the 16 columns of group f, 4 a lane
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = glu_fwd(acc[i][f][k], acc[i][2 + f][k], g.act, g.limit, g.alpha);
        d[f][0] = pack_bf16(v[0], v[1]);
        d[f][1] = pack_bf16(v[2], v[3]);
      }
      // lanes of even 16s take their and the next 16s' columns of group 0, the others of group 1: 16 bytes each
      const auto x = __builtin_amdgcn_permlane16_swap(d[0][0], d[1][0], false, false);
      const auto y = __builtin_amdgcn_permlane16_swap(d[0][1], d[1][1], false, false);
      const int c = wave * WC + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
      if (c < ncol) *(u32x4_t*)((uint16_t*)g.out0 + pos * g.I + c0 + c) = u32x4_t{x[0], y[0], x[1], y[1]};
    } else {
      const float w = g.w_of_pos[pos];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int c = wave * WC + f * 16 + 4 * (lane >> 4);
        if (c < ncol) *(f32x4*)((float*)g.out0 + pos * g.H + c0 + c) = w * acc[i][f];
      }
    }
  }
}

// Two stages, and the tile's padded scales.
template <class C>
constexpr size_t mx_lds(int K) {
  const size_t sc = (size_t)C::BN * (K / 32);
  return 4 * C::HALF * sizeof(uint16_t) + sc + (sc >> 7) * 4 + 16;
}

template <class C, bool GATE_UP>
hipError_t launch(const GemmProblem& pb, MxArgs p, const char* name, hipStream_t s) {
  constexpr int BC = GATE_UP ? C::BN / 2 : C::BN;
  const int K = GATE_UP ? pb.H : pb.I, N = GATE_UP ? pb.I : pb.H;
  const GArgs b = base_args(pb, C::BM);
  p.g.offsets = b.offsets; p.g.tile_prefix = b.tile_prefix; p.g.tok_of_pos = b.tok_of_pos; p.g.w_of_pos = b.w_of_pos;
  p.g.T = b.T; p.g.H = b.H; p.g.I = b.I; p.g.E = b.E; p.g.K = b.K; p.g.S = b.S;
  p.g.act = b.act; p.g.layout = b.layout; p.g.limit = b.limit; p.g.alpha = b.alpha;
  p.g.ntn = (N + BC - 1) / BC;
  const size_t lds = mx_lds<C>(K);
  static std::atomic<uint64_t> raised{0};   // devices whose limit of dynamic LDS is raised
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev > 63 || !(raised.load() >> dev & 1)) {
    err = hipFuncSetAttribute((const void*)mx_gemm_kernel<C, GATE_UP>, hipFuncAttributeMaxDynamicSharedMemorySize,
                              MX_MAX_LDS);
    if (err != hipSuccess) return err;
    if (dev <= 63) raised.fetch_or(uint64_t(1) << dev);
  }
  return run_kernel(name, s, [&] {
    mx_gemm_kernel<C, GATE_UP><<<(int)row_grid(pb, C::BM, p.g.ntn), C::NT, lds, s>>>(p);
  });
}

// Tiles of 32 positions for experts of at most 16 on average, where reading
// the weights is all of the time (gpt-oss-shaped layer at 256 tokens, 8 an
// expert, 392 us against 413; 512 tokens 430 against 442), else of 64 (1024
// tokens 503 us against 516, 4096 tokens 0.98 ms against 1.14).  Tiles of
// 128 positions x 512 rows on 8 waves move a third less through the load path,
// but one workgroup a CU leaves its waits and its ends uncovered: 1.01 ms at
// 4096 tokens, 3.32 against 3.37 ms at 16384.  The average decides for every
// expert: with Zipf(1.2) routing, whose largest expert has 382 of 2048 slots
// (3063 of 16384), 512 tokens take 428 us (uniform 414) and 4096 1.00 ms (0.98).
template <bool GATE_UP>
hipError_t launch_by_rows(const GemmProblem& pb, const MxArgs& p, const char* name, hipStream_t s) {
  if ((long)pb.S <= 16L * pb.E) return launch<MxCfg<32>, GATE_UP>(pb, p, name, s);
  return launch<MxCfg<64>, GATE_UP>(pb, p, name, s);
}

}  // namespace

hipError_t launch_mx_gate_up(const GemmProblem& pb, const MxWeights& w, const void* X, void* a, hipStream_t s) {
  MxArgs p = {};
  p.g.A = X;
  p.g.out0 = a;
  p.gu_g = w.gu_g; p.gu_u = w.gu_u; p.gus_g = w.gus_g; p.gus_u = w.gus_u;
  p.gu_es = w.gu_es; p.gu_rs = w.gu_rs;
  return launch_by_rows<true>(pb, p, "mx_gate_up", s);
}

hipError_t launch_mx_down(const GemmProblem& pb, const MxWeights& w, const void* a, float* Yp, hipStream_t s) {
  MxArgs p = {};
  p.g.A = a;
  p.g.out0 = Yp;
  p.Wd = w.Wd; p.sd = w.sd;
  return launch_by_rows<false>(pb, p, "mx_down", s);
}

}  // namespace moe
