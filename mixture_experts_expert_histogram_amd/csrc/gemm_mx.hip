// Grouped products on microscaled 4-bit expert weights, for more tokens than
// the few-token kernels take: the gate_up projection with its activation and
// the down projection with the routing weight, over the routed positions.
//
// One workgroup (4 waves) computes 128 positions x 256 weight rows of one
// expert on v_mfma_f32_32x32x16_bf16, 128 x 64 a wave, fp32 accumulators.
//
// * The weights go from global memory straight to registers as codes: a lane
//   holds 64 consecutive k of one weight row per 128-k stage (32 bytes, two
//   scales), and each 8 of them become a bf16 fragment by four conversions
//   that apply the scale (exact).  No two waves share weight rows, so LDS
//   would only add a copy, and a wave's 128 rows of activations per converted
//   fragment keep the conversions at a quarter of the matrix cores' time.
// * The activations (4 times the weights' bytes per element) are shared by the
//   4 waves through LDS, two stages of 128 k moved by buffer loads to LDS.
//   Lane half g of a fragment takes k = 64 g + 8 q of the stage in step q,
//   where the lane's weight codes are.
// * Rows past an expert's positions, weight rows past the matrix and k past
//   its end are loads past their buffer's end, which give zeros.
// * A tile's 32-row blocks without a position are skipped (the count is the
//   same for all waves), so a tile of few rows costs few products.
// * A stage's loads are issued one stage ahead; two workgroups a CU cover each
//   other's waits.
#include "gemm_mx.h"
#include "mx.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_vp;

constexpr uint32_t kPast = 0x80000000u;   // byte offset past every buffer

struct MxCfg {
  static constexpr int BM = 128, BN = 256, BK = 128, NW = 4, NT = NW * 64;
  static constexpr int WTM = 128, WTN = 64, FM = 4, FN = 2;
  static constexpr int SUB = BM * 64;   // elements of a 64-k half of a stage
  static constexpr int NB = BM / 8 / NW;   // 1 KB loads of a wave per 64-k half (8 rows of 128 bytes)
};
using C = MxCfg;

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

// A 64-k half tile is [row][64] with 16-byte chunk c of row r at slot
// c ^ ((r / 2) % 8): 16 lanes that read one chunk of 16 consecutive rows hit
// 16 bank groups.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// The activation rows of a tile: load j of wave w covers rows 8 (w NB + j) ..
// +8 of a half; off[j] is this lane's row in bytes (kPast: no such row).
struct ActRows {
  u32x4_t rs;
  uint32_t off[C::NB];
  int kc[C::NB];   // first k of this lane's chunk within a half
  __device__ __forceinline__ void issue(int kt, int K, uint16_t* stage, int wave) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) {
        const int k = kt * C::BK + h * 64 + kc[j];
        dma16(rs, k < K && off[j] != kPast ? off[j] + 2 * k : kPast, stage + h * C::SUB + (wave * C::NB + j) * 512);
      }
  }
};

// The weight rows of a wave: fragment f's row lane % 32; off / soff in bytes
// from the tile's first gate (f = 0) and up (f = 1) row, or output row.
struct WRows {
  __amdgpu_buffer_rsrc_t w[2], s[2];
  uint32_t off[2], soff[2];
};
// One stage of a wave's weights: 64 k a lane (two 16-byte loads) and the two scales.
// A row of an odd number of blocks ends with a lane that has one: its scale
// comes as a byte of its own (t), so that no byte past the row is read.
struct WStage {
  u32x4_t c[2][2];
  uint32_t s[2], t[2];
};
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void load_weights(const WRows& r, int kt, int nb, int lane, WStage& st) {
  const int b = kt * 4 + 2 * (lane >> 5);   // this lane's first block of 32 k
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    st.c[f][0] = load16(r.w[f], b < nb ? r.off[f] + b * 16 : kPast);
    st.c[f][1] = load16(r.w[f], b + 1 < nb ? r.off[f] + b * 16 + 16 : kPast);
    st.s[f] = __builtin_amdgcn_raw_buffer_load_b16(r.s[f], b + 1 < nb ? r.soff[f] + b : kPast, 0, 0);
    st.t[f] = 0;
    if (nb & 1) st.t[f] = __builtin_amdgcn_raw_buffer_load_b8(r.s[f], b + 1 == nb ? r.soff[f] + b : kPast, 0, 0);
  }
}

// acc += one stage, for the tile's first NF blocks of 32 rows.
template <int NF>
__device__ __forceinline__ void stage_products(const uint16_t* stage, const WStage& st, f32x16 (&acc)[C::FM][C::FN],
                                               int lane) {
  const uint16_t* half = stage + (lane >> 5) * C::SUB;
  const int r32 = lane & 31;
  float sc[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const uint32_t s = st.s[f] | st.t[f];
    sc[f][0] = mx_scale(s & 255);
    sc[f][1] = mx_scale(s >> 8 & 255);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    bf16x8_t a[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int row = i * 32 + r32;
      a[i] = *(const bf16x8_t*)(half + row * 64 + ((q ^ swz(row)) << 3));
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const uint32_t code = st.c[f][q >> 2][q & 3];
      const bf16x8_t b = mx_expand(code, sc[f][q >> 2]);
#pragma unroll
      for (int i = 0; i < NF; ++i) acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a[i], acc[i][f], 0, 0, 0);
    }
  }
}

template <int NF>
__device__ __forceinline__ void mainloop(const ActRows& ar, const WRows& wr, int K, uint16_t* lds,
                                         f32x16 (&acc)[C::FM][C::FN], int wave, int lane) {
  constexpr int STAGE = 2 * C::SUB;
  const int nb = K >> 5, nk = (nb + 3) >> 2;
  WStage st[2];
  load_weights(wr, 0, nb, lane, st[0]);
  ar.issue(0, K, lds, wave);
  for (int kt = 0; kt < nk; kt += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (kt + u < nk) {
        __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0): the stage's own loads and the last one's reads
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + u + 1 < nk) {
          load_weights(wr, kt + u + 1, nb, lane, st[1 - u]);
          ar.issue(kt + u + 1, K, lds + (1 - u) * STAGE, wave);
        }
        stage_products<NF>(lds + u * STAGE, st[u], acc, lane);
      }
    }
  }
}

template <bool GATE_UP>
__global__ __launch_bounds__(C::NT, 2) void mx_gemm_kernel(MxArgs p) {
  __shared__ __align__(1024) uint16_t lds[2 * 2 * C::SUB];
  const GArgs& g = p.g;
  int e, m0, rows, nt;
  if (!row_tile<C::BM>(g, e, m0, rows, nt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = GATE_UP ? g.H : g.I;
  ActRows ar;
  ar.rs = buffer_words(GATE_UP ? g.A : (const void*)((const uint16_t*)g.A + (size_t)m0 * g.I));
#pragma unroll
  for (int j = 0; j < C::NB; ++j) {
    const int row = (wave * C::NB + j) * 8 + (lane >> 3);
    ar.kc[j] = ((lane & 7) ^ swz(row)) * 8;
    const uint32_t r = row < rows ? (GATE_UP ? (uint32_t)g.tok_of_pos[m0 + row] : (uint32_t)row) : 0u;
    ar.off[j] = row < rows ? r * (uint32_t)(K * 2) : kPast;
  }
  WRows wr;
  const int n0 = GATE_UP ? nt * (C::BN / 2) + wave * 32 : nt * C::BN + wave * 64;   // the wave's first column
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    if (GATE_UP) {
      const size_t at = (size_t)p.gu_es * e + (size_t)p.gu_rs * min(n0, g.I - 1);
      const int j = min(n0 + (lane & 31), g.I - 1) - min(n0, g.I - 1);
      wr.w[f] = buffer_of((const char*)(f ? p.gu_u : p.gu_g) + at);
      wr.s[f] = buffer_of((const char*)(f ? p.gus_u : p.gus_g) + at / 16);
      wr.off[f] = (uint32_t)(p.gu_rs * j);
    } else {
      const size_t rb = g.I / 2;
      const size_t at = ((size_t)g.H * e + min(n0, g.H - 1)) * rb;
      const int j = min(n0 + f * 32 + (lane & 31), g.H - 1) - min(n0, g.H - 1);
      wr.w[f] = buffer_of((const char*)p.Wd + at);
      wr.s[f] = buffer_of((const char*)p.sd + at / 16);
      wr.off[f] = (uint32_t)(rb * j);
    }
    wr.soff[f] = wr.off[f] / 16;
  }
  f32x16 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int f = 0; f < C::FN; ++f)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][f][v] = 0.f;
  const int nf = (rows + 31) >> 5;
  if (nf > 2) mainloop<4>(ar, wr, K, lds, acc, wave, lane);
  else if (nf == 2) mainloop<2>(ar, wr, K, lds, acc, wave, lane);
  else mainloop<1>(ar, wr, K, lds, acc, wave, lane);
  if (GATE_UP) epi_gate_up<C, uint16_t, true, false>(g, acc, m0, rows, nt * (C::BN / 2), 0, wave, lane);
  else epi_down<C>(g, acc, m0, rows, nt * C::BN, 0, wave, lane);
}

}  // namespace

hipError_t launch_mx_gate_up(const GemmProblem& pb, const MxWeights& w, const void* X, void* a, hipStream_t s) {
  MxArgs p = {};
  p.g = base_args(pb, C::BM);
  p.g.A = X;
  p.g.out0 = a;
  p.g.ntn = (pb.I + C::BN / 2 - 1) / (C::BN / 2);
  p.gu_g = w.gu_g; p.gu_u = w.gu_u; p.gus_g = w.gus_g; p.gus_u = w.gus_u;
  p.gu_es = w.gu_es; p.gu_rs = w.gu_rs;
  return run_kernel("mx_gate_up", s, [&] {
    mx_gemm_kernel<true><<<(int)row_grid(pb, C::BM, p.g.ntn), C::NT, 0, s>>>(p);
  });
}

hipError_t launch_mx_down(const GemmProblem& pb, const MxWeights& w, const void* a, float* Yp, hipStream_t s) {
  MxArgs p = {};
  p.g = base_args(pb, C::BM);
  p.g.A = a;
  p.g.out0 = Yp;
  p.g.ntn = (pb.H + C::BN - 1) / C::BN;
  p.Wd = w.Wd; p.sd = w.sd;
  return run_kernel("mx_down", s, [&] {
    mx_gemm_kernel<false><<<(int)row_grid(pb, C::BM, p.g.ntn), C::NT, 0, s>>>(p);
  });
}

}  // namespace moe
