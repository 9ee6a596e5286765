// Mainloop of the dense products (feed-forward block, Newton-Schulz steps):
// one workgroup of 4 waves, one a SIMD, computes a 64 FM x 64 FN tile of
// A . B^T in FM x FN fragments of 32 x 32 a wave (2 x 2 waves).
//
// With 256 x 256 tiles a wave holds 128 x 128 results, so a k-step of 64
// reads 128 KB of operands out of LDS for 2048 cycles of matrix work, where 8
// waves of 128 x 64 read 192 KB.  One wave a SIMD has nobody to cover its
// waits, so the loop covers them itself:
//
// * Operands come straight into LDS (buffer loads to LDS, 1 KB a load, whole
//   128-byte lines) through a ring of NS stages of 64 k.
// * Fragments are read from LDS two slices of 16 k ahead of their products.
//   A stage is therefore read to its end half a step before its products are
//   done, and one barrier in the middle of a step stands for both "this stage
//   may be refilled" and "the next stage has landed" (every wave waits for its
//   own loads and reads before it).
// * Reads and loads are issued one at a time between the products.
//
// Operands contiguous along k are tiles [row][64 k]; operands contiguous
// along m or n (weights of an input gradient, both sides of a weight gradient)
// are panels [64 k][64 columns], read with ds_read_b64_tr_b16.  Both have rows
// of 128 bytes, whose 16-byte chunks are permuted against bank conflicts by
// permuting what each lane loads.  A k or a row that does not exist is read as
// zero (k) or as the last one (row, column; those results are not stored).
#pragma once
#include "gemm_common.h"

namespace moe {
namespace dense {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_vp_t;

constexpr uint32_t kNone = 0x80000000u;   // byte offset past every buffer: loads zero

template <int FM_, int FN_, int NS_>
struct Cfg {
  static constexpr int FM = FM_, FN = FN_, NS = NS_, BK = 64;
  static constexpr int BM = 64 * FM, BN = 64 * FN, NT = 256;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int NBA = 2 * FM, NBB = 2 * FN, PER = NBA + NBB;   // loads of a wave and step
  static_assert(NS * STAGE <= 160 * 1024, "the ring fits in LDS");
};

__device__ __forceinline__ u32x4 buffer(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) & 0xffffu, kNone, 0x00027000u};
}

// 16 bytes a lane from the buffer to LDS at byte dst + 16 lane.  In one asm
// block (the load has no output register) so that the compiler does not wait
// for every load in flight before each transposing LDS read; the mainloop
// waits for them itself.
__device__ __forceinline__ void load_lds(u32x4 rs, uint32_t off, uint32_t dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(off), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(dst))
      : "memory", "m0");
}

// s_waitcnt immediate: vmcnt <= n, lgkmcnt = 0 (gfx9 encoding).
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// An operand contiguous along k.  ROWS: where tile row r starts: a functor
// (r, side) -> byte offset from the buffer of its side; loads j and tile rows
// 8 (w NB + j) .. + 7 belong together, and side = j % 2 where there are two
// buffers (gate and up rows in turns of 8).
template <int NB, bool TWO = false>
struct KSrc {
  u32x4 rs[TWO ? 2 : 1];
  uint32_t off[NB];
  int kl;   // first k of this lane's chunk in a step
  template <class F>
  __device__ __forceinline__ void init(const void* b0, const void* b1, F row_off, int wave, int lane) {
    rs[0] = buffer(b0);
    if constexpr (TWO) rs[1] = buffer(b1);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int r = (wave * NB + j) * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ ((r >> 1) & 7);
      off[j] = row_off(r) + chunk * 16;
    }
    // (r / 2) % 8 of row 8 b + lane / 8 is 4 (b % 2) + lane / 16
    kl = ((lane & 7) ^ (lane >> 4)) * 8;
  }
  __device__ __forceinline__ void begin(int, int) {}
  // load j of the step whose first k is k0
  __device__ __forceinline__ void issue(int j, int k0, int K, uint32_t dst, int wave) const {
    const int k = k0 + (kl ^ ((j & 1) << 5));
    load_lds(rs[TWO ? j & 1 : 0], k < K ? off[j] + k0 * 2 : kNone, dst + (wave * NB + j) * 1024);
  }
  static constexpr bool MN = false;
};

// An operand contiguous along m or n: element (k, c) at base + k ld + c.
template <int NB>
struct CSrc {
  const char* base;
  u32x4 rs;
  uint32_t off[NB];
  uint32_t step;   // bytes of 64 k
  int kl[2];       // k of this lane's rows in a step: even and odd ... loads
  __device__ __forceinline__ void init(const void* b, long ld, int c0, int ncols, int wave, int lane) {
    base = (const char*)b;
    step = (uint32_t)(ld * 128);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int q = wave * NB + j;
      const int kr = (q & 7) * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ ((((kr >> 1) & 1) << 2) | (((kr >> 3) & 1) << 1));
      const int col = min(c0 + (q >> 3) * 64 + chunk * 8, ncols - 8);
      off[j] = (uint32_t)(kr * ld * 2) + col * 2;
    }
  }
  // the descriptor of the step whose first k is k0
  __device__ __forceinline__ void begin(int k0, int) { rs = buffer(base + (size_t)(k0 >> 6) * step); }
  __device__ __forceinline__ void issue(int j, int k0, int K, uint32_t dst, int wave) const {
    const int q = wave * NB + j;
    const int kr = (q & 7) * 8 + ((threadIdx.x & 63) >> 3);
    load_lds(rs, k0 + kr < K ? off[j] : kNone, dst + q * 1024);
  }
  static constexpr bool MN = true;
};

// Fragment reads of one side: F fragments of 32 rows (or columns) from tile row
// base on.  Fragment layout: lane -> row lane % 32, k = 8 (lane / 32) + 0 .. 7.
template <int F, bool MN>
struct FragSrc {
  uint32_t off[MN ? F : 4];
  __device__ __forceinline__ void init(uint32_t side, int base, int lane) {
    if constexpr (MN) {
      const int g = lane >> 4, s = lane & 15;
      const int kr = ((g >> 1) << 3) + (s >> 2);
      const int x = (((kr >> 1) & 1) << 2) | (((kr >> 3) & 1) << 1);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const int q = (base >> 5) + i;
        const int chunk = ((q & 1) << 2) + ((g & 1) << 1) + ((s & 3) >> 1);
        off[i] = side + (q >> 1) * 8192 + kr * 128 + ((chunk ^ x) << 4) + (s & 1) * 8;
      }
    } else {
      const int r = base + (lane & 31);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) off[kk] = side + r * 128 + (((kk * 2 + (lane >> 5)) ^ ((r >> 1) & 7)) << 4);
    }
  }
  // fragment i of slice kk of the stage at byte `stage` of lds
  template <typename V>
  __device__ __forceinline__ V read(const lds_char* lds, int stage, int kk, int i) const {
    if constexpr (MN) {
      const lds_char* p = lds + off[i] + (stage + kk * 2048);
      struct { s16x4_t h[2]; } r;
      r.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      r.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 512));
      return __builtin_bit_cast(V, r);
    } else {
      typedef __attribute__((address_space(3))) const V lds_v;
      return *(lds_v*)(lds + off[kk] + (stage + i * 4096));
    }
  }
};

__device__ __forceinline__ f32x16 mma32(bf16x8_t a, bf16x8_t b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f16x8_t a, f16x8_t b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// acc = A . B^T over K.  Accumulator element v of fragment (i, j) is tile row
// wm 32 FM + 32 i + lane % 32, column wn 32 FN + 32 j + acc_col4(v / 4, lane)
// + v % 4.  At the end every load and read of LDS is done, in all waves.
template <class C, typename V, class AS, class BS>
__device__ __forceinline__ void mainloop(AS& as, BS& bs, int K, char* lds_mem, f32x16 (&acc)[C::FM][C::FN], int wave,
                                         int lane) {
  constexpr int FM = C::FM, FN = C::FN, NS = C::NS, NP = FM * FN, NR = FM + FN;
  const lds_char* lds = (const lds_char*)lds_mem;
  const uint32_t at = (uint32_t)(uintptr_t)(lds_vp_t)lds_mem;
  const int wm = wave >> 1, wn = wave & 1;
  FragSrc<FM, AS::MN> fa;
  FragSrc<FN, BS::MN> fb;
  fa.init(0, wm * 32 * FM, lane);
  fb.init(C::A_BYTES, wn * 32 * FN, lane);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  const int nk = (K + 63) >> 6;
  const auto issue = [&](int n, int k0, int stage) {   // load n of a step: A's, then B's
    if (n < C::NBA) as.issue(n, k0, K, at + stage, wave);
    else bs.issue(n - C::NBA, k0, K, at + stage + C::A_BYTES, wave);
  };
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    as.begin(min(s, nk - 1) << 6, K);
    bs.begin(min(s, nk - 1) << 6, K);
#pragma unroll
    for (int n = 0; n < C::PER; ++n) issue(n, s << 6, s * C::STAGE);
  }
  V a[4][FM], b[4][FN];
  const auto read = [&](int n, int kk, int stage) {   // fragment n of a slice
    if (n < FM) a[kk][n] = fa.template read<V>(lds, stage, kk, n);
    else b[kk][n - FM] = fb.template read<V>(lds, stage, kk, n - FM);
  };
  __builtin_amdgcn_s_waitcnt(wait_vm((NS - 1) * C::PER));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int n = 0; n < NR; ++n) read(n, kk, 0);

  // Step t on stage st (its ring position): products of slices 0 .. 3; reads
  // of slices 2, 3 and the next step's 0, 1; loads of step t + NS.
  const auto step = [&](int t, int st, int sn) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk == 2) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_vm((NS - 2) * C::PER));   // step t + 1 has landed, stage st is read
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        as.begin(min(t + NS, nk - 1) << 6, K);
        bs.begin(min(t + NS, nk - 1) << 6, K);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = p / FN, j = (i & 1) ? FN - 1 - p % FN : p % FN;
        acc[i][j] = mma32(b[kk][j], a[kk][i], acc[i][j]);
        // NR reads and, in the second half, PER / 2 loads of the slice spread over its products
#pragma unroll
        for (int n = p * NR / NP; n < (p + 1) * NR / NP; ++n) read(n, (kk + 2) & 3, kk < 2 ? st : sn);
        if (kk >= 2) {
#pragma unroll
          for (int n = p * NR / NP; n < (p + 1) * NR / NP; ++n) issue((kk - 2) * NR + n, (t + NS) << 6, st);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int t = 0;
  for (; t + NS <= nk; t += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) step(t + u, u * C::STAGE, (u + 1) % NS * C::STAGE);
  }
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (t + u < nk) step(t + u, u * C::STAGE, (u + 1) % NS * C::STAGE);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The tile of workgroup w out of `total`, or -1: dealt to the XCDs (workgroup w
// runs on XCD w % 8) in chunks of up to 32 consecutive tiles, which an XCD's 32
// CUs hold at once, sharing their operands in its L2.
__device__ __forceinline__ int deal(int w, int total) {
  const int chunk = min(32, (total + 7) >> 3);
  const int j = w >> 3;
  const int t = ((j / chunk) * 8 + (w & 7)) * chunk + j % chunk;
  return t < total ? t : -1;
}
// Workgroups that hold `total` tiles.
inline int deal_grid(long total) {
  const long chunk = (total + 7) / 8 < 32 ? (total + 7) / 8 : 32;
  return (int)((total + 8 * chunk - 1) / (8 * chunk) * (8 * chunk));
}
// Tile t of an mtiles x ntiles grid, in groups of 8 row tiles, column by column:
// 32 consecutive ones are 8 row tiles by 4 column tiles.
__device__ __forceinline__ void tile_at(int t, int mtiles, int ntiles, int& mt, int& nt) {
  const int per = 8 * ntiles, grp = t / per, rem = t - grp * per;
  const int gm = min(8, mtiles - grp * 8);
  nt = rem / gm;
  mt = grp * 8 + rem - nt * gm;
}
__device__ __forceinline__ bool tile_of(int w, int mtiles, int ntiles, int& mt, int& nt) {
  const int t = deal(w, mtiles * ntiles);
  if (t >= 0) tile_at(t, mtiles, ntiles, mt, nt);
  return t >= 0;
}
inline int tile_grid(long mtiles, long ntiles) { return deal_grid(mtiles * ntiles); }

}  // namespace dense
}  // namespace moe
