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
//   128-byte lines) through rings of NSA and NSB stages of 64 k.
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
//
// Bound by the card's power in large products: 8192 x 4096 over 16384 takes 757
// us (1452 TFLOP/s) with the matrix cores 87 % busy at 1.56 GHz, where matrix
// instructions alone, on random operands, reach 1830 TFLOP/s at 1.89 GHz (2400
// on zeros).  Instructions of 16 x 16 results drew the same power.
#pragma once
#include <type_traits>

#include "gemm_common.h"

namespace moe {
namespace dense {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_vp_t;

constexpr uint32_t kNone = 0x80000000u;   // byte offset past every buffer: loads zero

// Tile of FM x FN (times 64), rings of NSA and NSB stages for A and B.
template <int FM_, int FN_, int NSA_, int NSB_>
struct Cfg {
  static constexpr int FM = FM_, FN = FN_, NSA = NSA_, NSB = NSB_, BK = 64;
  static constexpr int BM = 64 * FM, BN = 64 * FN, NT = 256;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, LDS = NSA * A_BYTES + NSB * B_BYTES;
  static constexpr int NBA = 2 * FM, NBB = 2 * FN, PER = NBA + NBB;   // loads of a wave and step
  static_assert(NSA >= 3 && NSB >= 2 && NSA >= NSB && LDS <= 160 * 1024, "the rings fit in LDS");
};

__device__ __forceinline__ u32x4 buffer(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) & 0xffffu, kNone, 0x00027000u};
}

// 16 bytes a lane from byte off + soff of the buffer to LDS at byte dst + 16 lane.  In one asm
// block (the load has no output register) so that the compiler does not wait
// for every load in flight before each transposing LDS read; the mainloop
// waits for them itself.
__device__ __forceinline__ void load_lds(u32x4 rs, uint32_t off, uint32_t soff, uint32_t dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, %3 offen lds"
      :
      : "v"(off), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(dst)), "s"(soff)
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
  __device__ __forceinline__ void begin(int) {}
  // load j of the step whose first k is k0; FULL: all of its 64 k exist
  template <bool FULL>
  __device__ __forceinline__ void issue(int j, int k0, int K, uint32_t dst, int wave) const {
    const u32x4 b = rs[TWO ? j & 1 : 0];
    dst += (wave * NB + j) * 1024;
    if constexpr (FULL) load_lds(b, off[j], k0 * 2, dst);
    else load_lds(b, k0 + (kl ^ ((j & 1) << 5)) < K ? off[j] + k0 * 2 : kNone, 0, dst);
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
  __device__ __forceinline__ void begin(int k0) { rs = buffer(base + (size_t)(k0 >> 6) * step); }
  template <bool FULL>
  __device__ __forceinline__ void issue(int j, int k0, int K, uint32_t dst, int wave) const {
    const int q = wave * NB + j;
    if constexpr (FULL) load_lds(rs, off[j], 0, dst + q * 1024);
    else load_lds(rs, k0 + (q & 7) * 8 + (int)((threadIdx.x & 63) >> 3) < K ? off[j] : kNone, 0, dst + q * 1024);
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
  // fragment i of slice kk of the stage at byte `stage` of this side
  template <typename V>
  __device__ __forceinline__ V read(const lds_char* lds, int stage, int kk, int i) const {
    uint32_t o = off[MN ? i : kk];
    if (stage >= 49152) {   // past what an instruction's offset reaches: one addition for all of a slice's reads
      o += stage;
      asm("" : "+v"(o));
      stage = 0;
    }
    if constexpr (MN) {
      const lds_char* p = lds + o + (stage + kk * 2048);
      struct { s16x4_t h[2]; } r;
      r.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      r.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 512));
      return __builtin_bit_cast(V, r);
    } else {
      typedef __attribute__((address_space(3))) const V lds_v;
      return *(lds_v*)(lds + o + (stage + i * 4096));
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
//
// Step t, with barrier B_t in its middle:
//
//   slices 0, 1: their products, reads of slices 2, 3, loads of A(t - 1 + NSA)
//   B_t:         own reads of step t and own loads of step t + 1 are done
//   slices 2, 3: their products, reads of step t + 1's slices 0, 1, loads of B(t + NSB)
//
// so A(t - 1 + NSA) goes where A(t - 1) was, which B_{t-1} saw read, and
// B(t + NSB) where B(t) was.  A ring one longer for A than for B keeps every
// load at least half a step ahead of its wait while they are issued evenly: a
// load occupies the path to LDS for 16 cycles, and all of them behind one half
// of the products held the waves up (8192^3: 1203 TFLOP/s).
template <class C, typename V, class AS, class BS>
__device__ __forceinline__ void mainloop(AS& as, BS& bs, int K, char* lds_mem, f32x16 (&acc)[C::FM][C::FN], int wave,
                                         int lane) {
  constexpr int FM = C::FM, FN = C::FN, NSA = C::NSA, NSB = C::NSB, NP = FM * FN, NR = FM + FN;
  // loads that may be in flight at B_t and before the first reads: those issued behind step t + 1's (step 0's)
  constexpr int FLIGHT = NSA > NSB ? (NSB - 2) * C::PER + C::NBA : (NSA - 2) * C::PER;
  constexpr int FIRST = NSA > NSB ? (NSB - 1) * C::PER : (NSA - 2) * C::PER + C::NBB;
  const lds_char* lds = (const lds_char*)lds_mem;
  const uint32_t at = (uint32_t)(uintptr_t)(lds_vp_t)lds_mem;
  const int wm = wave >> 1, wn = wave & 1;
  FragSrc<FM, AS::MN> fa;
  FragSrc<FN, BS::MN> fb;
  fa.init(0, wm * 32 * FM, lane);
  fb.init(NSA * C::A_BYTES, wn * 32 * FN, lane);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  const int nk = (K + 63) >> 6;
  // load n of A or B of step t into its ring position s
  const auto load_a = [&](auto full, int n, int t, int s) {
    as.template issue<decltype(full)::value>(n, t << 6, K, at + s * C::A_BYTES, wave);
  };
  const auto load_b = [&](auto full, int n, int t, int s) {
    bs.template issue<decltype(full)::value>(n, t << 6, K, at + NSA * C::A_BYTES + s * C::B_BYTES, wave);
  };
#pragma unroll
  for (int q = -NSA; q < 0; ++q) {   // in the order in which the steps would have issued them
    if (q + NSB >= 0) {
      bs.begin(min(q + NSB, nk - 1) << 6);
#pragma unroll
      for (int n = 0; n < C::NBB; ++n) load_b(std::false_type{}, n, q + NSB, q + NSB);
    }
    if (q < -1) {
      as.begin(min(q + NSA, nk - 1) << 6);
#pragma unroll
      for (int n = 0; n < C::NBA; ++n) load_a(std::false_type{}, n, q + NSA, q + NSA);
    }
  }
  V a[4][FM], b[4][FN];
  const auto read = [&](int n, int kk, int sa, int sb) {   // fragment n of a slice
    if (n < FM) a[kk][n] = fa.template read<V>(lds, sa * C::A_BYTES, kk, n);
    else b[kk][n - FM] = fb.template read<V>(lds, sb * C::B_BYTES, kk, n - FM);
  };
  __builtin_amdgcn_s_waitcnt(wait_vm(FIRST));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int n = 0; n < NR; ++n) read(n, kk, 0, 0);

  // u: t modulo the rings' lengths.  A product takes the matrix core 32 cycles,
  // 8 issue slots of the wave: reads go one behind each of a slice's first
  // products, loads evenly behind all.
  const auto step = [&](auto full, int t, int u) {
    const int sa = u % NSA, sb = u % NSB;
    as.begin(min(t - 1 + NSA, nk - 1) << 6);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk == 2) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_vm(FLIGHT));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        bs.begin(min(t + NSB, nk - 1) << 6);
        __builtin_amdgcn_sched_barrier(0);
      }
      constexpr int LA = FM, LB = FN;   // loads of a slice
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = p / FN, j = (i & 1) ? FN - 1 - p % FN : p % FN;
        acc[i][j] = mma32(b[kk][j], a[kk][i], acc[i][j]);
#pragma unroll
        for (int n = 0; n < NR; ++n)
          if (n * NP / (2 * NR) == p) read(n, (kk + 2) & 3, kk < 2 ? sa : (sa + 1) % NSA, kk < 2 ? sb : (sb + 1) % NSB);
        if (kk < 2) {
#pragma unroll
          for (int n = 0; n < LA; ++n)
            if ((2 * n + 1) * NP / (2 * LA) == p) load_a(full, kk * LA + n, t - 1 + NSA, (sa + NSA - 1) % NSA);
        } else {
#pragma unroll
          for (int n = 0; n < LB; ++n)
            if ((2 * n + 1) * NP / (2 * LB) == p) load_b(full, (kk - 2) * LB + n, t + NSB, sb);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  constexpr int U = NSA % NSB == 0 ? NSA : NSA * NSB;   // steps after which both rings are back
  int t = 0;
  for (; (t + U + (NSA - 1 > NSB ? NSA - 1 : NSB)) * 64 <= K; t += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) step(std::true_type{}, t + u, u);
  }
  for (; t + U <= nk; t += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) step(std::false_type{}, t + u, u);
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (t + u < nk) step(std::false_type{}, t + u, u);
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
// Tile t of an mtiles x ntiles grid, in groups of 4 row tiles, column by column:
// 32 consecutive ones are 4 row tiles by 8 column tiles.  With 8 by 4 the
// columns' operand came round later than the memory side cache kept it
// (8192 x 16384 x 4096: 1024 us against 837; 2 by 16 815, but slower at long k).
__device__ __forceinline__ void tile_at(int t, int mtiles, int ntiles, int& mt, int& nt) {
  const int per = 4 * ntiles, grp = t / per, rem = t - grp * per;
  const int gm = min(4, mtiles - grp * 4);
  nt = rem / gm;
  mt = grp * 4 + rem - nt * gm;
}
__device__ __forceinline__ bool tile_of(int w, int mtiles, int ntiles, int& mt, int& nt) {
  const int t = deal(w, mtiles * ntiles);
  if (t >= 0) tile_at(t, mtiles, ntiles, mt, nt);
  return t >= 0;
}
inline int tile_grid(long mtiles, long ntiles) { return deal_grid(mtiles * ntiles); }

}  // namespace dense
}  // namespace moe
