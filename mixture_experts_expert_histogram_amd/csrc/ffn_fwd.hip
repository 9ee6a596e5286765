// Forward products of the gated feed-forward block:
//
//   a = phi(x Wg^T, x Wu^T),   out = add + sigmoid(gate) (a Wd^T)
//
// a is rounded to bf16 as the second product's operand (2.35e-3 from 64 bits in
// the 2-norm, 1.66e-3 by the output's own rounding); the gate and up values are
// kept in fp32 for the backward pass.
#include "ffn_tiles.h"

namespace moe {
namespace dense {

// Tile rows of B take gate and up rows in turns of 8, so that accumulator
// groups v / 4 = 0, 2 are gate and 1, 3 up values of the same 8 columns and phi
// needs no exchange between lanes.  8192 tokens, H 4096, I 8192, gate and up
// values kept: 857 us (1283 TFLOP/s; matrix cores 74 % busy, for the tiles' ends
// store 1.2 GB with nothing beside them).  512 tokens, H 4096, I 2048: 24 us
// (728 TFLOP/s), bound by what reaches LDS from L2 (about 20 TB/s in small tiles).
// ACT: 0 swiglu, 1 clamped; A, Z: which results are written
template <class C, int ACT, bool A, bool Z>
__global__ __launch_bounds__(256, 1) void ffn_gate_up_kernel(FfnArgs p) {
  FFN_PROLOGUE(C)
  const int j0 = nt * (C::BN / 2);
  KSrc<C::NBA> as;
  KSrc<C::NBB, true> bs;
  init_rows(as, p.x, m0, p.T, p.H, wave, lane);
  const long at = p.gu_rs * j0;
  bs.init((const uint16_t*)p.gu_g + at, (const uint16_t*)p.gu_u + at,
          [&](int r) { return (uint32_t)(min(((r >> 4) << 3) + (r & 7), p.I - 1 - j0) * (int)p.gu_rs * 2); }, wave, lane);
  mainloop<C, bf16x8_t>(as, bs, p.H, lds, acc, wave, lane);
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row0 = m0 + wm * 32 * C::FM + 32 * i, row = row0 + (lane & 31);
    if (row0 >= p.T) break;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int c = j0 + (wn * C::FN + j) * 16;
      if (c >= p.I) break;
      float av[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float g[4], u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = acc[i][j][8 * q + e];
          u[e] = acc[i][j][8 * q + 4 + e];
          if (A) av[q][e] = glu_fwd_t<ACT>(g[e], u[e], p.limit, p.alpha);
        }
        if (Z && c + 8 * q < p.I) {
          *(float4*)z_block(p.z, row0, c + 8 * q, p.I, 0, lane) = make_float4(g[0], g[1], g[2], g[3]);
          *(float4*)z_block(p.z, row0, c + 8 * q, p.I, 1, lane) = make_float4(u[0], u[1], u[2], u[3]);
        }
      }
      if (A) {
        const u32x4 v = pack_pair(av[0], av[1]);
        const int cc = c + 8 * (lane >> 5);
        if (row < p.T && cc < p.I) *(u32x4*)((uint16_t*)p.a + (size_t)row * p.I + cc) = v;
      }
    }
  }
}

// 8192 tokens, H 4096, I 8192: 392 us (1402 TFLOP/s, matrix cores 83 % busy); 512
// tokens, H 4096, I 2048: 16 us.  What add holds is loaded 8 fragments ahead.
template <class C>
__global__ __launch_bounds__(256, 1) void ffn_down_kernel(FfnArgs p) {
  FFN_PROLOGUE(C)
  KSrc<C::NBA> as;
  KSrc<C::NBB> bs;
  init_rows(as, p.a, m0, p.T, p.I, wave, lane);
  init_rows(bs, p.wd, n0, p.H, p.I, wave, lane);
  mainloop<C, bf16x8_t>(as, bs, p.I, lds, acc, wave, lane);
  const int r0 = m0 + wm * 32 * C::FM + (lane & 31), c00 = n0 + wn * 32 * C::FN, c4 = 4 * (lane >> 5);
  float s[C::FM];
#pragma unroll
  for (int i = 0; i < C::FM; ++i) s[i] = row_gate(p.gate, min(r0 + 32 * i, p.T - 1));
  struct Add { uint2 v[4]; };
  each_fragment<C, Add, 8>(
      [&](int i, int j, Add& ad) __attribute__((always_inline)) {   // rows and columns past the last read the last one
        if (!p.add) return;
        const uint16_t* row = (const uint16_t*)p.add + (size_t)min(r0 + 32 * i, p.T - 1) * p.H;
#pragma unroll
        for (int v = 0; v < 4; ++v) ad.v[v] = *(const uint2*)(row + min(c00 + 32 * j + 8 * v, p.H - 8) + c4);
      },
      [&](int i, int j, const Add& ad) __attribute__((always_inline)) {
        const int row = r0 + 32 * i;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = e < 2 ? ad.v[2 * q + h].x : ad.v[2 * q + h].y;
              const float x = s[i] * acc[i][j][8 * q + 4 * h + e];
              v[h][e] = p.add ? x + __builtin_bit_cast(float, e & 1 ? w & 0xffff0000u : w << 16) : x;
            }
          const u32x4 o = pack_pair(v[0], v[1]);
          const int cc = c00 + 32 * j + 16 * q + 2 * c4;
          if (row < p.T && cc < p.H) *(u32x4*)((uint16_t*)p.out + (size_t)row * p.H + cc) = o;
        }
      });
}

template <class C, bool A, bool Z>
hipError_t run_gate_up(const FfnArgs& p, hipStream_t s) {
  const auto k = p.act && A ? ffn_gate_up_kernel<C, 1, A, Z> : ffn_gate_up_kernel<C, 0, A, Z>;
  return run_kernel("ffn_gate_up", s, [&] { k<<<tile_grid(p.mt, p.nt), C::NT, 0, s>>>(p); });
}

}  // namespace dense

using namespace dense;

hipError_t launch_ffn_gate_up(FfnArgs p, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.T, 2 * p.I, p.H), [&](auto c) {
    using C = decltype(c);
    p.mt = (p.T + C::BM - 1) / C::BM;
    p.nt = (2 * p.I + C::BN - 1) / C::BN;
    e = !p.z ? run_gate_up<C, true, false>(p, s) : p.a ? run_gate_up<C, true, true>(p, s) : run_gate_up<C, false, true>(p, s);
  });
  return e;
}

hipError_t launch_ffn_down(FfnArgs p, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.T, p.H, p.I), [&](auto c) {
    using C = decltype(c);
    p.mt = (p.T + C::BM - 1) / C::BM;
    p.nt = (p.H + C::BN - 1) / C::BN;
    const auto k = ffn_down_kernel<C>;
    e = run_kernel("ffn_down", s, [&] { k<<<tile_grid(p.mt, p.nt), C::NT, 0, s>>>(p); });
  });
  return e;
}

}  // namespace moe
