// Device pieces shared by the dense products of the feed-forward block.
#pragma once
#include "dense_tiles.h"
#include "ffn.h"

namespace moe {
namespace dense {

// Block of 32 rows x 8 columns of the saved gate (up = 0) and up values: 256
// floats, lane l's four at 4 l, the order in which the accumulators hold them,
// so that both passes move whole kilobytes.
__device__ __forceinline__ float* z_block(float* z, int row, int col, int I, int up, int lane) {
  return z + (((size_t)(row >> 5) * (I >> 3) + (col >> 3)) * 2 + up) * 256 + lane * 4;
}

__device__ __forceinline__ float row_gate(const float* gate, int row) { return gate ? 1.f / (1.f + expf(-gate[row])) : 1.f; }

// s (1 - s) from the logit: with s as it is rounded, 1 - s loses its digits where
// s is near one (0.5 % at a logit of 12, everything from 17.4 on).
__device__ __forceinline__ float gate_slope(float logit) {
  const float t = expf(-fabsf(logit)), u = 1.f + t;
  return t / (u * u);
}

// A workgroup's tile, its wave's place in it and the results.
#define FFN_PROLOGUE(C)                                                              \
  __shared__ __align__(1024) char lds[C::LDS];                             \
  int mt, nt;                                                                        \
  if (!tile_of(blockIdx.x, p.mt, p.nt, mt, nt)) return;                              \
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); \
  const int wm = wave >> 1, wn = wave & 1, m0 = mt * C::BM, n0 = nt * C::BN;         \
  f32x16 acc[C::FM][C::FN];

// Rows r0 .. of a matrix [rows][K] of bf16.
template <class S>
__device__ __forceinline__ void init_rows(S& s, const void* b, int r0, int rows, int K, int wave, int lane) {
  s.init((const uint16_t*)b + (size_t)r0 * K, nullptr, [&](int r) { return (uint32_t)(min(r, rows - 1 - r0) * K * 2); }, wave,
         lane);
}

}  // namespace dense
}  // namespace moe
