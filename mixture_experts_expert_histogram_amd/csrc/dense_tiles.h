// Pieces of the dense products' epilogues, and the choice of their tiles.
#pragma once
#include <type_traits>
#include <utility>

#include "dense.h"

namespace moe {
namespace dense {

// Four fp32 values each of two 4-column groups (columns c .. and c + 8 .. of a
// row, c = 4 (lane / 32)) as bf16, so that every lane ends with 8 consecutive
// columns: lanes below 32 columns 0 .. 7, the others 8 .. 15 of the 16.
__device__ __forceinline__ u32x4 pack_pair(const float* lo, const float* hi) {
  const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(lo[0], lo[1]), pack_bf16(hi[0], hi[1]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(lo[2], lo[3]), pack_bf16(hi[2], hi[3]), false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}

// A wave's FM x FN result fragments in turn, use(i, j, r) with what fetch(i, j,
// r) loaded for each DEPTH fragments earlier, so that an epilogue waits for
// memory once and not once a fragment.
template <class C, class R, int D, class Fetch, class Use, int... F>
__device__ __forceinline__ void each_fragment_of(Fetch fetch, Use use, std::integer_sequence<int, F...>) {
  R ring[D];
#pragma unroll
  for (int f = 0; f < D; ++f) fetch(f / C::FN, f % C::FN, ring[f]);
  __builtin_amdgcn_sched_barrier(0);
  ([&]() __attribute__((always_inline)) {   // not a loop: every index into the results has to be a constant
    use(F / C::FN, F % C::FN, ring[F % D]);
    if constexpr (F + D < (int)sizeof...(F)) fetch((F + D) / C::FN, (F + D) % C::FN, ring[F % D]);
    __builtin_amdgcn_sched_barrier(0);
  }(), ...);
}
template <class C, class R, int DEPTH, class Fetch, class Use>
__device__ __forceinline__ void each_fragment(Fetch fetch, Use use) {
  constexpr int N = C::FM * C::FN;
  each_fragment_of<C, R, (DEPTH < N ? DEPTH : N)>(fetch, use, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------------------ tiles
// Kernels exist for these tiles (rows x columns / 64).  Times in us of a step
// of 64 k with one workgroup a CU and with per_cu of them, and of a tile's
// start and end, from products that fill the card's rounds (8192 x 4096 x 8192:
// 398 us on 256 x 256 tiles, 455 on 256 x 192; 4096 x 2880 x 5760: 130 and 110;
// 5760 x 2880 x 4096: 185 on 256 x 256, 135 on 192 x 192; 512 x 4096 x 4096: 27
// on 128 x 128, 24 on 128 x 64, 26 on 64 x 64; 130 x 4096 x 4096: 24, 20, 13).
struct TileKind {
  int fm, fn, per_cu;
  float solo, full, ends;
};
constexpr TileKind kTiles[] = {
    {4, 4, 1, 1.50f, 1.50f, 8.f}, {4, 3, 1, 1.17f, 1.17f, 7.f}, {3, 3, 1, 0.92f, 0.92f, 6.f},
    {2, 2, 1, 0.45f, 0.45f, 4.f}, {2, 1, 2, 0.31f, 0.57f, 4.f}, {1, 1, 2, 0.155f, 0.34f, 3.5f},
};
constexpr int N_TILES = 6;

// Time of `tiles` tiles of a kind over K: rounds of 256 CUs; fewer workgroups
// than CUs each run faster (clocks and memory are shared by fewer: 144 tiles of
// 256 x 256 took 0.83 of a round's time, 64 of 128 x 128 0.73).
inline float tile_time(const TileKind& k, long tiles, long K) {
  const float nk = (float)((K + 63) / 64);
  if (tiles <= 256) return (nk * k.solo + k.ends) * (0.65f + 0.35f * (float)tiles / 256.f);
  const long slots = 256 * k.per_cu;
  return (float)((tiles + slots - 1) / slots) * (nk * k.full + k.ends);
}

// The kind of tile that an M x N product over K, `batch` times, is done with
// soonest, of those from `first` on whose tiles a launch holds (the entry points
// refuse calls whose tiles of the first kind are too many).
inline int tile_kind(long M, long N, long K, long batch = 1, int first = 0) {
  int best = first;
  float least = 0.f;
  for (int i = first; i < N_TILES; ++i) {
    const TileKind& k = kTiles[i];
    const long tiles = batch * ((M + 64 * k.fm - 1) / (64 * k.fm)) * ((N + 64 * k.fn - 1) / (64 * k.fn));
    const float t = tile_time(k, tiles, K);
    if (i == first || (t < least && tiles <= MAX_TILES)) best = i, least = t;
  }
  return best;
}

// Calls launch(Cfg) for a tile kind.
template <class F>
inline void with_tile(int kind, F launch) {
  switch (kind) {
    case 0: return launch(Cfg<4, 4, 3, 2>{});
    case 1: return launch(Cfg<4, 3, 3, 2>{});
    case 2: return launch(Cfg<3, 3, 3, 3>{});
    case 3: return launch(Cfg<2, 2, 3, 3>{});
    case 4: return launch(Cfg<2, 1, 3, 3>{});
    default: return launch(Cfg<1, 1, 5, 5>{});
  }
}

// The same for the square kinds, over the tiles on and above the diagonal of
// `batch` symmetric S x S products.
inline int square_tile_kind(long S, long K, long batch) {
  int best = -1;
  float least = 0.f;
  for (int i = 0; i < N_TILES; ++i) {
    const TileKind& k = kTiles[i];
    if (k.fm != k.fn) continue;
    const long side = (S + 64 * k.fm - 1) / (64 * k.fm), tiles = batch * side * (side + 1) / 2;
    const float t = tile_time(k, tiles, K);
    if (best < 0 || (t < least && tiles <= MAX_TILES)) best = i, least = t;
  }
  return best;
}
template <class F>
inline void with_square_tile(int kind, F launch) {
  switch (kind) {
    case 0: return launch(Cfg<4, 4, 3, 2>{});
    case 2: return launch(Cfg<3, 3, 3, 3>{});
    case 3: return launch(Cfg<2, 2, 3, 3>{});
    default: return launch(Cfg<1, 1, 5, 5>{});
  }
}

}  // namespace dense
}  // namespace moe
