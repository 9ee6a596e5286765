// The choice of the dense products' tiles, and their launches.
#pragma once
#include <type_traits>

#include "dense.h"

namespace moe {
namespace dense {

// ------------------------------------------------------------------ tiles
// Kernels exist for these tiles (rows x columns / 64, stages).  Time of a step
// of 64 k and of a tile's start and end in us, as timed with 256 workgroups
// that fill the card (T11 and T22: two a CU, so per pair of them).
struct TileKind {
  int fm, fn, stages, per_cu;
  float step, ends;
};
constexpr TileKind kTiles[] = {
    {4, 4, 2, 1, 1.77f, 8.f}, {4, 3, 2, 1, 1.25f, 7.f}, {3, 3, 3, 1, 0.92f, 6.f}, {2, 2, 2, 2, 0.96f, 5.f}, {1, 1, 4, 2, 0.38f, 4.f},
};
constexpr int N_TILES = 5;

// The kind of tile that an M x N product over K, `batch` times, is done with
// soonest: rounds of workgroups over 256 CUs times the time of one.
inline int tile_kind(long M, long N, long K, long batch = 1) {
  int best = 0;
  float least = 0.f;
  for (int i = 0; i < N_TILES; ++i) {
    const TileKind& k = kTiles[i];
    const long tiles = batch * ((M + 64 * k.fm - 1) / (64 * k.fm)) * ((N + 64 * k.fn - 1) / (64 * k.fn));
    const float nk = (float)((K + 63) / 64);
    // a CU with one of the small tiles takes about half a pair's time
    const long slots = 256 * k.per_cu;
    const float one = k.per_cu == 2 && tiles <= 256 ? 0.5f : 1.f;
    const float t = (float)((tiles + slots - 1) / slots) * (nk * k.step * one + k.ends);
    if (i == 0 || t < least) best = i, least = t;
  }
  return best;
}

// Calls launch(Cfg) for a tile kind.
template <class F>
inline void with_tile(int kind, F launch) {
  switch (kind) {
    case 0: return launch(Cfg<4, 4, 2>{});
    case 1: return launch(Cfg<4, 3, 2>{});
    case 2: return launch(Cfg<3, 3, 3>{});
    case 3: return launch(Cfg<2, 2, 2>{});
    default: return launch(Cfg<1, 1, 4>{});
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
    const long side = (S + 64 * k.fm - 1) / (64 * k.fm), tiles = batch * side * (side + 1) / 2, slots = 256 * k.per_cu;
    const float one = k.per_cu == 2 && tiles <= 256 ? 0.5f : 1.f;
    const float t = (float)((tiles + slots - 1) / slots) * ((float)((K + 63) / 64) * k.step * one + k.ends);
    if (best < 0 || t < least) best = i, least = t;
  }
  return best;
}
template <class F>
inline void with_square_tile(int kind, F launch) {
  switch (kind) {
    case 0: return launch(Cfg<4, 4, 2>{});
    case 2: return launch(Cfg<3, 3, 3>{});
    case 3: return launch(Cfg<2, 2, 2>{});
    default: return launch(Cfg<1, 1, 4>{});
  }
}

}  // namespace dense
}  // namespace moe
