// The vocabulary's division over the CTAs and tiles of the streaming kernel.
#pragma once

#include <cuda_runtime.h>

namespace flce {

constexpr int TILE_ROWS = 256;
constexpr int UNIT_ROWS = 16;

// This CTA's tiles: units [u0, u1) of 16 rows, spread evenly over its tiles (a
// short last tile would fill the ring's stages with few bytes: one token at
// 4096 x 128256 177 us against 166).
struct Range {
  int u0, u1, tiles;
  __device__ __forceinline__ int start(int i) const {   // first row of tile i (also: the end of tile i - 1)
    const int n = u1 - u0;   // (a division of 64 bits takes several times one of 32)
    return (u0 + (n < (1 << 15) ? n * i / tiles : static_cast<int>(static_cast<long long>(n) * i / tiles))) * UNIT_ROWS;
  }
};

__device__ __forceinline__ Range range_of(int V, int ctas, int cta) {
  const unsigned units = (static_cast<unsigned>(V) + UNIT_ROWS - 1) / UNIT_ROWS, c = cta, n = ctas;
  Range r;
  if (units < (1u << 23) && n < (1u << 9)) {
    r.u0 = static_cast<int>(units * c / n);
    r.u1 = static_cast<int>(units * (c + 1) / n);
  } else {
    r.u0 = static_cast<int>(static_cast<unsigned long long>(units) * c / n);
    r.u1 = static_cast<int>(static_cast<unsigned long long>(units) * (c + 1) / n);
  }
  r.tiles = (r.u1 - r.u0 + TILE_ROWS / UNIT_ROWS - 1) / (TILE_ROWS / UNIT_ROWS);
  return r;
}

}  // namespace flce
