// Workgroup -> (K slice, row tile, column tile) of a tiled product, and the sum of its K slices.
#pragma once

#include "device_common.h"

namespace awq {

struct TileAt {
  uint32_t slice, tm, tn;
};

// Each XCD (workgroup number % 8, its own L2) takes a run of consecutive tiles. Tiles are ordered
// slice-major and in bands of BAND row tiles, so that the 32 or 64 tiles an XCD works on at a time
// share BAND row panels and a few column panels. Every tile is taken once for any grid size.
template <uint32_t BAND>
__device__ __forceinline__ TileAt tile_order(uint32_t tilesM, uint32_t tilesN) {
  const uint32_t xcd = blockIdx.x & 7u, per = gridDim.x >> 3, rem = gridDim.x & 7u;
  const uint32_t id = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const uint32_t tiles = tilesM * tilesN;
  const uint32_t slice = id / tiles;
  const uint32_t tile = id - slice * tiles;
  const uint32_t band = tile / (BAND * tilesN), in_band = tile - band * BAND * tilesN;
  const uint32_t left = tilesM - band * BAND, bh = left < BAND ? left : BAND;
  const uint32_t tn = in_band / bh;
  // the divisions run on the vector unit: say that the results are the same in every lane
  TileAt t;
  t.slice = __builtin_amdgcn_readfirstlane(slice);
  t.tn = __builtin_amdgcn_readfirstlane(tn);
  t.tm = __builtin_amdgcn_readfirstlane(band * BAND + (in_band - tn * bh));
  return t;
}

// Four values of S slices, `stride` floats apart, added in slice order; eight slices' loads in
// flight.
__device__ __forceinline__ floatx4 sum_slices(const float* P, int S, int64_t stride) {
  constexpr int kC = 8;
  floatx4 t = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < S; j0 += kC) {
    floatx4 v[kC];
#pragma unroll
    for (int u = 0; u < kC; ++u)
      v[u] = *reinterpret_cast<const floatx4*>(P + (j0 + u < S ? j0 + u : 0) * stride);
#pragma unroll
    for (int u = 0; u < kC; ++u)
      if (j0 + u < S) t = (j0 + u == 0) ? v[u] : t + v[u];
  }
  return t;
}

}  // namespace awq
