// Tiles of rows sorted by expert, found by the block that takes one.
#pragma once

#include <algorithm>

#include "ops.h"

namespace ds4 {

// The expert and the run of its rows that row tile `tile` of the call covers:
// an expert with n rows has ceil(n / bm) tiles, in the experts' order.
// Offsets are held within [0, n] and taken as empty where they descend, so a
// bad one reads and writes nothing out of range.
struct RowTile {
  int e, lo, cnt;  // rows lo .. lo + cnt - 1 (cnt <= bm)
};
__device__ inline RowTile find_tile(const int32_t* offsets, int E, int n, int bm, int tile, int* lds) {
  RowTile r{0, tile * bm, min(bm, n - tile * bm)};
  if (!offsets) return r;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int per = (E + blockDim.x - 1) / blockDim.x, e0 = tid * per;
  int tiles = 0;
  for (int i = 0; i < per; ++i) {
    if (e0 + i >= E) break;
    const int lo = min(max(offsets[e0 + i], 0), n), hi = min(max(offsets[e0 + i + 1], 0), n);
    tiles += hi > lo ? (hi - lo + bm - 1) / bm : 0;
  }
  int x = tiles;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) lds[wave] = x;
  if (tid == 0) lds[8] = -1;
  __syncthreads();
  int first = x - tiles;
  for (int w = 0; w < nw; ++w)
    if (w < wave) first += lds[w];
  if (tile >= first && tile < first + tiles) {
    int left = tile - first;
    for (int i = 0; i < per; ++i) {
      const int lo = min(max(offsets[e0 + i], 0), n), hi = min(max(offsets[e0 + i + 1], 0), n);
      const int m = hi > lo ? (hi - lo + bm - 1) / bm : 0;
      if (left < m) {
        lds[8] = e0 + i;
        lds[9] = lo + left * bm;
        lds[10] = min(bm, hi - lo - left * bm);
        break;
      }
      left -= m;
    }
  }
  __syncthreads();
  r.e = lds[8];
  r.lo = lds[9];
  r.cnt = r.e < 0 ? 0 : lds[10];
  return r;
}

// Row tiles a call can have at most.
inline int64_t max_tiles(int64_t n, int E, bool grouped, int bm) {
  if (!grouped) return (n + bm - 1) / bm;
  return std::min<int64_t>(n, n / bm + std::min<int64_t>(E, n));
}

}  // namespace ds4
