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
  int e, lo, cnt;  // rows lo .. lo + cnt - 1 (cnt <= bm; 0: no work)
  int part;        // which of the tile's column parts
};
// The tile and part of item `local` of an expert with m tiles: kPartGroup
// parts of all its tiles before the next parts, a tile's neighbouring parts
// next to each other.
constexpr int kPartGroup = 8;
__device__ inline void split_item(int local, int m, int parts, int& tile, int& part) {
  const int g = local / (m * kPartGroup), left = local - g * m * kPartGroup;
  const int wide = min(kPartGroup, parts - g * kPartGroup);
  tile = left / wide;
  part = g * kPartGroup + left - tile * wide;
}

// The work item of this block among (row tile, part) pairs, `parts` to a row
// tile.  Blocks are dealt to the 8 XCDs in turn; here each XCD takes a
// contiguous run of the items there are, in which a few parts' weights meet
// all tiles of their expert before the next parts', so that what runs
// together shares both through the XCD's L2.  Items are counted in 64 bits:
// runs of bad offsets may overlap and add up to more than the rows have.
__device__ inline bool block_item(int64_t count, int64_t& item) {
  const int b = blockIdx.x, x = b & 7, i = b >> 3;
  const int64_t base = count >> 3;
  const int rem = (int)(count & 7);
  item = x * base + min(x, rem) + i;
  return b < count;
}

// lds: 16 ints.
__device__ inline RowTile find_tile(const int32_t* offsets, int E, int n, int bm, int parts, int* lds) {
  RowTile r{0, 0, 0, 0};
  int64_t item;
  int t;
  if (!offsets) {
    const int m = (n + bm - 1) / bm;
    if (!block_item((int64_t)m * parts, item)) return r;
    split_item((int)item, m, parts, t, r.part);
    r.lo = t * bm;
    r.cnt = min(bm, n - r.lo);
    return r;
  }
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
  __syncthreads();
  int first = x - tiles, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < wave) first += lds[w];
    total += lds[w];
  }
  if (!block_item((int64_t)total * parts, item)) return r;
  const int64_t mine = item - (int64_t)first * parts;  // from this thread's first tile on
  if (mine >= 0 && mine < (int64_t)tiles * parts) {
    int64_t left = mine;
    for (int i = 0; i < per; ++i) {
      const int lo = min(max(offsets[e0 + i], 0), n), hi = min(max(offsets[e0 + i + 1], 0), n);
      const int m = hi > lo ? (hi - lo + bm - 1) / bm : 0;
      if (left < (int64_t)m * parts) {
        int part;
        split_item((int)left, m, parts, t, part);
        lds[8] = e0 + i;
        lds[9] = lo + t * bm;
        lds[10] = min(bm, hi - lo - t * bm);
        lds[11] = part;
        break;
      }
      left -= (int64_t)m * parts;
    }
  }
  __syncthreads();
  // the same in every lane: keep them in scalar registers
  r.e = __builtin_amdgcn_readfirstlane(lds[8]);
  r.lo = __builtin_amdgcn_readfirstlane(lds[9]);
  r.cnt = __builtin_amdgcn_readfirstlane(lds[10]);
  r.part = __builtin_amdgcn_readfirstlane(lds[11]);
  return r;
}

// Row tiles a call can have at most.
inline int64_t max_tiles(int64_t n, int E, bool grouped, int bm) {
  if (!grouped) return (n + bm - 1) / bm;
  return std::min<int64_t>(n, n / bm + std::min<int64_t>(E, n));
}

}  // namespace ds4
