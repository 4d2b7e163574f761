// Rows grouped by expert: how a workgroup finds the expert and the rows it works on. The group
// boundaries (offsets) are device data that the host never sees: a launch is sized for the most tiles
// that M rows in E groups can make, M / BM + min(E, M), and every wave finds its tile by itself from the
// offsets, 64 experts at a time (one load and one wave-wide prefix sum per 64 experts, served from
// cache), so no table, second launch or workspace is needed. Row ranges are clamped to 0 .. rows, so
// offsets that break the rules cannot lead outside the arguments' buffers.
#pragma once

#include "common.hpp"

namespace splr {

struct Groups {
  const int32_t* offsets;  // [experts + 1]
  int experts;
  int rows;                // M
};

__host__ inline int64_t most_group_tiles(int64_t rows, int64_t experts, int64_t tile) {
  return rows / tile + (experts < rows ? experts : rows);
}

#ifdef __HIPCC__
namespace {

// One expert's part of the rows, as a wave-uniform value: rows lo .. lo + rows - 1, cut into `tiles`
// row tiles, of which the first is number `first` of all experts'. expert < 0: no such tile.
struct GroupTile {
  int expert, lo, rows, first, tiles;
};

__device__ __forceinline__ void group_rows(const Groups& g, int e, int& lo, int& rows) {
  lo = min(max(g.offsets[e], 0), g.rows);
  rows = min(max(g.offsets[e + 1], lo), g.rows) - lo;
}

// How many row tiles all experts have together.
template <int BM>
__device__ __forceinline__ int group_tiles_total(const Groups& g) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int e = lane; e < g.experts; e += 64) {
    int lo, rows;
    group_rows(g, e, lo, rows);
    sum += (rows + BM - 1) / BM;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  return __builtin_amdgcn_readfirstlane(sum);
}

// The expert that holds row tile `t`. Called by whole waves with a uniform t.
template <int BM>
__device__ __forceinline__ GroupTile find_group_tile(const Groups& g, int t) {
  const int lane = threadIdx.x & 63;
  int first = 0;
  for (int base = 0; base < g.experts; base += 64) {
    int lo = 0, rows = 0;
    if (base + lane < g.experts) group_rows(g, base + lane, lo, rows);
    const int tiles = (rows + BM - 1) / BM;
    int upto = tiles;  // inclusive prefix sum over the lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(upto, off);
      if (lane >= off) upto += v;
    }
    const uint64_t after = __ballot(first + upto > t);
    if (after) {
      const int l = __builtin_ctzll(after);
      const int n = __builtin_amdgcn_readlane(tiles, l);
      return GroupTile{base + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(rows, l),
                       first + __builtin_amdgcn_readlane(upto, l) - n, n};
    }
    first += __builtin_amdgcn_readlane(upto, 63);
  }
  return GroupTile{-1, 0, 0, 0, 0};
}

}  // namespace
#endif
}  // namespace splr
