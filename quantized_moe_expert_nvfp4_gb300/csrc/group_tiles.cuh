// Row tiles of a grouped product whose rows are sorted by group: group g has rows
// [offsets[g], offsets[g + 1]), and the rows from offsets[G] on, a last "group" G, belong to no
// matrix.  Every CTA derives the tiles from the offsets itself, so no launch builds a work list.
#pragma once

#include "internal.cuh"

namespace moe {

constexpr int kMaxGroups = kMaxE + 1;

struct GroupTiles {
  int off[kMaxGroups + 2];     // row bounds; off[G + 1] = M
  int first[kMaxGroups + 2];   // first tile of each group; first[G + 1] = number of tiles
  int warp_sum[32];
  int bad;
};

struct RowTile {
  int group, row, rows;        // group G: rows without a matrix
};

// Fills `g` with all threads of the CTA (a multiple of 32); ends with a barrier.  offsets == NULL:
// one group of all M rows.  Offsets that do not start at 0, decrease or end beyond M are
// reported, and every row then counts as one without a matrix.
__device__ __forceinline__ void build_group_tiles(GroupTiles& g, const int32_t* offsets, int G, int M, int tile_rows,
                                                  int32_t* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) g.bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i <= G + 1; i += blockDim.x) {
    int v = M;
    if (i <= G) {
      v = offsets ? __ldg(offsets + i) : (i == 0 ? 0 : M);
      const int before = i == 0 ? 0 : offsets ? __ldg(offsets + i - 1) : 0;
      if (v < before || v > M || (i == 0 && v != 0)) g.bad = 1;
    }
    g.off[i] = v;
  }
  __syncthreads();
  if (g.bad) {
    for (int i = threadIdx.x; i <= G; i += blockDim.x) g.off[i] = 0;
    if (threadIdx.x == 0) report_device_error(status, kDevBadIndex);
    __syncthreads();
  }
  const int n = G + 1, per = (n + blockDim.x - 1) / blockDim.x;
  const int a = min(n, static_cast<int>(threadIdx.x) * per), b = min(n, a + per);
  int sum = 0;
  for (int i = a; i < b; ++i) sum += (g.off[i + 1] - g.off[i] + tile_rows - 1) / tile_rows;
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) g.warp_sum[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += g.warp_sum[w];
  for (int i = a; i < b; ++i) {
    g.first[i] = run;
    run += (g.off[i + 1] - g.off[i] + tile_rows - 1) / tile_rows;
  }
  if (b == n && a < n) g.first[n] = run;
  __syncthreads();
}

__device__ __forceinline__ RowTile group_tile(const GroupTiles& g, int G, int tile, int tile_rows) {
  int lo = 0, hi = G;          // the last group whose first tile is at most `tile`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  RowTile r;
  r.group = lo;
  r.row = g.off[lo] + (tile - g.first[lo]) * tile_rows;
  r.rows = min(tile_rows, g.off[lo + 1] - r.row);
  return r;
}

// The same by a whole warp in two probes: 33 keys apart, then the 33 in between (a probe of shared
// memory takes 100 cycles and more while the tensor cores read their operands from it).
__device__ __forceinline__ RowTile group_tile_warp(const GroupTiles& g, int G, int tile, int tile_rows, int lane) {
  static_assert(kMaxGroups + 1 <= 33 * 32, "two probes of 32");
  int at = lane * 33;
  unsigned below = __ballot_sync(0xffffffffu, at <= G && g.first[min(at, G)] <= tile);
  at = (__popc(below) - 1) * 33 + 1 + lane;
  below = __ballot_sync(0xffffffffu, at <= G && g.first[min(at, G)] <= tile);
  RowTile r;
  r.group = at - 1 - lane + __popc(below);
  r.row = g.off[r.group] + (tile - g.first[r.group]) * tile_rows;
  r.rows = min(tile_rows, g.off[r.group + 1] - r.row);
  return r;
}

}  // namespace moe
