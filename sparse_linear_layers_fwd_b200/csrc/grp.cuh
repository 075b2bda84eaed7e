// Rows grouped by expert: the work list of the grouped kernels.
//
// The rows of expert e are offsets[e] .. offsets[e + 1] - 1, known on the
// device only (a router wrote them), so every CTA builds the same work list
// in shared memory: sanitized offsets (clamped to the rows that exist and
// made non-decreasing, so that no offsets can lead outside a buffer) and the
// running count of row tiles before each expert.
#pragma once

#include "common.cuh"

namespace sbn {

constexpr int kGrpMaxExperts = 1024;

struct GrpParams {
  const int32_t* offsets;   // [experts + 1], or NULL: one group of all rows
  int experts;
  int rows;
};

SBN_DEVFN int warp_scan_max(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = max(v, o);
  }
  return v;
}
SBN_DEVFN int warp_scan_add(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// One warp: sanitized offsets into off[0 .. E] and the tiles before expert e
// into first[0 .. E], an expert of t rows having ceil(t / tile_rows) *
// per_row_tile tiles (at least `empty_tiles` for one without rows).
SBN_DEVFN void grp_build(const GrpParams& p, int tile_rows, int per_row_tile, int empty_tiles, int* off, int* first) {
  const int lane = threadIdx.x & 31;
  int top = 0, tiles = 0;   // carried: largest offset so far, tiles so far
  // an entry's raw offset, loaded a round ahead
  auto load = [&](int e) { return p.offsets && e <= p.experts ? p.offsets[e] : e >= p.experts ? p.rows : 0; };
  int next = load(lane);
  for (int e0 = 0; e0 <= p.experts; e0 += 32) {
    const int e = e0 + lane;
    int v = min(max(next, 0), p.rows);
    next = load(e + 32);
    v = max(warp_scan_max(v, lane), top);
    const int prev = __shfl_up_sync(0xffffffffu, v, 1);
    const int before = lane ? prev : top;   // offset of expert e - 1's first row
    // tiles of expert e - 1, which ends at offset v
    int t = 0;
    if (e >= 1 && e <= p.experts) {
      const int n = v - before;
      t = n > 0 ? (n + tile_rows - 1) / tile_rows * per_row_tile : empty_tiles;
    }
    const int sum = warp_scan_add(t, lane) + tiles;
    if (e <= p.experts) {
      off[e] = v;
      first[e] = sum;
    }
    top = __shfl_sync(0xffffffffu, v, 31);
    tiles = __shfl_sync(0xffffffffu, sum, 31);
  }
}

// The expert of a tile: the e with first[e] <= tile < first[e + 1].
SBN_DEVFN int grp_find(const int* first, int experts, int tile) {
  int lo = 0, hi = experts;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace sbn
