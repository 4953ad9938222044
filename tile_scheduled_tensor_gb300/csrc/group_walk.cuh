// The work list of the block-scaled kernels' persistent CTAs, light enough for registers: the next
// tile and, grouped, its group, found in a table in shared memory.
//
// work_next (tile_sched.h) finds the group of the next tile by reading the groups' row counts
// from global memory one after another, in 64-bit sums: 2000 to 2900 cycles per tile in a warp of
// a block-scaled kernel, whose whole tile takes 15000.  Here each CTA first sums the counts into a
// table of every group's first tile, first row and rows, once, and each role finds the next tile's
// group in it by comparisons.  The items are those of work_next for whole tiles (static, persistent
// or grouped with shared N and K, at most kWalkGroups groups).
#pragma once
#include <stdint.h>

#include "kernel_params.h"
#include "tile_sched.h"

namespace tst {

constexpr int kWalkGroups = kBsWalkGroups;   // groups that a table holds
constexpr int kWalkBytes = (3 * kWalkGroups + 4) * 4;

struct GroupTable {
  int32_t* tile0;   // groups + 1: first linear tile of each group, then all tiles
  int32_t* row0;    // groups: first row, at most INT32_MAX
  int32_t* rows;    // groups
  __device__ __forceinline__ explicit GroupTable(void* base)
      : tile0(static_cast<int32_t*>(base)), row0(tile0 + kWalkGroups + 1), rows(row0 + kWalkGroups) {}
};

// One whole warp fills the table; the CTA's barrier makes it visible.
__device__ __forceinline__ void fill_group_table(const Sched& s, const GroupTable& t) {
  const int lane = threadIdx.x & 31;
  constexpr int64_t most = 0x7FFFFFFF, most_tiles = int64_t(1) << 30;
  int64_t tiles = 0, row = 0;
  for (int32_t b = 0; b < s.groups; b += 32) {
    const int32_t g = b + lane;
    const int64_t r = g < s.groups ? group_row_count(s, g) : 0;
    const int64_t n = g < s.groups ? group_tile_count(s, g, r) : 0;
    int64_t sum_n = n, sum_r = r;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t on = __shfl_up_sync(0xFFFFFFFFu, sum_n, d);
      const int64_t orow = __shfl_up_sync(0xFFFFFFFFu, sum_r, d);
      if (lane >= d) { sum_n += on; sum_r += orow; }
    }
    if (g < s.groups) {
      const int64_t first = tiles + sum_n - n, first_row = row + sum_r - r;
      t.tile0[g] = static_cast<int32_t>(first < most_tiles ? first : most_tiles);
      t.row0[g] = static_cast<int32_t>(first_row < most ? first_row : most);
      t.rows[g] = static_cast<int32_t>(r);
    }
    tiles += __shfl_sync(0xFFFFFFFFu, sum_n, 31);
    row += __shfl_sync(0xFFFFFFFFu, sum_r, 31);
  }
  if (lane == 0) t.tile0[s.groups] = static_cast<int32_t>(tiles < most_tiles ? tiles : most_tiles);
}

// What a tile needs of its work item (every tile takes the whole K, and N columns are the output's).
struct Tile {
  int32_t index, m, n;   // linear tile, its place in the group's grid
  int32_t group;
  int32_t row0, row_end; // first row in A and the output; rows from row_end on are not the tile's
  bool clamped;          // the group's rows end past the matrix
};

// A role's walk, by one thread (next) or by a converged warp (next_warp).
struct Walk {
  const Sched& s;
  GroupTable t;
  int32_t at, g;   // the next linear tile, the current group
  __device__ __forceinline__ Walk(const Sched& sched, const GroupTable& table, int32_t unit)
      : s(sched), t(table), at(unit), g(0) {}
  __device__ __forceinline__ void take(Tile& w) {
    w.index = at;
    w.group = g;
    if (s.groups == 0) {
      tile_coord(s, at, w.m, w.n);
      w.row0 = w.m * s.bm;
      w.row_end = s.rows;
      w.clamped = false;
    } else {
      const int32_t rows = t.rows[g];
      Sched sg;
      sg.map_kind = s.map_kind;
      sg.mt = (rows + s.bm - 1) / s.bm;
      sg.nt = s.nt;
      sg.group = s.group;
      sg.order = nullptr;
      tile_coord(sg, at - t.tile0[g], w.m, w.n);
      const int64_t row0 = static_cast<int64_t>(t.row0[g]) + static_cast<int64_t>(w.m) * s.bm;
      const int64_t end = static_cast<int64_t>(t.row0[g]) + rows;
      w.clamped = end > s.rows;
      w.row0 = static_cast<int32_t>(row0 < s.rows ? row0 : s.rows);
      w.row_end = static_cast<int32_t>(end < s.rows ? end : s.rows);
    }
    at += s.grid;
  }
  __device__ __forceinline__ bool next(Tile& w) {
    if (s.groups == 0) {
      if (at >= s.dp_tiles) return false;
    } else {
      if (at >= t.tile0[s.groups]) return false;
      int32_t past;
      do {   // four groups' ends at once: their loads' latency passes once
        past = 0;
#pragma unroll
        for (int32_t i = 1; i <= 4; ++i) past += at >= t.tile0[g + i < s.groups ? g + i : s.groups] ? 1 : 0;
        g += past;
      } while (past == 4);
    }
    take(w);
    return true;
  }
  // for roles that count tiles only
  __device__ __forceinline__ bool skip() {
    if (at >= (s.groups == 0 ? s.dp_tiles : t.tile0[s.groups])) return false;
    at += s.grid;
    return true;
  }
  __device__ __forceinline__ bool next_warp(Tile& w) {
    if (s.groups == 0) {
      if (at >= s.dp_tiles) return false;
    } else {
      if (at >= t.tile0[s.groups]) return false;
      const int lane = threadIdx.x & 31;
      for (;; g += 32) {
        const int32_t e = g + 1 + lane;
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, e <= s.groups && t.tile0[e] > at);
        if (past != 0u) {
          g += __ffs(past) - 1;
          break;
        }
      }
    }
    take(w);
    return true;
  }
};

}  // namespace tst
