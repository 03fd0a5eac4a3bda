// group_tiles.hpp -- from a workgroup's number to its tile where rows come in groups of
// ragged sizes, known on the device only (by their offsets).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "experts.hpp"
#include "tile_order.hpp"

namespace mcg {

// Rows [r0, r1) of a group.  Offsets that leave 0 .. M or decrease are read as the nearest
// that do not, so that no access leaves the operands.
struct GroupRows {
  int64_t r0, r1;
};
__host__ __device__ inline GroupRows group_rows(const int32_t* offsets, int g, int64_t M) {
  const int64_t a = offsets[g], b = offsets[g + 1];
  const int64_t r0 = a < 0 ? 0 : a > M ? M : a;
  return GroupRows{r0, b < r0 ? r0 : b > M ? M : b};
}

// Tiles of tm rows of a group.  (Launches are smaller than MANY_TILES: only offsets that decrease, and so
// count rows often, reach it.)
__host__ __device__ inline int tiles_of(const GroupRows& r, int tm) {
  const int64_t n = (r.r1 - r.r0 + tm - 1) / tm;
  return n < MANY_TILES ? (int)n : MANY_TILES;
}
__host__ __device__ inline int add_tiles(int a, int b) { return a + b < (1 << 30) ? a + b : 1 << 30; }  // (b: of 64 groups)

// What the wavefronts of a workgroup work on: tile t of group g.  Every wavefront finds it
// by itself, a group per lane.
struct GroupTile {
  int g;
  int64_t r0, r1;  // the group's rows; none (r0 == r1) if no group has the tile
  int t;
};

// Inclusive sum over the lanes.
__device__ __forceinline__ int lanes_sum(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    x += lane >= d ? y : 0;
  }
  return x;
}

// Tiles of TM rows of all groups.
template <int TM>
__device__ __forceinline__ int count_tiles(const int32_t* offsets, int G, int64_t M, int lane) {
  int total = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    int n = 0;
    if (g0 + lane < G) n = tiles_of(group_rows(offsets, g0 + lane, M), TM);
    total = add_tiles(total, __shfl(lanes_sum(n, lane), 63));
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// The tile with this number in the sequence of all groups' tiles (0 .. count_tiles - 1).
template <int TM>
__device__ __forceinline__ GroupTile find_tile(const int32_t* offsets, int G, int64_t M, int tile, int lane) {
  int before = 0;  // tiles of the groups before g0
  GroupTile w{0, 0, 0, 0};
  for (int g0 = 0; g0 < G; g0 += 64) {
    GroupRows r{0, 0};
    if (g0 + lane < G) r = group_rows(offsets, g0 + lane, M);
    const int n = tiles_of(r, TM), upto = lanes_sum(n, lane);
    const uint64_t past = __ballot(before + upto > tile);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      w.g = __builtin_amdgcn_readfirstlane(g0 + src);
      w.r0 = __builtin_amdgcn_readfirstlane((int)__shfl((int)r.r0, src));
      w.r1 = __builtin_amdgcn_readfirstlane((int)__shfl((int)r.r1, src));
      w.t = __builtin_amdgcn_readfirstlane(tile - before - __shfl(upto - n, src));
      return w;
    }
    before = add_tiles(before, __shfl(upto, 63));
  }
  return w;
}

// Workgroup bid of n -> its place in the sequence of tiles: workgroups go round-robin to the
// 8 XCDs, and those of one XCD take consecutive tiles, which share operands in its L2.
__host__ __device__ inline int xcd_order(int bid, int n) {
  const int x = bid & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (bid >> 3);
}

// The pipelined kernels' order of tiles.  A group's tiles at one column read the same part of its B, so
// they run next to each other on one XCD, whose L2 then reads it once; groups' weights are most
// of what these products read.  The columns are cut into 8 slices (or 4, 2, 1: as many as divide their
// number), one for each XCD, or for 2, 4, 8 of them, which then take the slice's tiles in turn parts.
// Every XCD so gets the long and the short groups alike.  A slice's tiles go group by group, and in a
// group column by column through 8 tile rows at a time.
struct Slices {
  int count, columns;  // slices, tile columns in one
  __host__ __device__ explicit Slices(int tiles_n) {
    count = tiles_n % 8 == 0 ? 8 : tiles_n % 4 == 0 ? 4 : tiles_n % 2 == 0 ? 2 : 1;
    columns = tiles_n / count;
  }
  // tiles of an XCD, of `tiles` tile rows in all
  __host__ __device__ int64_t part(int64_t tiles) const {
    const int64_t xcds = 8 / count;
    return (tiles * columns + xcds - 1) / xcds;
  }
};
// Workgroups that take all tiles.
__host__ __device__ inline int64_t slice_blocks(int64_t tiles, int tiles_n) { return 8 * Slices(tiles_n).part(tiles); }

// The tile of workgroup bid: rows from m0 on of group g, which end at r1, and tile column tn.  m0 == r1:
// no tile.
struct PipeTile {
  int g, tn;
  int64_t m0, r1;
};
template <int TM>
__device__ __forceinline__ PipeTile pipe_tile(const int32_t* offsets, int G, int64_t M, int tiles_n, int bid, int lane) {
  PipeTile w{0, 0, 0, 0};
  const int tiles = count_tiles<TM>(offsets, G, M, lane);
  const Slices s(tiles_n);
  if ((int64_t)tiles * s.columns > MANY_TILES) return w;  // (offsets that decrease: launches are smaller)
  const int all = tiles * s.columns, part = (int)s.part(tiles);
  const int x = bid & 7, slice = x % s.count;
  const int at = (x / s.count) * part + (bid >> 3);  // the tile's number in its slice
  if ((bid >> 3) >= part || at >= all) return w;
  int before = 0;  // the slice's tiles in the groups before g0
  for (int g0 = 0; g0 < G; g0 += 64) {
    GroupRows r{0, 0};
    if (g0 + lane < G) r = group_rows(offsets, g0 + lane, M);
    const int mine = tiles_of(r, TM), upto = lanes_sum(mine, lane) * s.columns;
    const uint64_t past = __ballot(before + upto > at);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const int rows = __builtin_amdgcn_readfirstlane(__shfl(mine, src));
      const int in_group = __builtin_amdgcn_readfirstlane(at - before - __shfl(upto - mine * s.columns, src));
      w.g = __builtin_amdgcn_readfirstlane(g0 + src);
      int tm, tn;
      fast::grouped_tile<8>(in_group, rows, s.columns, tm, tn);
      w.tn = slice * s.columns + tn;
      w.r1 = __builtin_amdgcn_readfirstlane((int)__shfl((int)r.r1, src));
      w.m0 = __builtin_amdgcn_readfirstlane((int)__shfl((int)r.r0, src)) + (int64_t)tm * TM;
      return w;
    }
    before += __shfl(upto, 63);
  }
  return w;
}

// f(n) with n = 0 .. N as a compile-time constant, for a wave-uniform n (0 if below).
template <int N, class F>
__device__ __forceinline__ void with_live(int n, F&& f) {
  if constexpr (N == 0) f(std::integral_constant<int, 0>{});
  else if (n >= N) f(std::integral_constant<int, N>{});
  else with_live<N - 1>(n, static_cast<F&&>(f));
}

}  // namespace mcg
