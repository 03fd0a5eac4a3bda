// group_tiles.hpp -- from a workgroup's number to its tile where rows come in groups of
// ragged sizes, known on the device only (by their offsets).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// Tiles of tm rows of a group, and the most tiles that are counted in all: launches are
// smaller, so that only offsets that decrease, and so count rows often, reach it.
constexpr int MANY_TILES = 1 << 23;
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

}  // namespace mcg
