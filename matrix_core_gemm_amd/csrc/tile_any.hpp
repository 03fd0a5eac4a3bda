// tile_any.hpp -- register-staged operand tiles for the 8-bit linear layer's
// general kernels: HBM -> registers -> LDS at any pointer and leading dimension.
//
// The tiles have the LDS layout of tile_io.hpp (TileGeom, swz), so its fragment
// readers apply.  gfx950 reads global memory at any byte address, so a chunk that
// lies inside the matrix is one 16-byte load at any alignment; only the chunks
// that cross the matrix's end are read by element.
#pragma once
#include "tile_io.hpp"

namespace mcg {

// 16 bytes from any address.
__device__ __forceinline__ i32x4 load16_any(const char* p) {
  struct __attribute__((packed, aligned(1))) U { int w[4]; };
  const U u = *(const U*)p;
  return i32x4{u.w[0], u.w[1], u.w[2], u.w[3]};
}

// The first `left` bytes (0..15) of the 16 at p, the rest zero.  The 16 bytes that end
// with them are loaded and shifted down: reading by element costs 8 to 16 loads and
// branches in every wavefront of an edge tile (500 x 1536 x 4096 with an
// MN-contiguous A: 221 us by element, 174 so).  base: the matrix's first byte; only a
// chunk that lies closer than 16 bytes to it is read by byte.
__device__ __forceinline__ i32x4 load_part(const char* base, const char* p, int left) {
  const char* q = p + left - 16;
  if (q >= base) {
    const i32x4 v = load16_any(q);
    const uint64_t lo = (uint64_t)(uint32_t)v[0] | ((uint64_t)(uint32_t)v[1] << 32);
    const uint64_t hi = (uint64_t)(uint32_t)v[2] | ((uint64_t)(uint32_t)v[3] << 32);
    const int s = 8 * (16 - left);  // bits to drop: 8..128
    const uint64_t l = s < 64 ? (lo >> s) | (hi << (64 - s)) : s < 128 ? hi >> (s - 64) : 0;
    const uint64_t h = s < 64 ? hi >> s : 0;
    return i32x4{(int)(uint32_t)l, (int)(uint32_t)(l >> 32), (int)(uint32_t)h, (int)(uint32_t)(h >> 32)};
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 15; ++e)
    if (e < left) w[e / 4] |= (uint32_t) * (const uint8_t*)(p + e) << (8 * (e & 3));
  return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// 16 bytes at p of a row that ends `left` bytes further, zeros past its end.
__device__ __forceinline__ i32x4 load_chunk(const char* base, const char* p, int64_t left) {
  if (left >= 16) return load16_any(p);
  if (left <= 0) return i32x4{0, 0, 0, 0};
  return load_part(base, p, (int)left);
}

// One operand tile by NT threads: storage rows [row0, row0 + R) and contiguous
// elements [col0, ...) of a matrix; rows past rlim and elements past clim are zero.
template <int EB, int LAYOUT, int ROWS_MN, int NT>
struct AnyLoader {
  using G = TileGeom<EB, LAYOUT, ROWS_MN>;
  static constexpr int PER_THREAD = G::CHUNKS / NT;
  static_assert(G::CHUNKS % NT == 0, "tile chunks must divide evenly among threads");
  i32x4 regs[PER_THREAD];

  __device__ __forceinline__ void load(const char* base, int64_t ld, int64_t row0, int64_t col0, int64_t rlim,
                                       int64_t clim, int tid) {
#pragma unroll
    for (int t = 0; t < PER_THREAD; ++t) {
      const int q = tid + t * NT;
      const int64_t gr = row0 + q / G::CPR, gc = col0 + (int64_t)(q % G::CPR) * (16 / EB);
      regs[t] = load_chunk(base, base + (gr * ld + gc) * EB, gr < rlim ? (clim - gc) * EB : 0);
    }
  }
  __device__ __forceinline__ void store(lds_char* tile, int tid) const {
#pragma unroll
    for (int t = 0; t < PER_THREAD; ++t) {
      const int q = tid + t * NT;
      const int r = q / G::CPR, cc = q % G::CPR;
      lds_write_b128(tile, r * G::W + ((cc ^ swz<EB, LAYOUT, G::CPR>(r)) * 16), regs[t]);
    }
  }
};

// Output tile of workgroup pid, grouped by 8 tile rows for L2 reuse.
__device__ __forceinline__ void general_tile(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int group = 8;
  const int tiles_in_group = group * tiles_n;
  const int first_m = pid / tiles_in_group * group;
  const int gsize = min(tiles_m - first_m, group);
  tm = first_m + (pid % tiles_in_group) % gsize;
  tn = (pid % tiles_in_group) / gsize;
}

// K ranges for `tiles` workgroups of nk K tiles each, from the time model
//   rounds * (kt_us * ceil(nk / s) + 3) + s * M * N * slot_us + (s > 1: 5), in us,
// where a range's partial results make one trip through the workspace.
inline int64_t plan_ranges(int64_t tiles, int64_t nk, int64_t out_elems, int num_cu, double kt_us,
                           int64_t max_splits, double* us) {
  constexpr double ROUND_US = 3.0, SLOT_US = 2.5e-6, SPLIT_US = 5.0;
  auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  int64_t best = 1;
  double best_t = 0;
  for (int64_t s = 1; s == 1 || (s <= max_splits && s <= nk / 2 + 1); ++s) {
    if (s > 1 && cdiv(nk, cdiv(nk, s)) != s) continue;  // every range non-empty
    const double t = (double)cdiv(tiles * s, num_cu) * (kt_us * (double)cdiv(nk, s) + ROUND_US) +
                     (s > 1 ? (double)s * (double)out_elems * SLOT_US + SPLIT_US : 0.0);
    if (s == 1 || t < best_t) {
      best = s;
      best_t = t;
    }
  }
  *us = best_t;
  return best;
}

}  // namespace mcg
