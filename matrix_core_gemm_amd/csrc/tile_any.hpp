// tile_any.hpp -- register-staged operand tiles for the 8-bit linear layer's
// general kernels: HBM -> registers -> LDS at any pointer and leading dimension.
//
// The tiles have the LDS layout of tile_io.hpp (TileGeom, swz), so its fragment
// readers apply.  gfx950 reads global memory at any byte address, so a chunk that
// lies inside the matrix is one 16-byte load at any alignment; a chunk that crosses
// a row's end is read as the row's last 16 bytes and shifted.
#pragma once
#include "tile_io.hpp"

namespace mcg {

// Global memory's address space is stated where the compiler cannot see it: a generic
// load counts as an LDS access too, and every wait after it waits for all of them.
typedef __attribute__((address_space(1))) float global_f32;
// 16 bytes from any address of global memory.
__device__ __forceinline__ i32x4 load16_any(const char* p) {
  typedef int v4 __attribute__((ext_vector_type(4), aligned(1)));
  return *(const __attribute__((address_space(1))) v4*)p;
}
__device__ __forceinline__ i32x4 shift_chunk(const i32x4& v, int bytes) {  // down by 0..15 bytes
  const uint64_t lo = (uint64_t)(uint32_t)v[0] | ((uint64_t)(uint32_t)v[1] << 32);
  const uint64_t hi = (uint64_t)(uint32_t)v[2] | ((uint64_t)(uint32_t)v[3] << 32);
  const int s = 8 * bytes;
  const uint64_t l = s == 0 ? lo : s < 64 ? (lo >> s) | (hi << (64 - s)) : hi >> (s - 64);
  const uint64_t h = s < 64 ? hi >> s : 0;
  return i32x4{(int)(uint32_t)l, (int)(uint32_t)(l >> 32), (int)(uint32_t)h, (int)(uint32_t)(h >> 32)};
}
// The 16 bytes at p of a row that ends `left` bytes further, zeros past its end.  A
// partial chunk is read as the 16 bytes that end with the row, and shifted (by
// element it costs 8 to 16 loads and branches); only one that starts closer than
// that to base, the matrix's first byte, is read by byte.
__device__ __forceinline__ i32x4 load_chunk(const char* base, const char* p, int left) {
  if (left >= 16) return load16_any(p);
  if (left <= 0) return i32x4{0, 0, 0, 0};
  if (p + left - 16 >= base) return shift_chunk(load16_any(p + left - 16), 16 - left);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 15; ++e)
    if (e < left) w[e / 4] |= (uint32_t) * (const uint8_t*)(p + e) << (8 * (e & 3));
  return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// Workgroup barrier that waits for this wave's LDS accesses only: global loads stay in flight.
__device__ __forceinline__ void barrier_tiles() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// What loads of K tiles past a range's end read.
static __device__ const int load_nothing[4] = {0, 0, 0, 0};

// One operand's K tiles by NT threads: KTB bytes of K of ROWS_MN rows (or columns)
// from mn0 on, of an operand with `mn` rows and K values of k, at least 16 bytes in
// all.  k past K is zero; rows past mn hold anything, since only outputs that are not
// stored see them.
//
// Loads have no conditions, at whose ends the compiler copies the registers and so
// waits for loads that should stay in flight: rows and chunks past the end are read at
// the last valid one's address, a row's partial chunk at the row's last 16 bytes (or
// the matrix's first), and K tiles past the range (live false) at a constant's.  What
// that leaves in the registers is set right before they are used, in the tiles that
// have an edge only.
template <int EB, int LAYOUT, int ROWS_MN, int NT, int KTB = KT_BYTES>
struct AnyLoader {
  using G = TileGeom<EB, LAYOUT, ROWS_MN, KTB>;
  static constexpr int PER_THREAD = G::CHUNKS / NT, RPI = NT / G::CPR;  // LDS rows per step of NT chunks
  static constexpr int KE = KTB / EB;                                   // values of k per tile
  static_assert(G::CHUNKS % NT == 0 && NT % G::CPR == 0, "tile chunks must divide evenly among threads");
  using Regs = i32x4[PER_THREAD];
  const char* base;
  int64_t off0, ldb, istride, kstride, K;  // off0: this thread's first chunk in K tile 0
  int r0, c16;  // this thread's first LDS row, and its chunk's byte in the row
  int mn_left;  // rows of the operand from mn0, at most the tile's
  int last;     // K tile with k's end
  int end;      // bytes of a row in the tile that has its end
  int back;     // bytes that the address of this thread's chunk moves down by there

  __device__ __forceinline__ void init(const char* b, int64_t ld, int64_t mn0, int64_t mn, int64_t K_, int tid) {
    base = b;
    K = K_;
    ldb = ld * EB;
    r0 = tid / G::CPR;
    c16 = 16 * (tid % G::CPR);
    mn_left = (int)min(mn - mn0, (int64_t)ROWS_MN);
    last = (int)((K - 1) / KE);
    end = (LAYOUT == LAYOUT_K ? (int)(K - (int64_t)last * KE) : mn_left) * EB;
    back = c16 + 16 <= end ? 0 : c16 < end ? c16 + 16 - end : c16 + max(0, 16 - end);
    kstride = LAYOUT == LAYOUT_K ? (int64_t)KTB : KE * ldb;
    istride = RPI * ldb;
    off0 = (LAYOUT == LAYOUT_K ? mn0 * ldb : mn0 * EB) + r0 * ldb + c16;
  }
  // values of k in K tile kt
  __device__ __forceinline__ int k_here(int kt) const { return (int)min(K - (int64_t)kt * KE, (int64_t)KE); }
  __device__ __forceinline__ int rows(int kt) const { return LAYOUT == LAYOUT_K ? mn_left : k_here(kt); }
  // whether rows end in K tile kt of this tile
  __device__ __forceinline__ bool ends(int kt) const { return LAYOUT == LAYOUT_MN || kt == last; }
  // offset of chunk t of K tile kt, and the bytes its address moves down by
  __device__ __forceinline__ int64_t offset(int kt, int t) const {
    int64_t off = off0 + kt * kstride + t * istride;
    if (LAYOUT == LAYOUT_K || kt >= last) off -= max(r0 + t * RPI - (rows(kt) - 1), 0) * ldb;
    return off;
  }
  __device__ __forceinline__ int moved(int64_t off) const { return off < back ? (int)off : back; }
  __device__ __forceinline__ void load(Regs& regs, int kt, bool live) const {
    const bool e = ends(kt);
#pragma unroll
    for (int t = 0; t < PER_THREAD; ++t) {
      const int64_t off = offset(kt, t);
      regs[t] = load16_any(live ? base + (off - (e ? moved(off) : 0)) : (const char*)load_nothing);
    }
  }
  // Corrects the registers of K tile kt, before they are used.
  __device__ __forceinline__ void settle(Regs& regs, int kt) const {
    if (ends(kt) && end < G::W) {
      const int valid = end - c16;  // bytes of this thread's chunks that are in the row
#pragma unroll
      for (int t = 0; t < PER_THREAD; ++t) {
        if (valid > 0) regs[t] = shift_chunk(regs[t], moved(offset(kt, t)));
        if (LAYOUT == LAYOUT_K) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int n = valid - 4 * w;
            regs[t][w] = n >= 4 ? regs[t][w] : n <= 0 ? 0 : (int)((uint32_t)regs[t][w] & (0xffffffffu >> (32 - 8 * n)));
          }
        }
      }
    }
    if (LAYOUT == LAYOUT_MN && kt >= last) {
#pragma unroll
      for (int t = 0; t < PER_THREAD; ++t)
        if (r0 + t * RPI >= rows(kt)) regs[t] = i32x4{0, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void store(const Regs& regs, lds_char* tile) const {
#pragma unroll
    for (int t = 0; t < PER_THREAD; ++t) {
      const int r = r0 + t * RPI, cc = c16 / 16;
      lds_write_b128(tile, r * G::W + ((cc ^ swz<EB, LAYOUT, G::CPR>(r)) * 16), regs[t]);
    }
  }
};

// Whether AnyLoader takes an operand of rows x cols elements of eb bytes.
inline bool any_operand_ok(int64_t eb, int64_t rows, int64_t cols, int64_t ld) {
  return rows > 0 && cols > 0 && ((rows - 1) * ld + cols) * eb >= 16;
}
// f(0), f(1), ... as compile-time constants: register sets of successive K tiles.
template <int N, class F, int I = 0>
__device__ __forceinline__ void for_each_set(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    for_each_set<N, F, I + 1>(static_cast<F&&>(f));
  }
}

// Rows of the general kernels' tiles: the fewest that hold M, up to 128 (32 x 4096 x
// 4096 from 8-bit weights 15.9 us with 32 rows, 25 with 128; 64 rows 21.4 and 25; a
// second row of tiles would read B twice).
inline int general_rows(int64_t M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }
// The 4 wavefronts' blocks of 16 x 16 in a BM x 128 tile: 2 x 2 wavefronts, or 1 x 4.
template <int BM>
struct WaveGrid {
  static constexpr int WTM = BM == 128 ? 4 : 2, WTN = BM == 32 ? 2 : 4;
  __device__ static __forceinline__ int row(int wave) { return BM == 32 ? 0 : (wave >> 1) * (BM / 2); }
  __device__ static __forceinline__ int col(int wave) { return BM == 32 ? wave * 32 : (wave & 1) * 64; }
};

// The epilogue's way from accumulators to rows: the workgroup's BM x 128 block through
// LDS (stage: BM * 512 bytes), then f(row, column, four values) with 32 threads along a
// row, in a loop.  The code runs once in a workgroup, and fetching it costs more than
// running it (stores unrolled over the accumulators: 200 x 1024 x 1024 from 8-bit
// weights to binary32 20 us, so 15).
template <class WG, int BM, class V4, class F>
__device__ __forceinline__ void store_tile_rows(lds_char* stage, const V4 (&acc)[WG::WTM][WG::WTN], int tid, F f) {
  typedef __attribute__((address_space(3))) V4 lds_v4;
  using ACC = frag::Acc<frag::ACC_16x16>;
  const int lane = tid & 63, wave = tid >> 6;
  const int r0 = WG::row(wave) + ACC::coord(lane, 0).j, c0 = WG::col(wave) + ACC::coord(lane, 0).i;
#pragma unroll
  for (int i = 0; i < WG::WTM; ++i)
#pragma unroll
    for (int j = 0; j < WG::WTN; ++j) {  // a lane holds 4 consecutive columns of a row
      const int r = r0 + 16 * i, c = (c0 + 16 * j) / 4;
      *(lds_v4*)(stage + r * 512 + ((c ^ (r & 31)) << 4)) = acc[i][j];
    }
  barrier_tiles();
  const int c = tid & 31;
#pragma unroll 2
  for (int r = tid >> 5; r < BM; r += 8) {
    const V4 v = *(const lds_v4*)(stage + r * 512 + ((c ^ (r & 31)) << 4));
    f(r, 4 * c, v);
  }
}

// Sum over the K ranges, in their order, of four consecutive elements of an M x N
// matrix: SUM_BATCH loads in flight (one at a time, 13 ranges took 6 us).  w: the
// elements in the first range; n + 4 may pass N.
constexpr int SUM_BATCH = 8;
template <class V4, class T>
__device__ __forceinline__ V4 sum_ranges4(const T* w, int64_t slot, int splits, int64_t n, int64_t N) {
  V4 acc = {0, 0, 0, 0};
  for (int s0 = 0; s0 < splits; s0 += SUM_BATCH) {
    V4 v[SUM_BATCH];
#pragma unroll
    for (int u = 0; u < SUM_BATCH; ++u) {
      const T* src = w + min(s0 + u, splits - 1) * slot;
      if (N % 4 == 0) {
        v[u] = *(const V4*)src;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = src[min((int64_t)e, N - 1 - n)];
      }
    }
#pragma unroll
    for (int u = 0; u < SUM_BATCH; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += s0 + u < splits ? v[u][e] : (T)0;
  }
  return acc;
}

// Output tile of workgroup pid, grouped by 8 tile rows for L2 reuse.
__device__ __forceinline__ void general_tile(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int group = 8;
  const int tiles_in_group = group * tiles_n;
  const int first_m = pid / tiles_in_group * group;
  const int gsize = min(tiles_m - first_m, group);
  tm = first_m + (pid % tiles_in_group) % gsize;
  tn = (pid % tiles_in_group) / gsize;
}

// A general kernel, in us: a K tile of a workgroup alone on its compute unit, the time
// each of several takes of it, how many fit (their LDS), and the rest of a workgroup
// (the first tiles' latency, the code's first fetch, the epilogue)
// where it stores D.
struct TileCost {
  double alone, shared;
  int resident;
  double fixed;
};

// K ranges for `tiles` workgroups of nk K tiles each, from the time model
//   max(alone * rounds, shared * workgroups per unit) * ceil(nk / s)
//   + (s > 1 ? 7.5 + s * M * N * slot_us : fixed * rounds), in us,
// where a range's partial results make one trip through the workspace.
inline int64_t plan_ranges(int64_t tiles, int64_t nk, int64_t out_elems, int num_cu, const TileCost& c,
                           int64_t max_splits, double* us) {
  constexpr double SPLIT_FIXED_US = 3.0, SLOT_US = 3.2e-6, SPLIT_US = 4.5;
  auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  int64_t best = 1;
  double best_t = 0;
  for (int64_t s = 1; s == 1 || (s <= max_splits && s <= nk / 2 + 1); ++s) {
    if (s > 1 && cdiv(nk, cdiv(nk, s)) != s) continue;  // every range non-empty
    const int64_t per_cu = cdiv(tiles * s, num_cu), rounds = cdiv(per_cu, c.resident);
    const double kt = c.alone * (double)rounds > c.shared * (double)per_cu ? c.alone * (double)rounds : c.shared * (double)per_cu;
    const double t = kt * (double)cdiv(nk, s) + (s > 1 ? SPLIT_FIXED_US : c.fixed * (double)rounds) +
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
