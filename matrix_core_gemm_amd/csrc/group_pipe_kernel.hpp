// group_pipe_kernel.hpp -- the pipelined 16-bit products by group, for operands with
// 16-byte rows:
//
//   rows   D[r][j] = sum_k A[r][k] B_g[k][j]               for the rows r of group g
//   grad   D_g[i][j] = sum_{r in g} A[r][i] B[r][j] + beta C_g[i][j]
//
// Tile TB x TB by 8 (TB 256) or 4 (TB 128) wavefronts, each (TB / 2) x 64 outputs as 32 x 32 x
// 16 instructions.  K tiles of 128 bytes of each row in two LDS stages (three of B), filled by
// buffer_load ... lds.  A wavefront walks down its rows 32 by 32: the next rows' fragments
// are read from LDS while 8 instructions (64 columns, whose fragments stay in registers) run
// on these.  The K tile's barrier stands two rows of instructions before its end, where
// the last fragments are in registers: its stage is then free for the K tile after next, and
// the instructions that are left cover the barrier and the DMA's issue.
//
// Bound: the matrix pipe within a long tile (one group of 8192 rows, 8192 x 8192, 833 us, 1320 TFLOP/s; its
// weight gradient 838); beside it a tile's prologue and epilogue, short last tiles and the last round
// (8192 rows over 16 ragged groups, 4096 x 4096, 315 us, 253 with 512 rows each; their weight gradients, 8 K tiles
// to a tile, 374).
#pragma once
#include "fast_tiles.hpp"
#include "group_epilogue.hpp"
#include "group_tiles.hpp"

namespace mcg {
namespace gpipe {

using namespace fast;

constexpr int KTB = 128, KE = KTB / 2;  // bytes and values of k of a K tile

// Fragments of N blocks of 32 rows (or columns) from rb on, all four instructions of a K tile.
template <int LAYOUT, int TB, int N>
__device__ __forceinline__ void read_frags(const lds_char* tile, int rb, int lane, i32x4 (&f)[N][4]) {
  using R = Reader<2, LAYOUT, TB, KTB>;
  const int g = lane >> 5;
  if constexpr (LAYOUT == LAYOUT_K) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int s = 0; s < 4; ++s) f[n][s] = R::read16k(tile, rb + 32 * n, 32 * s + 16 * g, lane);
  } else {
    constexpr int W = 2 * TB;  // bytes per LDS row (one k)
    uint32_t ad[2 * N];
    i32x2 r[2 * N][4];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) ad[2 * n + h] = R::mn_addr(tile, rb + 32 * n, 64 * h + 16 * g, lane);
    lds_read_tr_x4<2, 4 * W, 16 * W, 20 * W>(ad, r);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[n][2 * h] = i32x4{r[2 * n + h][0].x, r[2 * n + h][0].y, r[2 * n + h][1].x, r[2 * n + h][1].y};
        f[n][2 * h + 1] = i32x4{r[2 * n + h][2].x, r[2 * n + h][2].y, r[2 * n + h][3].x, r[2 * n + h][3].y};
      }
  }
}

// LDS stages of K tiles: a tile of half as many rows as columns has room for a third, which a group's
// short last tile needs, since its instructions do not cover a load's way.
template <int TBM, int TB>
struct Ring {
  static constexpr int STAGE_A = TBM * KTB, STAGE_B = TB * KTB;
  static constexpr int NA = TBM < TB ? 3 : 2, NB = 3, BYTES = NA * STAGE_A + NB * STAGE_B;
};

// The tile TBM x TB of D from row m0 (those below m_end) and column n0 on: TB / 32 wavefronts, two
// down the rows.  A: its first row of m0 = 0 (K-contiguous) or of k = 0.
template <class Op, int LA, int LB, int TBM, int TB, bool GRAD>
__device__ __forceinline__ void pipe_tile_work(const GroupArgs& p, lds_char* smem, const char* A, const char* B, int64_t K,
                                               int64_t m0, int64_t m_end, int64_t n0, int64_t dbase, int wave, int lane) {
  constexpr int NWAVES = TB / 32, WN = TB / 64;  // wavefronts, 2 x WN of them
  constexpr int WTM = TBM / 64, WTN = 2;         // 32 x 32 blocks of a wavefront
  using RG = Ring<TBM, TB>;
  constexpr int NA = RG::NA, NB = RG::NB;
  using DmaA = LineLoader<2, LA, TBM, KTB>;
  using DmaB = LineLoader<2, LB, TB, KTB>;
  constexpr int HALVES = NWAVES / 4, IA = DmaA::INSTR / HALVES, IB = DmaB::INSTR / HALVES;  // instructions per wavefront and K tile
  const int q = wave & 3, half = wave >> 2;
  const int rbA = (wave / WN) * (TBM / 2), rbB = (wave % WN) * 64;
  const int nk = (int)((K + KE - 1) / KE);

  f32x16 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j) acc[i][j] = f32x16{};

  if (!GRAD || nk > 0) {  // (a gradient's group may be empty: its sums are zero)
    DmaA da;
    DmaB db;
    if constexpr (LA == LAYOUT_K)
      da.init(A + m0 * p.lda * 2, (uint32_t)(min(m_end - m0, (int64_t)TBM) * p.lda * 2), p.lda, K, q, lane);
    else
      da.init(A + m0 * 2, mn_window(K, p.lda, m_end, m0, 2), p.lda, K, q, lane);
    if constexpr (LB == LAYOUT_K)
      db.init(B + n0 * p.ldb * 2, (uint32_t)(min(p.N - n0, (int64_t)TB) * p.ldb * 2), p.ldb, K, q, lane);
    else
      db.init(B + n0 * 2, mn_window(K, p.ldb, p.N, n0, 2), p.ldb, K, q, lane);
    auto stage_a = [&](int t) { return smem + (t % NA) * RG::STAGE_A; };
    auto stage_b = [&](int t) { return smem + NA * RG::STAGE_A + (t % NB) * RG::STAGE_B; };
    // (K tiles past the end: zeros)
    auto issue_a = [&](int t) { da.issue(stage_a(t), t, IA * half, IA, q); };
    auto issue_b = [&](int t) { db.issue(stage_b(t), t, IB * half, IB, q); };
    // loads of a wavefront that are younger than those of K tile t + 1 once K tiles t + NA - 1 of A and
    // t + NB - 1 of B are on their way (A before B of the same step)
    constexpr int NEWER = (NA - 2) * IA + (NB - 2) * IB;
#pragma unroll
    for (int t = 0; t < NB - NA; ++t) issue_b(t);
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      issue_a(t);
      issue_b(t + NB - NA);
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NA - 1) * (IA + IB) + (NB > NA ? IB : 0)) : "memory");  // own loads of K tile 0
    barrier_lds();
    i32x4 fb[WTN][4], fa[1][4], next[1][4];
    read_frags<LB, TB, WTN>(stage_b(0), rbB, lane, fb);
    read_frags<LA, TBM, 1>(stage_a(0), rbA, lane, next);
    // The K tiles, with LIVE of the wavefront's WTM blocks of rows inside the tile: a group's last
    // tile costs the instructions of its own rows only.  All wavefronts take the same barriers.
    auto k_loop = [&](auto live) {
      constexpr int LIVE = decltype(live)::value, LAST = LIVE > 2 ? LIVE - 2 : 0;
      for (int t = 0; t < nk; ++t) {
#pragma unroll
        for (int i = 0; i < (LIVE > 0 ? LIVE : 1); ++i) {
          if (i < LIVE) {
#pragma unroll
            for (int s = 0; s < 4; ++s) fa[0][s] = next[0][s];
          }
          if (i + 1 < LIVE) read_frags<LA, TBM, 1>(stage_a(t), rbA + 32 * (i + 1), lane, next);
          if (i == LAST) {
            // the last fragments are on their way: this stage is free once every wavefront is here,
            // and K tile t + 1 has landed once all but the newest loads have
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NEWER) : "memory");
            barrier_lds();
            issue_a(t + NA);
            issue_b(t + NB);
          }
          if (i < LIVE) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int j = 0; j < WTN; ++j) Op::mma(acc[i][j], fb[j][s], fa[0][s]);
          }
        }
        if (LIVE > 0) {
          read_frags<LA, TBM, 1>(stage_a(t + 1), rbA, lane, next);
          read_frags<LB, TB, WTN>(stage_b(t + 1), rbB, lane, fb);  // (past the end: zeros, not used)
        }
      }
    };
    const int64_t left = (m_end - m0 - rbA + 31) / 32;
    if constexpr (GRAD) k_loop(std::integral_constant<int, WTM>{});
    else with_live<WTM>(left < WTM ? (int)left : WTM, k_loop);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no LDS DMA outstanding at exit
    barrier_lds();
  }

  // Epilogue: register 4 u + e of lane l of block (i, j) is D[32 i + l % 32][32 j + 8 u + 4 (l / 32) + e].
  // 32 rows of a wavefront at a time go through its 8 KiB of LDS, so that 16 lanes then store a
  // row's 64 columns.
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  lds_char* wbuf = smem + wave * 8192;
  const int wr = lane & 31, rr = lane >> 4, cc = lane & 15;
#pragma unroll
  for (int i = 0; i < WTM; ++i) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < WTN; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int ch = 8 * j + 2 * u + (lane >> 5);
        *(lds_f32x4*)(wbuf + wr * 256 + ((ch ^ (wr & 15)) << 4)) =
            f32x4{acc[i][j][4 * u], acc[i][j][4 * u + 1], acc[i][j][4 * u + 2], acc[i][j][4 * u + 3]};
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    f32x4 v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int r = 4 * t + rr;
      v[t] = *(const lds_f32x4*)(wbuf + r * 256 + ((cc ^ (r & 15)) << 4));
    }
    const int64_t m = m0 + rbA + 32 * i + rr, n = n0 + rbB + 4 * cc;
    group_store_rows(p, dbase, m, m_end, n, v);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// TBM x TB tiles (256 x 256, 128 x 128, 64 x 128); with TBM = TB a group's last one of up to TB / 2 rows is
// TB / 2 x TB.
template <class Op, int LA, int LB, int TBM, int TB, bool GRAD>
__global__ __launch_bounds__(2 * TB) __attribute__((amdgpu_waves_per_eu(2, 2))) void group_pipe_kernel(GroupArgs p) {
  constexpr int LDS = Ring<TBM, TB>::BYTES;
  static_assert(LDS >= Ring<TB / 2, TB>::BYTES, "ring of a short tile");
  __shared__ __attribute__((aligned(1024))) char smem_raw[LDS];
  lds_char* smem = (lds_char*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if constexpr (GRAD) {
    // (groups one after the other, each spread over the XCDs: with whole groups on an XCD, the one with
    // the longest group ends last: 8192 rows over 16 experts, 4096 x 4096 515 us, so 385)
    const int tiles = p.tiles_m * p.tiles_n, g = blockIdx.x / tiles;
    int tm, tn;
    grouped_tile<4>(xcd_order(blockIdx.x - g * tiles, tiles), p.tiles_m, p.tiles_n, tm, tn);
    const GroupRows r = group_rows(p.offsets, g, p.K);
    pipe_tile_work<Op, LA, LB, TB, TB, true>(p, smem, p.A + r.r0 * p.lda * 2, p.B + r.r0 * p.ldb * 2, r.r1 - r.r0, (int64_t)tm * TB,
                                             p.M, (int64_t)tn * TB, g * p.strideD, wave, lane);
  } else {
    const PipeTile w = pipe_tile<TBM>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, lane);
    if (w.m0 >= w.r1) return;  // (the whole workgroup)
    const char* B = p.B + w.g * p.strideB * 2;
    if (TBM == TB && w.r1 - w.m0 > TB / 2)
      pipe_tile_work<Op, LA, LB, TB, TB, false>(p, smem, p.A, B, p.K, w.m0, w.r1, (int64_t)w.tn * TB, 0, wave, lane);
    else
      pipe_tile_work<Op, LA, LB, TB / 2, TB, false>(p, smem, p.A, B, p.K, w.m0, w.r1, (int64_t)w.tn * TB, 0, wave, lane);
  }
}

template <class Op, int LA, int LB, int TBM, int TB, bool GRAD>
hipError_t launch_one(const GroupArgs& a0, hipStream_t s) {
  GroupArgs a = a0;
  a.tiles_m = (int)(GRAD ? (a.M + TBM - 1) / TBM : most_tiles(a.M, a.groups, TBM, true));
  a.tiles_n = (int)((a.N + TB - 1) / TB);
  const int64_t blocks = GRAD ? (int64_t)a.tiles_m * a.tiles_n * a.groups : slice_blocks(a.tiles_m, a.tiles_n);
  if (blocks >= MANY_TILES) return hipErrorInvalidValue;
  hipLaunchKernelGGL((group_pipe_kernel<Op, LA, LB, TBM, TB, GRAD>), dim3((unsigned)blocks), dim3(2 * TB), 0, s, a);
  return hipGetLastError();
}

template <class Op, int TBM, int TB>
hipError_t launch_rows(int lb, const GroupArgs& a, hipStream_t s) {
  return lb == LAYOUT_K ? launch_one<Op, LAYOUT_K, LAYOUT_K, TBM, TB, false>(a, s)
                        : launch_one<Op, LAYOUT_K, LAYOUT_MN, TBM, TB, false>(a, s);
}
// tile: 256 and 128, square tiles; 64: (rows) 64 x 128
template <class Op>
hipError_t launch_op(int lb, bool grad, int tile, const GroupArgs& a, hipStream_t s) {
  if (grad)
    return tile == 256 ? launch_one<Op, LAYOUT_MN, LAYOUT_MN, 256, 256, true>(a, s)
                       : launch_one<Op, LAYOUT_MN, LAYOUT_MN, 128, 128, true>(a, s);
  return tile == 256   ? launch_rows<Op, 256, 256>(lb, a, s)
         : tile == 128 ? launch_rows<Op, 128, 128>(lb, a, s)
                       : launch_rows<Op, 64, 128>(lb, a, s);
}

}  // namespace gpipe
}  // namespace mcg
