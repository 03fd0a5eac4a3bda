// group_pipe_kernel.hpp -- the pipelined 16-bit products by group, for operands with
// 16-byte rows:
//
//   rows   D[r][j] = sum_k A[r][k] B_g[k][j]               for the rows r of group g
//   grad   D_g[i][j] = sum_{r in g} A[r][i] B[r][j] + beta C_g[i][j]
//
// Tile TB x TB by 8 (TB 256) or 4 (TB 128) wavefronts, each (TB / 2) x 64 outputs as 32 x 32 x
// 16 instructions.  K tiles of 128 bytes of each row in two LDS stages, filled by
// buffer_load ... lds.  A wavefront walks down its rows 32 by 32: the next rows' fragments
// are read from LDS while 8 instructions (64 columns, whose fragments stay in registers) run
// on these.  The K tile's barrier stands two rows of instructions before its end, where
// the last fragments are in registers: its stage is then free for the K tile after next, and
// the instructions that are left cover the barrier and the DMA's issue.
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

template <class Op, int LA, int LB, int TB, bool GRAD>
__global__ __launch_bounds__(2 * TB) __attribute__((amdgpu_waves_per_eu(2, 2))) void group_pipe_kernel(GroupArgs p) {
  constexpr int NWAVES = TB / 32, WN = TB / 64;  // wavefronts, 2 x WN of them
  constexpr int WTM = TB / 64, WTN = 2;          // 32 x 32 blocks of a wavefront
  constexpr int STAGE = TB * KTB;
  using DmaA = LineLoader<2, LA, TB, KTB>;
  using DmaB = LineLoader<2, LB, TB, KTB>;
  constexpr int HALVES = NWAVES / 4, IA = DmaA::INSTR / HALVES;  // instructions per wavefront, operand and K tile
  static_assert(DmaA::INSTR == DmaB::INSTR, "square tiles");
  __shared__ __attribute__((aligned(1024))) char smem_raw[4 * STAGE];
  lds_char* smem = (lds_char*)smem_raw;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = wave & 3, half = wave >> 2;
  const int rbA = (wave / WN) * (TB / 2), rbB = (wave % WN) * 64;

  // the tile: rows [m0, m_end) and columns from n0 on, over K values of k
  int tm, tn;
  int64_t m0, m_end = p.M, K = p.K, dbase = 0;
  const char *A = p.A, *B = p.B;
  if constexpr (GRAD) {
    const int tiles = p.tiles_m * p.tiles_n, pid = xcd_order(blockIdx.x, tiles * p.groups);
    const int g = __builtin_amdgcn_readfirstlane(pid / tiles);
    grouped_tile<4>(pid - g * tiles, p.tiles_m, p.tiles_n, tm, tn);
    const GroupRows r = group_rows(p.offsets, g, p.K);
    m0 = (int64_t)tm * TB;
    K = r.r1 - r.r0;
    A += r.r0 * p.lda * 2;
    B += r.r0 * p.ldb * 2;
    dbase = g * p.strideD;
  } else {
    const int tiles = count_tiles<TB>(p.offsets, p.groups, p.M, lane);
    if ((int64_t)blockIdx.x >= (int64_t)tiles * p.tiles_n) return;  // (the whole workgroup)
    grouped_tile<4>(xcd_order(blockIdx.x, tiles * p.tiles_n), tiles, p.tiles_n, tm, tn);
    const GroupTile w = find_tile<TB>(p.offsets, p.groups, p.M, tm, lane);
    m0 = w.r0 + (int64_t)w.t * TB;
    m_end = w.r1;
    if (m0 >= m_end) return;
    B += w.g * p.strideB * 2;
  }
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int64_t n0 = (int64_t)tn * TB;
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
      da.init(A + m0 * p.lda * 2, (uint32_t)(min(m_end - m0, (int64_t)TB) * p.lda * 2), p.lda, K, q, lane);
    else
      da.init(A + m0 * 2, mn_window(K, p.lda, m_end, m0, 2), p.lda, K, q, lane);
    if constexpr (LB == LAYOUT_K)
      db.init(B + n0 * p.ldb * 2, (uint32_t)(min(p.N - n0, (int64_t)TB) * p.ldb * 2), p.ldb, K, q, lane);
    else
      db.init(B + n0 * 2, mn_window(K, p.ldb, p.N, n0, 2), p.ldb, K, q, lane);
    auto stage = [&](int t) { return smem + (t & 1) * (2 * STAGE); };
    auto issue = [&](int t) {  // (K tiles past the end: zeros)
      da.issue(stage(t), t, IA * half, IA, q);
      db.issue(stage(t) + STAGE, t, IA * half, IA, q);
    };
    issue(0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    barrier_lds();
    issue(1);
    i32x4 fb[WTN][4], fa[1][4], next[1][4];
    read_frags<LB, TB, WTN>(stage(0) + STAGE, rbB, lane, fb);
    read_frags<LA, TB, 1>(stage(0), rbA, lane, next);
    for (int t = 0; t < nk; ++t) {
#pragma unroll
      for (int i = 0; i < WTM; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) fa[0][s] = next[0][s];
        if (i + 1 < WTM) read_frags<LA, TB, 1>(stage(t), rbA + 32 * (i + 1), lane, next);
        if (i == WTM - 2) {
          // the last fragments are on their way: this stage is free once every wavefront is here,
          // and K tile t + 1 (whose loads went out a K tile ago) has landed
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          barrier_lds();
          issue(t + 2);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < WTN; ++j) Op::mma(acc[i][j], fb[j][s], fa[0][s]);
      }
      read_frags<LA, TB, 1>(stage(t + 1), rbA, lane, next);
      read_frags<LB, TB, WTN>(stage(t + 1) + STAGE, rbB, lane, fb);  // (past the end: zeros, not used)
    }
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
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (m + 4 * t < m_end && n < p.N) group_store4(p, dbase, m + 4 * t, n, v[t]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <class Op, int LA, int LB, int TB, bool GRAD>
hipError_t launch_one(const GroupArgs& a0, hipStream_t s) {
  GroupArgs a = a0;
  a.tiles_m = (int)(GRAD ? (a.M + TB - 1) / TB : most_tiles(a.M, a.groups, TB, true));
  a.tiles_n = (int)((a.N + TB - 1) / TB);
  const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n * (GRAD ? a.groups : 1);
  if (blocks >= MANY_TILES) return hipErrorInvalidValue;
  hipLaunchKernelGGL((group_pipe_kernel<Op, LA, LB, TB, GRAD>), dim3((unsigned)blocks), dim3(2 * TB), 0, s, a);
  return hipGetLastError();
}

template <class Op, int TB>
hipError_t launch_kinds(int lb, bool grad, const GroupArgs& a, hipStream_t s) {
  if (grad) return launch_one<Op, LAYOUT_MN, LAYOUT_MN, TB, true>(a, s);
  return lb == LAYOUT_K ? launch_one<Op, LAYOUT_K, LAYOUT_K, TB, false>(a, s)
                        : launch_one<Op, LAYOUT_K, LAYOUT_MN, TB, false>(a, s);
}

}  // namespace gpipe
}  // namespace mcg
