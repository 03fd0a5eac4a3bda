// f8_blocks_kernel.hpp -- the pipelined product of block-scaled 8-bit floats, for
// operands with 16-byte rows, over all rows or by group:
//
//   D[i][j] = sum_b sa[i][b] sb[b][j] sum_{k in b} A[i][k] B[k][j] + beta C[i][j]
//
// The scales change with every block of 128 k, so a block's sum has to leave the matrix
// instruction before it is scaled.  One 16 x 16 x 128 instruction is one block of a 16 x 16
// tile, and its result four registers: p = A B (with no accumulator), then
// acc += (sa sb) p on the vector unit, 4 fused steps of 4 cycles for an instruction of 32
// cycles, which run beside the matrix core (the next row of instructions is
// issued first).  With 32 x 32 x 64 instructions a block is a chain of two and its result 16
// registers, which do not fit beside 128 accumulators and the fragments.
//
// Tile TB x TB by 8 (TB 256) or 4 (TB 128) wavefronts, each (TB / 2) x 64 outputs.  A K tile
// is one block: 128 bytes of each row, in two LDS stages filled by buffer_load ... lds (16
// bytes per lane), with its scales of the tile's rows and columns (one 4-byte load per lane).
// A wavefront walks down its rows 16 by 16: the next 16 rows' fragment is read from LDS
// while 4 instructions (64 columns, whose fragments stay in registers) run on this one.
// The K tile's barrier stands two rows of instructions before its end, where the last
// fragments are in registers: its stage is then free for the K tile after next, and the
// instructions that are left cover the barrier and the DMA's issue.
//
// For D in bf16 the products run on the 8-bit instruction, which keeps about 13 bits below the
// largest of 8 consecutive products: off by 2^-12 of D, typically, where bf16 rounds at
// 2^-8.  For f16 and binary32 D the codes are widened exactly to bf16 (WIDE), four
// instructions of 32 k for a block.
//
// Bound: the matrix and the vector pipe together.  8192^3 to bf16 takes 527 us (2090 TFLOP/s), 494 with scales
// that stay in registers, 418 with none; a weight gradient 4096^2 x 8192 to binary32 277 us (993
// TFLOP/s).  Smaller calls: 500 x 4096 x 4096 in one round of 64 x 128 tiles 20.9 us, of which a K tile takes
// 0.5; 8192 rows over 32 groups, 4096 x 4096, 234 us (the bytes alone 125).
#pragma once
#include "f8_block_ops.hpp"
#include "fast_tiles.hpp"
#include "group_epilogue.hpp"
#include "group_tiles.hpp"

namespace mcg {
namespace f8b {

using namespace fast;

constexpr int KT = SCALE_BLOCK;  // k (and bytes) of a K tile

// LDS rows of MN-contiguous tiles (one k each, TB bytes): 16-byte chunks are XOR-ed so that the
// transposing reads of 16 columns, 8 k from each of two lane groups 16 k apart in a cycle, fall
// in distinct banks.  The pattern repeats every 32 rows.
template <int TB>
__device__ __forceinline__ int mn_swz(int row) {
  static_assert(TB == 256 || TB == 128 || TB == 64, "tile");
  if constexpr (TB == 256) return (row & 7) | (8 * ((row >> 4) & 1));
  else if constexpr (TB == 128) return ((row >> 1) & 3) | (4 * ((row >> 4) & 1));
  else return ((row >> 2) & 1) | (2 * ((row >> 4) & 1));
}

// HBM -> LDS loader of one operand's K tiles: wavefront q of 4 writes LDS bytes
// [(i * 4 + q) * 1024, +1024) in instruction i, INSTR instructions in all.
template <int LAYOUT, int TB>
struct TileDma {
  static constexpr int INSTR = TB * KT / 4096;
  LineLoader<1, LAYOUT_K, TB, KT> line;  // K-contiguous
  __amdgpu_buffer_rsrc_t rsrc;           // MN-contiguous
  uint32_t voff[2], istride, kstride;

  // base: the operand's first row (or column) of the tile; rows of it that exist: mn
  __device__ __forceinline__ void init(const char* base, int64_t ld, int64_t mn, int64_t x0, int64_t K, int q, int lane) {
    if constexpr (LAYOUT == LAYOUT_K) {
      line.init(base + x0 * ld, (uint32_t)(min(mn - x0, (int64_t)TB) * ld), ld, K, q, lane);
    } else {
      rsrc = make_rsrc(base + x0, mn_window(K, ld, mn, x0, 1));
      constexpr int CPR = TB / 16, RPI = 256 / CPR;  // chunks per LDS row, rows per instruction
      const int c = q * 64 + lane, r = c / CPR;
      voff[0] = (uint32_t)(r * ld + 16 * ((c % CPR) ^ mn_swz<TB>(r)));
      voff[1] = (uint32_t)(r * ld + 16 * ((c % CPR) ^ mn_swz<TB>(r + RPI)));
      istride = __builtin_amdgcn_readfirstlane((uint32_t)(RPI * ld));
      kstride = __builtin_amdgcn_readfirstlane((uint32_t)(KT * ld));
    }
  }
  // instructions [i0, i0 + n) of K tile kt (past the end: zeros)
  template <int N>
  __device__ __forceinline__ void issue(lds_char* dst, int kt, int i0, int q) const {
    if constexpr (LAYOUT == LAYOUT_K) {
      line.issue(dst, kt, i0, N, q);
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int i = i0 + u;
        // (i0 is even: u tells which half of the pattern's 32 rows)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(dst + (i * 4 + q) * 1024), 16,
                                                 voff[TB == 256 ? u & 1 : 0] + (uint32_t)kt * kstride + (uint32_t)i * istride, 0, 0, 0);
      }
    }
  }
};

// Fragments: 32 k of a row (or column) in each lane, lane group g = lane / 16 with k 16 g .. 16 g +
// 15 and 64 + 16 g .. 64 + 16 g + 15 of the K tile.
template <int LAYOUT, int TB, int N>
__device__ __forceinline__ void read_frags(const lds_char* tile, int rb, int lane, i32x8 (&f)[N]) {
  const int g = lane >> 4;
  if constexpr (LAYOUT == LAYOUT_K) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = rb + 16 * n + (lane & 15), s = (r >> 1) & 7;
      const i32x4 x = lds_read_b128(tile, r * KT + ((g ^ s) << 4)), y = lds_read_b128(tile, r * KT + (((g + 4) ^ s) << 4));
      f[n] = i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
  } else {
    const int L = lane & 15, row = 16 * g + (L >> 1);
    uint32_t ad[N];
    i32x2 r[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) ad[n] = lds_addr(tile + row * TB + (((rb / 16 + n) ^ mn_swz<TB>(row)) << 4) + 8 * (L & 1));
    lds_read_tr_x4<1, 8 * TB, 64 * TB, 72 * TB>(ad, r);
#pragma unroll
    for (int n = 0; n < N; ++n)
      f[n] = i32x8{r[n][0].x, r[n][0].y, r[n][1].x, r[n][1].y, r[n][2].x, r[n][2].y, r[n][3].x, r[n][3].y};
  }
}

// LDS stages of K tiles, codes and scales: a tile of half as many rows as columns has room for a third,
// which a group's short last tile needs, since its instructions do not cover a load's way.
template <int TBM, int TB>
struct Ring {
  static constexpr int STAGE_A = TBM * KT, CODES = STAGE_A + TB * KT, STAGE = CODES + (TBM + TB) * 4;
  static constexpr int NS = TBM < TB ? 3 : 2, BYTES = NS * STAGE;
};

// The tile TBM x TB of D from row m0 (those below m_end) and column n0 on: TB / 32 wavefronts, two
// down the rows.  BLKB: columns of B under one scale (128 or 1).
template <class Op, int LA, int LB, int BLKB, int TBM, int TB>
__device__ __forceinline__ void f8_tile_work(const GroupArgs& p, lds_char* smem, const char* B, const float* sb, int64_t m0,
                                             int64_t m_end, int64_t n0, int wave, int lane) {
  constexpr int NWAVES = TB / 32, WN = TB / 64;  // wavefronts, 2 x WN of them
  constexpr int WTM = TBM / 32, WTN = 4;         // 16 x 16 blocks of a wavefront
  using RG = Ring<TBM, TB>;
  constexpr int NS = RG::NS;
  using DmaA = TileDma<LA, TBM>;
  using DmaB = TileDma<LB, TB>;
  constexpr int HALVES = NWAVES / 4, IA = DmaA::INSTR / HALVES, IB = DmaB::INSTR / HALVES;
  constexpr int NL = IA + IB + 1;  // load instructions per wavefront and K tile
  typedef __attribute__((address_space(3))) float lds_f32;
  const int q = wave & 3, half = wave >> 2;
  const int rbA = (wave / WN) * (TBM / 2), rbB = (wave % WN) * 64;
  const int nk = (int)((p.K + KT - 1) / KT);

  DmaA da;
  DmaB db;
  da.init(p.A, p.lda, m_end, m0, p.K, q, lane);
  db.init(B, p.ldb, p.N, n0, p.K, q, lane);
  // Scales of a K tile: the first wavefronts load those of the rows, the next those of the
  // columns, one for each lane, the others (of a tile of few rows) the same as the last of these.
  // (Past the end of either: zeros or another's, for outputs that are not stored.)
  const int ws = min(wave, (TBM + TB) / 64 - 1);
  const bool of_rows = ws < TBM / 64;
  const int sc = (of_rows ? ws : ws - TBM / 64) * 64 + lane;  // row or column of the tile
  __amdgpu_buffer_rsrc_t srs;
  uint32_t soff, sstride;
  {
    const int64_t nb = (p.N + BLKB - 1) / BLKB, c0 = n0 / BLKB;
    const int64_t cnt = of_rows ? min(m_end - m0, (int64_t)TBM) : min(nb - c0, (int64_t)(TB / BLKB));
    const int64_t ld = of_rows ? p.ldsa : p.ldsb, x0 = of_rows ? m0 : c0;
    const float* base = of_rows ? p.sa : sb;
    const int x = of_rows ? sc : sc / BLKB;
    if ((of_rows ? LA : LB) == LAYOUT_K) {
      srs = make_rsrc(base + x0 * ld, (uint32_t)(((cnt - 1) * ld + nk) * 4));
      soff = (uint32_t)(x * ld * 4);
      sstride = 4;
    } else {
      srs = make_rsrc(base + x0, (uint32_t)(((nk - 1) * ld + cnt) * 4));
      soff = (uint32_t)(x * 4);
      sstride = (uint32_t)(ld * 4);
    }
  }
  auto stage = [&](int t) { return smem + (t % NS) * RG::STAGE; };
  auto issue = [&](int t) {  // (K tiles past the end: zeros)
    lds_char* st = stage(t);
    da.template issue<IA>(st, t, IA * half, q);
    db.template issue<IB>(st + RG::STAGE_A, t, IB * half, q);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(srs, (__attribute__((address_space(3))) void*)(st + RG::CODES + ws * 256), 4,
                                             t < nk ? soff + (uint32_t)t * sstride : BUF_OOB, 0, 0, 0);
  };

  f32x4 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

#pragma unroll
  for (int t = 0; t < NS; ++t) issue(t);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * NL) : "memory");  // own loads of K tile 0
  barrier_lds();
  typename Op::frag_t fb[WTN];
  i32x8 rawa[1];
  auto read_b = [&](int t) {
    i32x8 r[WTN];
    read_frags<LB, TB, WTN>(stage(t) + RG::STAGE_A, rbB, lane, r);
#pragma unroll
    for (int j = 0; j < WTN; ++j) fb[j] = Op::b(r[j]);
  };
  read_b(0);
  read_frags<LA, TBM, 1>(stage(0), rbA, lane, rawa);
  // The K tiles, with LIVE of the wavefront's WTM blocks of rows inside the tile (in pairs): a
  // group's last tile costs the instructions of its own rows only.  All wavefronts take the same
  // barriers.
  auto k_loop = [&](auto pairs) {
    constexpr int LIVE = 2 * decltype(pairs)::value, LAST = LIVE > 2 ? LIVE - 2 : 0;
    for (int t = 0; t < nk; ++t) {
      const lds_char* st = stage(t);
      const lds_f32* ssa = (const lds_f32*)(st + RG::CODES);
      const lds_f32* ssb = ssa + TBM;
      float fs[LIVE > 0 ? LIVE : 1];
      f32x4 cs[BLKB == 1 ? WTN : 1];
      if (LIVE > 0) {
        const float sbu = BLKB == 1 ? 1.0f : ssb[rbB];
#pragma unroll
        for (int i = 0; i < LIVE; ++i) fs[i] = ssa[rbA + 16 * i + (lane & 15)] * sbu;
        if constexpr (BLKB == 1) {
          typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
#pragma unroll
          for (int j = 0; j < WTN; ++j) cs[j] = *(const lds_f32x4*)(ssb + rbB + 16 * j + 4 * (lane >> 4));
        }
      }
      f32x4 part[2][WTN];
      auto add = [&](int i) {
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = BLKB == 1 ? fs[i] * cs[BLKB == 1 ? j : 0][e] : fs[i];
            acc[i][j][e] = __builtin_fmaf(part[i & 1][j][e], s, acc[i][j][e]);
          }
      };
#pragma unroll
      for (int i = 0; i < (LIVE > 0 ? LIVE : 1); ++i) {
        typename Op::frag_t fa;
        if (i < LIVE) fa = Op::a(rawa[0]);
        if (i + 1 < LIVE) read_frags<LA, TBM, 1>(st, rbA + 16 * (i + 1), lane, rawa);
        if (i == LAST) {
          // the last fragments are on their way: this stage is free once every wavefront is here,
          // and K tile t + 1 has landed once all but the NS - 2 newest K tiles' loads have
          asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * NL) : "memory");
          barrier_lds();
          issue(t + NS);
        }
        if (i < LIVE) {
#pragma unroll
          for (int j = 0; j < WTN; ++j) part[i & 1][j] = Op::block(fb[j], fa);
          if (i > 0) add(i - 1);
        }
      }
      if (LIVE > 0) {
        read_frags<LA, TBM, 1>(stage(t + 1), rbA, lane, rawa);
        read_b(t + 1);  // (past the end: zeros, not used)
        add(LIVE - 1);
      }
    }
  };
  const int64_t left = (m_end - m0 - rbA + 31) / 32;
  if constexpr (LA == LAYOUT_MN) k_loop(std::integral_constant<int, WTM / 2>{});  // (no groups)
  else with_live<WTM / 2>(left < WTM / 2 ? (int)left : WTM / 2, k_loop);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no LDS DMA outstanding at exit
  barrier_lds();

  // Epilogue: lane l of block (i, j) holds D[16 i + l % 16][16 j + 4 (l / 16) .. + 3].  32 rows of a
  // wavefront at a time go through its 8 KiB of LDS, so that 16 lanes then store a row's 64 columns.
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  lds_char* wbuf = smem + wave * 8192;
  const int rr = lane >> 4, cc = lane & 15;
#pragma unroll
  for (int i = 0; i < WTM; i += 2) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < WTN; ++j) {
        const int r = 16 * h + cc, ch = 4 * j + rr;
        *(lds_f32x4*)(wbuf + r * 256 + ((ch ^ (r & 15)) << 4)) = acc[i + h][j];
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    f32x4 v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int r = 4 * t + rr;
      v[t] = *(const lds_f32x4*)(wbuf + r * 256 + ((cc ^ (r & 15)) << 4));
    }
    const int64_t m = m0 + rbA + 16 * i + rr, n = n0 + rbB + 4 * cc;
    group_store_rows(p, 0, m, m_end, n, v);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// TBM x TB tiles (256 x 256, 128 x 128, 64 x 128); with TBM = TB a group's last one of up to TB / 2 rows is
// TB / 2 x TB.
template <class Op, int LA, int LB, int BLKB, int TBM, int TB>
__global__ __launch_bounds__(2 * TB) __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_blocks_kernel(GroupArgs p) {
  constexpr bool GROUPS = LA == LAYOUT_K;  // (the weight gradient has none)
  constexpr int LDS = !GROUPS || Ring<TBM, TB>::BYTES > Ring<TB / 2, TB>::BYTES ? Ring<TBM, TB>::BYTES : Ring<TB / 2, TB>::BYTES;
  __shared__ __attribute__((aligned(1024))) char smem_raw[LDS];
  lds_char* smem = (lds_char*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (GROUPS && p.offsets) {
    const PipeTile w = pipe_tile<TBM>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, lane);
    if (w.m0 >= w.r1) return;  // (the whole workgroup)
    const char* B = p.B + w.g * p.strideB;
    const float* sb = p.sb + w.g * p.strideSB;
    if (TBM == TB && w.r1 - w.m0 > TB / 2)
      f8_tile_work<Op, LA, LB, BLKB, TB, TB>(p, smem, B, sb, w.m0, w.r1, (int64_t)w.tn * TB, wave, lane);
    else
      f8_tile_work<Op, LA, LB, BLKB, TB / 2, TB>(p, smem, B, sb, w.m0, w.r1, (int64_t)w.tn * TB, wave, lane);
  } else {
    int tm, tn;
    grouped_tile<4>(xcd_order(blockIdx.x, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, tm, tn);
    f8_tile_work<Op, LA, LB, BLKB, TBM, TB>(p, smem, p.B, p.sb, (int64_t)tm * TBM, p.M, (int64_t)tn * TB, wave, lane);
  }
}

template <class Op, int LA, int LB, int BLKB, int TBM, int TB>
hipError_t launch_one(const GroupArgs& a0, hipStream_t s) {
  GroupArgs a = a0;
  a.tiles_m = (int)most_tiles(a.M, a.groups, TBM, a.offsets != nullptr);
  a.tiles_n = (int)((a.N + TB - 1) / TB);
  const int64_t blocks = a.offsets ? slice_blocks(a.tiles_m, a.tiles_n) : (int64_t)a.tiles_m * a.tiles_n;
  if (blocks >= MANY_TILES) return hipErrorInvalidValue;
  hipLaunchKernelGGL((f8_blocks_kernel<Op, LA, LB, BLKB, TBM, TB>), dim3((unsigned)blocks), dim3(2 * TB), 0, s, a);
  return hipGetLastError();
}

// A layer's output, its input gradient and its weight gradient.
template <class Op, int TBM, int TB>
hipError_t launch_kinds(int la, int lb, const GroupArgs& a, hipStream_t s) {
  // (256 x 256 tiles of the weight gradient, with two products more for each scale, spill in the K loop:
  // 8192^3 1112 us, 672 in 128 x 128)
  if constexpr (TB == 128)
    if (la == LAYOUT_MN) return launch_one<Op, LAYOUT_MN, LAYOUT_MN, 1, TBM, TB>(a, s);
  return lb == LAYOUT_K ? launch_one<Op, LAYOUT_K, LAYOUT_K, 128, TBM, TB>(a, s)
                        : launch_one<Op, LAYOUT_K, LAYOUT_MN, 128, TBM, TB>(a, s);
}

}  // namespace f8b
}  // namespace mcg
