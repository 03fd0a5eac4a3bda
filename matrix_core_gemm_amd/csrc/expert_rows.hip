// expert_rows.hip -- products of few rows, by group or over all rows, for K-contiguous
// operands with 16-byte rows: a decoding batch, bound by reading B once.
//
// A workgroup computes 16 RB rows x 32 columns; its 8 wavefronts share K, each a run of the
// 128-byte K tiles, and add their sums through LDS at the end, in their order.  Fragments go
// from memory to registers: a 16 x 16 instruction's lane holds 16 bytes of a row at a time,
// so that four lanes read 64 consecutive bytes of each row of B, and nothing is staged, waited
// for together or shared between wavefronts on the way.  A wavefront has up to U K tiles in flight (the
// compiler holds fewer, in 45 to 70 registers, for 7 or 8 wavefronts on a SIMD; all U at once, on 4 of
// them, took 85 us instead of 75 for 64 rows over 32 8-bit experts of 4096 x 4096).
//
// Bound: HBM where a group has one tile of 16 rows (8-bit, one row x 8192 x 8192 14.6 us, 4.6 TB/s;
// 23 of 32 experts in use, 75 us, 5.1 TB/s).  More rows: every workgroup reads its rows of A from L2
// beside 32 columns of B, at 28 KB a us and compute unit in all (32 rows x 8192 x 8192 24 us).
//
// 8-bit operands: a K tile is one block, whose sum is scaled as it is added (see
// f8_blocks_kernel.hpp).
#include "f8_blocks_kernel.hpp"

namespace mcg {
namespace few {

using namespace fast;
using f8b::Native;
using f8b::Wide;

constexpr int W = 8, CB = 2;  // wavefronts, 16-column blocks of a workgroup
constexpr int COLS = 16 * CB;

struct Bf16Op {
  static constexpr int EB = 2;
  __device__ static __forceinline__ f32x4 mma(const i32x4& b, const i32x4& a, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bit_cast<bf16x8>(b), bit_cast<bf16x8>(a), c, 0, 0, 0);
  }
};
struct F16Op {
  static constexpr int EB = 2;
  __device__ static __forceinline__ f32x4 mma(const i32x4& b, const i32x4& a, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(bit_cast<f16x8>(b), bit_cast<f16x8>(a), c, 0, 0, 0);
  }
};
template <class Block>
struct F8Op {
  static constexpr int EB = 1;
  using block_t = Block;
};

constexpr int AUX_NT = 2;  // non-temporal: B is read once, A by every workgroup
template <int AUX>
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return bit_cast<i32x4>(__builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, AUX));
}

template <class Op, int RB, int U>
__global__ __launch_bounds__(64 * W) void rows_kernel(GroupArgs p) {
  constexpr int EB = Op::EB;
  constexpr bool SCALED = EB == 1;
  __shared__ __attribute__((aligned(16))) f32x4 sums[W][RB * CB * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;

  int64_t m0, m_end = p.M, n0;
  const char* B = p.B;
  const float* sb = p.sb;
  if (p.offsets) {
    const PipeTile w = pipe_tile<16 * RB>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, lane);
    if (w.m0 >= w.r1) return;  // (the whole workgroup)
    m0 = w.m0;
    m_end = w.r1;
    n0 = (int64_t)w.tn * COLS;
    B += w.g * p.strideB * EB;
    if constexpr (SCALED) sb += w.g * p.strideSB;
  } else {
    const int pid = xcd_order(blockIdx.x, p.tiles_m * p.tiles_n);
    m0 = (int64_t)(pid % p.tiles_m) * (16 * RB);
    n0 = (int64_t)(pid / p.tiles_m) * COLS;
  }
  // K tiles [kt, end) of this wavefront
  const uint32_t kbytes = (uint32_t)(p.K * EB);
  const int nk = (int)((kbytes + 127) / 128);
  int kt = wave * nk / W;
  const int end = (wave + 1) * nk / W;

  const uint32_t lda = (uint32_t)(p.lda * EB), ldb = (uint32_t)(p.ldb * EB);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + m0 * p.lda * EB, (uint32_t)min(m_end - m0, (int64_t)(16 * RB)) * lda);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(B + n0 * p.ldb * EB, (uint32_t)min(p.N - n0, (int64_t)COLS) * ldb);
  // scales of rows c, c + 16, .. and of the workgroup's columns (all under one scale)
  __amdgpu_buffer_rsrc_t rs = ra;
  const float* sbk = nullptr;
  if constexpr (SCALED) {
    rs = make_rsrc(p.sa + m0 * p.ldsa, (uint32_t)(((min(m_end - m0, (int64_t)(16 * RB)) - 1) * p.ldsa + nk) * 4));
    sbk = sb + n0 / SCALE_BLOCK * p.ldsb;
  }
  f32x4 acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  for (; kt < end; kt += U) {
    i32x4 a[U][RB][2], b[U][CB][2];
    float s[SCALED ? U : 1][RB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t kb = (uint32_t)(kt + u) * 128 + 64 * h + 16 * g;
        const bool in = kt + u < end && kb < kbytes;
#pragma unroll
        for (int j = 0; j < CB; ++j) b[u][j][h] = load16<AUX_NT>(rb, in ? (c + 16 * j) * ldb + kb : BUF_OOB);
#pragma unroll
        for (int i = 0; i < RB; ++i) a[u][i][h] = load16<0>(ra, in ? (c + 16 * i) * lda + kb : BUF_OOB);
      }
      if constexpr (SCALED) {
        const int t = min(kt + u, end - 1);
        const float sbt = sbk[t];
#pragma unroll
        for (int i = 0; i < RB; ++i)
          s[u][i] = bit_cast<float>(__builtin_amdgcn_raw_buffer_load_b32(rs, (int)((c + 16 * i) * (uint32_t)p.ldsa * 4 + t * 4), 0, 0)) * sbt;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (SCALED) {
        using Block = typename Op::block_t;
        if (kt + u >= end) break;  // (zeros times a scale that may be no number)
        typename Block::frag_t fb[CB];
#pragma unroll
        for (int j = 0; j < CB; ++j)
          fb[j] = Block::b(i32x8{b[u][j][0].x, b[u][j][0].y, b[u][j][0].z, b[u][j][0].w, b[u][j][1].x, b[u][j][1].y, b[u][j][1].z, b[u][j][1].w});
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const auto fa =
              Block::a(i32x8{a[u][i][0].x, a[u][i][0].y, a[u][i][0].z, a[u][i][0].w, a[u][i][1].x, a[u][i][1].y, a[u][i][1].z, a[u][i][1].w});
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            const f32x4 v = Block::block(fb[j], fa);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(v[e], s[u][i], acc[i][j][e]);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) acc[i][j] = Op::mma(b[u][j][h], a[u][i][h], acc[i][j]);
      }
    }
  }

  // lane l of block (i, j): D[16 i + l % 16][16 j + 4 (l / 16) .. + 3]
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) sums[wave][(i * CB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int x = threadIdx.x; x < RB * CB * 64; x += 64 * W) {
    f32x4 v = sums[0][x];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w][x];
    const int l = x & 63, blk = x >> 6;
    const int64_t m = m0 + 16 * (blk / CB) + (l & 15), n = n0 + 16 * (blk % CB) + 4 * (l >> 4);
    if (m < m_end && n < p.N) group_store4(p, 0, m, n, v);
  }
}

template <class Op, int RB, int U>
static hipError_t launch_one(const GroupArgs& a0, hipStream_t s) {
  GroupArgs a = a0;
  a.tiles_m = (int)most_tiles(a.M, a.groups, 16 * RB, a.offsets != nullptr);
  a.tiles_n = (int)((a.N + COLS - 1) / COLS);
  const int64_t blocks = a.offsets ? slice_blocks(a.tiles_m, a.tiles_n) : (int64_t)a.tiles_m * a.tiles_n;
  if (blocks >= MANY_TILES) return hipErrorInvalidValue;
  hipLaunchKernelGGL((rows_kernel<Op, RB, U>), dim3((unsigned)blocks), dim3(64 * W), 0, s, a);
  return hipGetLastError();
}
template <class Op>
static hipError_t launch_op(int rows, const GroupArgs& a, hipStream_t s) {
  if (rows == 16) return launch_one<Op, 1, 4>(a, s);
  if constexpr (Op::EB == 1)
    if (rows == 64) return launch_one<Op, 4, 2>(a, s);
  return launch_one<Op, 2, 4>(a, s);
}

}  // namespace few

hipError_t launch_few_rows(int dt, int rows, bool wide, const GroupArgs& a, hipStream_t s) {
  using namespace few;
  if (dt == DT_BF16) return launch_op<Bf16Op>(rows, a, s);
  if (dt == DT_F16) return launch_op<F16Op>(rows, a, s);
  if (dt == DT_E4M3) return wide ? launch_op<F8Op<Wide<0>>>(rows, a, s) : launch_op<F8Op<Native<0>>>(rows, a, s);
  return wide ? launch_op<F8Op<Wide<1>>>(rows, a, s) : launch_op<F8Op<Native<1>>>(rows, a, s);
}

}  // namespace mcg
