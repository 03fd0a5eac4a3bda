// expert_general.hip -- general kernels of the products by group and of block-scaled
// 8-bit floats: any size, pointer and leading dimension.
//
//   rows   D[r][j] = sum_k A[r][k] B_g[k][j]             for the rows r of group g
//   grad   D_g[i][j] = sum_{r in g} A[r][i] B[r][j] + beta C_g[i][j]
//   8-bit  D[i][j] = sum_b sa[i][b] sb[b][j] sum_{k in b} A[i][k] B[k][j] + beta C[i][j]
//                                                        (blocks b of 128 k; also by rows)
//
// Tiles of 128 (16-bit), 64 or 32 rows x 128 columns, 4 wavefronts; the loaders of tile_any.hpp
// (two K tiles ahead in registers, two stages in LDS).  A K tile of 8-bit values is one
// block of 128, whose sum leaves the matrix instructions before it is scaled and added
// (f8_block_ops.hpp: the 8-bit instruction for a bf16 D, else products widened to bf16).
//
// Bound: the general kernels' loop (one barrier per K tile between register-staged
// tiles), about half the matrix rate of the pipelined kernels: 8-bit 5658 x 1472 x 4672 from rows of odd lengths 172
// us; weight gradients of 777 rows over 5 groups, 1990 x 1147, 31 us.
#include "experts.hpp"
#include "f8_block_ops.hpp"
#include "group_epilogue.hpp"
#include "group_tiles.hpp"
#include "tile_any.hpp"

namespace mcg {

// 8-bit operands: Block is f8b::Native or f8b::Wide.
template <class Block>
struct OpBlocks {
  static constexpr int ELEM_BYTES = 1, STEPS = 1;
};
template <class Op>
struct IsScaled {
  static constexpr bool value = false;
  using block_t = void;
};
template <class Block>
struct IsScaled<OpBlocks<Block>> {
  static constexpr bool value = true;
  using block_t = Block;
};

template <class Op, int LA, int LB, int BM, bool GRAD>
__global__ __launch_bounds__(256, 2) void group_general_kernel(GroupArgs p) {
  constexpr int EB = Op::ELEM_BYTES, BN = 128, NT = 256, KE = KT_BYTES / EB;
  constexpr bool SCALED = IsScaled<Op>::value;
  using WG = WaveGrid<BM>;
  constexpr int WTM = WG::WTM, WTN = WG::WTN;
  using GA = TileGeom<EB, LA, BM>;
  using GB = TileGeom<EB, LB, BN>;
  using RA = FragReader<EB, SCALED ? 32 : 16, LA, BM>;
  using RB = FragReader<EB, SCALED ? 32 : 16, LB, BN>;
  constexpr int STAGE = GA::BYTES + GB::BYTES + (SCALED ? NT * 4 : 0);  // codes, and a scale from each thread
  __shared__ __attribute__((aligned(16))) char smem_raw[2 * STAGE];
  lds_char* smem = (lds_char*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rm = WG::row(wave), rn = WG::col(wave);

  // the tile: rows [m0, m_end) and columns from n0 on; for grad of group g's D, over K rows from r0
  int64_t m0, m_end, K = p.K, dbase = 0;
  const char *A = p.A, *B = p.B;
  const float* sb = p.sb;
  int tm, tn;
  if constexpr (GRAD) {
    const GroupRows r = group_rows(p.offsets, blockIdx.y, p.K);
    general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    m0 = (int64_t)tm * BM;
    m_end = p.M;
    K = r.r1 - r.r0;
    A += r.r0 * p.lda * EB;
    B += r.r0 * p.ldb * EB;
    dbase = (int64_t)blockIdx.y * p.strideD;
  } else if (p.offsets) {
    const int tiles = count_tiles<BM>(p.offsets, p.groups, p.M, lane);
    if ((int64_t)blockIdx.x >= (int64_t)tiles * p.tiles_n) return;  // (the whole workgroup)
    general_tile(blockIdx.x, tiles, p.tiles_n, tm, tn);
    const GroupTile w = find_tile<BM>(p.offsets, p.groups, p.M, tm, lane);
    m0 = w.r0 + (int64_t)w.t * BM;
    m_end = w.r1;
    if (m0 >= m_end) return;
    B += w.g * p.strideB * EB;
    if constexpr (SCALED) sb += w.g * p.strideSB;
  } else {
    general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    m0 = (int64_t)tm * BM;
    m_end = p.M;
  }
  const int64_t n0 = (int64_t)tn * BN;
  const int nk = (int)((K + KE - 1) / KE);

  f32x4 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  if (nk > 0) {  // (a gradient's group may be empty: its sums are zero)
    using LdA = AnyLoader<EB, LA, BM, NT>;
    using LdB = AnyLoader<EB, LB, BN, NT>;
    LdA la;
    LdB lb;
    la.init(A, p.lda, m0, m_end, K, tid);
    lb.init(B, p.ldb, n0, p.N, K, tid);
    constexpr int SETS = 2;
    typename LdA::Regs ra[SETS];
    typename LdB::Regs rb[SETS];
    // 8-bit: threads 0 .. 127 load the scales of the tile's columns, the others those of its rows (past
    // either's end: the last one's), zero for K tiles past the end.
    typedef __attribute__((address_space(3))) float lds_f32;
    const global_f32* scale = nullptr;
    int64_t scale_step = 1;
    float rs[SETS];
    if constexpr (SCALED) {
      if (tid < BN) {
        const int64_t n = min(n0 + tid, p.N - 1), c = p.blockB == 1 ? n : n / SCALE_BLOCK;
        scale = (const global_f32*)(sb + (LB == LAYOUT_K ? c * p.ldsb : c));
        if (LB == LAYOUT_MN) scale_step = p.ldsb;
      } else {
        const int64_t m = min(m0 + (tid - BN) % BM, m_end - 1);
        scale = (const global_f32*)(p.sa + (LA == LAYOUT_K ? m * p.ldsa : m));
        if (LA == LAYOUT_MN) scale_step = p.ldsa;
      }
    }
    auto load_tile = [&](auto set_c, int kt) {
      constexpr int set = decltype(set_c)::value;
      la.load(ra[set], kt, kt < nk);
      lb.load(rb[set], kt, kt < nk);
      if constexpr (SCALED) rs[set] = kt < nk ? scale[kt * scale_step] : *(const global_f32*)(const float*)load_nothing;
    };
    auto store_tile = [&](auto set_c, int kt) {
      constexpr int set = decltype(set_c)::value;
      lds_char* st = smem + (set & 1) * STAGE;
      la.settle(ra[set], kt);
      lb.settle(rb[set], kt);
      la.store(ra[set], st);
      lb.store(rb[set], st + GA::BYTES);
      if constexpr (SCALED) *(lds_f32*)(st + GA::BYTES + GB::BYTES + 4 * tid) = rs[set];
    };
    using ACC = frag::Acc<frag::ACC_16x16>;
    const int am = ACC::coord(lane, 0).j, an = ACC::coord(lane, 0).i;  // row and first of 4 columns in a block
    auto step = [&](auto set_c, int kt) {
      constexpr int set = decltype(set_c)::value;
      const lds_char* cur = smem + (set & 1) * STAGE;
      store_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1);
      load_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1 + SETS);
      if constexpr (SCALED) {
        using Block = typename IsScaled<Op>::block_t;
        const lds_f32* ssb = (const lds_f32*)(cur + GA::BYTES + GB::BYTES);
        const lds_f32* ssa = ssb + BN;
        typename Block::frag_t fb[WTN];
#pragma unroll
        for (int j = 0; j < WTN; ++j) fb[j] = Block::b(RB::read(cur + GA::BYTES, rn + j * 16, 0, lane));
#pragma unroll
        for (int i = 0; i < WTM; ++i) {
          const auto fa = Block::a(RA::read(cur, rm + i * 16, 0, lane));
          const float sa = ssa[rm + 16 * i + am];
#pragma unroll
          for (int j = 0; j < WTN; ++j) {
            typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
            const f32x4 part = Block::block(fb[j], fa), sc = *(const lds_f32x4*)(ssb + rn + 16 * j + an);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[e], sa * sc[e], acc[i][j][e]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < Op::STEPS; ++s) {
          i32x4 fa[WTM], fb[WTN];
#pragma unroll
          for (int i = 0; i < WTM; ++i) fa[i] = RA::read(cur, rm + i * 16, s, lane);
#pragma unroll
          for (int j = 0; j < WTN; ++j) fb[j] = RB::read(cur + GA::BYTES, rn + j * 16, s, lane);
#pragma unroll
          for (int i = 0; i < WTM; ++i)
#pragma unroll
            for (int j = 0; j < WTN; ++j) acc[i][j] = Op::mma(fb[j], fa[i], acc[i][j]);
        }
      }
      barrier_tiles();
    };
    for_each_set<SETS>([&](auto set) { load_tile(set, set); });
    store_tile(std::integral_constant<int, 0>{}, 0);
    load_tile(std::integral_constant<int, 0>{}, SETS);
    barrier_tiles();
    for (int kt = 0; kt < nk; kt += SETS) for_each_set<SETS>([&](auto set) { step(set, kt + set); });
  }
  static_assert(BM * 512 <= 2 * STAGE, "epilogue stage");
  store_tile_rows<WG, BM>(smem, acc, tid, [&](int r, int c, const f32x4& v) {
    if (m0 + r < m_end && n0 + c < p.N) group_store4(p, dbase, m0 + r, n0 + c, v);
  });
}

// Operands whose rows are shorter than a 16-byte load, and empty sums: one output per
// thread, the sums of a block of scales apart as elsewhere.
template <int DT>
__device__ __forceinline__ float tiny_value(const char* p, int64_t i) {
  if constexpr (DT == DT_BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
  else if constexpr (DT == DT_F16) return f16_bits_to_f32(((const uint16_t*)p)[i]);
  else if constexpr (DT == DT_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)(uint8_t)p[i], 0);
  else return __builtin_amdgcn_cvt_f32_bf8((int)(uint8_t)p[i], 0);
}
template <int DTA, int DTB>
__global__ __launch_bounds__(256) void group_tiny_kernel(GroupArgs p, int la, int lb, int grad) {
  constexpr bool SCALED = DTA == DT_E4M3 || DTA == DT_E5M2;
  constexpr int EB = SCALED ? 1 : 2;
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= p.N) return;
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    int64_t k0 = 0, k1 = p.K, dbase = 0;
    const char* B = p.B;
    const float* sb = p.sb;
    if (grad) {
      if (p.K > 0) {
        const GroupRows r = group_rows(p.offsets, blockIdx.z, p.K);
        k0 = r.r0;
        k1 = r.r1;
      }
      dbase = (int64_t)blockIdx.z * p.strideD;
    } else if (p.offsets) {
      int lo = 0, hi = p.groups;  // the last group that starts at or before m
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.offsets[mid] <= m) lo = mid;
        else hi = mid;
      }
      const GroupRows r = group_rows(p.offsets, lo, p.M);
      if (m < r.r0 || m >= r.r1) continue;
      B += lo * p.strideB * EB;
      if (SCALED) sb += lo * p.strideSB;
    }
    float acc = 0.0f, part = 0.0f;
    for (int64_t k = k0; k < k1; ++k) {
      const float a = tiny_value<DTA>(p.A, la == LAYOUT_K ? m * p.lda + k : k * p.lda + m);
      const float b = tiny_value<DTB>(B, lb == LAYOUT_K ? n * p.ldb + k : k * p.ldb + n);
      part = __builtin_fmaf(a, b, part);
      if constexpr (SCALED) {
        if (k + 1 < k1 && (k + 1) % SCALE_BLOCK != 0) continue;
        const int64_t blk = k / SCALE_BLOCK, c = p.blockB == 1 ? n : n / SCALE_BLOCK;
        const float s = p.sa[la == LAYOUT_K ? m * p.ldsa + blk : blk * p.ldsa + m] *
                        sb[lb == LAYOUT_K ? c * p.ldsb + blk : blk * p.ldsb + c];
        acc = __builtin_fmaf(part, s, acc);
        part = 0.0f;
      }
    }
    combine_store(p.C, p.D, dbase + m * p.ldc + n, SCALED ? acc : part, 1.0f, p.beta, p.use_c, p.out);
  }
}

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
}  // namespace

template <class Op, int LA, int LB, int BM, bool GRAD>
static hipError_t launch_one(const GroupArgs& a0, hipStream_t s) {
  GroupArgs a = a0;
  a.tiles_m = (int)(GRAD ? cdiv(a.M, BM) : most_tiles(a.M, a.groups, BM, a.offsets != nullptr));
  a.tiles_n = (int)cdiv(a.N, 128);
  const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n;
  if (blocks * (GRAD ? a.groups : 1) >= MANY_TILES) return hipErrorInvalidValue;
  hipLaunchKernelGGL((group_general_kernel<Op, LA, LB, BM, GRAD>), dim3((unsigned)blocks, GRAD ? (unsigned)a.groups : 1u),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}
template <class Op, int LA, int LB, bool GRAD>
static hipError_t launch_rows(const GroupArgs& a, int tile, hipStream_t s) {
  return tile == 32   ? launch_one<Op, LA, LB, 32, GRAD>(a, s)
         : tile == 64 ? launch_one<Op, LA, LB, 64, GRAD>(a, s)
                      : launch_one<Op, LA, LB, 128, GRAD>(a, s);
}
template <class Op>
static hipError_t launch_16(int lb, bool grad, const GroupArgs& a, int tile, hipStream_t s) {
  if (grad) return launch_rows<Op, LAYOUT_MN, LAYOUT_MN, true>(a, tile, s);
  return lb == LAYOUT_K ? launch_rows<Op, LAYOUT_K, LAYOUT_K, false>(a, tile, s)
                        : launch_rows<Op, LAYOUT_K, LAYOUT_MN, false>(a, tile, s);
}
// (8-bit tiles of 128 rows spill over 100 registers, or leave a compute unit with one workgroup: 5658 x 1472 x
// 4672 from rows of odd lengths 396 us, 172 in tiles of 64 rows)
template <class Op, int LA, int LB>
static hipError_t launch_rows8(const GroupArgs& a, int tile, hipStream_t s) {
  return tile == 32 ? launch_one<Op, LA, LB, 32, false>(a, s) : launch_one<Op, LA, LB, 64, false>(a, s);
}
template <class Op>
static hipError_t launch_8(int la, int lb, const GroupArgs& a, int tile, hipStream_t s) {
  if (la == LAYOUT_K)
    return lb == LAYOUT_K ? launch_rows8<Op, LAYOUT_K, LAYOUT_K>(a, tile, s)
                          : launch_rows8<Op, LAYOUT_K, LAYOUT_MN>(a, tile, s);
  return lb == LAYOUT_K ? launch_rows8<Op, LAYOUT_MN, LAYOUT_K>(a, tile, s)
                        : launch_rows8<Op, LAYOUT_MN, LAYOUT_MN>(a, tile, s);
}

hipError_t launch_group_general(int dt, int la, int lb, bool grad, const GroupArgs& a, int tile, hipStream_t s) {
  using f8b::Native;
  using f8b::Wide;
  if (dt == DT_BF16) return launch_16<OpBF16>(lb, grad, a, tile, s);
  if (dt == DT_F16) return launch_16<OpF16>(lb, grad, a, tile, s);
  const bool wide = a.out != OUT_BF16;
  if (dt == DT_E4M3) return wide ? launch_8<OpBlocks<Wide<0>>>(la, lb, a, tile, s) : launch_8<OpBlocks<Native<0>>>(la, lb, a, tile, s);
  return wide ? launch_8<OpBlocks<Wide<1>>>(la, lb, a, tile, s) : launch_8<OpBlocks<Native<1>>>(la, lb, a, tile, s);
}

hipError_t launch_group_tiny(int dt, int la, int lb, bool grad, const GroupArgs& a, hipStream_t s) {
  const int64_t cols = cdiv(a.N, 256), z = grad ? a.groups : 1;
  if (cols * z > MANY_TILES) return hipErrorInvalidValue;
  const int64_t most = MANY_TILES / (cols * z), rows = a.M < most ? a.M : most;
  const dim3 grid((unsigned)cols, (unsigned)(rows < 4096 ? rows : 4096), (unsigned)z);
  if (dt == DT_BF16) hipLaunchKernelGGL((group_tiny_kernel<DT_BF16, DT_BF16>), grid, dim3(256), 0, s, a, la, lb, (int)grad);
  else if (dt == DT_F16) hipLaunchKernelGGL((group_tiny_kernel<DT_F16, DT_F16>), grid, dim3(256), 0, s, a, la, lb, (int)grad);
  else if (dt == DT_E4M3) hipLaunchKernelGGL((group_tiny_kernel<DT_E4M3, DT_E4M3>), grid, dim3(256), 0, s, a, la, lb, (int)grad);
  else hipLaunchKernelGGL((group_tiny_kernel<DT_E5M2, DT_E4M3>), grid, dim3(256), 0, s, a, la, lb, (int)grad);
  return hipGetLastError();
}

}  // namespace mcg
