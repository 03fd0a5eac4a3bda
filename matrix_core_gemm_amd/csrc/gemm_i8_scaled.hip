// gemm_i8_scaled.hip -- int8 matrix product with a scale for each row of A (token)
// and each column of B (channel): D[i][j] = sa[i] * sb[j] * sum_k A[i][k] B[k][j] + bias[j].
//
// The sum is the exact int32 of the MFMA int8 instructions (K is limited so that
// it cannot wrap); it is rounded once to binary32, multiplied by sa and by sb,
// added to the bias and rounded to D's type.
//
// General kernel: tiles of 128, 64 or 32 rows (general_rows) x 128 columns, 4
// wavefronts, any size, pointer and leading dimension; the structure of
// dense_general.hpp with the loaders of tile_any.hpp.  K may be cut into
// ranges (few tiles, long K): each range leaves its int32 sums in the workspace and a
// second kernel adds them and applies the epilogue.
#include <algorithm>

#include "scaled_epilogue.hpp"
#include "tile_any.hpp"

namespace mcg {

template <int LB, int BM>
__global__ __launch_bounds__(256, 2) void scaled_general_kernel(ScaledArgs p) {
  constexpr int BN = 128, NT = 256;
  using WG = WaveGrid<BM>;
  constexpr int WTM = WG::WTM, WTN = WG::WTN;
  using Op = OpI8;
  using GA = TileGeom<1, LAYOUT_K, BM>;
  using GB = TileGeom<1, LB, BN>;
  using RA = FragReader<1, 16, LAYOUT_K, BM>;
  using RB = FragReader<1, 16, LB, BN>;
  __shared__ __attribute__((aligned(16))) char smem_raw[2 * (GA::BYTES + GB::BYTES)];
  lds_char* smem = (lds_char*)smem_raw;
  lds_char* ldsA[2] = {smem, smem + GA::BYTES + GB::BYTES};
  lds_char* ldsB[2] = {smem + GA::BYTES, smem + 2 * GA::BYTES + GB::BYTES};
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rm = WG::row(wave), rn = WG::col(wave);
  int tm, tn;
  general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nk_all = (int)((p.K + KT_BYTES - 1) / KT_BYTES);
  const int kt0 = (int)blockIdx.y * p.kt_per_split;
  const int nk = min(nk_all - kt0, p.kt_per_split);

  // SETS K tiles ahead in registers, two stages in LDS.  (One tile ahead, with loads the
  // compiler waited for at the end of every condition around them: one token x 8000 x
  // 8000, rows 8003 apart, 29 us; so 17.4, the streaming kernel's time for aligned rows.)
  using LdA = AnyLoader<1, LAYOUT_K, BM, NT>;
  using LdB = AnyLoader<1, LB, BN, NT>;
  LdA la;
  LdB lb;
  la.init(p.A, p.lda, m0, p.M, p.K, tid);
  lb.init(p.B, p.ldb, n0, p.N, p.K, tid);
  constexpr int SETS = 2;
  typename LdA::Regs ra[SETS];
  typename LdB::Regs rb[SETS];
  auto load_tile = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value;
    la.load(ra[set], kt0 + kt, kt < nk);
    lb.load(rb[set], kt0 + kt, kt < nk);
  };
  auto store_tile = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value;
    la.settle(ra[set], kt0 + kt);
    lb.settle(rb[set], kt0 + kt);
    la.store(ra[set], ldsA[set & 1]);
    lb.store(rb[set], ldsB[set & 1]);
  };
  i32x4 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // K tile kt, in stage kt % 2; tile kt + 1 goes from its registers to the other stage.
  // Tiles past the range are zeros, so that the last steps need no conditions.
  auto step = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value, cur = set & 1;
    store_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1);
    load_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1 + SETS);
#pragma unroll
    for (int s = 0; s < Op::STEPS; ++s) {
      i32x4 fa[WTM], fb[WTN];
#pragma unroll
      for (int i = 0; i < WTM; ++i) fa[i] = RA::read(ldsA[cur], rm + i * 16, s, lane);
#pragma unroll
      for (int j = 0; j < WTN; ++j) fb[j] = RB::read(ldsB[cur], rn + j * 16, s, lane);
#pragma unroll
      for (int i = 0; i < WTM; ++i)
#pragma unroll
        for (int j = 0; j < WTN; ++j) acc[i][j] = Op::mma(fb[j], fa[i], acc[i][j]);
    }
    barrier_tiles();
  };
  for_each_set<SETS>([&](auto set) { load_tile(set, set); });
  store_tile(std::integral_constant<int, 0>{}, 0);
  load_tile(std::integral_constant<int, 0>{}, SETS);
  barrier_tiles();
  for (int kt = 0; kt < nk; kt += SETS) for_each_set<SETS>([&](auto set) { step(set, kt + set); });
  static_assert(BM * 512 <= 2 * (GA::BYTES + GB::BYTES), "epilogue stage");
  if (p.splits > 1) {
    store_tile_rows<WG, BM>(smem, acc, tid, [&](int r, int c, const i32x4& v) {
      if (m0 + r < p.M && n0 + c < p.N) scaled_part4(p, blockIdx.y, m0 + r, n0 + c, v);
    });
    return;
  }
  const ScaledCols cols = scaled_cols(p, min(n0 + 4 * (tid & 31), p.N - 1));
  store_tile_rows<WG, BM>(smem, acc, tid, [&](int r, int c, const i32x4& v) {
    if (m0 + r < p.M && n0 + c < p.N) scaled_store4(p, m0 + r, n0 + c, v, p.sa[m0 + r], cols);
  });
}

// Operands of fewer than 16 bytes, which the general kernel's loads do not take, and
// empty sums: one output per thread.
template <int LB>
__global__ __launch_bounds__(256) void scaled_tiny_kernel(ScaledArgs p) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= p.N) return;
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    int acc = 0;
    for (int64_t k = 0; k < p.K; ++k)
      acc += (int)(int8_t)p.A[m * p.lda + k] * (int)(int8_t)p.B[LB == LAYOUT_K ? n * p.ldb + k : k * p.ldb + n];
    const float o[4] = {scaled_value(acc, p.sa[m], p.sb[n], p.bias ? p.bias[n] : 0.0f), 0, 0, 0};
    scaled_put4(p.D, m * p.ldc + n, p.out, o, false, 1);
  }
}

// Adds the K ranges' sums and applies the epilogue: 4 consecutive columns per thread.
__global__ __launch_bounds__(256) void scaled_finish_kernel(ScaledArgs p) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= p.N) return;
  const ScaledCols cols = scaled_cols(p, n);
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    const i32x4 acc = sum_ranges4<i32x4>((const int32_t*)p.ws + m * p.N + n, p.M * p.N, p.splits, n, p.N);
    scaled_store4(p, m, n, acc, p.sa[m], cols);
  }
}

namespace {
// K tiles of 128 values of the general kernel (fitted from 1 to 300 rows, 1000 to 8192
// columns and K 512 to 8192, rows 3 bytes longer than K, K in 1 to 16 ranges)
TileCost general_cost(int rows) {
  return rows == 32   ? TileCost{0.65, 0.65, 4, 3.0}
         : rows == 64 ? TileCost{0.85, 0.7, 3, 4.0}
                      : TileCost{1.2, 0.8, 2, 9.0};
}
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t round_up(int64_t x, int64_t y) { return cdiv(x, y) * y; }
constexpr int64_t LIM = (int64_t)1 << 31;  // buffer offsets stay below it
// Operands that the pipelined and streaming kernels take: 16-byte chunks, K whole
// chunks, and every offset (K tiles up to 4 past the end) below LIM.
bool offsets_ok(int64_t K, int64_t lda, int lb, int64_t ldb) {
  return 256 * lda < LIM && (lb == LAYOUT_K ? 256 : K + 4 * KT_BYTES) * ldb < LIM;
}
bool chunks_ok(const ScaledArgs& a, int lb) {
  return a.K > 0 && a.K % 16 == 0 && a.lda % 16 == 0 && a.ldb % 16 == 0 && (uintptr_t)a.A % 16 == 0 &&
         (uintptr_t)a.B % 16 == 0 && offsets_ok(a.K, a.lda, lb, a.ldb);
}
// Streaming kernel.  A compute unit keeps about 20 bytes per ns of B in flight, so B
// comes at HBM's rate only when every one has a block: the K ranges follow from
//   rounds * K tiles * STREAM_KT_US * rows + [s > 1] (SUM_US + s * M * N trips of 8 bytes),
// with at least STREAM_MIN_KT K tiles in a range.
constexpr double STREAM_KT_US = 0.2 / 32, STREAM_SUM_US = 4.0;  // per row of a block and K tile
constexpr int64_t STREAM_MIN_KT = 8;
constexpr int64_t PANEL_STEP = 256;  // columns of a panel come in whole tiles

// The pipelined problem on the copies of A and of a panel of B with nc columns.
ScaledArgs panel_args(int lb, const ScaledArgs& a, int64_t n0, int64_t nc) {
  ScaledArgs d = a;
  d.A = (const char*)a.ws;
  d.lda = a.kp;
  d.B = d.A + a.M * a.kp;
  d.ldb = lb == LAYOUT_K ? a.kp : a.ldb2;
  d.K = a.kp;
  d.N = nc;
  d.sb = a.sb + n0;
  d.bias = a.bias ? a.bias + n0 : nullptr;
  d.D = (char*)a.D + n0 * (a.out == OUT_32 ? 4 : 2);
  return d;
}
int64_t panel_bytes(int lb, const ScaledArgs& a) { return a.kp * (lb == LAYOUT_K ? a.panel_n : a.ldb2); }

// Fills the panel fields for ws_bytes of workspace: the modelled time and the bytes
// used, or a negative time when offsets or the workspace rule it out.
double plan_panels(int lb, ScaledArgs& a, int num_cu, int64_t ws_bytes, int64_t* used) {
  a.kp = round_up(a.K, 16);
  const int64_t fixed = a.M * a.kp;
  if (fixed >= ws_bytes || fixed / 16 >= LIM) return -1.0;
  // the widest panel that fits, cut into equal ones
  const int64_t most = std::min((ws_bytes - fixed) / a.kp, (LIM - 1) / (a.kp + 4 * KT_BYTES)) / 16 * 16;
  if (most < round_up(a.N, 16) && most < PANEL_STEP) return -1.0;
  const int64_t count = most >= round_up(a.N, 16) ? 1 : cdiv(a.N, most / PANEL_STEP * PANEL_STEP);
  a.panel_n = count == 1 ? a.N : round_up(cdiv(a.N, count), PANEL_STEP);
  a.ldb2 = round_up(a.panel_n, 16);
  if (!offsets_ok(a.kp, a.kp, lb, lb == LAYOUT_K ? a.kp : a.ldb2)) return -1.0;
  const int64_t bytes = fixed + panel_bytes(lb, a);
  ScaledArgs d = panel_args(lb, a, 0, a.panel_n);
  const PipePlan pp = plan_pipe(DT_I8, d, num_cu, ws_bytes - bytes);
  a.kernel = KERNEL_FAST;
  a.tile = pp.tile;
  a.sk_tiles = d.sk_tiles;
  // the last panel is narrower, and may take a stream-K split where the others do not
  ScaledArgs last = panel_args(lb, a, 0, a.N - (cdiv(a.N, a.panel_n) - 1) * a.panel_n);
  *used = bytes + std::max(pp.ws, plan_pipe(DT_I8, last, num_cu, ws_bytes - bytes).ws);
  constexpr double BYTE_US = 1 / 4.5e6, LAUNCH_US = 4.0;  // of the copies
  return 2.0 * fixed * BYTE_US + cdiv(a.N, a.panel_n) * (2.0 * panel_bytes(lb, a) * BYTE_US + LAUNCH_US + pp.us);
}
}  // namespace

// Fills the plan's fields and returns the workspace bytes it takes (at most ws_bytes).
//   - up to 32 rows in 16-byte chunks: the streaming kernel (reads B once);
//   - more rows: the pipelined kernel (whole tiles or stream-K; operands without
//     16-byte chunks go there as copies), or the general kernel, which reads any
//     operands in place and cuts K where there are few tiles; the modelled times
//     decide (4096^3, rows 4099 apart: 145 us in place, 79 with copies; 64 x 4096 x 4096:
//     14.7 and 28)
int64_t plan_scaled(ScaledArgs& a, int lb, int num_cu, int64_t ws_bytes) {
  const int64_t nk = cdiv(a.K, KT_BYTES);
  const int64_t slot = a.M * a.N * 4;
  const int64_t most = slot > 0 ? ws_bytes / slot : 1;
  a.splits = 1;
  a.kt_per_split = (int)(nk > 0 ? nk : 1);
  a.dp_tiles = a.sk_tiles = a.sk_wgs = 0;
  a.panel_n = 0;
  auto ranges = [&](int64_t s) {
    a.kt_per_split = (int)(nk > 0 ? cdiv(nk, s) : 1);
    a.splits = (int)(nk > 0 ? cdiv(nk, a.kt_per_split) : 1);
    return a.splits > 1 ? a.splits * slot : 0;
  };
  if (a.M <= 32 && chunks_ok(a, lb)) {
    a.kernel = KERNEL_STREAM;
    a.stream_bw = a.N >= 64 * (int64_t)num_cu || lb == LAYOUT_MN ? 128 : 32;
    const int64_t blocks = cdiv(a.N, a.stream_bw);
    int64_t best = 1;
    double best_us = 0.0;
    for (int64_t s = 1; s == 1 || (s <= most && nk / s >= STREAM_MIN_KT); ++s) {
      const double us = cdiv(blocks * s, num_cu) * cdiv(nk, s) * STREAM_KT_US * a.stream_bw +
                        (s > 1 ? STREAM_SUM_US + 2.0 * s * slot / 4.5e6 : 0.0);
      if (s == 1 || us < best_us) {
        best = s;
        best_us = us;
      }
    }
    return ranges(best);
  }
  const int rows = general_rows(a.M);
  const int64_t tiles_m = cdiv(a.M, rows), tiles_n = cdiv(a.N, 128);
  double general_us;
  const int64_t s = plan_ranges(tiles_m * tiles_n, nk, a.M * a.N, num_cu, general_cost(rows), most < 64 ? most : 64, &general_us);
  if (chunks_ok(a, lb)) {
    const PipePlan pp = plan_pipe(DT_I8, a, num_cu, ws_bytes);
    if (pp.us < general_us) {
      a.kernel = KERNEL_FAST;
      a.tile = pp.tile;
      return pp.ws;
    }
  } else if (a.K > 0) {
    int64_t used = 0;
    const double us = plan_panels(lb, a, num_cu, ws_bytes, &used);
    if (us > 0.0 && us < general_us) return used;
  }
  a.kernel = any_operand_ok(1, a.M, a.K, a.lda) && any_operand_ok(1, lb == LAYOUT_K ? a.N : a.K, lb == LAYOUT_K ? a.K : a.N, a.ldb)
                 ? KERNEL_GENERAL
                 : KERNEL_TINY;
  a.panel_n = 0;
  a.dp_tiles = a.sk_tiles = a.sk_wgs = 0;
  a.tile = rows;
  a.tiles_m = (int)tiles_m;
  a.tiles_n = (int)tiles_n;
  return ranges(a.kernel == KERNEL_TINY ? 1 : s);
}

static hipError_t launch_pipe(int lb, const ScaledArgs& a, hipStream_t s) {
  return a.tile == 256 ? launch_scaled_fast(lb, a, s) : a.tile == 128 ? launch_scaled_mid(lb, a, s) : launch_scaled_half(lb, a, s);
}

static hipError_t launch_panels(int lb, const ScaledArgs& a, int num_cu, hipStream_t s) {
  hipError_t e = hipSuccess;
  const AlignRows copy_a{a.A, a.lda, a.M, a.K, (char*)a.ws, a.kp, a.M};
  const int64_t bytes = a.M * a.kp + panel_bytes(lb, a);
  for (int64_t n0 = 0; n0 < a.N && e == hipSuccess; n0 += a.panel_n) {
    const int64_t nc = std::min(a.panel_n, a.N - n0);
    ScaledArgs d = panel_args(lb, a, n0, nc);
    const AlignRows copy_b = lb == LAYOUT_K ? AlignRows{a.B + n0 * a.ldb, a.ldb, nc, a.K, (char*)d.B, a.kp, nc}
                                            : AlignRows{a.B + n0, a.ldb, a.K, nc, (char*)d.B, a.ldb2, a.kp};
    e = n0 == 0 ? launch_align_rows(copy_a, s, &copy_b) : launch_align_rows(copy_b, s);
    if (e != hipSuccess) break;
    d.ws = (char*)a.ws + bytes;
    d.tile = plan_pipe(DT_I8, d, num_cu, a.ws_bytes - bytes).tile;
    e = launch_pipe(lb, d, s);
  }
  return e;
}

template <int BM>
static void launch_general(int lb, const ScaledArgs& a, dim3 grid, hipStream_t s) {
  if (lb == LAYOUT_K) hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_K, BM>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_MN, BM>), grid, dim3(256), 0, s, a);
}

hipError_t launch_scaled(int layoutB, const ScaledArgs& a, int num_cu, hipStream_t s) {
  if (a.panel_n > 0) return launch_panels(layoutB, a, num_cu, s);
  if (a.kernel == KERNEL_FAST) return launch_pipe(layoutB, a, s);
  hipError_t e;
  if (a.kernel == KERNEL_TINY) {
    const dim3 grid((unsigned)cdiv(a.N, 256), (unsigned)std::min<int64_t>(a.M, 65535));
    if (layoutB == LAYOUT_K) hipLaunchKernelGGL(scaled_tiny_kernel<LAYOUT_K>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(scaled_tiny_kernel<LAYOUT_MN>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (a.kernel == KERNEL_STREAM) {
    e = launch_scaled_stream(layoutB, a, s);
  } else {
    const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n;
    if (blocks > 0xffffff) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
    const dim3 grid((unsigned)blocks, (unsigned)a.splits);
    if (a.tile == 32) launch_general<32>(layoutB, a, grid, s);
    else if (a.tile == 64) launch_general<64>(layoutB, a, grid, s);
    else launch_general<128>(layoutB, a, grid, s);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(scaled_finish_kernel, dim3((unsigned)cdiv(a.N, 1024), (unsigned)(a.M < 4096 ? a.M : 4096)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}

}  // namespace mcg
