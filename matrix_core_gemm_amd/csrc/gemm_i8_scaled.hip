// gemm_i8_scaled.hip -- int8 matrix product with a scale for each row of A (token)
// and each column of B (channel): D[i][j] = sa[i] * sb[j] * sum_k A[i][k] B[k][j] + bias[j].
//
// The sum is the exact int32 of the MFMA int8 instructions (K is limited so that
// it cannot wrap); it is rounded once to binary32, multiplied by sa and by sb,
// added to the bias and rounded to D's type.
//
// General kernel: 128 x 128 tiles, 4 wavefronts, any size, pointer and leading
// dimension; the structure of dense_general.hpp with the loaders of tile_any.hpp.
// K may be cut into ranges (few tiles, long K): each range leaves its int32 sums
// in the workspace and a second kernel adds them and applies the epilogue.
#include <algorithm>

#include "scaled_epilogue.hpp"
#include "tile_any.hpp"

namespace mcg {

template <int LB>
__global__ __launch_bounds__(256) void scaled_general_kernel(ScaledArgs p) {
  constexpr int BM = 128, BN = 128, NT = 256, WT = 4;
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
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nk_all = (int)((p.K + KT_BYTES - 1) / KT_BYTES);
  const int kt0 = (int)blockIdx.y * p.kt_per_split;
  const int nk = min(nk_all - kt0, p.kt_per_split);

  AnyLoader<1, LAYOUT_K, BM, NT> la;
  AnyLoader<1, LB, BN, NT> lb;
  auto load_tiles = [&](int kt) {
    const int64_t k0 = (int64_t)(kt0 + kt) * KT_BYTES;
    la.load(p.A, p.lda, m0, k0, p.M, p.K, tid);
    if constexpr (LB == LAYOUT_K) lb.load(p.B, p.ldb, n0, k0, p.N, p.K, tid);
    else lb.load(p.B, p.ldb, k0, n0, p.K, p.N, tid);
  };
  i32x4 acc[WT][WT];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int j = 0; j < WT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  if (nk > 0) {
    load_tiles(0);
    la.store(ldsA[0], tid);
    lb.store(ldsB[0], tid);
    __syncthreads();
  }
  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < nk) load_tiles(kt + 1);
#pragma unroll
    for (int s = 0; s < Op::STEPS; ++s) {
      i32x4 fa[WT], fb[WT];
#pragma unroll
      for (int i = 0; i < WT; ++i) fa[i] = RA::read(ldsA[cur], wm * 64 + i * 16, s, lane);
#pragma unroll
      for (int j = 0; j < WT; ++j) fb[j] = RB::read(ldsB[cur], wn * 64 + j * 16, s, lane);
#pragma unroll
      for (int i = 0; i < WT; ++i)
#pragma unroll
        for (int j = 0; j < WT; ++j) acc[i][j] = Op::mma(fb[j], fa[i], acc[i][j]);
    }
    if (kt + 1 < nk) {
      la.store(ldsA[cur ^ 1], tid);
      lb.store(ldsB[cur ^ 1], tid);
    }
    __syncthreads();
  }
  // a lane holds 4 consecutive columns of one row of each 16 x 16 block
  using ACC = frag::Acc<frag::ACC_16x16>;
  const int acc_m = ACC::coord(lane, 0).j, acc_n = ACC::coord(lane, 0).i;
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    const int64_t m = m0 + wm * 64 + i * 16 + acc_m;
    if (m >= p.M) continue;
    const float sa = p.splits > 1 ? 0.0f : p.sa[m];
#pragma unroll
    for (int j = 0; j < WT; ++j) {
      const int64_t n = n0 + wn * 64 + j * 16 + acc_n;
      if (n >= p.N) continue;
      if (p.splits > 1) scaled_part4(p, blockIdx.y, m, n, acc[i][j]);
      else scaled_store4(p, m, n, acc[i][j], sa);
    }
  }
}

// Adds the K ranges' sums and applies the epilogue: 4 consecutive columns per thread.
__global__ __launch_bounds__(256) void scaled_finish_kernel(ScaledArgs p) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= p.N) return;
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    i32x4 acc = {0, 0, 0, 0};
    for (int s = 0; s < p.splits; ++s) {
      const int32_t* w = (const int32_t*)p.ws + ((int64_t)s * p.M + m) * p.N + n;
      if (p.N % 4 == 0) {
        const i32x4 v = *(const i32x4*)w;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) acc[e] += w[e];
      }
    }
    scaled_store4(p, m, n, acc, p.sa[m]);
  }
}

namespace {
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
// Streaming kernel: blocks of 32 channels until there are 64 per compute unit.
constexpr int64_t STREAM_MIN_BLOCKS = 128, STREAM_MIN_KT = 16;
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
  *used = bytes + pp.ws;
  return pass_us(2.0 * fixed) + cdiv(a.N, a.panel_n) * (pass_us(2.0 * panel_bytes(lb, a)) + pp.us);
}
}  // namespace

// Fills the plan's fields and returns the workspace bytes it takes (at most ws_bytes).
//   - up to 32 rows in 16-byte chunks: the streaming kernel (reads B once);
//   - more rows in 16-byte chunks: the pipelined kernel, whole tiles or stream-K;
//   - other operands: the general kernel reads them in place at any alignment, or
//     copies with 16-byte chunks go to the pipelined kernel; the modelled times
//     decide: PANEL_NOTE
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
  if (chunks_ok(a, lb)) {
    if (a.M <= 32) {
      a.kernel = KERNEL_STREAM;
      a.stream_bw = a.N >= 64 * (int64_t)num_cu || lb == LAYOUT_MN ? 128 : 32;
      const int64_t blocks = cdiv(a.N, a.stream_bw);
      int64_t s = 1;
      if (blocks < STREAM_MIN_BLOCKS)
        s = std::max<int64_t>(1, std::min(cdiv(STREAM_MIN_BLOCKS, blocks), nk / STREAM_MIN_KT));
      return ranges(std::max<int64_t>(1, std::min(s, most)));
    }
    const PipePlan pp = plan_pipe(DT_I8, a, num_cu, ws_bytes);
    a.kernel = KERNEL_FAST;
    a.tile = pp.tile;
    return pp.ws;
  }
  a.kernel = KERNEL_GENERAL;
  a.tiles_m = (int)cdiv(a.M, 128);
  a.tiles_n = (int)cdiv(a.N, 128);
  double general_us;
  const int64_t s = plan_ranges((int64_t)a.tiles_m * a.tiles_n, nk, a.M * a.N, num_cu, 1.0, most < 64 ? most : 64, &general_us);
  if (a.K > 0) {
    int64_t used = 0;
    const double us = plan_panels(lb, a, num_cu, ws_bytes, &used);
    if (us > 0.0 && us < general_us) return used;
    a.panel_n = 0;
    a.dp_tiles = a.sk_tiles = a.sk_wgs = 0;
  }
  return ranges(s);
}

static hipError_t launch_pipe(int lb, const ScaledArgs& a, hipStream_t s) {
  return a.tile == 256 ? launch_scaled_fast(lb, a, s) : a.tile == 128 ? launch_scaled_mid(lb, a, s) : launch_scaled_half(lb, a, s);
}

static hipError_t launch_panels(int lb, const ScaledArgs& a, int num_cu, hipStream_t s) {
  hipError_t e = launch_align_rows(a.A, a.lda, a.M, a.K, a.ws, a.kp, a.M, s);
  const int64_t bytes = a.M * a.kp + panel_bytes(lb, a);
  for (int64_t n0 = 0; n0 < a.N && e == hipSuccess; n0 += a.panel_n) {
    const int64_t nc = std::min(a.panel_n, a.N - n0);
    ScaledArgs d = panel_args(lb, a, n0, nc);
    e = lb == LAYOUT_K ? launch_align_rows(a.B + n0 * a.ldb, a.ldb, nc, a.K, (void*)d.B, a.kp, nc, s)
                       : launch_align_rows(a.B + n0, a.ldb, a.K, nc, (void*)d.B, a.ldb2, a.kp, s);
    if (e != hipSuccess) break;
    d.ws = (char*)a.ws + bytes;
    d.tile = plan_pipe(DT_I8, d, num_cu, a.ws_bytes - bytes).tile;
    e = launch_pipe(lb, d, s);
  }
  return e;
}

hipError_t launch_scaled(int layoutB, const ScaledArgs& a, int num_cu, hipStream_t s) {
  if (a.panel_n > 0) return launch_panels(layoutB, a, num_cu, s);
  if (a.kernel == KERNEL_FAST) return launch_pipe(layoutB, a, s);
  hipError_t e;
  if (a.kernel == KERNEL_STREAM) {
    e = launch_scaled_stream(layoutB, a, s);
  } else {
    const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n;
    if (blocks > 0xffffff) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
    const dim3 grid((unsigned)blocks, (unsigned)a.splits);
    if (layoutB == LAYOUT_K) hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_K>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_MN>), grid, dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(scaled_finish_kernel, dim3((unsigned)cdiv(a.N, 1024), (unsigned)(a.M < 4096 ? a.M : 4096)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}

}  // namespace mcg
