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
#include "tile_any.hpp"
#include "linear8.hpp"

namespace mcg {

// D of one output from its exact sum.
__device__ __forceinline__ float scaled_value(int acc, float sa, float sb, float bias) {
  return __builtin_fmaf((float)acc * sa, sb, bias);
}
// Four consecutive outputs at (m, n); n + 4 may pass N.
__device__ __forceinline__ void scaled_store4(const ScaledArgs& p, int64_t m, int64_t n, const i32x4& acc, float sa) {
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = n + e < p.N ? n + e : p.N - 1;
    o[e] = scaled_value(acc[e], sa, p.sb[c], p.bias ? p.bias[c] : 0.0f);
  }
  const int64_t off = m * p.ldd + n;
  const bool full = p.vec_d && n + 4 <= p.N;
  if (p.out == OUT_32) {
    float* D = (float*)p.D + off;
    if (full) *(f32x4*)D = f32x4{o[0], o[1], o[2], o[3]};
    else
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) D[e] = o[e];
  } else {
    uint16_t* D = (uint16_t*)p.D + off;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = to_out_bits(p.out, o[e]);
    if (full) *(i32x2*)D = i32x2{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
    else
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) D[e] = (uint16_t)b[e];
  }
}

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
      if (p.splits > 1) {
        int32_t* w = p.ws + ((int64_t)blockIdx.y * p.M + m) * p.N + n;
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) w[e] = acc[i][j][e];
      } else {
        scaled_store4(p, m, n, acc[i][j], sa);
      }
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
      const int32_t* w = p.ws + ((int64_t)s * p.M + m) * p.N + n;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) acc[e] += w[e];
    }
    scaled_store4(p, m, n, acc, p.sa[m]);
  }
}

// Fills the plan's fields and returns the workspace bytes it takes (at most ws_bytes).
int64_t plan_scaled(ScaledArgs& a, int, int num_cu, int64_t ws_bytes) {
  const int64_t nk = (a.K + KT_BYTES - 1) / KT_BYTES;
  a.tiles_m = (int)((a.M + 127) / 128);
  a.tiles_n = (int)((a.N + 127) / 128);
  const int64_t slot = a.M * a.N * 4;
  const int64_t most = slot > 0 ? ws_bytes / slot : 1;
  const int64_t s = plan_ranges((int64_t)a.tiles_m * a.tiles_n, nk, a.M * a.N, num_cu, 1.0, most < 64 ? most : 64);
  a.kt_per_split = (int)(nk > 0 ? (nk + s - 1) / s : 1);
  a.splits = (int)s;
  return s > 1 ? s * slot : 0;
}

hipError_t launch_scaled(int layoutB, const ScaledArgs& a, hipStream_t s) {
  const unsigned rows = (unsigned)(a.M < 4096 ? a.M : 4096);
  const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n;
  if (blocks > 0xffffff) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
  const dim3 grid((unsigned)blocks, (unsigned)a.splits);
  if (layoutB == LAYOUT_K) hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_K>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((scaled_general_kernel<LAYOUT_MN>), grid, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(scaled_finish_kernel, dim3((unsigned)((a.N + 1023) / 1024), rows), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mcg
