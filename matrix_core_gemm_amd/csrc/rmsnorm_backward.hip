// rmsnorm_backward.hip -- backward pass of y = x * rstd * w, rstd = (mean(x^2) + eps)^(-1/2)
// over rows of n elements:
//
//   g = dy * w,  c = rstd^2 / n * sum(g x)
//   dx = rstd * (g - c x) + dr          (dr: the gradient of the residual stream)
//   dw = sum over the rows of dy * x * rstd
//
// x comes in the type of dy or as an 8-bit checkpoint (codes and one scale per row).
//
// A row's threads hold it in registers between the sum and dx (rows of 8 to 8192
// columns; others are read again).  dw is a sum over
// rows: each workgroup walks rows a fixed stride apart, adds its threads' columns
// in registers, and leaves one partial row in the workspace; a second kernel adds
// the partial rows in a fixed order (no atomics: the result does not depend on
// timing).  Everything is summed in binary32.
//
// Bound: memory (8 bytes per element with 16-bit x and dr).  8192 x 4096 bf16: 55 us
// (4.9 TB/s), of which the sum of the partial rows takes 4; with 1024 partial rows,
// summed by 8 threads a column one element at a time, and no loads ahead 87 us.  Rows
// above 8192 columns read x and dy twice for dx and once for dw: 8192 x 16384 bf16 329
// us, 3.3 TB/s of the bytes that it cannot do without.
#include "row_vec.hpp"

namespace mcg {
namespace rows {

constexpr int64_t MAX_PARTS = 512;   // partial rows of dw: workgroups of the row kernels
constexpr int64_t MAX_BLOCKS = 1 << 20;  // workgroups along the rows (a launch holds less than 2^32 threads)

// Elements between the partial rows: whole 16-byte vectors.
__host__ __device__ inline int64_t part_stride(int64_t n) { return (n + 3) & ~(int64_t)3; }

template <int TPR>
__device__ __forceinline__ float row_sum(float x, int phase) {
  x = wave_sum(x);
  if constexpr (TPR > 64) {
    constexpr int NWV = TPR / 64;
    __shared__ float ls[2][NWV];  // by turns: a wavefront may be one row ahead
    if ((threadIdx.x & 63) == 0) ls[phase][threadIdx.x >> 6] = x;
    __syncthreads();
    x = ls[phase][0];
#pragma unroll
    for (int i = 1; i < NWV; ++i) x += ls[phase][i];
  }
  return x;
}

// c of the formulas: rstd^2 / n * sum, one factor rstd at a time (its square leaves
// binary32 for rows of about 1e-19 and less, or 1e19 and more; sum * rstd has the size
// of n g).
__device__ __forceinline__ float row_factor(float sum, float rstd, int64_t n) { return sum * rstd / (float)n * rstd; }

template <int DT, int DTX>
__device__ __forceinline__ void load_x(const NormGradArgs& p, int64_t row, int64_t c, float (&x)[8]) {
  widen8<DTX>(load8<DTX>(p.X + row * p.ldx * elem_size<DTX>(), c, p.N), x);
  if constexpr (DTX == DT_I8) {
    const float s = p.xscale[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
  }
}

// dx of one vector from g and x.
template <int DT>
__device__ __forceinline__ void store_dx(const NormGradArgs& p, int64_t row, int64_t c, float rstd, float k,
                                         const float (&g)[8], const float (&x)[8]) {
  constexpr int ES = elem_size<DT>();
  float d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) d[e] = rstd * __builtin_fmaf(-k, x[e], g[e]);
  if (p.dR) {
    float r[8];
    widen8<DT>(load8<DT>(p.dR + row * p.lddr * ES, c, p.N), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] += r[e];
  }
  store8<DT>(p.dX + row * p.lddx * ES, c, p.N, narrow8<DT>(d));
}

// One row per TPR threads, NV vectors of eight elements per thread; a workgroup
// walks the rows a grid apart, the next row's loads in flight while it reduces this
// one (dX may be dY or dR, so that the compiler itself would keep them behind the
// stores), and leaves one partial row of dw.  Rows of at least 8 elements.
template <int DT, int DTX, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(NormGradArgs p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  constexpr int ES = elem_size<DT>();
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * RPW;
  RowVec at[NV];
  float dw[NV][8];
  Raw8<DT> w[NV], dy[NV], dr[NV];
  Raw8<DTX> xr[NV];
  float rstd = 0.0f, xs = 1.0f;
  auto load_row = [&](int64_t m) {
    rstd = p.rstd[m];
    if constexpr (DTX == DT_I8) xs = p.xscale[m];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      dy[v] = load_vec<DT>(p.dY + m * p.lddy * ES, at[v]);
      xr[v] = load_vec<DTX>(p.X + m * p.ldx * elem_size<DTX>(), at[v]);
      if (p.dR) dr[v] = load_vec<DT>(p.dR + m * p.lddr * ES, at[v]);
    }
  };
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    at[v] = row_vec((int64_t)(v * TPR + t) * 8, p.N);
    if (p.W) w[v] = load_vec<DT>(p.W, at[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  }
  int64_t row = (int64_t)blockIdx.x * RPW + sub;
  if (row < p.M) load_row(row);
  for (int phase = 0; row < p.M; row += step, phase ^= 1) {
    const float rs = rstd;
    float g[NV][8], x[NV][8], d[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      widen8<DT>(dy[v], g[v]);
      widen8<DTX>(xr[v], x[v]);
      if (p.dR) widen8<DT>(dr[v], d[v]);
      if constexpr (DTX == DT_I8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= xs;
      }
    }
    if (row + step < p.M) load_row(row + step);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      mask_vec(g[v], at[v]);
      mask_vec(x[v], at[v]);
      float wv[8];
      if (p.W) widen8<DT>(w[v], wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = __builtin_fmaf(g[v][e] * rs, x[v][e], dw[v][e]);
        if (p.W) g[v][e] *= wv[e];
        sum = __builtin_fmaf(g[v][e], x[v][e], sum);
      }
    }
    sum = row_sum<TPR>(sum, phase);
    const float k = row_factor(sum, rs, p.N);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = rs * __builtin_fmaf(-k, x[v][e], g[v][e]);
        if (p.dR) o[e] += d[v][e];
      }
      store_vec<DT>(p.dX + row * p.lddx * ES, at[v], narrow8<DT>(o));
    }
  }
  if (!p.dW) return;
  if constexpr (RPW > 1) {
    // the workgroup's wavefronts each hold rows of their own: one partial row of them
    __shared__ float acc[RPW][TPR * NV * 8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[sub][(v * 8 + e) * TPR + t] = dw[v][e];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 1; i < RPW; ++i) dw[v][e] += acc[i][(v * 8 + e) * TPR + t];
  }
  char* part = (char*)(p.part + blockIdx.x * part_stride(p.N));
#pragma unroll
  for (int v = 0; v < NV; ++v) store_vec<DT_F32>(part, at[v], narrow8<DT_F32>(dw[v]));
}

// Rows of any other length (above 8192, or under a vector): dx with the row read twice, and dw's partial rows column by
// column (blockIdx.y is the part, threads along the columns).
template <int DT, int DTX>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGradArgs p) {
  constexpr int ES = elem_size<DT>();
  int phase = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, phase ^= 1) {
    const float rstd = p.rstd[row];
    auto load = [&](int64_t c, float(&g)[8], float(&x)[8]) {
      load_x<DT, DTX>(p, row, c, x);
      widen8<DT>(load8<DT>(p.dY + row * p.lddy * ES, c, p.N), g);
      if (p.W) {
        float w[8];
        widen8<DT>(load8<DT>(p.W, c, p.N), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= w[e];
      }
    };
    float sum = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.N; c += 8192) {
      float g[8], x[8];
      load(c, g, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(g[e], x[e], sum);
    }
    sum = row_sum<1024>(sum, phase);
    const float k = row_factor(sum, rstd, p.N);
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.N; c += 8192) {
      float g[8], x[8];
      load(c, g, x);
      store_dx<DT>(p, row, c, rstd, k, g, x);
    }
  }
}
template <int DT, int DTX>
__global__ __launch_bounds__(256) void norm_grad_long_dw_kernel(NormGradArgs p) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= p.N) return;
  float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t row = blockIdx.y; row < p.M; row += p.parts) {
    float g[8], x[8];
    load_x<DT, DTX>(p, row, c, x);
    widen8<DT>(load8<DT>(p.dY + row * p.lddy * elem_size<DT>(), c, p.N), g);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = __builtin_fmaf(g[e] * rstd, x[e], dw[e]);
  }
  store8<DT_F32>((char*)(p.part + (int64_t)blockIdx.y * part_stride(p.N)), c, p.N, narrow8<DT_F32>(dw));
}

// dw = sum of the partial rows, 32 columns (one 128-byte line of a row) per
// workgroup: 32 groups of 8 threads take every 32nd part, SUM_BATCH loads in
// flight, and the groups' sums are added in order through LDS.
constexpr int SUM_BATCH = 8;
__global__ __launch_bounds__(256) void norm_grad_sum_kernel(NormGradArgs p) {
  const int c4 = threadIdx.x & 7, sub = threadIdx.x >> 3;
  const int64_t n = (int64_t)blockIdx.x * 32 + 4 * c4, stride = part_stride(p.N);
  __shared__ float ls[32][33];
  float s[4] = {0, 0, 0, 0};
  if (n < p.N) {
    const float* src = p.part + n;  // 16-byte aligned; past N the row's padding
    for (int64_t g0 = sub; g0 < p.parts; g0 += 32 * SUM_BATCH) {
      f32x4 v[SUM_BATCH];
#pragma unroll
      for (int u = 0; u < SUM_BATCH; ++u) {
        const int64_t g = g0 + 32 * u;
        v[u] = g < p.parts ? *(const f32x4*)(src + g * stride) : f32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int u = 0; u < SUM_BATCH; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[u][e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) ls[sub][4 * c4 + e] = s[e];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && col < p.N) {
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) d += ls[i][threadIdx.x];
    p.dW[col] = d;
  }
}

template <int DT, int DTX, int TPR, int NV>
static void launch_one(const NormGradArgs& a, hipStream_t s) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  hipLaunchKernelGGL((norm_grad_kernel<DT, DTX, TPR, NV>), dim3((unsigned)a.parts), dim3(RPW * TPR), 0, s, a);
}

template <int DT, int DTX>
static hipError_t launch_dt(const NormGradArgs& a, hipStream_t s) {
  const int64_t n = a.N;
  if (a.M > 0) {
    if (n >= 8 && n <= 512) launch_one<DT, DTX, 64, 1>(a, s);
    else if (n >= 8 && n <= 1024) launch_one<DT, DTX, 64, 2>(a, s);
    else if (n >= 8 && n <= 2048) launch_one<DT, DTX, 256, 1>(a, s);
    else if (n >= 8 && n <= 4096) launch_one<DT, DTX, 256, 2>(a, s);
    // (as one of 8192, 4999 columns took 89 us instead of 86 for 8000 rows)
    else if (n >= 8 && n <= 6144) launch_one<DT, DTX, 384, 2>(a, s);
    else if (n >= 8 && n <= 8192) launch_one<DT, DTX, 512, 2>(a, s);
    // (two vectors in each of 1024 threads, which have 128 registers, spilled 110 to 157
    // of them: bf16 1 x 8200 40 us, 8192 x 12288 1089, 8192 x 16384 1143; so 9, 244 and 329)
    else {
      if (a.dW) {  // first: dX may be the memory of dY
        const dim3 grid((unsigned)((n + 2047) / 2048), (unsigned)a.parts);
        hipLaunchKernelGGL((norm_grad_long_dw_kernel<DT, DTX>), grid, dim3(256), 0, s, a);
      }
      const unsigned blocks = (unsigned)(a.M < MAX_BLOCKS ? a.M : MAX_BLOCKS);
      hipLaunchKernelGGL((norm_grad_long_kernel<DT, DTX>), dim3(blocks), dim3(1024), 0, s, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dW) hipLaunchKernelGGL(norm_grad_sum_kernel, dim3((unsigned)((n + 31) / 32)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace rows

// Rows of the kernel's workgroups: 4 wavefronts with a row each up to 1024 columns.
int64_t norm_grad_parts(int64_t M, int64_t N) {
  const int64_t groups = N <= 1024 ? (M + 3) / 4 : M;
  return groups < rows::MAX_PARTS ? groups : rows::MAX_PARTS;
}
// (stated for one row per workgroup, whatever the kernel)
int64_t norm_grad_workspace(int64_t M, int64_t N) {
  return (M < rows::MAX_PARTS ? M : rows::MAX_PARTS) * rows::part_stride(N) * 4;
}

hipError_t launch_norm_grad(int dt, bool x8, const NormGradArgs& a0, hipStream_t s) {
  NormGradArgs a = a0;
  a.parts = norm_grad_parts(a.M, a.N);
  if (dt == DT_BF16)
    return x8 ? rows::launch_dt<DT_BF16, DT_I8>(a, s) : rows::launch_dt<DT_BF16, DT_BF16>(a, s);
  if (dt == DT_F16) return x8 ? rows::launch_dt<DT_F16, DT_I8>(a, s) : rows::launch_dt<DT_F16, DT_F16>(a, s);
  return x8 ? rows::launch_dt<rows::DT_F32, DT_I8>(a, s) : rows::launch_dt<rows::DT_F32, rows::DT_F32>(a, s);
}

}  // namespace mcg
