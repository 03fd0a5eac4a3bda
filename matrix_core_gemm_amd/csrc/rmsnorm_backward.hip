// rmsnorm_backward.hip -- backward pass of y = x * rstd * w, rstd = (mean(x^2) + eps)^(-1/2)
// over rows of n elements:
//
//   g = dy * w,  c = rstd^2 / n * sum(g x)
//   dx = rstd * (g - c x) + dr          (dr: the gradient of the residual stream)
//   dw = sum over the rows of dy * x * rstd
//
// x comes in the type of dy or as an 8-bit checkpoint (codes and one scale per row).
//
// A row's threads hold it in registers between the sum and dx.  dw is a sum over
// rows: each workgroup walks rows a fixed stride apart, adds its threads' columns
// in registers, and leaves one partial row in the workspace; a second kernel adds
// the partial rows in a fixed order (no atomics: the result does not depend on
// timing).  Everything is summed in binary32.
//
// Bound: memory (8 bytes per element with 16-bit x and dr).
#include "row_vec.hpp"

namespace mcg {
namespace rows {

constexpr int64_t MAX_PARTS = 1024;  // partial rows of dw
constexpr int64_t MAX_BLOCKS = 1 << 20;  // workgroups along the rows (a launch holds less than 2^32 threads)

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

template <int DT, int DTX, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(NormGradArgs p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  constexpr int ES = elem_size<DT>();
  const int t = threadIdx.x % TPR;
  const int64_t first = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  if (first >= p.parts) return;  // whole wavefronts, and only where a row is one wavefront
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (p.W) {
      widen8<DT>(load8<DT>(p.W, (int64_t)(v * TPR + t) * 8, p.N), w[v]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[v][e] = 1.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  }
  int phase = 0;
  for (int64_t row = first; row < p.M; row += p.parts, phase ^= 1) {
    const float rstd = p.rstd[row];
    float g[NV][8], x[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = (int64_t)(v * TPR + t) * 8;
      load_x<DT, DTX>(p, row, c, x[v]);
      widen8<DT>(load8<DT>(p.dY + row * p.lddy * ES, c, p.N), g[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = __builtin_fmaf(g[v][e] * rstd, x[v][e], dw[v][e]);
        g[v][e] *= w[v][e];
        sum = __builtin_fmaf(g[v][e], x[v][e], sum);
      }
    sum = row_sum<TPR>(sum, phase);
    const float k = sum * (rstd * rstd) / (float)p.N;
#pragma unroll
    for (int v = 0; v < NV; ++v) store_dx<DT>(p, row, (int64_t)(v * TPR + t) * 8, rstd, k, g[v], x[v]);
  }
  if (p.dW) {
    char* part = (char*)(p.part + first * p.N);
#pragma unroll
    for (int v = 0; v < NV; ++v) store8<DT_F32>(part, (int64_t)(v * TPR + t) * 8, p.N, narrow8<DT_F32>(dw[v]));
  }
}

// Rows of any length: dx with the row read twice, and dw's partial rows column by
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
    const float k = sum * (rstd * rstd) / (float)p.N;
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
  store8<DT_F32>((char*)(p.part + (int64_t)blockIdx.y * p.N), c, p.N, narrow8<DT_F32>(dw));
}

// dw = sum of the partial rows, 32 columns per workgroup: 8 threads of a column
// take every eighth part, and their sums are added in order through LDS.
__global__ __launch_bounds__(256) void norm_grad_sum_kernel(NormGradArgs p) {
  const int col = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + col;
  __shared__ float ls[8][32];
  float s = 0.0f;
  if (n < p.N)
    for (int64_t g = sub; g < p.parts; g += 8) s += p.part[g * p.N + n];
  ls[sub][col] = s;
  __syncthreads();
  if (sub == 0 && n < p.N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += ls[i][col];
    p.dW[n] = s;
  }
}

template <int DT, int DTX, int TPR, int NV>
static void launch_one(const NormGradArgs& a, hipStream_t s) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  const int64_t blocks = (a.parts + RPW - 1) / RPW;
  hipLaunchKernelGGL((norm_grad_kernel<DT, DTX, TPR, NV>), dim3((unsigned)blocks), dim3(RPW * TPR), 0, s, a);
}

template <int DT, int DTX>
static hipError_t launch_dt(const NormGradArgs& a, hipStream_t s) {
  const int64_t n = a.N;
  if (a.M > 0) {
    if (n <= 512) launch_one<DT, DTX, 64, 1>(a, s);
    else if (n <= 1024) launch_one<DT, DTX, 64, 2>(a, s);
    else if (n <= 2048) launch_one<DT, DTX, 256, 1>(a, s);
    else if (n <= 4096) launch_one<DT, DTX, 256, 2>(a, s);
    else if (n <= 8192) launch_one<DT, DTX, 512, 2>(a, s);
    else if (n <= 16384) launch_one<DT, DTX, 1024, 2>(a, s);
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

int64_t norm_grad_parts(int64_t M, int64_t) { return M < rows::MAX_PARTS ? M : rows::MAX_PARTS; }

hipError_t launch_norm_grad(int dt, bool x8, const NormGradArgs& a0, hipStream_t s) {
  NormGradArgs a = a0;
  a.parts = norm_grad_parts(a.M, a.N);
  if (dt == DT_BF16)
    return x8 ? rows::launch_dt<DT_BF16, DT_I8>(a, s) : rows::launch_dt<DT_BF16, DT_BF16>(a, s);
  if (dt == DT_F16) return x8 ? rows::launch_dt<DT_F16, DT_I8>(a, s) : rows::launch_dt<DT_F16, DT_F16>(a, s);
  return x8 ? rows::launch_dt<rows::DT_F32, DT_I8>(a, s) : rows::launch_dt<rows::DT_F32, rows::DT_F32>(a, s);
}

}  // namespace mcg
