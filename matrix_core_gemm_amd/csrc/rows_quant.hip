// rows_quant.hip -- rows of a matrix to 8 bits with one scale each, after the
// root-mean-square norm (rmsnorm_quant) or as they are (quantize_rows), and back
// (dequantize_rows).
//
//   h = x + r,  rstd = (mean(h^2) + eps)^(-1/2),  y = h * w * rstd
//   scale = max|y| / 127,  q = rint(127 y / max|y|)
//
// rstd > 0 is common to the row, so max|y| = rstd * max|h w| and y / (max|y| / 127) =
// 127 h w / max|h w|: both reductions (the sum of squares and the largest
// |h w|) run over the same values at once, and the codes need no rstd.  A row is
// read once and kept in registers between its reductions and its stores.
// Statistics and products are binary32; h is rounded once, to be stored, and the
// norm is taken of the unrounded sum.
//
// Bound: memory (7 bytes per element with a 16-bit residual, 3 without).  8192 x
// 8192 bf16 with a residual: 93 us, 5.0 TB/s (a copy: 5.1); binary32 176 us, 4.95; rows
// above 16384 columns are read twice (4096 x 20480 bf16 161 us, 3.6).
#include "row_vec.hpp"

namespace mcg {
namespace rows {

constexpr float QMAX = 127.0f;
constexpr int64_t WG_PER_CU = 8;       // workgroups per compute unit that walk the rows
constexpr int64_t MAX_BLOCKS = 1 << 20;  // workgroups along the rows (a launch holds less than 2^32 threads)

// Sum and largest pattern over the TPR threads of a row, in all of them.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& ss, uint32_t& top, int phase) {
  ss = wave_sum(ss);
  top = wave_umax(top);
  if constexpr (TPR > 64) {
    constexpr int NWV = TPR / 64;
    __shared__ float ls[2][NWV];  // by turns: a wavefront may be one row ahead
    __shared__ uint32_t lt[2][NWV];
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      ls[phase][wave] = ss;
      lt[phase][wave] = top;
    }
    __syncthreads();
    ss = ls[phase][0];
    top = lt[phase][0];
#pragma unroll
    for (int i = 1; i < NWV; ++i) {
      ss += ls[phase][i];
      top = top > lt[phase][i] ? top : lt[phase][i];
    }
  }
}

// A row's statistics from its reductions: the factor 127 / max of its codes, its
// scale and rstd.  A row with a NaN or an infinity, whose squares overflow, or whose
// mean square plus eps is below the normal numbers (an eps of 0: squares lose their
// bits there, and rstd ends infinite) gets the scale NaN and codes 0; a row of zeros
// the scale 0.
struct RowStat {
  double inv;
  float scale, rstd;
};
template <bool NORM>
__device__ __forceinline__ RowStat row_stat(float ss, uint32_t top, int64_t n, float eps) {
  RowStat s;
  const float t = bit_cast<float>(top);
  s.rstd = 1.0f;
  bool finite = top < 0x7f800000u;
  if constexpr (NORM) {
    const float mean = (n > 0 ? ss / (float)n : 0.0f) + eps;
    s.rstd = 1.0f / __builtin_sqrtf(mean);
    finite = finite && ss < __builtin_inff() && (mean >= 0x1p-126f || top == 0);
  }
  s.inv = finite && t > 0.0f ? (double)QMAX / (double)t : 0.0;
  if (!finite) s.scale = __builtin_nanf("");
  else s.scale = t > 0.0f ? t * s.rstd / QMAX : 0.0f;
  return s;
}

// Codes of eight values: 127 y / max|y| in binary64, rounded to binary32 and then to
// the nearest integer, ties to even.  The binary64 product is off by at most 2^-52 of
// its value, so the binary32 one is that of the exact quotient but within 2^-52 of the
// middle of two: a tie of integers (63.5 for half the largest value, common in 16-bit
// rows) stays one, and no other quotient of 16-bit values comes nearer to one than
// 2^-20, so that their codes are exact.  (As y * (127 / max) in binary32, 632 of 16384
// codes of f16 rows that hold that half were the other neighbour.)
// At most 127 in magnitude: 127 (1 + 2^-52) rounds to it.  Adding 1.5 * 2^23 rounds to
// an integer whose two's complement is in the low bits of the sum; with the two
// conversions four instructions a code, as in binary32 with a clamp.
// inv == 0 (see RowStat) gives zeros: the values may then be infinite or NaN.
__device__ __forceinline__ Raw8<DT_I8> codes8(const float (&y)[8], const RowStat& s) {
  Raw8<DT_I8> v;
  if (s.inv == 0.0) {
    v.w[0] = v.w[1] = 0;
    return v;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = bit_cast<uint32_t>((float)((double)y[4 * i + e] * s.inv) + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    v.w[i] = lo | hi;
  }
  return v;
}

// One vector of a row: h (widened sum) and its products with the weights.
template <int DT, bool NORM>
__device__ __forceinline__ void load_h(const RowsQuantArgs& p, const char* x, const char* r, int64_t c, float (&h)[8]) {
  widen8<DT>(load8<DT>(x, c, p.N), h);
  if (NORM && r) {
    float y[8];
    widen8<DT>(load8<DT>(r, c, p.N), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] += y[e];
  }
}
template <int DT, bool NORM>
__device__ __forceinline__ void weigh(const RowsQuantArgs& p, int64_t c, float (&h)[8]) {
  if (NORM && p.W) {
    float w[8];
    widen8<DT>(load8<DT>(p.W, c, p.N), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= w[e];
  }
}
__device__ __forceinline__ void stat8(const float (&h)[8], float& ss) {
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[e], h[e], ss);
}
__device__ __forceinline__ void top8(const float (&y)[8], uint32_t& top) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = bit_cast<uint32_t>(y[e]) & 0x7fffffffu;
    top = top > b ? top : b;
  }
}

// TPR threads per row (a wavefront or a workgroup), NV vectors of eight elements
// per thread: rows of 8 to 8 * TPR * NV elements.  A workgroup walks rows a grid
// apart: the weights stay in its registers, and the next row's loads go out before
// this row's stores (which the compiler would otherwise keep them behind, since H
// may be X).  With the loads of every row behind the previous stores, 8192 x 8192
// bf16 with a residual took 270 us.
template <int DT, bool NORM, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rows_quant_kernel(RowsQuantArgs p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  constexpr int ES = elem_size<DT>();
  const int t = threadIdx.x % TPR;
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  if (row >= p.M) return;  // whole wavefronts, and only where a row is one wavefront
  RowVec at[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) at[v] = row_vec((int64_t)(v * TPR + t) * 8, p.N);
  Raw8<DT> x[NV], r[NORM ? NV : 1], w[NORM ? NV : 1];
  auto load_row = [&](int64_t m) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v] = load_vec<DT>(p.X + m * p.ldx * ES, at[v]);
      if constexpr (NORM)
        if (p.R) r[v] = load_vec<DT>(p.R + m * p.ldr * ES, at[v]);
    }
  };
  if constexpr (NORM) {
    if (p.W) {
#pragma unroll
      for (int v = 0; v < NV; ++v) w[v] = load_vec<DT>(p.W, at[v]);
    }
  }
  load_row(row);
  // whole wavefronts leave the loop together, whole workgroups where a row is a workgroup's
  for (int phase = 0; row < p.M; row += step, phase ^= 1) {
    float y[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      widen8<DT>(x[v], y[v]);
      if constexpr (NORM) {
        if (p.R) {
          float z[8];
          widen8<DT>(r[v], z);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[v][e] += z[e];
        }
      }
    }
    if (row + step < p.M) load_row(row + step);
    float ss = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      mask_vec(y[v], at[v]);
      if constexpr (NORM) {
        if (p.H) store_vec<DT>(p.H + row * p.ldh * ES, at[v], narrow8<DT>(y[v]));
        stat8(y[v], ss);
        if (p.W) {
          float z[8];
          widen8<DT>(w[v], z);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[v][e] *= z[e];
        }
      }
      top8(y[v], top);
    }
    row_reduce<TPR>(ss, top, phase);
    const RowStat s = row_stat<NORM>(ss, top, p.N, p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) store_vec<DT_I8>((char*)p.Q + row * p.ldq, at[v], codes8(y[v], s));
    if (t == 0) {
      p.scale[row] = s.scale;
      if (NORM && p.rstd) p.rstd[row] = s.rstd;
    }
  }
}

// Rows of any other length: the row is read a second time (through the caches) for
// its codes.  H is written in the second pass, by the thread that has just read the
// same elements of X and R, so it may be either of them.
template <int DT, bool NORM>
__global__ __launch_bounds__(1024) void rows_quant_long_kernel(RowsQuantArgs p) {
  constexpr int ES = elem_size<DT>();
  int phase = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, phase ^= 1) {
    const char* x = p.X + row * p.ldx * ES;
    const char* r = p.R ? p.R + row * p.ldr * ES : nullptr;
    float ss = 0.0f;
    uint32_t top = 0;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.N; c += 8192) {
      float h[8];
      load_h<DT, NORM>(p, x, r, c, h);
      if constexpr (NORM) {
        stat8(h, ss);
        weigh<DT, NORM>(p, c, h);
      }
      top8(h, top);
    }
    row_reduce<1024>(ss, top, phase);
    const RowStat s = row_stat<NORM>(ss, top, p.N, p.eps);
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.N; c += 8192) {
      float h[8];
      load_h<DT, NORM>(p, x, r, c, h);
      if constexpr (NORM) {
        if (p.H) store8<DT>(p.H + row * p.ldh * ES, c, p.N, narrow8<DT>(h));
        weigh<DT, NORM>(p, c, h);
      }
      store8<DT_I8>((char*)p.Q + row * p.ldq, c, p.N, codes8(h, s));
    }
    if (threadIdx.x == 0) {
      p.scale[row] = s.scale;
      if (NORM && p.rstd) p.rstd[row] = s.rstd;
    }
  }
}

// The values of 8-bit rows: one vector of eight codes per thread, columns along x;
// short rows share a workgroup, `rows` of `vecs` vectors (8000 x 300: 6.2 us with a
// workgroup each, 3.9 so).
template <int DT>
__global__ __launch_bounds__(256) void rows_dequant_kernel(RowsDequantArgs p, int vecs, int rows) {
  const int sub = threadIdx.x / vecs;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x % vecs) * 8;
  if (c >= p.N || sub >= rows) return;
  for (int64_t row = (int64_t)blockIdx.y * rows + sub; row < p.M; row += (int64_t)gridDim.y * rows) {
    float x[8];
    widen8<DT_I8>(load8<DT_I8>((const char*)p.Q + row * p.ldq, c, p.N), x);
    const float s = p.scale[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
    store8<DT>(p.D + row * p.ldd * elem_size<DT>(), c, p.N, narrow8<DT>(x));
  }
}

template <int DT, bool NORM, int TPR, int NV>
static hipError_t launch_one(const RowsQuantArgs& a, int num_cu, hipStream_t s) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  const int64_t blocks = min((a.M + RPW - 1) / RPW, (int64_t)num_cu * WG_PER_CU);
  hipLaunchKernelGGL((rows_quant_kernel<DT, NORM, TPR, NV>), dim3((unsigned)blocks), dim3(RPW * TPR), 0, s, a);
  return hipGetLastError();
}

template <int DT, bool NORM>
static hipError_t launch_dt(const RowsQuantArgs& a, int num_cu, hipStream_t s) {
  const int64_t n = a.N;
  if (n >= 8) {
    if (n <= 512) return launch_one<DT, NORM, 64, 1>(a, num_cu, s);
    if (n <= 1024) return launch_one<DT, NORM, 64, 2>(a, num_cu, s);
    if (n <= 2048) return launch_one<DT, NORM, 256, 1>(a, num_cu, s);
    if (n <= 4096) return launch_one<DT, NORM, 256, 2>(a, num_cu, s);
    // (as one of 8192, 5000 columns took 55 us instead of 48 for 8000 rows)
    if (n <= 6144 && a.M > num_cu) return launch_one<DT, NORM, 256, 3>(a, num_cu, s);
    if (n <= 8192) return a.M <= num_cu ? launch_one<DT, NORM, 1024, 1>(a, num_cu, s) : launch_one<DT, NORM, 256, 4>(a, num_cu, s);
    if (n <= 16384) return launch_one<DT, NORM, 1024, 2>(a, num_cu, s);
  }
  hipLaunchKernelGGL((rows_quant_long_kernel<DT, NORM>), dim3((unsigned)min(a.M, MAX_BLOCKS)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <bool NORM>
static hipError_t launch_norm(int dt, const RowsQuantArgs& a, int num_cu, hipStream_t s) {
  if (dt == DT_BF16) return launch_dt<DT_BF16, NORM>(a, num_cu, s);
  if (dt == DT_F16) return launch_dt<DT_F16, NORM>(a, num_cu, s);
  return launch_dt<DT_F32, NORM>(a, num_cu, s);
}

}  // namespace rows

hipError_t launch_rows_quant(int dt, bool norm, const RowsQuantArgs& a, int num_cu, hipStream_t s) {
  return norm ? rows::launch_norm<true>(dt, a, num_cu, s) : rows::launch_norm<false>(dt, a, num_cu, s);
}

hipError_t launch_rows_dequant(int dt, const RowsDequantArgs& a, hipStream_t s) {
  const int vecs = a.N < 2048 ? (int)((a.N + 7) / 8) : 256, rows = 256 / vecs;
  const int64_t groups = (a.M + rows - 1) / rows;
  const dim3 grid((unsigned)((a.N + 2047) / 2048), (unsigned)(groups < 65535 ? groups : 65535));
  if (dt == DT_BF16) hipLaunchKernelGGL((rows::rows_dequant_kernel<DT_BF16>), grid, dim3(256), 0, s, a, vecs, rows);
  else if (dt == DT_F16) hipLaunchKernelGGL((rows::rows_dequant_kernel<DT_F16>), grid, dim3(256), 0, s, a, vecs, rows);
  else hipLaunchKernelGGL((rows::rows_dequant_kernel<rows::DT_F32>), grid, dim3(256), 0, s, a, vecs, rows);
  return hipGetLastError();
}

}  // namespace mcg
