// scaled_epilogue.hpp -- the epilogue of the int8 product with scales, shared by its
// kernels: D[m][n] = sa[m] * sb[n] * sum + bias[n].  The exact int32 sum is rounded
// to binary32, multiplied by sa, then by sb with the bias added in one fused step,
// and rounded to D's type.
#pragma once
#include "arch_gfx950.hpp"
#include "linear8.hpp"

namespace mcg {

__device__ __forceinline__ float scaled_value(int acc, float sa, float sb, float bias) {
  return __builtin_fmaf((float)acc * sa, sb, bias);
}
// Four values to consecutive elements of D (full: one aligned vector; else the first `left`).
__device__ __forceinline__ void scaled_put4(void* D, int64_t off, int out, const float (&o)[4], bool full, int64_t left) {
  if (out == OUT_32) {
    float* d = (float*)D + off;
    if (full) *(f32x4*)d = f32x4{o[0], o[1], o[2], o[3]};
    else
      for (int e = 0; e < 4; ++e)
        if (e < left) d[e] = o[e];
  } else {
    uint16_t* d = (uint16_t*)D + off;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = to_out_bits(out, o[e]);
    if (full) *(i32x2*)d = i32x2{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
    else
      for (int e = 0; e < 4; ++e)
        if (e < left) d[e] = (uint16_t)b[e];
  }
}
// The scales and biases of four consecutive columns; n + 4 may pass N.  Kernels that
// store several blocks load these first: behind a store, which might overwrite them
// for all the compiler knows, every block waits for its own loads (16 blocks: 10 us).
struct ScaledCols {
  float sb[4], bias[4];
};
__device__ __forceinline__ ScaledCols scaled_cols(const ScaledArgs& p, int64_t n) {
  ScaledCols c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t i = n + e < p.N ? n + e : p.N - 1;
    c.sb[e] = p.sb[i];
    c.bias[e] = p.bias ? p.bias[i] : 0.0f;
  }
  return c;
}
// Four consecutive outputs at (m, n); n + 4 may pass N.
__device__ __forceinline__ void scaled_store4(const ScaledArgs& p, int64_t m, int64_t n, const i32x4& acc, float sa,
                                              const ScaledCols& c) {
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = scaled_value(acc[e], sa, c.sb[e], c.bias[e]);
  scaled_put4(p.D, m * p.ldc + n, p.out, o, p.vec_cd && n + 4 <= p.N, p.N - n);
}
// Four consecutive sums of K range `range` to the workspace.
__device__ __forceinline__ void scaled_part4(const ScaledArgs& p, int range, int64_t m, int64_t n, const i32x4& acc) {
  int32_t* w = (int32_t*)p.ws + ((int64_t)range * p.M + m) * p.N + n;
  if (p.N % 4 == 0) *(i32x4*)w = acc;
  else
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) w[e] = acc[e];
}

}  // namespace mcg
