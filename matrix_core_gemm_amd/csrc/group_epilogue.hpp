// group_epilogue.hpp -- the epilogue of the products by group and of block-scaled 8-bit
// floats: D = v + beta * C, rounded once to D's type, four consecutive elements at a time.
#pragma once
#include "arch_gfx950.hpp"
#include "experts.hpp"

namespace mcg {

// Four elements at any alignment of theirs: the instructions take it (one by one, as rows of odd
// lengths would else be stored: weight gradients of 3000 rows over 32 groups, 1500 x 2001 to binary32,
// 234 us, so 197).
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// base: first element of the group's D and C.  n + 4 may pass N.
__device__ __forceinline__ void group_store4(const GroupArgs& p, int64_t base, int64_t m, int64_t n, const f32x4& v) {
  const int64_t off = base + m * p.ldc + n;
  const bool full = n + 4 <= p.N;
  if (full && p.out == OUT_32) {
    f32x4 o = v;
    if (p.use_c) {
      const f32x4 c = *(const f32x4_any*)((const float*)p.C + off);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(p.beta, c[e], v[e]);
    }
    *(f32x4_any*)((float*)p.D + off) = o;
  } else if (full) {
    i32x2 c = {0, 0};
    if (p.use_c) c = *(const i32x2_any*)((const uint16_t*)p.C + off);
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ce = from_out_bits(p.out, ((uint32_t)c[e / 2] >> (16 * (e & 1))) & 0xffffu);
      b[e] = to_out_bits(p.out, p.use_c ? __builtin_fmaf(p.beta, ce, v[e]) : v[e]);
    }
    *(i32x2_any*)((uint16_t*)p.D + off) = i32x2{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
  } else {
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) combine_store(p.C, p.D, off + e, v[e], 1.0f, p.beta, p.use_c, p.out);
  }
}

// Two binary32 values in a 16-bit format, to nearest even.
__device__ __forceinline__ int pack2(int out, float x, float y) {
  if (out == OUT_BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return bit_cast<int>(bf16x2{(__bf16)x, (__bf16)y});
  }
  return (int)(f32_to_f16_bits(x) | (f32_to_f16_bits(y) << 16));
}

// Eight rows 4 apart, m, m + 4, .. (those below m_end), at columns n .. n + 3.  The form of the
// store is chosen once, and C's loads go out together.
__device__ __forceinline__ void group_store_rows(const GroupArgs& p, int64_t base, int64_t m, int64_t m_end, int64_t n,
                                                 const f32x4 (&v)[8]) {
  if (n >= p.N) return;
  const int rows = (int)min((m_end - m + 3) / 4, (int64_t)8);
  const int64_t off = base + m * p.ldc + n, step = 4 * p.ldc;
  if (n + 4 > p.N) {
    for (int t = 0; t < 8; ++t) {  // (v's indices are constants)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) x = u == t ? v[u][e] : x;
        if (t < rows && n + e < p.N) combine_store(p.C, p.D, off + t * step + e, x, 1.0f, p.beta, p.use_c, p.out);
      }
    }
  } else if (p.out == OUT_32) {
    float* d = (float*)p.D + off;
    f32x4 c[8];
    if (p.use_c) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < rows) c[t] = *(const f32x4_any*)((const float*)p.C + off + t * step);
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[t][e] = __builtin_fmaf(p.beta, c[t][e], v[t][e]);
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) c[t] = v[t];
    }
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < rows) *(f32x4_any*)(d + t * step) = c[t];
  } else {
    uint16_t* d = (uint16_t*)p.D + off;
    i32x2 o[8];
    if (p.use_c) {
      i32x2 c[8];
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < rows) c[t] = *(const i32x2_any*)((const uint16_t*)p.C + off + t * step);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = __builtin_fmaf(p.beta, from_out_bits(p.out, ((uint32_t)c[t][e / 2] >> (16 * (e & 1))) & 0xffffu), v[t][e]);
        o[t] = i32x2{pack2(p.out, x[0], x[1]), pack2(p.out, x[2], x[3])};
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) o[t] = i32x2{pack2(p.out, v[t][0], v[t][1]), pack2(p.out, v[t][2], v[t][3])};
    }
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < rows) *(i32x2_any*)(d + t * step) = o[t];
  }
}

}  // namespace mcg
