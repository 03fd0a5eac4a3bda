// group_epilogue.hpp -- the epilogue of the products by group and of block-scaled 8-bit
// floats: four consecutive elements D = v + beta * C, rounded once to D's type.
#pragma once
#include "arch_gfx950.hpp"
#include "experts.hpp"

namespace mcg {

// base: first element of the group's D and C.  n + 4 may pass N.
__device__ __forceinline__ void group_store4(const GroupArgs& p, int64_t base, int64_t m, int64_t n, const f32x4& v) {
  const int64_t off = base + m * p.ldc + n;
  const bool full = p.vec_cd && n + 4 <= p.N;
  if (full && p.out == OUT_32) {
    f32x4 o = v;
    if (p.use_c) {
      const f32x4 c = *(const f32x4*)((const float*)p.C + off);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(p.beta, c[e], v[e]);
    }
    *(f32x4*)((float*)p.D + off) = o;
  } else if (full) {
    i32x2 c = {0, 0};
    if (p.use_c) c = *(const i32x2*)((const uint16_t*)p.C + off);
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ce = from_out_bits(p.out, ((uint32_t)c[e / 2] >> (16 * (e & 1))) & 0xffffu);
      b[e] = to_out_bits(p.out, p.use_c ? __builtin_fmaf(p.beta, ce, v[e]) : v[e]);
    }
    *(i32x2*)((uint16_t*)p.D + off) = i32x2{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
  } else {
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) combine_store(p.C, p.D, off + e, v[e], 1.0f, p.beta, p.use_c, p.out);
  }
}

}  // namespace mcg
