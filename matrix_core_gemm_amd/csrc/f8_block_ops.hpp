// f8_block_ops.hpp -- the product of a block of 128 k of 8-bit floats, 16 x 16 outputs: on the
// 8-bit instruction, or exactly, widened to bf16.
#pragma once
#include "arch_gfx950.hpp"

namespace mcg {
namespace f8b {

// A block's product of 16 x 16 outputs.  FA: format of A; B is E4M3.
template <int FA>
struct Native {
  using frag_t = i32x8;
  static constexpr bool WIDE = false;
  __device__ static __forceinline__ frag_t a(const i32x8& v) { return v; }
  __device__ static __forceinline__ frag_t b(const i32x8& v) { return v; }
  __device__ static __forceinline__ f32x4 block(const frag_t& fb, const frag_t& fa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, f32x4{0, 0, 0, 0}, 0, FA, 0, 0, 0, 0);
  }
};
struct WideFrag {
  i32x4 s[4];  // 8 bf16 values for each of 4 instructions
};
template <int FA>
struct Wide {
  using frag_t = WideFrag;
  static constexpr bool WIDE = true;
  template <int FMT>
  __device__ static __forceinline__ frag_t widen(const i32x8& v) {
    frag_t f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 x;
        if constexpr (FMT == 0) {
          x = h & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + h / 2], 1.0f, true)
                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + h / 2], 1.0f, false);
        } else {
          x = h & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[2 * s + h / 2], 1.0f, true)
                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[2 * s + h / 2], 1.0f, false);
        }
        f.s[s][h] = bit_cast<int>(x);
      }
    }
    return f;
  }
  __device__ static __forceinline__ frag_t a(const i32x8& v) { return widen<FA>(v); }
  __device__ static __forceinline__ frag_t b(const i32x8& v) { return widen<0>(v); }
  __device__ static __forceinline__ f32x4 block(const frag_t& fb, const frag_t& fa) {
    f32x4 p = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bit_cast<bf16x8>(fb.s[s]), bit_cast<bf16x8>(fa.s[s]), p, 0, 0, 0);
    return p;
  }
};

}  // namespace f8b
}  // namespace mcg
