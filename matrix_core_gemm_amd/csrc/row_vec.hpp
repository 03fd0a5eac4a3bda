// row_vec.hpp -- eight consecutive elements of a row as binary32 values, for the
// row-wise kernels, and their reductions over the threads of a row.
//
// Rows may start at any element: gfx950 loads and stores global memory at any
// byte address (the vector types below carry the element's alignment only), so
// one 16-byte access serves aligned and unaligned rows alike, and no element
// path is needed but for a row's last, partial vector.
#pragma once
#include "arch_gfx950.hpp"
#include "linear8.hpp"

namespace mcg {
namespace rows {

// element formats of the row kernels (mcg_dtype values; DT_BF16, DT_F16, DT_I8 as elsewhere)
enum : int { DT_F32 = 5 };

template <int DT>
constexpr int elem_size() {
  return DT == DT_F32 ? 4 : DT == DT_I8 ? 1 : 2;
}

// Raw bits of eight elements: 8, 16 or 32 bytes.
template <int DT>
struct Raw8 {
  static constexpr int DWORDS = 2 * elem_size<DT>();
  uint32_t w[DWORDS];
};

// Elements [c, c + 8) of a row of n elements; zeros past its end.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const char* row, int64_t c, int64_t n) {
  constexpr int ES = elem_size<DT>();
  Raw8<DT> v;
  if (c + 8 <= n) {
    struct __attribute__((packed, aligned(ES))) U { uint32_t w[Raw8<DT>::DWORDS]; };
    const U u = *(const U*)(row + c * ES);
#pragma unroll
    for (int i = 0; i < Raw8<DT>::DWORDS; ++i) v.w[i] = u.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < Raw8<DT>::DWORDS; ++i) v.w[i] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e >= n) continue;
      const char* p = row + (c + e) * ES;
      if constexpr (ES == 4) v.w[e] = *(const uint32_t*)p;
      else if constexpr (ES == 2) v.w[e / 2] |= (uint32_t) * (const uint16_t*)p << (16 * (e & 1));
      else v.w[e / 4] |= (uint32_t) * (const uint8_t*)p << (8 * (e & 3));
    }
  }
  return v;
}

template <int DT>
__device__ __forceinline__ void store8(char* row, int64_t c, int64_t n, const Raw8<DT>& v) {
  constexpr int ES = elem_size<DT>();
  if (c + 8 <= n) {
    struct __attribute__((packed, aligned(ES))) U { uint32_t w[Raw8<DT>::DWORDS]; };
    U u;
#pragma unroll
    for (int i = 0; i < Raw8<DT>::DWORDS; ++i) u.w[i] = v.w[i];
    *(U*)(row + c * ES) = u;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e >= n) continue;
      char* p = row + (c + e) * ES;
      if constexpr (ES == 4) *(uint32_t*)p = v.w[e];
      else if constexpr (ES == 2) *(uint16_t*)p = (uint16_t)(v.w[e / 2] >> (16 * (e & 1)));
      else *(uint8_t*)p = (uint8_t)(v.w[e / 4] >> (8 * (e & 3)));
    }
  }
}

// The row kernels' vectors of a row of n >= 8 elements.  The one that starts at c is
// loaded without a condition (at whose end the compiler copies its registers and waits
// for every load in flight: 8000 rows of 7999 bf16, the norm's gradient 205 us, of
// 8000 106), at the row's last 8 elements if it passes the end: its first `skip`
// elements are then another thread's, and are masked (in place they may be changing).
struct RowVec {
  int64_t at;  // first element in memory
  int skip;    // elements that are not this vector's: 0, 1..7 (partial) or 8 (past the end)
};
__device__ __forceinline__ RowVec row_vec(int64_t c, int64_t n) {
  const int64_t at = c < n - 8 ? c : n - 8;
  return RowVec{at, (int)(c - at < 8 ? c - at : 8)};
}
template <int DT>
__device__ __forceinline__ Raw8<DT> load_vec(const char* row, const RowVec& r) {
  constexpr int ES = elem_size<DT>();
  struct __attribute__((packed, aligned(ES))) U { uint32_t w[Raw8<DT>::DWORDS]; };
  const U u = *(const U*)(row + r.at * ES);
  Raw8<DT> v;
#pragma unroll
  for (int i = 0; i < Raw8<DT>::DWORDS; ++i) v.w[i] = u.w[i];
  return v;
}
__device__ __forceinline__ void mask_vec(float (&x)[8], const RowVec& r) {
  if (r.skip == 0) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = e < r.skip ? 0.0f : x[e];
}
template <int DT>
__device__ __forceinline__ void store_vec(char* row, const RowVec& r, const Raw8<DT>& v) {
  constexpr int ES = elem_size<DT>();
  if (r.skip == 0) {
    struct __attribute__((packed, aligned(ES))) U { uint32_t w[Raw8<DT>::DWORDS]; };
    U u;
#pragma unroll
    for (int i = 0; i < Raw8<DT>::DWORDS; ++i) u.w[i] = v.w[i];
    *(U*)(row + r.at * ES) = u;
  } else if (r.skip < 8) {
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      if (e < r.skip) continue;
      char* p = row + (r.at + e) * ES;
      if constexpr (ES == 4) *(uint32_t*)p = v.w[e];
      else if constexpr (ES == 2) *(uint16_t*)p = (uint16_t)(v.w[e / 2] >> (16 * (e & 1)));
      else *(uint8_t*)p = (uint8_t)(v.w[e / 4] >> (8 * (e & 3)));
    }
  }
}

// Exact widening of the raw elements (8-bit codes: their integer values).
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (DT == DT_F32) x[e] = bit_cast<float>(v.w[e]);
    else if constexpr (DT == DT_BF16) x[e] = bit_cast<float>((e & 1) ? v.w[e / 2] & 0xffff0000u : v.w[e / 2] << 16);
    else if constexpr (DT == DT_F16) x[e] = f16_bits_to_f32((v.w[e / 2] >> (16 * (e & 1))) & 0xffffu);
    else x[e] = (float)(int)(int8_t)(v.w[e / 4] >> (8 * (e & 3)));
  }
}

// One rounding, to nearest even.
template <int DT>
__device__ __forceinline__ Raw8<DT> narrow8(const float (&x)[8]) {
  Raw8<DT> v;
#pragma unroll
  for (int i = 0; i < Raw8<DT>::DWORDS; ++i) {
    if constexpr (DT == DT_F32) {
      v.w[i] = bit_cast<uint32_t>(x[i]);
    } else if constexpr (DT == DT_BF16) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      v.w[i] = bit_cast<uint32_t>(bf16x2{(__bf16)x[2 * i], (__bf16)x[2 * i + 1]});
    } else if constexpr (DT == DT_F16) {
      v.w[i] = f32_to_f16_bits(x[2 * i]) | (f32_to_f16_bits(x[2 * i + 1]) << 16);
    }
  }
  return v;
}

// Sum over the lanes of a wavefront, in every lane; a fixed order.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}
// Largest bit pattern over the lanes: the largest magnitude of binary32 values
// without their signs, where a NaN exceeds every number and so is never lost.
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) {
    const uint32_t y = (uint32_t)__shfl_xor((int)x, m);
    x = x > y ? x : y;
  }
  return x;
}

}  // namespace rows
}  // namespace mcg
