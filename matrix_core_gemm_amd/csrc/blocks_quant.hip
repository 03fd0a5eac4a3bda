// blocks_quant.hip -- a matrix in 8-bit floats with one scale for each block of 128
// values of a row (1 x 128), of a column (128 x 1), or 128 x 128, and back.
//
//   scale = max|x| / L,  q = the 8-bit float nearest to L x / max|x|  (ties to even)
//
// with L the format's largest value (E4M3 448, E5M2 57344), so that no code overflows.
// A block is read once and stays in registers between its maximum and its codes: 16
// lanes hold 128 columns (8 each), a thread RPT rows 16 apart.
//
// The quotient L x / max|x| is formed as fl((L x)) / max|x| correctly rounded to binary32
// and then rounded to 8 bits.  Of 16-bit x, L x is exact (L has three significant bits) and
// no quotient of such values comes nearer than 2^-20 to the middle of two codes without
// being it, so the codes are those of the exact quotient.  The quotient is
// computed as (double)(L x) * (1 / max|x|) rounded to binary32: the binary64 product is off by
// 2^-52, and a quotient of two 24-bit values is never that near to the middle of two
// binary32 values.
//
// Bound: memory (3 bytes per 16-bit element, 5 per binary32 one, each way): 8192 x 8192 bf16, 1 x 128 blocks,
// and back 82 us, 4.96 TB/s (a copy 5.1).  A small matrix waits for its workgroups' one chain of loads, maximum
// and stores: f16 333 x 2047, 128 x 1 blocks, and back 8.9 us, of which two launches are 6.
#include "experts.hpp"
#include "row_vec.hpp"

namespace mcg {
namespace blocks {

using namespace rows;

constexpr int COLS = 128;             // columns of a workgroup: 16 lanes of 8
constexpr int THREADS = 256, TY = THREADS / 16;  // rows at a time

enum : int { ROW_BLOCKS = 0, COL_BLOCKS = 1, SQUARE_BLOCKS = 2 };  // 1 x 128, 128 x 1, 128 x 128

template <int DTQ>
constexpr float largest() {
  return DTQ == DT_E4M3 ? 448.0f : 57344.0f;
}

// What turns a block's values into codes, from its largest magnitude (a bit pattern).
struct BlockStat {
  float lead;   // L times a power of two that keeps L x normal
  double inv;   // what that leaves of 1 / max|x|; 0: all codes are zero
  float scale;
};
template <int DTQ>
__device__ __forceinline__ BlockStat block_stat(uint32_t top) {
  constexpr float L = largest<DTQ>();
  const float t = bit_cast<float>(top);
  BlockStat s{L, 0.0, 0.0f};
  if (top >= 0x7f800000u) {  // a NaN or an infinity
    s.scale = __builtin_nanf("");
  } else if (top > 0) {
    // L x must not overflow, and must not lose bits below the normal numbers
    double shift = 1.0;
    if (t >= 0x1p64f) shift = 0x1p64;
    else if (t < 0x1p-64f) shift = 0x1p-64;
    s.lead = (float)(L / shift);
    s.inv = shift / (double)t;
    s.scale = t / L;
  }
  return s;
}
// Eight codes, two dwords.
template <int DTQ>
__device__ __forceinline__ i32x2 codes8(const float (&x)[8], const float (&lead)[8], const double (&inv)[8]) {
  i32x2 q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double i = inv[4 * w + e];
      y[e] = i == 0.0 ? 0.0f : (float)((double)(x[4 * w + e] * lead[4 * w + e]) * i);
    }
    int v = 0;
    if constexpr (DTQ == DT_E4M3) {
      v = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], v, false);
      v = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], v, true);
    } else {
      v = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], v, false);
      v = __builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], v, true);
    }
    q[w] = v;
  }
  return q;
}
template <int DTQ>
__device__ __forceinline__ void values8(const Raw8<DT_I8>& v, float (&x)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    f32x2 lo, hi;
    if constexpr (DTQ == DT_E4M3) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.w[w], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.w[w], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.w[w], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.w[w], true);
    }
    x[4 * w] = lo.x;
    x[4 * w + 1] = lo.y;
    x[4 * w + 2] = hi.x;
    x[4 * w + 3] = hi.y;
  }
}

// A thread's vectors of 8 columns: of rows of 8 and more, the one that would pass the
// row's end is the row's last 8 elements, the first `skip` of them another thread's.
template <int DT, bool SHORT>
__device__ __forceinline__ Raw8<DT> get(const char* row, int64_t c, int64_t n, const RowVec& at) {
  if constexpr (SHORT) return load8<DT>(row, c, n);
  else return load_vec<DT>(row, at);
}
template <int DT, bool SHORT>
__device__ __forceinline__ void put(char* row, int64_t c, int64_t n, const RowVec& at, const Raw8<DT>& v) {
  if constexpr (SHORT) store8<DT>(row, c, n, v);
  else store_vec<DT>(row, at, v);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Largest over the 16 lanes that hold a row's 128 columns.
__device__ __forceinline__ uint32_t row_umax(uint32_t x) {
#pragma unroll
  for (int m = 8; m; m >>= 1) x = umax(x, (uint32_t)__shfl_xor((int)x, m));
  return x;
}

// Workgroup (blockIdx.x, blockIdx.y): 128 columns by RPT * 16 rows (all 128 of a block for
// blocks of 128 rows).
template <int DT, int DTQ, int KIND, int RPT, bool SHORT>
__global__ __launch_bounds__(THREADS) void blocks_quant_kernel(BlocksArgs p) {
  constexpr int ES = elem_size<DT>();
  static_assert(KIND == ROW_BLOCKS || RPT * TY == SCALE_BLOCK, "a block of 128 rows per workgroup");
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * COLS + 8 * tx;
  const RowVec at = SHORT ? RowVec{c, c < p.N ? 0 : 8} : row_vec(c, p.N);
  for (int64_t m0 = (int64_t)blockIdx.y * (RPT * TY); m0 < p.M; m0 += (int64_t)gridDim.y * (RPT * TY)) {
    Raw8<DT> raw[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {  // (rows past the end: the last row again)
      const int64_t m = min(m0 + ty + TY * r, p.M - 1);
      raw[r] = get<DT, SHORT>(p.X + m * p.ldx * ES, c, p.N, at);
    }
    uint32_t top[8] = {};  // COL_BLOCKS: of each column
    uint32_t mine = 0;       // ROW_BLOCKS: of row tx of this thread's RPT
    BlockStat s[1];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      float x[8];
      widen8<DT>(raw[r], x);
      if (KIND == ROW_BLOCKS)
#pragma unroll
        for (int e = 0; e < 8; ++e) top[e] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = bit_cast<uint32_t>(x[e]) & 0x7fffffffu;
        // another thread's columns count in no row's maximum; in a column's they are not used
        top[e] = umax(top[e], KIND != COL_BLOCKS && e < at.skip ? 0u : b);
      }
      if constexpr (KIND == ROW_BLOCKS) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = umax(t, top[e]);
        t = row_umax(t);
        mine = tx == r ? t : mine;
      }
    }
    float lead[8], row_lead[RPT];
    double inv[8], row_inv[RPT];
    if constexpr (KIND == ROW_BLOCKS) {
      // (each of a row's lanes finds another row's scale, and hands it to all 16)
      s[0] = block_stat<DTQ>(mine);
      const int64_t m = m0 + ty + TY * tx;
      if (tx < RPT && m < p.M) p.scale[m * p.lds + blockIdx.x] = s[0].scale;
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        row_lead[r] = __shfl(s[0].lead, r, 16);
        row_inv[r] = __shfl(s[0].inv, r, 16);
      }
    } else {
      __shared__ uint32_t lt[TY][COLS];
      __syncthreads();  // (a walk's earlier blocks have been read)
      if constexpr (KIND == SQUARE_BLOCKS) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = umax(t, top[e]);
        t = row_umax(t);
        if (tx == 0) lt[ty][0] = t;
        __syncthreads();
        t = 0;
#pragma unroll
        for (int r = 0; r < TY; ++r) t = umax(t, lt[r][0]);
        s[0] = block_stat<DTQ>(t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lead[e] = s[0].lead;
          inv[e] = s[0].inv;
        }
        if (threadIdx.x == 0) p.scale[m0 / SCALE_BLOCK * p.lds + blockIdx.x] = s[0].scale;
      } else {
        // columns, 8 by 8 as the lanes hold them (a shifted vector's are its own); a thread finds the scale of
        // one (all 8 in each thread, with as many binary64 quotients: 333 x 2047 7.1 us, so 5.1)
        __shared__ __attribute__((aligned(16))) double linv[COLS];
        __shared__ __attribute__((aligned(16))) float llead[COLS];
#pragma unroll
        for (int e = 0; e < 8; ++e) lt[ty][8 * tx + e] = top[e];
        __syncthreads();
        if (threadIdx.x < COLS) {
          const int slot = threadIdx.x, e = slot & 7;
          uint32_t t = 0;
#pragma unroll
          for (int r = 0; r < TY; ++r) t = umax(t, lt[r][slot]);
          s[0] = block_stat<DTQ>(t);
          linv[slot] = s[0].inv;
          llead[slot] = s[0].lead;
          const int64_t c8 = (int64_t)blockIdx.x * COLS + (slot - e);
          const RowVec mine = SHORT ? RowVec{c8, c8 < p.N ? 0 : 8} : row_vec(c8, p.N);
          const int64_t n = mine.at + e;
          if (e >= mine.skip && n < p.N) p.scale[m0 / SCALE_BLOCK * p.lds + n] = s[0].scale;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lead[e] = llead[8 * tx + e];
          inv[e] = linv[8 * tx + e];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int64_t m = m0 + ty + TY * r;
      if (m >= p.M) continue;
      float x[8];
      widen8<DT>(raw[r], x);
      if constexpr (KIND == ROW_BLOCKS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lead[e] = row_lead[r];
          inv[e] = row_inv[r];
        }
      }
      const i32x2 q = codes8<DTQ>(x, lead, inv);
      put<DT_I8, SHORT>(p.Y + m * p.ldy, c, p.N, at, Raw8<DT_I8>{{(uint32_t)q[0], (uint32_t)q[1]}});
    }
  }
}

// Values of codes: scale * q in binary32, rounded to DT.
template <int DT, int DTQ, int KIND, int RPT, bool SHORT>
__global__ __launch_bounds__(THREADS) void blocks_dequant_kernel(BlocksArgs p) {
  constexpr int ES = elem_size<DT>();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * COLS + 8 * tx;
  const RowVec at = SHORT ? RowVec{c, c < p.N ? 0 : 8} : row_vec(c, p.N);
  const int64_t first = SHORT ? c : at.at;
  for (int64_t m0 = (int64_t)blockIdx.y * (RPT * TY); m0 < p.M; m0 += (int64_t)gridDim.y * (RPT * TY)) {
    Raw8<DT_I8> raw[RPT];
    float s[KIND == COL_BLOCKS ? 8 : RPT];
    if constexpr (KIND == COL_BLOCKS) {
      // (the rows of a step lie in one block; a whole vector in two loads: each scale by its own, for every
      // row, 8192 x 4096 63 us, so 16)
      static_assert(SCALE_BLOCK % (RPT * TY) == 0, "rows of one block");
      const float* sc = p.scale + m0 / SCALE_BLOCK * p.lds;
      if constexpr (SHORT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = sc[min(first + e, p.N - 1)];
      } else {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        const f32x4_any lo = *(const f32x4_any*)(sc + first), hi = *(const f32x4_any*)(sc + first + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = lo[e], s[4 + e] = hi[e];
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int64_t m = min(m0 + ty + TY * r, p.M - 1);
      raw[r] = get<DT_I8, SHORT>(p.X + m * p.ldx, c, p.N, at);
      if constexpr (KIND != COL_BLOCKS) s[r] = p.scale[(KIND == ROW_BLOCKS ? m : m / SCALE_BLOCK) * p.lds + blockIdx.x];
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int64_t m = m0 + ty + TY * r;
      if (m >= p.M) continue;
      float x[8];
      values8<DTQ>(raw[r], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= s[KIND == COL_BLOCKS ? e : r];
        // (else the compiler joins the product and the conversion in an instruction that rounds once,
        // for f16 alone)
        if constexpr (DT == DT_F16) asm volatile("" : "+v"(x[e]));
      }
      put<DT, SHORT>(p.Y + m * p.ldy * ES, c, p.N, at, narrow8<DT>(x));
    }
  }
}

template <bool QUANT, int DT, int DTQ, int KIND, int RPT>
static hipError_t launch(const BlocksArgs& a, hipStream_t s) {
  const int64_t cols = (a.N + COLS - 1) / COLS, rows = (a.M + RPT * TY - 1) / (RPT * TY);
  const dim3 grid((unsigned)cols, (unsigned)(rows < 65535 ? rows : 65535));
  if constexpr (QUANT) {
    if (a.N < 8) hipLaunchKernelGGL((blocks_quant_kernel<DT, DTQ, KIND, RPT, true>), grid, dim3(THREADS), 0, s, a);
    else hipLaunchKernelGGL((blocks_quant_kernel<DT, DTQ, KIND, RPT, false>), grid, dim3(THREADS), 0, s, a);
  } else {
    if (a.N < 8) hipLaunchKernelGGL((blocks_dequant_kernel<DT, DTQ, KIND, RPT, true>), grid, dim3(THREADS), 0, s, a);
    else hipLaunchKernelGGL((blocks_dequant_kernel<DT, DTQ, KIND, RPT, false>), grid, dim3(THREADS), 0, s, a);
  }
  return hipGetLastError();
}
template <bool QUANT, int DT, int DTQ>
static hipError_t launch_kind(int bm, int bn, const BlocksArgs& a, hipStream_t s) {
  constexpr int RPT = SCALE_BLOCK / TY;
  // Codes of rows: 4 rows a thread where that leaves four workgroups for each compute unit (2048 x 4096 bf16 6.8 us, 7.8 with
  // 2 and 7.3 with 8; 333 x 2047 3.7, 3.2 with 2).
  if (QUANT && bm == 1 && (a.M + 4 * TY - 1) / (4 * TY) * ((a.N + COLS - 1) / COLS) >= 1024)
    return launch<QUANT, DT, DTQ, ROW_BLOCKS, QUANT ? 4 : 2>(a, s);
  if (bm == 1) return launch<QUANT, DT, DTQ, ROW_BLOCKS, 2>(a, s);
  return bn == 1 ? launch<QUANT, DT, DTQ, COL_BLOCKS, QUANT ? RPT : 4>(a, s)
                 : launch<QUANT, DT, DTQ, SQUARE_BLOCKS, QUANT ? RPT : 2>(a, s);
}
template <bool QUANT>
static hipError_t launch_types(int dt, int dtQ, int bm, int bn, const BlocksArgs& a, hipStream_t s) {
  if (dtQ == DT_E4M3)
    return dt == DT_BF16  ? launch_kind<QUANT, DT_BF16, DT_E4M3>(bm, bn, a, s)
           : dt == DT_F16 ? launch_kind<QUANT, DT_F16, DT_E4M3>(bm, bn, a, s)
                          : launch_kind<QUANT, DT_F32, DT_E4M3>(bm, bn, a, s);
  return dt == DT_BF16  ? launch_kind<QUANT, DT_BF16, DT_E5M2>(bm, bn, a, s)
         : dt == DT_F16 ? launch_kind<QUANT, DT_F16, DT_E5M2>(bm, bn, a, s)
                        : launch_kind<QUANT, DT_F32, DT_E5M2>(bm, bn, a, s);
}

}  // namespace blocks

hipError_t launch_blocks_quant(int dt, int dtQ, int bm, int bn, const BlocksArgs& a, hipStream_t s) {
  return blocks::launch_types<true>(dt, dtQ, bm, bn, a, s);
}
hipError_t launch_blocks_dequant(int dtQ, int dt, int bm, int bn, const BlocksArgs& a, hipStream_t s) {
  return blocks::launch_types<false>(dt, dtQ, bm, bn, a, s);
}

}  // namespace mcg
