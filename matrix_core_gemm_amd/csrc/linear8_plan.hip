// linear8_plan.hip -- what the two products of the 8-bit linear layer share on their
// way to the pipelined dense kernels: the choice of tile and stream-K split with a
// modelled time, and the copy that gives an operand 16-byte chunks.
#include <algorithm>

#include "linear8.hpp"
#include "tile_any.hpp"

namespace mcg {

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
// One round of tiles takes KT_US per 128-byte K tile and ROUND_US; stream-K's last
// round adds FIXUP_US and a trip of its slots through the workspace.
constexpr double KT_US_256_16BIT = 1.6, KT_US_256_8BIT = 0.85, KT_US_128 = 0.55, KT_US_64 = 0.38, ROUND_US = 4.0, FIXUP_US = 5.0;
constexpr int64_t MIN_TILES_256 = 128;  // 256 x 256 tiles from which that form is faster
}  // namespace

PipePlan plan_pipe(int dt, DenseArgs& a, int num_cu, int64_t ws_cap) {
  const int64_t nk = cdiv(a.K * (dt == DT_I8 ? 1 : 2), KT_BYTES);
  auto whole = [&](int64_t tm, int64_t tn, double kt) {
    return cdiv(cdiv(a.M, tm) * cdiv(a.N, tn), num_cu) * (kt * nk + ROUND_US);
  };
  PipePlan p;
  p.tile = cdiv(a.M, 256) * cdiv(a.N, 256) >= MIN_TILES_256 ? 256 : 128;
  const double kt = p.tile == 128 ? KT_US_128 : dt == DT_I8 ? KT_US_256_8BIT : KT_US_256_16BIT;
  p.us = whole(p.tile, p.tile, kt);
  p.ws = plan_streamk(dt, a, num_cu, p.tile);
  if (p.ws > 0 && p.ws <= ws_cap)
    p.us = cdiv(a.dp_tiles, num_cu) * (kt * nk + ROUND_US) + kt * a.sk_iters + ROUND_US + FIXUP_US + 2.0 * p.ws / 4.5e6;
  else p.ws = 0;
  const double half = whole(64, 128, KT_US_64);
  if (p.tile == 128 && half < p.us) {
    p.tile = 64;
    p.us = half;
    p.ws = 0;
  }
  if (p.ws == 0) a.dp_tiles = a.sk_tiles = a.sk_wgs = 0;
  return p;
}

// One 16-byte chunk of the destination per thread.
__global__ __launch_bounds__(256) void align_rows_kernel(const char* src, int64_t lds, int64_t rows, int64_t row_bytes,
                                                         char* dst, int64_t ldd, uint32_t cpr, uint32_t chunks) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t r = i / cpr, c = i % cpr;
  const int64_t left = r < rows ? row_bytes - 16 * (int64_t)c : 0;
  *(i32x4*)(dst + r * ldd + 16 * (int64_t)c) = load_chunk(src, src + r * lds + 16 * (int64_t)c, (int)min(left, (int64_t)16));
}

hipError_t launch_align_rows(const void* src, int64_t lds, int64_t rows, int64_t row_bytes, void* dst, int64_t ldd,
                             int64_t rows_d, hipStream_t s) {
  const int64_t cpr = ldd / 16, chunks = cpr * rows_d;
  if (chunks > 0xffffff00) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
  hipLaunchKernelGGL(align_rows_kernel, dim3((unsigned)cdiv(chunks, 256)), dim3(256), 0, s, (const char*)src, lds, rows,
                     row_bytes, (char*)dst, ldd, (uint32_t)cpr, (uint32_t)chunks);
  return hipGetLastError();
}

}  // namespace mcg
