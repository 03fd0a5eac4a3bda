// linear8_plan.hip -- what the two products of the 8-bit linear layer share on their
// way to the pipelined dense kernels: the choice of tile and stream-K split with a
// modelled time, and the copy that gives an operand 16-byte chunks.
#include <algorithm>

#include "linear8.hpp"
#include "tile_any.hpp"

namespace mcg {

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
// One round of tiles takes KT_US per 128-byte K tile and ROUND_US, most of it the
// epilogue (from 500 x 4096 x 4096 to 8192^3); stream-K's last round adds FIXUP_US and
// a trip of its slots through the workspace.  16-bit 5703 x 1344 x 4288: 138 tiles of
// 256 x 256 take 140 us, 495 of 128 x 128 85; int8 5536 x 768 x 832: 66 take 27, 264 20.
// One set serves int8 and 16-bit operands in either order: over 48 to 8192 rows, five
// N x K from 1024 x 4096 to 8192 x 8192 and five products (int8 in both orders, bf16 in
// both, a binary32 result), 175 problems with each form forced, the choice is on geometric
// mean 0.0 to 1.1% slower than the best and in three problems more than 10% (worst: binary32
// result 704 x 2048 x 8192, 118 us with the general kernel, 101 with stream-K).
struct TileTime {
  double kt_us, round_us;
};
constexpr TileTime TILE_256{1.45, 15.0}, TILE_128{0.5, 6.0}, TILE_64{0.38, 4.5};
constexpr double FIXUP_US = 5.0;
}  // namespace

PipePlan plan_pipe(int dt, DenseArgs& a, int num_cu, int64_t ws_cap) {
  const int64_t nk = cdiv(a.K * (dt == DT_I8 ? 1 : 2), KT_BYTES);
  PipePlan best{0, 0, 0.0};
  auto consider = [&](int tile, int64_t ws, double us) {
    if (best.tile == 0 || us < best.us) best = PipePlan{tile, ws, us};
  };
  auto whole = [&](int64_t tm, int64_t tn, const TileTime& t) {
    return cdiv(cdiv(a.M, tm) * cdiv(a.N, tn), num_cu) * (t.kt_us * nk + t.round_us);
  };
  for (int tile = 256; tile >= 128; tile /= 2) {
    const TileTime& t = tile == 256 ? TILE_256 : TILE_128;
    consider(tile, 0, whole(tile, tile, t));
    const int64_t ws = plan_streamk(dt, a, num_cu, tile);
    if (ws > 0 && ws <= ws_cap)
      consider(tile, ws,
               cdiv(a.dp_tiles, num_cu) * (t.kt_us * nk + t.round_us) + t.kt_us * a.sk_iters + t.round_us + FIXUP_US +
                   2.0 * ws / 4.5e6);
  }
  consider(64, 0, whole(64, 128, TILE_64));
  if (best.ws > 0) plan_streamk(dt, a, num_cu, best.tile);
  else a.dp_tiles = a.sk_tiles = a.sk_wgs = 0;
  return best;
}

// One 16-byte chunk of a destination per thread: first the first copy's chunks, then
// the second's (both operands of a product in one launch: 1024^3, rows 1027 apart, 14.5
// us with two launches, 12.8 with one).
__device__ __forceinline__ void align_chunk(const AlignRows& a, uint32_t i) {
  const uint32_t cpr = (uint32_t)(a.ldd / 16), r = i / cpr, c = i % cpr;
  const int64_t left = r < a.rows ? a.row_bytes - 16 * (int64_t)c : 0;
  *(i32x4*)(a.dst + r * a.ldd + 16 * (int64_t)c) =
      load_chunk(a.src, a.src + r * a.lds + 16 * (int64_t)c, (int)min(left, (int64_t)16));
}
__global__ __launch_bounds__(256) void align_rows_kernel(AlignRows a, AlignRows b, uint32_t chunks_a, uint32_t chunks) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i < chunks_a) align_chunk(a, i);
  else if (i < chunks) align_chunk(b, i - chunks_a);
}

hipError_t launch_align_rows(const AlignRows& a, hipStream_t s, const AlignRows* second) {
  const AlignRows b = second ? *second : AlignRows{};
  const int64_t chunks_a = a.ldd / 16 * a.rows_d, chunks = chunks_a + b.ldd / 16 * b.rows_d;
  if (chunks > 0xffffff00) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
  hipLaunchKernelGGL(align_rows_kernel, dim3((unsigned)cdiv(chunks, 256)), dim3(256), 0, s, a, b, (uint32_t)chunks_a,
                     (uint32_t)chunks);
  return hipGetLastError();
}

}  // namespace mcg
