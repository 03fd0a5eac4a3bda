// expert_plan.cpp -- the choice between the kernels of the products by group and of
// block-scaled 8-bit floats, from sizes, types and alignment, and their launch.
#include <algorithm>

#include "../../include/mcg.h"
#include "experts.hpp"

namespace mcg {

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t elem_bytes(int dt) { return dt == MCG_BF16 || dt == MCG_F16 ? 2 : 1; }
// Rows of at least one 16-byte load, as the general kernels' loaders need them.
bool rows_ok(int64_t eb, int64_t K, int64_t mn, int layout) { return (layout == MCG_K_CONTIG ? K : mn) * eb >= 16; }
bool aligned_to(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
constexpr int64_t LIM = (int64_t)1 << 31;  // buffer windows and offsets stay below it

// Operands that the pipelined kernels take: 16-byte rows (whole chunks of K where it is
// contiguous), and every offset into a tile's operands, K tiles up to `ahead` past the end, below LIM.
bool chunks_ok(int64_t eb, const GroupArgs& a, int la, int lb, int64_t ahead) {
  if (!aligned_to(a.A, 16) || !aligned_to(a.B, 16) || a.lda * eb % 16 || a.ldb * eb % 16 || a.strideB * eb % 16) return false;
  if ((la == MCG_K_CONTIG || lb == MCG_K_CONTIG) && a.K * eb % 16) return false;
  const int64_t k = a.K + ahead * (128 / eb);
  return (la == MCG_K_CONTIG ? 256 : k) * a.lda * eb < LIM && (lb == MCG_K_CONTIG ? 256 : k) * a.ldb * eb < LIM;
}

// The 8-bit kinds that f8_blocks_kernel has, and its scales' windows.
bool f8_pipe_ok(const GroupArgs& a, int la, int lb) {
  if (la == MCG_K_CONTIG ? a.blockB != SCALE_BLOCK : (lb == MCG_K_CONTIG || a.blockB != 1)) return false;
  const int64_t kb = cdiv(a.K, SCALE_BLOCK) + 2;
  return chunks_ok(1, a, la, lb, 2) && 4 * (la == MCG_K_CONTIG ? 256 : kb) * a.ldsa < LIM &&
         4 * (lb == MCG_K_CONTIG ? 256 : kb) * a.ldsb < LIM;
}

// Rows of the general kernels' tiles (see general_rows in tile_any.hpp).
int general_tile_rows(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// One round of a pipelined kernel's tiles: kt_us for each K tile of 128 bytes and fixed_us, most of it
// the epilogue.  Of the tiles with 128 columns a compute unit holds two: `alone` where it has one.
struct TileTime {
  int tile;
  double kt_us, alone_us, fixed_us;
};
constexpr TileTime TIMES_16[] = {{256, 1.45, 1.45, 12.0}, {128, 1.0, 0.62, 8.0}, {64, 0.75, 0.45, 6.0}};
constexpr TileTime TIMES_F8[] = {{256, 1.85, 1.85, 12.0}, {128, 1.2, 0.7, 8.0}, {64, 0.85, 0.5, 6.0}};
constexpr TileTime TIMES_WIDE[] = {{128, 2.0, 1.2, 8.0}, {64, 1.3, 0.8, 6.0}};

// tiles(t): tiles of t rows; nk K tiles each.
template <int N, class F>
GroupPlan best_tile(const TileTime (&times)[N], int64_t nk, int64_t cols, int num_cu, int least, F tiles) {
  GroupPlan best{KERNEL_GENERAL, 0};
  double best_us = 0.0;
  for (const TileTime& t : times) {
    if (t.tile < least) continue;
    const int64_t n = tiles(t.tile) * cdiv(cols, t.tile == 256 ? 256 : 128);
    const int64_t at_once = t.tile == 256 ? num_cu : 2 * (int64_t)num_cu;
    const double us = n <= num_cu ? t.alone_us * nk + t.fixed_us : cdiv(n, at_once) * (t.kt_us * nk + t.fixed_us);
    if (best.tile == 0 || us < best_us) {
      best = {t.tile == 256 ? KERNEL_FAST : t.tile == 128 ? KERNEL_MID : KERNEL_HALF, t.tile};
      best_us = us;
    }
  }
  return best;
}
// Tiles that the rows of groups of unknown sizes take: half a tile of each group's last one is empty.
int64_t likely_tiles(const GroupArgs& a, int64_t tile) {
  if (!a.offsets || a.groups == 1) return cdiv(a.M, tile);
  return cdiv(a.M, tile) + std::min<int64_t>(a.groups, a.M) / 2;
}
}  // namespace

GroupPlan plan_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || !rows_ok(eb, a.K, a.M, la) || !rows_ok(eb, a.K, a.N, lb)) return {KERNEL_TINY, 1};
  const int64_t nk = cdiv(a.K * eb, 128), rows = a.M / a.groups;
  auto tiles = [&](int t) { return likely_tiles(a, t); };
  if (rows > 32 && eb == 2 && chunks_ok(2, a, la, lb, 3)) return best_tile(TIMES_16, nk, a.N, num_cu, 64, tiles);
  if (rows > 32 && eb == 1 && f8_pipe_ok(a, la, lb))
    return a.out == OUT_BF16 ? best_tile(TIMES_F8, nk, a.N, num_cu, 64, tiles) : best_tile(TIMES_WIDE, nk, a.N, num_cu, 64, tiles);
  return {KERNEL_GENERAL, general_tile_rows(rows)};
}

GroupPlan plan_grouped_grad(int dt, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || a.M * eb < 16 || a.N * eb < 16) return {KERNEL_TINY, 1};
  if (chunks_ok(2, a, MCG_MN_CONTIG, MCG_MN_CONTIG, 3) && a.M >= 64 && a.N >= 64)
    return best_tile(TIMES_16, cdiv(a.K * eb, 128 * a.groups), a.N, num_cu, 128, [&](int t) { return a.groups * cdiv(a.M, t); });
  return {KERNEL_GENERAL, general_tile_rows(a.M)};
}

hipError_t launch_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped(dt, la, lb, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, la, lb, false, a, s);
  if (p.kernel == KERNEL_GENERAL) return launch_group_general(dt, la, lb, false, a, p.tile, s);
  if (elem_bytes(dt) == 2) return launch_group_pipe(dt, lb, false, p.tile, a, s);
  const bool wide = a.out != OUT_BF16;
  if (p.tile == 256) return launch_f8_blocks_256(dt, la, lb, a, s);
  return p.tile == 128 ? launch_f8_blocks_128(dt, la, lb, wide, a, s) : launch_f8_blocks_64(dt, la, lb, wide, a, s);
}

hipError_t launch_grouped_grad(int dt, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped_grad(dt, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, s);
  if (p.kernel == KERNEL_GENERAL) return launch_group_general(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, p.tile, s);
  return launch_group_pipe(dt, MCG_MN_CONTIG, true, p.tile, a, s);
}

}  // namespace mcg
