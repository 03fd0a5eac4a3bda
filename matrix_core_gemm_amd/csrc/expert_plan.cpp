// expert_plan.cpp -- the choice between the kernels of the products by group and of
// block-scaled 8-bit floats, from sizes, types and alignment, and their launch.
#include <algorithm>

#include "../../include/mcg.h"
#include "experts.hpp"

namespace mcg {

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t elem_bytes(int dt) { return dt == MCG_BF16 || dt == MCG_F16 ? 2 : 1; }
// An operand of at least one 16-byte load, as the general kernels' loaders need it.
bool load_ok(int64_t eb, int64_t K, int64_t mn, int64_t ld, int layout) {
  const int64_t rows = layout == MCG_K_CONTIG ? mn : K, cols = layout == MCG_K_CONTIG ? K : mn;
  return ((rows - 1) * ld + cols) * eb >= 16;
}
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

// A choice and its modelled time.
struct Timed {
  GroupPlan plan;
  double us;
};

// One round of a pipelined kernel's tiles: kt_us for each K tile of 128 bytes and fixed_us, most of it
// the epilogue.  Of the tiles with 128 columns a compute unit holds two: `alone` where it has one, a
// quarter less where most units have none.
struct TileTime {
  int tile;
  double kt_us, alone_us, fixed_us;
};
constexpr TileTime TIMES_16[] = {{256, 1.45, 1.45, 12.0}, {128, 1.0, 0.62, 8.0}, {64, 0.75, 0.45, 6.0}};
constexpr TileTime TIMES_F8[] = {{256, 1.85, 1.85, 12.0}, {128, 1.2, 0.7, 8.0}, {64, 0.85, 0.58, 5.0}};
constexpr TileTime TIMES_WIDE[] = {{128, 2.0, 1.2, 8.0}, {64, 1.3, 0.8, 6.0}};

// tiles(t), at_most(t): tiles of t rows, likely and at most; nk K tiles each.
template <int N, class F, class G>
Timed best_tile(const TileTime (&times)[N], int64_t nk, int64_t cols, int num_cu, int least, int most, F tiles, G at_most) {
  Timed best{{KERNEL_GENERAL, 0}, 0.0};
  for (const TileTime& t : times) {
    if (t.tile < least || t.tile > most || !tiles_fit(at_most(t.tile), cols, t.tile == 256 ? 256 : 128)) continue;
    const int64_t n = tiles(t.tile) * cdiv(cols, t.tile == 256 ? 256 : 128);
    const int64_t at_once = t.tile == 256 ? num_cu : 2 * (int64_t)num_cu;
    const double us = n <= num_cu ? t.alone_us * (0.75 + 0.25 * (double)n / num_cu) * nk + t.fixed_us
                                  : (double)cdiv(n, at_once) * (t.kt_us * nk + t.fixed_us);
    if (best.plan.tile == 0 || us < best.us)
      best = {{t.tile == 256 ? KERNEL_FAST : t.tile == 128 ? KERNEL_MID : KERNEL_HALF, t.tile}, us};
  }
  return best;
}
// Tiles that the rows of groups of unknown sizes take: half a tile of each group's last one is empty, and
// where there are few rows a quarter of the groups.
int64_t likely_tiles(const GroupArgs& a, int64_t tile) {
  if (!a.offsets || a.groups == 1) return cdiv(a.M, tile);
  const int64_t some = std::min<int64_t>(a.groups, a.M);
  return std::max(cdiv(a.M, tile) + some / 2, some * 3 / 4);
}
// Rows of the general kernels' tiles: the most that leave a workgroup for each compute unit (8-bit 276 x
// 5056 x 3776 from rows of odd lengths: 200 workgroups of 64 rows 76 us, 360 of 32 57; 2000 x 2001 x 2003: 512
// of 64 rows 39 us, 32 rows 57; bf16 2000 rows over 9 groups, 1003 x 1501: 168 of 128 rows 43 us, 288 of 64 34).
template <class F>
GroupPlan general_plan(int most, int64_t cols, int num_cu, F tiles) {
  for (int t = most; t > 32; t /= 2)
    if (tiles(t) * cdiv(cols, 128) >= num_cu) return {KERNEL_GENERAL, t};
  return {KERNEL_GENERAL, 32};
}
// The kernel for few rows: 28 KB a us and compute unit (see expert_rows.hip), and 0.7 us for a
// workgroup (10 rows over 28 groups, 6208 x 128: 20 us in workgroups of 32 columns, 8.6 in tiles of 64 x 128).
Timed best_few_rows(const GroupArgs& a, int64_t eb, int num_cu) {
  Timed best{{KERNEL_GENERAL, 0}, 0.0};
  for (int tile = 16; tile <= (eb == 1 ? 64 : 32); tile *= 2) {
    if (!tiles_fit(most_tiles(a.M, a.groups, tile, a.offsets != nullptr), a.N, 32)) continue;
    const double per_cu = (double)likely_tiles(a, tile) * (double)cdiv(a.N, 32) / num_cu;
    const double us = 6.0 + (per_cu < 1.0 ? 1.0 : per_cu) * (0.7 + (32 + tile) * (double)(a.K * eb) / 28e3);
    if (best.plan.tile == 0 || us < best.us) best = {{KERNEL_ROWS, tile}, us};
  }
  return best;
}
}  // namespace

GroupPlan plan_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || !load_ok(eb, a.K, a.M, a.lda, la) || !load_ok(eb, a.K, a.N, a.ldb, lb)) return {KERNEL_TINY, 1};
  const int64_t nk = cdiv(a.K * eb, 128), rows = a.M / a.groups;
  const bool chunks = chunks_ok(eb, a, la, lb, 3);
  const bool pipe = chunks && (eb == 2 || f8_pipe_ok(a, la, lb));
  const bool few = chunks && rows <= 64 && la == MCG_K_CONTIG && lb == MCG_K_CONTIG &&
                   (eb == 2 || (a.blockB == SCALE_BLOCK && 4 * 256 * a.ldsa < LIM));
  auto tiles = [&](int t) { return likely_tiles(a, t); };
  auto at_most = [&](int t) { return most_tiles(a.M, a.groups, t, a.offsets != nullptr); };
  Timed best{general_plan(general_rows((int)eb), a.N, num_cu, tiles), 0.0};
  if (pipe) {
    best = eb == 2              ? best_tile(TIMES_16, nk, a.N, num_cu, 64, 256, tiles, at_most)
           : a.out == OUT_BF16 ? best_tile(TIMES_F8, nk, a.N, num_cu, 64, la == MCG_K_CONTIG ? 256 : 128, tiles, at_most)
                               : best_tile(TIMES_WIDE, nk, a.N, num_cu, 64, 128, tiles, at_most);
    // (the weights of four groups in five come from HBM, at 4.3 TB/s in these kernels' tiles of few rows)
    const double weights_us = 5.0 + 0.8 * (double)std::min<int64_t>(a.groups, a.M) * (double)(a.N * a.K * eb) / 4.3e6;
    best.us = std::max(best.us, weights_us);
  }
  if (few) {
    const Timed t = best_few_rows(a, eb, num_cu);
    if (t.plan.tile && (best.plan.kernel == KERNEL_GENERAL || t.us < best.us)) best = t;
  }
  return best.plan;
}

GroupPlan plan_grouped_grad(int dt, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  // (a group may be one row, which is then the operand)
  if (a.K == 0 || a.M * eb < 16 || a.N * eb < 16) return {KERNEL_TINY, 1};
  auto tiles = [&](int t) { return a.groups * cdiv(a.M, t); };
  if (chunks_ok(2, a, MCG_MN_CONTIG, MCG_MN_CONTIG, 3) && a.M >= 64 && a.N >= 64)
    return best_tile(TIMES_16, cdiv(a.K * eb, 128 * a.groups), a.N, num_cu, 128, 256, tiles, tiles).plan;
  return general_plan(general_rows((int)eb), a.N, num_cu, tiles);
}

hipError_t launch_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped(dt, la, lb, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, la, lb, false, a, s);
  if (p.kernel == KERNEL_GENERAL) return launch_group_general(dt, la, lb, false, a, p.tile, s);
  const bool wide = a.out != OUT_BF16;
  if (p.kernel == KERNEL_ROWS) return launch_few_rows(dt, p.tile, wide, a, s);
  if (elem_bytes(dt) == 2) return launch_group_pipe(dt, lb, false, p.tile, a, s);
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
