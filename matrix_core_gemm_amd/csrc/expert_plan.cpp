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
}  // namespace

GroupPlan plan_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || !rows_ok(eb, a.K, a.M, la) || !rows_ok(eb, a.K, a.N, lb)) return {KERNEL_TINY, 1};
  if (eb == 1 && f8_pipe_ok(a, la, lb) && a.M / a.groups > 32) {
    if (a.out == OUT_BF16 && cdiv(a.M, 256) * cdiv(a.N, 256) >= num_cu / 2) return {KERNEL_FAST, 256};
    return {KERNEL_MID, 128};
  }
  if (eb == 2 && chunks_ok(2, a, la, lb, 2) && a.M / a.groups > 32) {
    const int tile = cdiv(a.M, 256) * cdiv(a.N, 256) >= num_cu / 2 ? 256 : 128;
    return {tile == 256 ? KERNEL_FAST : KERNEL_MID, tile};
  }
  return {KERNEL_GENERAL, general_tile_rows(a.M / a.groups)};
}

GroupPlan plan_grouped_grad(int dt, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || a.M * eb < 16 || a.N * eb < 16) return {KERNEL_TINY, 1};
  if (chunks_ok(2, a, MCG_MN_CONTIG, MCG_MN_CONTIG, 2) && a.M >= 64 && a.N >= 64) {
    const int tile = a.groups * cdiv(a.M, 256) * cdiv(a.N, 256) >= num_cu / 2 ? 256 : 128;
    return {tile == 256 ? KERNEL_FAST : KERNEL_MID, tile};
  }
  return {KERNEL_GENERAL, general_tile_rows(a.M)};
}

hipError_t launch_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped(dt, la, lb, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, la, lb, false, a, s);
  if (elem_bytes(dt) == 2 && p.kernel != KERNEL_GENERAL) return launch_group_pipe(dt, lb, false, p.tile, a, s);
  if (p.kernel == KERNEL_FAST) return launch_f8_blocks_256(dt, la, lb, a.blockB, a, s);
  if (p.kernel == KERNEL_MID) return launch_f8_blocks_128(dt, la, lb, a.blockB, a.out != OUT_BF16, a, s);
  return launch_group_general(dt, la, lb, false, a, p.tile, s);
}

hipError_t launch_grouped_grad(int dt, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped_grad(dt, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, s);
  if (p.kernel != KERNEL_GENERAL) return launch_group_pipe(dt, MCG_MN_CONTIG, true, p.tile, a, s);
  return launch_group_general(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, p.tile, s);
}

}  // namespace mcg
