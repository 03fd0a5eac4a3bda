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
// Rows of the general kernels' tiles (see general_rows in tile_any.hpp).
int general_tile_rows(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
}  // namespace

GroupPlan plan_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || !rows_ok(eb, a.K, a.M, la) || !rows_ok(eb, a.K, a.N, lb)) return {KERNEL_TINY, 1};
  return {KERNEL_GENERAL, general_tile_rows(a.M / a.groups)};
}

GroupPlan plan_grouped_grad(int dt, const GroupArgs& a, int num_cu) {
  const int64_t eb = elem_bytes(dt);
  if (a.K == 0 || a.M * eb < 16 || a.N * eb < 16) return {KERNEL_TINY, 1};
  return {KERNEL_GENERAL, general_tile_rows(a.M)};
}

hipError_t launch_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped(dt, la, lb, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, la, lb, false, a, s);
  return launch_group_general(dt, la, lb, false, a, p.tile, s);
}

hipError_t launch_grouped_grad(int dt, const GroupArgs& a, int num_cu, hipStream_t s) {
  const GroupPlan p = plan_grouped_grad(dt, a, num_cu);
  if (p.kernel == KERNEL_TINY) return launch_group_tiny(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, s);
  return launch_group_general(dt, MCG_MN_CONTIG, MCG_MN_CONTIG, true, a, p.tile, s);
}

}  // namespace mcg
