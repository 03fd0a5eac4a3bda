// experts.hpp -- kernel argument blocks and launchers of the products by group (the
// experts of a layer) and of block-scaled 8-bit floats.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear8.hpp"

namespace mcg {

constexpr int SCALE_BLOCK = 128;  // values of k under one scale: one K tile of 8-bit values

// Products by group and products with block scales.  The dense argument block (alpha is
// not used; ldc is of C and D) with the groups' offsets and the scales:
//   rows   D[r] = A[r] . B_g for the rows r of group g (offsets null: one group of all rows)
//   grad   D_g = A_g^T . B_g over the rows of group g (M x N of each D_g; K rows in all)
struct GroupArgs : DenseArgs {
  const int32_t* offsets;     // groups + 1, or null
  int groups;
  int64_t strideB, strideD;   // elements from one group's B (rows) or C and D (grad) to the next
  const float *sa, *sb;       // block scales of A and B (8-bit operands)
  int64_t ldsa, ldsb, strideSB;
  int blockB;                 // columns of B under one scale: 1 or 128
};

// Kernel of a call (mcg_grouped_path reports it): the dense kernels' codes, and
// KERNEL_HALF 64 x 128 tiles, KERNEL_TINY one output per thread, KERNEL_ROWS few rows, straight
// from memory to registers.
enum : int { KERNEL_ROWS = 17 };
struct GroupPlan {
  int kernel;
  int tile;  // rows of a tile
};

// Tiles of `tile` rows that M rows in G groups can need.
inline int64_t most_tiles(int64_t M, int64_t G, int64_t tile, bool grouped) {
  if (!grouped) return (M + tile - 1) / tile;
  const int64_t some = G < M ? G : M;  // groups that can hold a row; each has less than one tile of its own
  return (M - some) / tile + some;
}

// Tiles that a launch and its counters hold, and whether `rows` tile rows of N columns stay below
// (with what the pipelined kernels round their number up to).
constexpr int MANY_TILES = 1 << 23;
inline bool tiles_fit(int64_t rows, int64_t N, int64_t cols) { return rows * ((N + cols - 1) / cols) + 64 < MANY_TILES; }

// Rows of the general kernels' largest tiles (128 columns): a call whose tiles of that size do not fit is refused.
inline int general_rows(int elem_bytes) { return elem_bytes == 2 ? 128 : 64; }

// General kernels: any size, pointer and leading dimension (expert_general.hip).  dt: element
// type of A (bf16, f16, or an 8-bit float; B is then E4M3).
hipError_t launch_group_general(int dt, int la, int lb, bool grad, const GroupArgs& a, int tile, hipStream_t s);
hipError_t launch_group_tiny(int dt, int la, int lb, bool grad, const GroupArgs& a, hipStream_t s);

// Matrices in 8-bit floats with a scale per block (blocks_quant.hip): bm x bn of 1 x 128,
// 128 x 1 or 128 x 128.
struct BlocksArgs {
  const char* X;  // quantize: values; dequantize: codes
  char* Y;        // quantize: codes; dequantize: values
  float* scale;
  int64_t M, N, ldx, ldy, lds;  // leading dimensions in elements
};
hipError_t launch_blocks_quant(int dt, int dtQ, int bm, int bn, const BlocksArgs& a, hipStream_t s);
hipError_t launch_blocks_dequant(int dtQ, int dt, int bm, int bn, const BlocksArgs& a, hipStream_t s);

// The pipelined product of block-scaled 8-bit floats (f8_blocks_kernel.hpp), 256 x 256, 128 x 128 and
// 64 x 128 tiles: A and B K-contiguous or B MN-contiguous with blockB 128, or both MN-contiguous with
// blockB 1.  wide: exact products (f16 and binary32 D).
hipError_t launch_f8_blocks_256(int dtA, int la, int lb, const GroupArgs& a, hipStream_t s);
hipError_t launch_f8_blocks_128(int dtA, int la, int lb, bool wide, const GroupArgs& a, hipStream_t s);
hipError_t launch_f8_blocks_64(int dtA, int la, int lb, bool wide, const GroupArgs& a, hipStream_t s);

// The pipelined 16-bit products by group (group_pipe_kernel.hpp), 256 x 256, 128 x 128 or (rows) 64 x 128
// tiles.
hipError_t launch_group_pipe(int dt, int lb, bool grad, int tile, const GroupArgs& a, hipStream_t s);

// Few rows of K-contiguous operands (expert_rows.hip): tiles of 16, 32 or (8-bit) 64 rows.
hipError_t launch_few_rows(int dt, int rows, bool wide, const GroupArgs& a, hipStream_t s);

// The choice of a kernel, and its launch (expert_plan.cpp).
GroupPlan plan_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu);
GroupPlan plan_grouped_grad(int dt, const GroupArgs& a, int num_cu);
hipError_t launch_grouped(int dt, int la, int lb, const GroupArgs& a, int num_cu, hipStream_t s);
hipError_t launch_grouped_grad(int dt, const GroupArgs& a, int num_cu, hipStream_t s);

}  // namespace mcg
