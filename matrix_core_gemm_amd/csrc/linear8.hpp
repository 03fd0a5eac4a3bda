// linear8.hpp -- kernel argument blocks and launchers of the 8-bit linear layer:
// row quantisation, the root-mean-square norm around it, and the scaled int8 and
// mixed products.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_kernels.hpp"

namespace mcg {

// Rows to 8 bits, with or without the norm (rows_quant.hip).
struct RowsQuantArgs {
  const char* X;
  const char* R;  // residual, or null
  const char* W;  // norm weights, or null (ones)
  char* H;        // sum of X and R, or null
  int8_t* Q;
  float* scale;
  float* rstd;    // or null
  int64_t M, N, ldx, ldr, ldh, ldq;  // leading dimensions in elements
  float eps;
};
hipError_t launch_rows_quant(int dt, bool norm, const RowsQuantArgs& a, int num_cu, hipStream_t s);

struct RowsDequantArgs {
  const int8_t* Q;
  const float* scale;
  char* D;
  int64_t M, N, ldq, ldd;
};
hipError_t launch_rows_dequant(int dtD, const RowsDequantArgs& a, hipStream_t s);

// Backward pass of the norm (rmsnorm_backward.hip).
struct NormGradArgs {
  const char* dY;
  const char* X;        // 16/32-bit rows, or 8-bit codes with xscale
  const float* xscale;  // 8-bit X only
  const char* W;        // or null (ones)
  const float* rstd;
  const char* dR;       // or null
  char* dX;
  float* dW;            // or null
  float* part;          // workspace of norm_grad_workspace(M, N) bytes: partial rows of dW
  int64_t M, N, lddy, ldx, lddr, lddx;
  int64_t parts;        // filled by the launcher
};
int64_t norm_grad_workspace(int64_t M, int64_t N);
hipError_t launch_norm_grad(int dt, bool x8, const NormGradArgs& a, hipStream_t s);

// D = (A . B) * sa_i * sb_j + bias_j, int8 operands (gemm_i8_scaled.hip): the dense
// argument block (A row-major; ldc is D's leading dimension, C and alpha / beta are
// not used) with the scales and the chosen kernel.  splits > 1: ws holds one M x N
// int32 matrix per K range; sk_tiles > 0: ws holds the stream-K slots.
struct ScaledArgs : DenseArgs {
  const float* sa;    // M
  const float* sb;    // N
  const float* bias;  // N, or null
  int kernel;         // KERNEL_TINY, KERNEL_GENERAL, KERNEL_STREAM, or KERNEL_FAST with
  int tile;           // PipePlan's tile; KERNEL_GENERAL: rows of a tile
  // copies of operands without 16-byte chunks, for the pipelined kernel: panels of
  // panel_n columns (0: no copies), K padded with zeros to kp
  int64_t panel_n, kp, ldb2;
  int64_t ws_bytes;
};
constexpr int KERNEL_HALF = 7, KERNEL_TINY = 16;  // (beside the dense kernels' codes; mcg_i8_scaled_path)
// Code of the pipelined kernel with this tile.
inline int pipe_kernel(int tile) { return tile == 256 ? KERNEL_FAST : tile == 128 ? KERNEL_MID : KERNEL_HALF; }
int64_t plan_scaled(ScaledArgs& a, int layoutB, int num_cu, int64_t ws_bytes);
hipError_t launch_scaled(int layoutB, const ScaledArgs& a, int num_cu, hipStream_t s);
// The pipelined kernel with tile x tile tiles (256 or 128) and the streaming kernel (M <= 32).
hipError_t launch_scaled_fast(int layoutB, const ScaledArgs& a, hipStream_t s);
hipError_t launch_scaled_mid(int layoutB, const ScaledArgs& a, hipStream_t s);
hipError_t launch_scaled_half(int layoutB, const ScaledArgs& a, hipStream_t s);  // 64 x 128 tiles
hipError_t launch_scaled_stream(int layoutB, const ScaledArgs& a, hipStream_t s);

// D = A . diag(s) . Q + beta C, A 16-bit and Q int8 (gemm_grad_i8.hip).
struct GradArgs {
  const char* A;       // M x K in layoutA
  const char* Q;       // K x N, row-major
  const float* sk;     // K
  const void* C;       // M x N in D's type, or null
  void* D;
  int64_t M, N, K, lda, ldq, ldd;  // ldd: of C and D
  float beta;
  int use_c;
  int out;
  int vec_d;
  // general kernel (panel_n == 0)
  int tiny;            // the form for operands of less than 16 bytes
  int tile;            // rows of a tile
  int tiles_m, tiles_n;
  int splits, kt_per_split;  // splits > 1: ws holds one M x N binary32 matrix per range
  // panels of Q widened in the workspace, for the pipelined dense kernels
  int64_t panel_n;     // columns per panel (a multiple of 256, or all of N)
  int64_t ldw;         // of a panel, elements
  int64_t ka;          // K of the dense product: K, or a multiple of 8 with zeros past K
  int64_t lda2;        // of the copy of A, or 0: A is read in place
  int pipe_tile, sk_tiles;  // of the first panel's product (each panel's is planned at its launch)
  void* ws;
  int64_t ws_bytes;
};
int64_t plan_grad(int dtA, int layoutA, GradArgs& a, int num_cu, int64_t ws_bytes);
hipError_t launch_grad(int dtA, int layoutA, const GradArgs& a, int num_cu, hipStream_t s);

// Form of the pipelined dense kernels for a problem whose operands they take
// (chunked and windowed as they need; M and N may be below the tile): the tile, the
// stream-K plan in a when it fits ws_cap, and the modelled time in us.
struct PipePlan {
  int tile;    // 256, 128, or 64 (64 x 128: launch_fast_half / launch_scaled_half)
  int64_t ws;
  double us;
};
// 16-bit A in layoutA, MN-contiguous B, 64 x 128 tiles.
hipError_t launch_fast_half(int dtA, int layoutA, const DenseArgs& a, hipStream_t s);
PipePlan plan_pipe(int dt, DenseArgs& a, int num_cu, int64_t ws_cap);
// A copy of rows of row_bytes bytes, lds apart, to rows of ldd bytes (a multiple of
// 16), zeros past row_bytes and past `rows` up to rows_d.
struct AlignRows {
  const char* src;
  int64_t lds, rows, row_bytes;
  char* dst;
  int64_t ldd, rows_d;
};
hipError_t launch_align_rows(const AlignRows& a, hipStream_t s, const AlignRows* second = nullptr);
// Time of a pass that moves `bytes` at the rate of a copy, with its launch, in us.
inline double pass_us(double bytes) { return 3.0 + bytes / 5.5e6; }

}  // namespace mcg
