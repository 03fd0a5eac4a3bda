// linear8.hpp -- kernel argument blocks and launchers of the 8-bit linear layer:
// row quantisation, the root-mean-square norm around it, and the scaled int8 and
// mixed products.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// D = (A . B) * sa_i * sb_j + bias_j, int8 operands (gemm_i8_scaled.hip).
struct ScaledArgs {
  const char* A;       // M x K, row-major
  const char* B;       // K x N in layoutB
  const float* sa;     // M
  const float* sb;     // N
  const float* bias;   // N, or null
  void* D;
  int64_t M, N, K, lda, ldb, ldd;
  int out;             // OUT_32, OUT_BF16, OUT_F16
  int vec_d;           // 4 consecutive elements of D can be stored as one vector
  int tiles_m, tiles_n;
  int splits, kt_per_split;  // K ranges multiplied by separate workgroups
  int32_t* ws;         // splits > 1: one M x N int32 matrix per range
};
int64_t plan_scaled(ScaledArgs& a, int layoutB, int num_cu, int64_t ws_bytes);
hipError_t launch_scaled(int layoutB, const ScaledArgs& a, hipStream_t s);

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
  int tiles_m, tiles_n;
  int splits, kt_per_split;
  float* ws;           // splits > 1: one M x N binary32 matrix per range
};
int64_t plan_grad(int dtA, int layoutA, GradArgs& a, int num_cu, int64_t ws_bytes);
hipError_t launch_grad(int dtA, int layoutA, const GradArgs& a, hipStream_t s);

}  // namespace mcg
