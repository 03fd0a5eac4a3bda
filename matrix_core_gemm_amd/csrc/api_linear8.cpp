// api_linear8.cpp -- the C ABI of the 8-bit linear layer (include/mcg.h): row
// quantisation, the root-mean-square norm and its gradient, the int8 product with
// scales per row and column, and the product of 16-bit with scaled 8-bit rows.
// Arguments are checked on the host before any HIP call.
#include <cfloat>

#include "api_util.hpp"
#include "gemm_kernels.hpp"
#include "linear8.hpp"

using namespace mcg::host;

namespace {

bool sizes_ok(int64_t a, int64_t b) { return a >= 0 && b >= 0 && a <= INT32_MAX && b <= INT32_MAX; }
bool ld_ok(int64_t ld, int64_t n) { return ld >= (n > 1 ? n : 1); }
int out_format(int dtypeD) {
  return dtypeD == MCG_BF16 ? mcg::OUT_BF16 : dtypeD == MCG_F16 ? mcg::OUT_F16 : mcg::OUT_32;
}

// Workspace argument checks common to the products.
int check_workspace(const void* ws, int64_t bytes) {
  if (bytes < 0) return MCG_ERR_INVALID_SIZE;
  return ws != nullptr && !aligned_to(ws, 16) ? MCG_ERR_MISALIGNED : MCG_SUCCESS;
}

mcg::ScaledArgs scaled_args(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                            int64_t ldd, int dtypeD, const void* D) {
  mcg::ScaledArgs a{};
  a.A = (const char*)A;
  a.B = (const char*)B;
  a.D = (void*)D;
  a.M = M;
  a.N = N;
  a.K = K;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldd;
  a.out = out_format(dtypeD);
  a.vec_cd = aligned_to(D, 4 * elem_bytes(dtypeD)) && ldd % 4 == 0;
  return a;
}

mcg::GradArgs grad_args(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Q, int64_t ldq,
                        const void* C, const void* D, int64_t ldd, int dtypeD, double beta) {
  mcg::GradArgs a{};
  a.A = (const char*)A;
  a.Q = (const char*)Q;
  a.C = C;
  a.D = (void*)D;
  a.M = M;
  a.N = N;
  a.K = K;
  a.lda = lda;
  a.ldq = ldq;
  a.ldd = ldd;
  a.beta = (float)beta;
  a.use_c = beta != 0.0;
  a.out = out_format(dtypeD);
  const int vb = 4 * elem_bytes(dtypeD);
  a.vec_d = aligned_to(D, vb) && (!a.use_c || aligned_to(C, vb)) && ldd % 4 == 0;
  return a;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ rows
int mcg_validate_rmsnorm_quant(int dtype, int64_t M, int64_t N, const void* X, int64_t ldx, const void* R,
                               int64_t ldr, const void* weight, double eps, const void* H, int64_t ldh,
                               const void* Q, int64_t ldq, const void* scale, const void* rstd) {
  if (!float_out(dtype)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N)) return MCG_ERR_INVALID_SIZE;
  if (!std::isfinite(eps) || eps < 0.0 || eps > FLT_MAX) return MCG_ERR_INVALID_VALUE;
  if (M == 0) return MCG_SUCCESS;
  if (!scale || (N > 0 && (!X || !Q))) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(ldx, N) || !ld_ok(ldq, N) || (R && !ld_ok(ldr, N)) || (H && !ld_ok(ldh, N))) return MCG_ERR_INVALID_LD;
  const int eb = elem_bytes(dtype);
  if (!aligned_to(X, eb) || !aligned_to(R, eb) || !aligned_to(weight, eb) || !aligned_to(H, eb) ||
      !aligned_to(scale, 4) || !aligned_to(rstd, 4))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int rmsnorm_quant(int dtype, int64_t M, int64_t N, const void* X, int64_t ldx, const void* R, int64_t ldr,
                  const void* weight, double eps, void* H, int64_t ldh, int8_t* Q, int64_t ldq, float* scale,
                  float* rstd, void* stream) {
  int st = mcg_validate_rmsnorm_quant(dtype, M, N, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, scale, rstd);
  if (st != MCG_SUCCESS || M == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::RowsQuantArgs a{};
  a.X = (const char*)X;
  a.R = (const char*)R;
  a.W = (const char*)weight;
  a.H = (char*)H;
  a.Q = Q;
  a.scale = scale;
  a.rstd = rstd;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldq = ldq;
  a.eps = (float)eps;
  return hip_status(mcg::launch_rows_quant(dtype, true, a, current_num_cu(), (hipStream_t)stream));
}

int mcg_validate_rmsnorm_backward(int dtype, int dtypeX, int64_t M, int64_t N, const void* dY, int64_t lddy,
                                  const void* X, int64_t ldx, const void* scaleX, const void* weight,
                                  const void* rstd, const void* dR, int64_t lddr, const void* dX, int64_t lddx,
                                  const void* dW, const void* workspace, int64_t workspace_bytes) {
  if (!float_out(dtype) || (dtypeX != dtype && dtypeX != MCG_I8)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N)) return MCG_ERR_INVALID_SIZE;
  int st = check_workspace(workspace, workspace_bytes);
  if (st != MCG_SUCCESS) return st;
  if (N == 0) return MCG_SUCCESS;
  if (M > 0) {
    if (!dY || !X || !rstd || !dX || (dtypeX == MCG_I8 && !scaleX)) return MCG_ERR_NULL_POINTER;
    if (!ld_ok(lddy, N) || !ld_ok(ldx, N) || !ld_ok(lddx, N) || (dR && !ld_ok(lddr, N))) return MCG_ERR_INVALID_LD;
    const int eb = elem_bytes(dtype);
    if (!aligned_to(dY, eb) || !aligned_to(X, elem_bytes(dtypeX)) || !aligned_to(weight, eb) ||
        !aligned_to(dR, eb) || !aligned_to(dX, eb) || !aligned_to(scaleX, 4) || !aligned_to(rstd, 4))
      return MCG_ERR_MISALIGNED;
  }
  if (dW) {
    if (!aligned_to(dW, 4)) return MCG_ERR_MISALIGNED;
    const int64_t need = mcg_rmsnorm_backward_workspace_bytes(M, N);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MCG_ERR_SCRATCH_LIMIT;
  }
  return MCG_SUCCESS;
}

int64_t mcg_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N) {
  return M <= 0 || N <= 0 ? 0 : mcg::norm_grad_workspace(M, N);
}

int rmsnorm_backward(int dtype, int dtypeX, int64_t M, int64_t N, const void* dY, int64_t lddy, const void* X,
                     int64_t ldx, const float* scaleX, const void* weight, const float* rstd, const void* dR,
                     int64_t lddr, void* dX, int64_t lddx, float* dW, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  int st = mcg_validate_rmsnorm_backward(dtype, dtypeX, M, N, dY, lddy, X, ldx, scaleX, weight, rstd, dR, lddr, dX,
                                         lddx, dW, workspace, workspace_bytes);
  if (st != MCG_SUCCESS || N == 0 || (M == 0 && !dW)) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::NormGradArgs a{};
  a.dY = (const char*)dY;
  a.X = (const char*)X;
  a.xscale = scaleX;
  a.W = (const char*)weight;
  a.rstd = rstd;
  a.dR = (const char*)dR;
  a.dX = (char*)dX;
  a.dW = dW;
  a.part = (float*)workspace;
  a.M = M;
  a.N = N;
  a.lddy = lddy;
  a.ldx = ldx;
  a.lddr = lddr;
  a.lddx = lddx;
  return hip_status(mcg::launch_norm_grad(dtype, dtypeX == MCG_I8, a, (hipStream_t)stream));
}

int mcg_validate_quantize_rows(int dtype, int64_t M, int64_t N, const void* X, int64_t ldx, const void* Q,
                               int64_t ldq, const void* scale) {
  if (!float_out(dtype)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N)) return MCG_ERR_INVALID_SIZE;
  if (M == 0) return MCG_SUCCESS;
  if (!scale || (N > 0 && (!X || !Q))) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(ldx, N) || !ld_ok(ldq, N)) return MCG_ERR_INVALID_LD;
  if (!aligned_to(X, elem_bytes(dtype)) || !aligned_to(scale, 4)) return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int quantize_rows(int dtype, int64_t M, int64_t N, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale,
                  void* stream) {
  int st = mcg_validate_quantize_rows(dtype, M, N, X, ldx, Q, ldq, scale);
  if (st != MCG_SUCCESS || M == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::RowsQuantArgs a{};
  a.X = (const char*)X;
  a.Q = Q;
  a.scale = scale;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldq = ldq;
  return hip_status(mcg::launch_rows_quant(dtype, false, a, current_num_cu(), (hipStream_t)stream));
}

int mcg_validate_dequantize_rows(int dtypeD, int64_t M, int64_t N, const void* Q, int64_t ldq, const void* scale,
                                 const void* D, int64_t ldd) {
  if (!float_out(dtypeD)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N)) return MCG_ERR_INVALID_SIZE;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!Q || !scale || !D) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(ldq, N) || !ld_ok(ldd, N)) return MCG_ERR_INVALID_LD;
  if (!aligned_to(D, elem_bytes(dtypeD)) || !aligned_to(scale, 4)) return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int dequantize_rows(int dtypeD, int64_t M, int64_t N, const int8_t* Q, int64_t ldq, const float* scale, void* D,
                    int64_t ldd, void* stream) {
  int st = mcg_validate_dequantize_rows(dtypeD, M, N, Q, ldq, scale, D, ldd);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::RowsDequantArgs a{};
  a.Q = Q;
  a.scale = scale;
  a.D = (char*)D;
  a.M = M;
  a.N = N;
  a.ldq = ldq;
  a.ldd = ldd;
  return hip_status(mcg::launch_rows_dequant(dtypeD, a, (hipStream_t)stream));
}

// -------------------------------------------------------------- products
int mcg_validate_i8_scaled(int layoutB, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                           const void* scaleA, const void* B, int64_t ldb, const void* scaleB, const void* bias,
                           const void* D, int64_t ldd, int dtypeD, const void* workspace, int64_t workspace_bytes) {
  if (!float_out(dtypeD) || !valid_layout(layoutB)) return MCG_ERR_UNSUPPORTED_DTYPE;
  // K * 128 * 128 must fit an int32
  if (!sizes_ok(M, N) || K < 0 || K > 131071) return MCG_ERR_INVALID_SIZE;
  const int st = check_workspace(workspace, workspace_bytes);
  if (st != MCG_SUCCESS) return st;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!scaleA || !scaleB || !D || (K > 0 && (!A || !B))) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(lda, K) || !ld_ok(ldb, layoutB == MCG_K_CONTIG ? K : N) || !ld_ok(ldd, N)) return MCG_ERR_INVALID_LD;
  if (!aligned_to(scaleA, 4) || !aligned_to(scaleB, 4) || !aligned_to(bias, 4) || !aligned_to(D, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int64_t mcg_i8_scaled_workspace_bytes(int layoutB, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                      const void* B, int64_t ldb) {
  if (!valid_layout(layoutB) || M <= 0 || N <= 0 || K <= 0 || !sizes_ok(M, N) || K > 131071) return 0;
  mcg::ScaledArgs a = scaled_args(M, N, K, A, lda, B, ldb, N, MCG_F32, nullptr);
  return mcg::plan_scaled(a, layoutB, current_num_cu(), INT64_MAX);
}

int mcg_i8_scaled_path(int layoutB, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                       int64_t ldb, int64_t workspace_bytes, int64_t* plan) {
  if (!valid_layout(layoutB) || M <= 0 || N <= 0 || K < 0 || !sizes_ok(M, N) || K > 131071) return -1;
  mcg::ScaledArgs a = scaled_args(M, N, K, A, lda, B, ldb, N, MCG_F32, nullptr);
  const int64_t used = mcg::plan_scaled(a, layoutB, current_num_cu(), workspace_bytes);
  if (plan) {
    plan[0] = a.panel_n;
    plan[1] = a.splits;
    plan[2] = a.sk_tiles;
    plan[3] = used;
  }
  return a.kernel == mcg::KERNEL_FAST ? mcg::pipe_kernel(a.tile) : a.kernel;
}

int gemm_i8_scaled(int layoutB, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* scaleA,
                   const int8_t* B, int64_t ldb, const float* scaleB, const float* bias, void* D, int64_t ldd,
                   int dtypeD, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = mcg_validate_i8_scaled(layoutB, M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, D, ldd, dtypeD, workspace,
                                  workspace_bytes);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::ScaledArgs a = scaled_args(M, N, K, A, lda, B, ldb, ldd, dtypeD, D);
  a.sa = scaleA;
  a.sb = scaleB;
  a.bias = bias;
  a.ws = workspace;
  a.ws_bytes = workspace ? workspace_bytes : 0;
  const int num_cu = current_num_cu();
  mcg::plan_scaled(a, layoutB, num_cu, a.ws_bytes);
  return hip_status(mcg::launch_scaled(layoutB, a, num_cu, (hipStream_t)stream));
}

int mcg_validate_grad_i8(int dtypeA, int layoutA, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                         const void* Q, int64_t ldq, const void* scaleK, const void* C, const void* D, int64_t ldd,
                         int dtypeD, double beta, const void* workspace, int64_t workspace_bytes) {
  if ((dtypeA != MCG_BF16 && dtypeA != MCG_F16) || (dtypeD != dtypeA && dtypeD != MCG_F32) || !valid_layout(layoutA))
    return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N) || !sizes_ok(K, 0)) return MCG_ERR_INVALID_SIZE;
  if (!std::isfinite((float)beta)) return MCG_ERR_INVALID_VALUE;
  const int st = check_workspace(workspace, workspace_bytes);
  if (st != MCG_SUCCESS) return st;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!D || (K > 0 && (!A || !Q || !scaleK)) || (beta != 0.0 && !C)) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(lda, layoutA == MCG_K_CONTIG ? K : M) || !ld_ok(ldq, N) || !ld_ok(ldd, N)) return MCG_ERR_INVALID_LD;
  if (!aligned_to(A, 2) || !aligned_to(scaleK, 4) || !aligned_to(D, elem_bytes(dtypeD)) ||
      !aligned_to(C, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int64_t mcg_grad_i8_workspace_bytes(int dtypeA, int layoutA, int64_t M, int64_t N, int64_t K, const void* A,
                                    int64_t lda, const void* Q, int64_t ldq, int dtypeD) {
  if ((dtypeA != MCG_BF16 && dtypeA != MCG_F16) || (dtypeD != dtypeA && dtypeD != MCG_F32) ||
      !valid_layout(layoutA) || M <= 0 || N <= 0 || K <= 0 || !sizes_ok(M, N) || !sizes_ok(K, 0))
    return 0;
  mcg::GradArgs a = grad_args(M, N, K, A, lda, Q, ldq, nullptr, nullptr, N, dtypeD, 0.0);
  return mcg::plan_grad(dtypeA, layoutA, a, current_num_cu(), INT64_MAX);
}

int mcg_grad_i8_path(int dtypeA, int layoutA, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                     const void* Q, int64_t ldq, int dtypeD, int64_t workspace_bytes, int64_t* plan) {
  if ((dtypeA != MCG_BF16 && dtypeA != MCG_F16) || (dtypeD != dtypeA && dtypeD != MCG_F32) ||
      !valid_layout(layoutA) || M <= 0 || N <= 0 || K < 0 || !sizes_ok(M, N) || !sizes_ok(K, 0))
    return -1;
  mcg::GradArgs a = grad_args(M, N, K, A, lda, Q, ldq, nullptr, nullptr, N, dtypeD, 0.0);
  const int64_t used = mcg::plan_grad(dtypeA, layoutA, a, current_num_cu(), workspace_bytes);
  const bool panels = a.panel_n > 0;
  if (plan) {
    plan[0] = a.panel_n;
    plan[1] = panels ? 1 : a.splits;
    plan[2] = panels ? a.sk_tiles : 0;
    plan[3] = used;
  }
  return a.tiny ? mcg::KERNEL_TINY : panels ? mcg::pipe_kernel(a.pipe_tile) : mcg::KERNEL_GENERAL;
}

int gemm_grad_i8(int dtypeA, int layoutA, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                 const int8_t* Q, int64_t ldq, const float* scaleK, const void* C, void* D, int64_t ldd, int dtypeD,
                 double beta, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = mcg_validate_grad_i8(dtypeA, layoutA, M, N, K, A, lda, Q, ldq, scaleK, C, D, ldd, dtypeD, beta, workspace,
                                workspace_bytes);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::GradArgs a = grad_args(M, N, K, A, lda, Q, ldq, C, D, ldd, dtypeD, beta);
  a.sk = scaleK;
  a.ws = workspace;
  a.ws_bytes = workspace ? workspace_bytes : 0;
  const int num_cu = current_num_cu();
  mcg::plan_grad(dtypeA, layoutA, a, num_cu, a.ws_bytes);
  return hip_status(mcg::launch_grad(dtypeA, layoutA, a, num_cu, (hipStream_t)stream));
}

}  // extern "C"
