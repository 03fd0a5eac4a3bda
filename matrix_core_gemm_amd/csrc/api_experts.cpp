// api_experts.cpp -- the C ABI of the products by group and of block-scaled 8-bit
// floats (include/mcg.h).  Arguments are checked on the host before any HIP call.
#include "api_util.hpp"
#include "experts.hpp"

using namespace mcg::host;

namespace {

constexpr int64_t MAX_GROUPS = 65535;  // (a grid's second dimension)
constexpr int64_t BLOCK = mcg::SCALE_BLOCK;
constexpr int64_t MAX_COLUMN_BLOCKS = (1 << 24) - 1;  // (a grid holds less than 2^32 threads along a dimension: 256 for each)

bool sizes_ok(int64_t a, int64_t b, int64_t c) {
  return a >= 0 && b >= 0 && c >= 0 && a <= INT32_MAX && b <= INT32_MAX && c <= INT32_MAX;
}
bool ld_ok(int64_t ld, int64_t n) { return ld >= (n > 1 ? n : 1); }
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
bool f16_type(int dt) { return dt == MCG_BF16 || dt == MCG_F16; }
bool f8_type(int dt) { return dt == MCG_FP8_E4M3 || dt == MCG_FP8_E5M2; }
bool block_ok(int bm, int bn) { return (bm == 1 && bn == BLOCK) || (bm == BLOCK && (bn == 1 || bn == BLOCK)); }

// Tiles of G groups of M rows, or (grouped false) of one product, by N columns, 16- or 8-bit operands.
bool tiles_ok(int eb, int64_t M, int64_t G, int64_t N, bool grouped) {
  return mcg::tiles_fit(mcg::most_tiles(M, G, mcg::general_rows(eb), grouped), N, 128);
}
bool grad_tiles_ok(int64_t G, int64_t M, int64_t N) { return mcg::tiles_fit(G * cdiv(M, mcg::general_rows(2)), N, 128); }

int out_format(int dtypeD) {
  return dtypeD == MCG_BF16 ? mcg::OUT_BF16 : dtypeD == MCG_F16 ? mcg::OUT_F16 : mcg::OUT_32;
}

mcg::GroupArgs group_args(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                          const void* C, const void* D, int64_t ldd, int dtypeD, double beta) {
  mcg::GroupArgs a{};
  a.A = (const char*)A;
  a.B = (const char*)B;
  a.C = C;
  a.D = (void*)D;
  a.M = M;
  a.N = N;
  a.K = K;
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldd;
  a.alpha = 1.0f;
  a.beta = (float)beta;
  a.alpha_i = 1;
  a.use_c = beta != 0.0;
  a.out = out_format(dtypeD);
  a.splits = 1;
  a.groups = 1;
  a.blockB = (int)BLOCK;
  return a;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------- matrices in blocks
int mcg_validate_quantize_blocks(int dtype, int dtypeQ, int blockM, int blockN, int64_t M, int64_t N, const void* X,
                                 int64_t ldx, const void* Q, int64_t ldq, const void* scale, int64_t lds) {
  if (!float_out(dtype) || !f8_type(dtypeQ)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!block_ok(blockM, blockN)) return MCG_ERR_INVALID_VALUE;
  if (!sizes_ok(M, N, 0) || cdiv(N, BLOCK) > MAX_COLUMN_BLOCKS) return MCG_ERR_INVALID_SIZE;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!X || !Q || !scale) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(ldx, N) || !ld_ok(ldq, N) || !ld_ok(lds, cdiv(N, blockN))) return MCG_ERR_INVALID_LD;
  if (!aligned_to(X, elem_bytes(dtype)) || !aligned_to(scale, 4)) return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int quantize_blocks(int dtype, int dtypeQ, int blockM, int blockN, int64_t M, int64_t N, const void* X, int64_t ldx,
                    void* Q, int64_t ldq, float* scale, int64_t lds, void* stream) {
  int st = mcg_validate_quantize_blocks(dtype, dtypeQ, blockM, blockN, M, N, X, ldx, Q, ldq, scale, lds);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  const mcg::BlocksArgs a{(const char*)X, (char*)Q, scale, M, N, ldx, ldq, lds};
  return hip_status(mcg::launch_blocks_quant(dtype, dtypeQ, blockM, blockN, a, (hipStream_t)stream));
}

int mcg_validate_dequantize_blocks(int dtypeQ, int dtypeD, int blockM, int blockN, int64_t M, int64_t N,
                                   const void* Q, int64_t ldq, const void* scale, int64_t lds, const void* D,
                                   int64_t ldd) {
  if (!f8_type(dtypeQ) || !float_out(dtypeD)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!block_ok(blockM, blockN)) return MCG_ERR_INVALID_VALUE;
  if (!sizes_ok(M, N, 0) || cdiv(N, BLOCK) > MAX_COLUMN_BLOCKS) return MCG_ERR_INVALID_SIZE;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!Q || !scale || !D) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(ldq, N) || !ld_ok(ldd, N) || !ld_ok(lds, cdiv(N, blockN))) return MCG_ERR_INVALID_LD;
  if (!aligned_to(D, elem_bytes(dtypeD)) || !aligned_to(scale, 4)) return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int dequantize_blocks(int dtypeQ, int dtypeD, int blockM, int blockN, int64_t M, int64_t N, const void* Q, int64_t ldq,
                      const float* scale, int64_t lds, void* D, int64_t ldd, void* stream) {
  int st = mcg_validate_dequantize_blocks(dtypeQ, dtypeD, blockM, blockN, M, N, Q, ldq, scale, lds, D, ldd);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  const mcg::BlocksArgs a{(const char*)Q, (char*)D, (float*)scale, M, N, ldq, ldd, lds};
  return hip_status(mcg::launch_blocks_dequant(dtypeQ, dtypeD, blockM, blockN, a, (hipStream_t)stream));
}

// ------------------------------------------------------------------ products
int mcg_validate_grouped(int dtype, int layoutB, int64_t G, int64_t M, int64_t N, int64_t K, const void* offsets,
                         const void* A, int64_t lda, const void* B, int64_t ldb, int64_t strideB, const void* D,
                         int64_t ldd, int dtypeD) {
  if (!f16_type(dtype) || (dtypeD != dtype && dtypeD != MCG_F32) || !valid_layout(layoutB))
    return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N, K) || G < 0 || G > MAX_GROUPS || strideB < 0) return MCG_ERR_INVALID_SIZE;
  if (G == 0 || M == 0 || N == 0) return MCG_SUCCESS;
  if (!tiles_ok(2, M, G, N, true)) return MCG_ERR_INVALID_SIZE;
  if (!offsets || !D || (K > 0 && (!A || !B))) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(lda, K) || !ld_ok(ldb, layoutB == MCG_K_CONTIG ? K : N) || !ld_ok(ldd, N)) return MCG_ERR_INVALID_LD;
  if (!aligned_to(offsets, 4) || !aligned_to(A, 2) || !aligned_to(B, 2) || !aligned_to(D, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int gemm_grouped(int dtype, int layoutB, int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                 const void* A, int64_t lda, const void* B, int64_t ldb, int64_t strideB, void* D, int64_t ldd,
                 int dtypeD, void* stream) {
  int st = mcg_validate_grouped(dtype, layoutB, G, M, N, K, offsets, A, lda, B, ldb, strideB, D, ldd, dtypeD);
  if (st != MCG_SUCCESS || G == 0 || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, nullptr, D, ldd, dtypeD, 0.0);
  a.offsets = offsets;
  a.groups = (int)G;
  a.strideB = strideB;
  return hip_status(mcg::launch_grouped(dtype, MCG_K_CONTIG, layoutB, a, current_num_cu(), (hipStream_t)stream));
}

int mcg_validate_grouped_grad(int dtype, int64_t G, int64_t M, int64_t N, int64_t K, const void* offsets,
                              const void* A, int64_t lda, const void* B, int64_t ldb, const void* C, const void* D,
                              int64_t ldd, int64_t strideD, int dtypeD, double beta) {
  if (!f16_type(dtype) || (dtypeD != dtype && dtypeD != MCG_F32)) return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N, K) || G < 0 || G > MAX_GROUPS) return MCG_ERR_INVALID_SIZE;
  if (!std::isfinite((float)beta)) return MCG_ERR_INVALID_VALUE;
  if (G == 0 || M == 0 || N == 0) return MCG_SUCCESS;
  if (!grad_tiles_ok(G, M, N)) return MCG_ERR_INVALID_SIZE;
  if (!D || (K > 0 && (!offsets || !A || !B)) || (beta != 0.0 && !C)) return MCG_ERR_NULL_POINTER;
  if (!ld_ok(lda, M) || !ld_ok(ldb, N) || !ld_ok(ldd, N) || (G > 1 && strideD < (M - 1) * ldd + N))
    return MCG_ERR_INVALID_LD;
  if (!aligned_to(offsets, 4) || !aligned_to(A, 2) || !aligned_to(B, 2) || !aligned_to(D, elem_bytes(dtypeD)) ||
      !aligned_to(C, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int gemm_grouped_grad(int dtype, int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets, const void* A,
                      int64_t lda, const void* B, int64_t ldb, const void* C, void* D, int64_t ldd, int64_t strideD,
                      int dtypeD, double beta, void* stream) {
  int st = mcg_validate_grouped_grad(dtype, G, M, N, K, offsets, A, lda, B, ldb, C, D, ldd, strideD, dtypeD, beta);
  if (st != MCG_SUCCESS || G == 0 || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, C, D, ldd, dtypeD, beta);
  a.offsets = K > 0 ? offsets : nullptr;
  a.groups = (int)G;
  a.strideD = strideD;
  return hip_status(mcg::launch_grouped_grad(dtype, a, current_num_cu(), (hipStream_t)stream));
}

int mcg_validate_f8_blocks(int dtypeA, int dtypeB, int layoutA, int layoutB, int blockB, int64_t M, int64_t N,
                           int64_t K, const void* A, int64_t lda, const void* scaleA, int64_t ldsa, const void* B,
                           int64_t ldb, const void* scaleB, int64_t ldsb, const void* C, const void* D, int64_t ldd,
                           int dtypeD, double beta) {
  if (!f8_type(dtypeA) || dtypeB != MCG_FP8_E4M3 || !float_out(dtypeD) || !valid_layout(layoutA) ||
      !valid_layout(layoutB))
    return MCG_ERR_UNSUPPORTED_DTYPE;
  if ((blockB != 1 && blockB != BLOCK) || !std::isfinite((float)beta)) return MCG_ERR_INVALID_VALUE;
  if (!sizes_ok(M, N, K)) return MCG_ERR_INVALID_SIZE;
  if (M == 0 || N == 0) return MCG_SUCCESS;
  if (!tiles_ok(1, M, 1, N, false)) return MCG_ERR_INVALID_SIZE;
  if (!D || (K > 0 && (!A || !B || !scaleA || !scaleB)) || (beta != 0.0 && !C)) return MCG_ERR_NULL_POINTER;
  const int64_t kb = cdiv(K, BLOCK), nb = cdiv(N, blockB);
  if (!ld_ok(lda, layoutA == MCG_K_CONTIG ? K : M) || !ld_ok(ldb, layoutB == MCG_K_CONTIG ? K : N) || !ld_ok(ldd, N) ||
      !ld_ok(ldsa, layoutA == MCG_K_CONTIG ? kb : M) || !ld_ok(ldsb, layoutB == MCG_K_CONTIG ? kb : nb))
    return MCG_ERR_INVALID_LD;
  if (!aligned_to(scaleA, 4) || !aligned_to(scaleB, 4) || !aligned_to(D, elem_bytes(dtypeD)) ||
      !aligned_to(C, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int gemm_f8_blocks(int dtypeA, int dtypeB, int layoutA, int layoutB, int blockB, int64_t M, int64_t N, int64_t K,
                   const void* A, int64_t lda, const float* scaleA, int64_t ldsa, const void* B, int64_t ldb,
                   const float* scaleB, int64_t ldsb, const void* C, void* D, int64_t ldd, int dtypeD, double beta,
                   void* stream) {
  int st = mcg_validate_f8_blocks(dtypeA, dtypeB, layoutA, layoutB, blockB, M, N, K, A, lda, scaleA, ldsa, B, ldb,
                                  scaleB, ldsb, C, D, ldd, dtypeD, beta);
  if (st != MCG_SUCCESS || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, C, D, ldd, dtypeD, beta);
  a.sa = scaleA;
  a.sb = scaleB;
  a.ldsa = ldsa;
  a.ldsb = ldsb;
  a.blockB = blockB;
  return hip_status(mcg::launch_grouped(dtypeA, layoutA, layoutB, a, current_num_cu(), (hipStream_t)stream));
}

int mcg_validate_grouped_f8_blocks(int dtypeA, int dtypeB, int layoutB, int64_t G, int64_t M, int64_t N, int64_t K,
                                   const void* offsets, const void* A, int64_t lda, const void* scaleA, int64_t ldsa,
                                   const void* B, int64_t ldb, int64_t strideB, const void* scaleB, int64_t ldsb,
                                   int64_t strideSB, const void* D, int64_t ldd, int dtypeD) {
  if (!f8_type(dtypeA) || dtypeB != MCG_FP8_E4M3 || !float_out(dtypeD) || !valid_layout(layoutB))
    return MCG_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(M, N, K) || G < 0 || G > MAX_GROUPS || strideB < 0 || strideSB < 0) return MCG_ERR_INVALID_SIZE;
  if (G == 0 || M == 0 || N == 0) return MCG_SUCCESS;
  if (!tiles_ok(1, M, G, N, true)) return MCG_ERR_INVALID_SIZE;
  if (!offsets || !D || (K > 0 && (!A || !B || !scaleA || !scaleB))) return MCG_ERR_NULL_POINTER;
  const int64_t kb = cdiv(K, BLOCK), nb = cdiv(N, BLOCK);
  if (!ld_ok(lda, K) || !ld_ok(ldb, layoutB == MCG_K_CONTIG ? K : N) || !ld_ok(ldd, N) || !ld_ok(ldsa, kb) ||
      !ld_ok(ldsb, layoutB == MCG_K_CONTIG ? kb : nb))
    return MCG_ERR_INVALID_LD;
  if (!aligned_to(offsets, 4) || !aligned_to(scaleA, 4) || !aligned_to(scaleB, 4) || !aligned_to(D, elem_bytes(dtypeD)))
    return MCG_ERR_MISALIGNED;
  return MCG_SUCCESS;
}

int gemm_grouped_f8_blocks(int dtypeA, int dtypeB, int layoutB, int64_t G, int64_t M, int64_t N, int64_t K,
                           const int32_t* offsets, const void* A, int64_t lda, const float* scaleA, int64_t ldsa,
                           const void* B, int64_t ldb, int64_t strideB, const float* scaleB, int64_t ldsb,
                           int64_t strideSB, void* D, int64_t ldd, int dtypeD, void* stream) {
  int st = mcg_validate_grouped_f8_blocks(dtypeA, dtypeB, layoutB, G, M, N, K, offsets, A, lda, scaleA, ldsa, B, ldb,
                                          strideB, scaleB, ldsb, strideSB, D, ldd, dtypeD);
  if (st != MCG_SUCCESS || G == 0 || M == 0 || N == 0) return st;
  st = check_arch();
  if (st != MCG_SUCCESS) return st;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, nullptr, D, ldd, dtypeD, 0.0);
  a.offsets = offsets;
  a.groups = (int)G;
  a.strideB = strideB;
  a.sa = scaleA;
  a.sb = scaleB;
  a.ldsa = ldsa;
  a.ldsb = ldsb;
  a.strideSB = strideSB;
  return hip_status(mcg::launch_grouped(dtypeA, MCG_K_CONTIG, layoutB, a, current_num_cu(), (hipStream_t)stream));
}

// The kernel of a call, with tiles of its rows in plan[0] (or NULL).
int mcg_grouped_path(int dtype, int layoutA, int layoutB, int64_t G, int64_t M, int64_t N, int64_t K, const void* A,
                     int64_t lda, const void* B, int64_t ldb, int64_t strideB, int blockB, int dtypeD, int64_t* plan) {
  const bool f8 = f8_type(dtype);
  if ((!f8 && !f16_type(dtype)) || !float_out(dtypeD) || !valid_layout(layoutA) || !valid_layout(layoutB) ||
      !sizes_ok(M, N, K) || M == 0 || N == 0 || G < 0 || G > MAX_GROUPS || !tiles_ok(f8 ? 1 : 2, M, G, N, G > 0))
    return -1;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, nullptr, nullptr, N, dtypeD, 0.0);
  static const int32_t some = 0;
  a.offsets = G > 0 ? &some : nullptr;  // (not read)
  a.groups = (int)(G > 0 ? G : 1);
  a.strideB = strideB;
  a.blockB = blockB;
  const mcg::GroupPlan p = mcg::plan_grouped(dtype, layoutA, layoutB, a, current_num_cu());
  if (plan) plan[0] = p.tile;
  return p.kernel;
}

int mcg_grouped_grad_path(int dtype, int64_t G, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                          const void* B, int64_t ldb, int dtypeD, int64_t* plan) {
  if (!f16_type(dtype) || (dtypeD != dtype && dtypeD != MCG_F32) || !sizes_ok(M, N, K) || M == 0 || N == 0 || G <= 0 ||
      G > MAX_GROUPS || !grad_tiles_ok(G, M, N))
    return -1;
  mcg::GroupArgs a = group_args(M, N, K, A, lda, B, ldb, nullptr, nullptr, N, dtypeD, 0.0);
  a.groups = (int)G;
  const mcg::GroupPlan p = mcg::plan_grouped_grad(dtype, a, current_num_cu());
  if (plan) plan[0] = p.tile;
  return p.kernel;
}

}  // extern "C"
