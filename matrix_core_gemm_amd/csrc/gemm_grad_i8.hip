// gemm_grad_i8.hip -- product of a 16-bit matrix with an 8-bit one whose rows carry
// a scale along the summed dimension:
//
//   D[i][j] = sum_k A[i][k] * (s[k] Q[k][j]) + beta * C[i][j]
//
// A linear layer's weight gradient from the 8-bit checkpoint of its input
// (A = dY^T, k the tokens) and its input gradient from 8-bit weights with a scale
// per output channel (A = dY, k the channels).
//
// s varies along k, so it cannot leave the sum; the value s[k] Q[k][j] is formed in
// binary32 and multiplied on the matrix cores in A's type:
//   - for a D of A's type it is rounded once to that type (as the activation was
//     before it was put in 8 bits): an error of at most half a step per product,
//     the size of the rounding of D itself;
//   - for a binary32 D it is split into two values of A's type (the rounded value
//     and the rounded rest) and multiplied twice, which leaves 2^-17 of bf16 and
//     2^-22 of f16 values, so that gradients summed over many calls do not collect
//     the operand's rounding.
// Sums are binary32.
//
// General kernel: 128 x 128 tiles, 4 wavefronts, any size, pointer and leading
// dimension.  Q's tile is widened on its way from the registers to LDS, where it is
// an ordinary 16-bit MN-contiguous tile.
#include <algorithm>

#include "linear8.hpp"
#include "row_vec.hpp"
#include "tile_any.hpp"

namespace mcg {

// 16 codes of one k row -> 16 values in A's type: hi, and with TWO the rest lo.
template <class Op, bool TWO>
__device__ __forceinline__ void widen16(const i32x4& codes, float s, i32x4 (&hi)[2], i32x4 (&lo)[2]) {
  constexpr int DT = std::is_same<Op, OpBF16>::value ? DT_BF16 : DT_F16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const rows::Raw8<DT_I8> r{{(uint32_t)codes[2 * h], (uint32_t)codes[2 * h + 1]}};
    float v[8];
    rows::widen8<DT_I8>(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s;
    const rows::Raw8<DT> a = rows::narrow8<DT>(v);
    hi[h] = i32x4{(int)a.w[0], (int)a.w[1], (int)a.w[2], (int)a.w[3]};
    if constexpr (TWO) {
      float b[8];
      rows::widen8<DT>(a, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] -= b[e];
      const rows::Raw8<DT> c = rows::narrow8<DT>(v);
      lo[h] = i32x4{(int)c.w[0], (int)c.w[1], (int)c.w[2], (int)c.w[3]};
    }
  }
}

// alpha = 1: D = v + beta * C, one rounding to D's type.
__device__ __forceinline__ void grad_store4(const GradArgs& p, int64_t m, int64_t n, const f32x4& v) {
  const int64_t off = m * p.ldd + n;
  const bool full = p.vec_d && n + 4 <= p.N;
  if (full && p.out == OUT_32) {
    f32x4 o = v;
    if (p.use_c) {
      const f32x4 c = *(const f32x4*)((const float*)p.C + off);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(p.beta, c[e], v[e]);
    }
    *(f32x4*)((float*)p.D + off) = o;
  } else if (full) {
    i32x2 c = {0, 0};
    if (p.use_c) c = *(const i32x2*)((const uint16_t*)p.C + off);
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ce = from_out_bits(p.out, ((uint32_t)c[e / 2] >> (16 * (e & 1))) & 0xffffu);
      b[e] = to_out_bits(p.out, p.use_c ? __builtin_fmaf(p.beta, ce, v[e]) : v[e]);
    }
    *(i32x2*)((uint16_t*)p.D + off) = i32x2{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
  } else {
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) combine_store(p.C, p.D, off + e, v[e], 1.0f, p.beta, p.use_c, p.out);
  }
}

template <class Op, int LA, bool TWO>
__global__ __launch_bounds__(256) void grad_general_kernel(GradArgs p) {
  constexpr int BM = 128, BN = 128, NT = 256, WT = 4, KE = KT_BYTES / 2;
  using GA = TileGeom<2, LA, BM>;
  using GB = TileGeom<2, LAYOUT_MN, BN>;
  using RA = FragReader<2, 16, LA, BM>;
  using RB = FragReader<2, 16, LAYOUT_MN, BN>;
  constexpr int STAGE = GA::BYTES + (TWO ? 2 : 1) * GB::BYTES;
  constexpr int QCPR = BN / 16, QPT = KE * QCPR / NT;  // 16-code chunks per row and per thread
  __shared__ __attribute__((aligned(16))) char smem_raw[2 * STAGE];
  lds_char* smem = (lds_char*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nk_all = (int)((p.K + KE - 1) / KE);
  const int kt0 = (int)blockIdx.y * p.kt_per_split;
  const int nk = min(nk_all - kt0, p.kt_per_split);

  AnyLoader<2, LA, BM, NT> la;
  i32x4 q[QPT];
  float s[QPT];
  auto load_tiles = [&](int kt) {
    const int64_t k0 = (int64_t)(kt0 + kt) * KE;
    if constexpr (LA == LAYOUT_K) la.load(p.A, p.lda, m0, k0, p.M, p.K, tid);
    else la.load(p.A, p.lda, k0, m0, p.K, p.M, tid);
#pragma unroll
    for (int t = 0; t < QPT; ++t) {
      const int c = tid + t * NT;
      const int64_t k = k0 + c / QCPR, n = n0 + 16 * (c % QCPR);
      q[t] = load_chunk(p.Q, p.Q + k * p.ldq + n, k < p.K ? p.N - n : 0);
      s[t] = k < p.K ? p.sk[k] : 0.0f;
    }
  };
  auto store_tiles = [&](lds_char* st) {
    la.store(st, tid);
    lds_char* tb = st + GA::BYTES;
#pragma unroll
    for (int t = 0; t < QPT; ++t) {
      const int c = tid + t * NT;
      const int r = c / QCPR, cc = 2 * (c % QCPR);
      const int sw = swz<2, LAYOUT_MN, GB::CPR>(r);
      i32x4 hi[2], lo[2];
      widen16<Op, TWO>(q[t], s[t], hi, lo);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds_write_b128(tb, r * GB::W + (((cc + h) ^ sw) * 16), hi[h]);
        if constexpr (TWO) lds_write_b128(tb + GB::BYTES, r * GB::W + (((cc + h) ^ sw) * 16), lo[h]);
      }
    }
  };
  f32x4 acc[WT][WT];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int j = 0; j < WT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  if (nk > 0) {
    load_tiles(0);
    store_tiles(smem);
    __syncthreads();
  }
  for (int kt = 0; kt < nk; ++kt) {
    lds_char* cur = smem + (kt & 1) * STAGE;
    if (kt + 1 < nk) load_tiles(kt + 1);
#pragma unroll
    for (int st = 0; st < Op::STEPS; ++st) {
      i32x4 fa[WT], fb[WT];
#pragma unroll
      for (int i = 0; i < WT; ++i) fa[i] = RA::read(cur, wm * 64 + i * 16, st, lane);
#pragma unroll
      for (int h = 0; h < (TWO ? 2 : 1); ++h) {
#pragma unroll
        for (int j = 0; j < WT; ++j) fb[j] = RB::read(cur + GA::BYTES + h * GB::BYTES, wn * 64 + j * 16, st, lane);
#pragma unroll
        for (int i = 0; i < WT; ++i)
#pragma unroll
          for (int j = 0; j < WT; ++j) acc[i][j] = Op::mma(fb[j], fa[i], acc[i][j]);
      }
    }
    if (kt + 1 < nk) store_tiles(smem + ((kt & 1) ^ 1) * STAGE);
    __syncthreads();
  }
  using ACC = frag::Acc<frag::ACC_16x16>;
  const int acc_m = ACC::coord(lane, 0).j, acc_n = ACC::coord(lane, 0).i;
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    const int64_t m = m0 + wm * 64 + i * 16 + acc_m;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < WT; ++j) {
      const int64_t n = n0 + wn * 64 + j * 16 + acc_n;
      if (n >= p.N) continue;
      if (p.splits > 1) {
        float* w = (float*)p.ws + ((int64_t)blockIdx.y * p.M + m) * p.N + n;
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) w[e] = acc[i][j][e];
      } else {
        grad_store4(p, m, n, acc[i][j]);
      }
    }
  }
}

// Adds the K ranges' sums in order (K ascending) and applies the epilogue.
__global__ __launch_bounds__(256) void grad_finish_kernel(GradArgs p) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= p.N) return;
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    f32x4 acc = {0, 0, 0, 0};
    for (int s = 0; s < p.splits; ++s) {
      const float* w = (const float*)p.ws + ((int64_t)s * p.M + m) * p.N + n;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) acc[e] += w[e];
    }
    grad_store4(p, m, n, acc);
  }
}

// A panel: columns [n0, n0 + nc) of s[k] Q[k][j] in A's type, ldw apart, zeros past nc
// and past row K; with TWO a second panel of the rests at lo.  16 codes per thread.
template <class Op, bool TWO>
__global__ __launch_bounds__(256) void grad_widen_kernel(const char* Q, const float* sk, int64_t K, int64_t ldq, int64_t n0,
                                                         int64_t nc, char* hi, char* lo, int64_t ldw, uint32_t cpr,
                                                         uint32_t chunks) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const int64_t k = i / cpr, c = 16 * (int64_t)(i % cpr);
  const float s = k < K ? sk[k] : 0.0f;
  i32x4 h[2], l[2];
  widen16<Op, TWO>(load_chunk(Q, Q + k * ldq + n0 + c, k < K ? nc - c : 0), s, h, l);
  char* d = hi + (k * ldw + c) * 2;
  *(i32x4*)d = h[0];
  *(i32x4*)(d + 16) = h[1];
  if constexpr (TWO) {
    d = lo + (k * ldw + c) * 2;
    *(i32x4*)d = l[0];
    *(i32x4*)(d + 16) = l[1];
  }
}

namespace {
int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t round_up(int64_t x, int64_t y) { return cdiv(x, y) * y; }
constexpr int64_t PANEL_STEP = 256;  // columns of a panel come in whole tiles

// Bytes of the copy of A and of the panels, at the workspace's start.
int64_t copy_bytes(int la, const GradArgs& a) { return a.lda2 ? a.lda2 * 2 * (la == LAYOUT_K ? a.M : a.K) : 0; }
int64_t panel_bytes(const GradArgs& a) { return a.ka * a.ldw * 2; }

// The dense product of A (or its copy) with a panel of nc columns.
DenseArgs dense_args(int la, const GradArgs& a, int64_t nc) {
  DenseArgs d{};
  d.A = a.lda2 ? (const char*)a.ws : a.A;
  d.lda = a.lda2 ? a.lda2 : a.lda;
  d.ldb = a.ldw;
  d.M = a.M;
  d.N = nc;
  d.K = a.ka;
  d.ldc = a.ldd;
  d.alpha = 1.0f;
  d.beta = a.beta;
  d.use_c = a.use_c;
  d.out = a.out;
  d.vec_cd = a.vec_d;
  return d;
}

// Fills the panel fields for ws_bytes of workspace: the modelled time and the bytes
// used, or a negative time when the operands' offsets or the workspace rule it out.
double plan_panels(int dtA, int la, GradArgs& a, int num_cu, int64_t ws_bytes, int64_t* used) {
  const int64_t two = a.out == OUT_32 ? 2 : 1;
  const bool chunks = (uintptr_t)a.A % 16 == 0 && a.lda % 8 == 0 && (la == LAYOUT_MN || a.K % 8 == 0);
  a.ka = chunks || la == LAYOUT_MN ? a.K : round_up(a.K, 8);
  a.lda2 = chunks ? 0 : round_up(la == LAYOUT_K ? a.K : a.M, 8);
  const int64_t fixed = copy_bytes(la, a), lim = (int64_t)1 << 31;
  const int64_t lda = a.lda2 ? a.lda2 : a.lda;
  if ((la == LAYOUT_K ? 256 * lda : (a.ka + 256) * lda) * 2 >= lim || fixed / 16 >= lim || fixed >= ws_bytes) return -1.0;
  // the widest panel that fits, cut into equal ones
  const int64_t fit = (ws_bytes - fixed) / (a.ka * 2 * two);
  const int64_t most = std::min((lim - 1) / ((a.ka + 256) * 2), fit) / 16 * 16;  // (a panel's offsets below 2 GiB)
  if (most < round_up(a.N, 16) && most < PANEL_STEP) return -1.0;
  const int64_t count = most >= round_up(a.N, 16) ? 1 : cdiv(a.N, most / PANEL_STEP * PANEL_STEP);
  a.panel_n = count == 1 ? a.N : round_up(cdiv(a.N, count), PANEL_STEP);
  a.ldw = round_up(a.panel_n, 16);
  const int64_t panels = fixed + two * panel_bytes(a);
  DenseArgs d = dense_args(la, a, a.panel_n);
  const PipePlan pp = plan_pipe(dtA, d, num_cu, ws_bytes - panels);
  *used = panels + pp.ws;
  const double widen = pass_us((double)a.ka * a.ldw * (1 + 2 * two));
  return (fixed > 0 ? pass_us(2.0 * fixed) : 0.0) + cdiv(a.N, a.panel_n) * (widen + two * pp.us);
}
}  // namespace

// Two ways: the general kernel widens Q's tiles on their way to LDS, once for every
// 128 rows of A, and takes any operands; panels widen Q once into the workspace (a
// copy's time for 3 or 5 bytes an element) and multiply on the pipelined dense
// kernels, at about half the time per product.  The modelled times decide: PANEL_NOTE
int64_t plan_grad(int dtA, int la, GradArgs& a, int num_cu, int64_t ws_bytes) {
  const int64_t nk = cdiv(a.K, KT_BYTES / 2);
  a.tiles_m = (int)cdiv(a.M, 128);
  a.tiles_n = (int)cdiv(a.N, 128);
  const int64_t slot = a.M * a.N * 4;
  const int64_t most = slot > 0 ? ws_bytes / slot : 1;
  double general_us;
  const int64_t s = plan_ranges((int64_t)a.tiles_m * a.tiles_n, nk, a.M * a.N, num_cu, a.out == OUT_32 ? 1.5 : 0.9,
                                most < 64 ? most : 64, &general_us);
  a.kt_per_split = (int)(nk > 0 ? cdiv(nk, s) : 1);
  a.splits = (int)s;
  if (a.K > 0) {
    int64_t used = 0;
    const double us = plan_panels(dtA, la, a, num_cu, ws_bytes, &used);
    if (us > 0.0 && us < general_us) return used;
  }
  a.panel_n = 0;
  return s > 1 ? s * slot : 0;
}

template <class Op>
static hipError_t launch_widen(const GradArgs& a, int64_t n0, int64_t nc, char* hi, char* lo, hipStream_t s) {
  const int64_t cpr = a.ldw / 16, chunks = cpr * a.ka;
  const dim3 grid((unsigned)cdiv(chunks, 256));
  if (lo)
    hipLaunchKernelGGL((grad_widen_kernel<Op, true>), grid, dim3(256), 0, s, a.Q, a.sk, a.K, a.ldq, n0, nc, hi, lo, a.ldw,
                       (uint32_t)cpr, (uint32_t)chunks);
  else
    hipLaunchKernelGGL((grad_widen_kernel<Op, false>), grid, dim3(256), 0, s, a.Q, a.sk, a.K, a.ldq, n0, nc, hi, lo, a.ldw,
                       (uint32_t)cpr, (uint32_t)chunks);
  return hipGetLastError();
}

// Panels: binary32 results take the product with the rests first, then add the other.
static hipError_t launch_panels(int dtA, int la, const GradArgs& a, int num_cu, hipStream_t s) {
  const bool two = a.out == OUT_32;
  const int64_t eo = two ? 4 : 2, fixed = copy_bytes(la, a);
  char* hi = (char*)a.ws + fixed;
  char* lo = two ? hi + panel_bytes(a) : nullptr;
  char* slots = hi + (two ? 2 : 1) * panel_bytes(a);
  hipError_t e = hipSuccess;
  if (a.lda2)
    e = la == LAYOUT_K ? launch_align_rows(a.A, a.lda * 2, a.M, a.K * 2, a.ws, a.lda2 * 2, a.M, s)
                       : launch_align_rows(a.A, a.lda * 2, a.K, a.M * 2, a.ws, a.lda2 * 2, a.K, s);
  for (int64_t n0 = 0; n0 < a.N && e == hipSuccess; n0 += a.panel_n) {
    const int64_t nc = std::min(a.panel_n, a.N - n0);
    e = dtA == DT_BF16 ? launch_widen<OpBF16>(a, n0, nc, hi, lo, s) : launch_widen<OpF16>(a, n0, nc, hi, lo, s);
    for (int part = two ? 0 : 1; part < 2 && e == hipSuccess; ++part) {
      DenseArgs d = dense_args(la, a, nc);
      d.B = part == 0 ? lo : hi;
      d.D = (char*)a.D + n0 * eo;
      d.C = a.use_c ? (const char*)a.C + n0 * eo : nullptr;
      if (two && part == 1) {
        d.C = d.D;
        d.beta = 1.0f;
        d.use_c = 1;
      }
      d.ws = slots;
      const PipePlan pp = plan_pipe(dtA, d, num_cu, a.ws_bytes - (slots - (char*)a.ws));
      e = pp.tile == 64 ? launch_fast_half(dtA, la, d, s)
          : pp.ws > 0   ? launch_fast_sk(dtA, dtA, la, LAYOUT_MN, d, s, pp.tile)
                        : launch_fast(dtA, dtA, la, LAYOUT_MN, d, s, pp.tile);
    }
  }
  return e;
}

template <class Op>
static void launch_general(int la, const GradArgs& a, dim3 grid, hipStream_t s) {
  const bool two = a.out == OUT_32;
  if (la == LAYOUT_K) {
    if (two) hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_K, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_K, false>), grid, dim3(256), 0, s, a);
  } else {
    if (two) hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_MN, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_MN, false>), grid, dim3(256), 0, s, a);
  }
}

hipError_t launch_grad(int dtA, int layoutA, const GradArgs& a, int num_cu, hipStream_t s) {
  if (a.panel_n > 0) return launch_panels(dtA, layoutA, a, num_cu, s);
  const int64_t blocks = (int64_t)a.tiles_m * a.tiles_n;
  if (blocks > 0xffffff) return hipErrorInvalidValue;  // (a launch holds less than 2^32 threads)
  const dim3 grid((unsigned)blocks, (unsigned)a.splits);
  if (dtA == DT_BF16) launch_general<OpBF16>(layoutA, a, grid, s);
  else launch_general<OpF16>(layoutA, a, grid, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(grad_finish_kernel, dim3((unsigned)((a.N + 1023) / 1024), (unsigned)(a.M < 4096 ? a.M : 4096)),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mcg
