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
// General kernel: tiles of 128, 64 or 32 rows x 128 columns, 4 wavefronts, any size,
// pointer and leading dimension.  Q's tile is widened on its way from the registers to LDS, where it is
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

template <class Op, int LA, bool TWO, int BM>
__global__ __launch_bounds__(256, TWO && BM == 128 ? 1 : 2) void grad_general_kernel(GradArgs p) {
  constexpr int BN = 128, NT = 256, KE = KT_BYTES / 2;
  using WG = WaveGrid<BM>;
  constexpr int WTM = WG::WTM, WTN = WG::WTN;
  using GA = TileGeom<2, LA, BM>;
  using GB = TileGeom<2, LAYOUT_MN, BN>;
  using RA = FragReader<2, 16, LA, BM>;
  using RB = FragReader<2, 16, LAYOUT_MN, BN>;
  constexpr int STAGE = GA::BYTES + (TWO ? 2 : 1) * GB::BYTES;
  __shared__ __attribute__((aligned(16))) char smem_raw[2 * STAGE];
  lds_char* smem = (lds_char*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rm = WG::row(wave), rn = WG::col(wave);
  int tm, tn;
  general_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nk_all = (int)((p.K + KE - 1) / KE);
  const int kt0 = (int)blockIdx.y * p.kt_per_split;
  const int nk = min(nk_all - kt0, p.kt_per_split);

  // SETS K tiles ahead in registers, two stages in LDS (see gemm_i8_scaled.hip).
  using LdA = AnyLoader<2, LA, BM, NT>;
  using LdQ = AnyLoader<1, LAYOUT_MN, BN, NT, KE>;
  constexpr int QPT = LdQ::PER_THREAD;
  LdA la;
  LdQ lq;
  la.init(p.A, p.lda, m0, p.M, p.K, tid);
  lq.init(p.Q, p.ldq, n0, p.N, p.K, tid);
  constexpr int SETS = 2;
  typename LdA::Regs ra[SETS];
  typename LdQ::Regs q[SETS];
  float sk[SETS][QPT];
  auto load_tile = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value;
    la.load(ra[set], kt0 + kt, kt < nk);
    lq.load(q[set], kt0 + kt, kt < nk);
    const global_f32* src = (const global_f32*)(kt < nk ? p.sk + (int64_t)(kt0 + kt) * KE : (const float*)load_nothing);
    const int top = kt < nk ? lq.rows(kt0 + kt) - 1 : 0;  // (rows past K: their codes are zero)
#pragma unroll
    for (int t = 0; t < QPT; ++t) sk[set][t] = src[min(lq.r0 + t * LdQ::RPI, top)];
  };
  auto store_tile = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value;
    lds_char* st = smem + (set & 1) * STAGE;
    la.settle(ra[set], kt0 + kt);
    lq.settle(q[set], kt0 + kt);
    la.store(ra[set], st);
    lds_char* tb = st + GA::BYTES;
#pragma unroll
    for (int t = 0; t < QPT; ++t) {
      const int r = lq.r0 + t * LdQ::RPI, cc = lq.c16 / 8;  // a chunk of codes widens to two
      const int sw = swz<2, LAYOUT_MN, GB::CPR>(r);
      i32x4 hi[2], lo[2];
      widen16<Op, TWO>(q[set][t], sk[set][t], hi, lo);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds_write_b128(tb, r * GB::W + (((cc + h) ^ sw) * 16), hi[h]);
        if constexpr (TWO) lds_write_b128(tb + GB::BYTES, r * GB::W + (((cc + h) ^ sw) * 16), lo[h]);
      }
    }
  };
  f32x4 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto step = [&](auto set_c, int kt) {
    constexpr int set = decltype(set_c)::value;
    lds_char* cur = smem + (set & 1) * STAGE;
    store_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1);
    load_tile(std::integral_constant<int, (set + 1) % SETS>{}, kt + 1 + SETS);
#pragma unroll
    for (int st = 0; st < Op::STEPS; ++st) {
      i32x4 fa[WTM], fb[WTN];
#pragma unroll
      for (int i = 0; i < WTM; ++i) fa[i] = RA::read(cur, rm + i * 16, st, lane);
#pragma unroll
      for (int h = 0; h < (TWO ? 2 : 1); ++h) {
#pragma unroll
        for (int j = 0; j < WTN; ++j) fb[j] = RB::read(cur + GA::BYTES + h * GB::BYTES, rn + j * 16, st, lane);
#pragma unroll
        for (int i = 0; i < WTM; ++i)
#pragma unroll
          for (int j = 0; j < WTN; ++j) acc[i][j] = Op::mma(fb[j], fa[i], acc[i][j]);
      }
    }
    barrier_tiles();
  };
  for_each_set<SETS>([&](auto set) { load_tile(set, set); });
  store_tile(std::integral_constant<int, 0>{}, 0);
  load_tile(std::integral_constant<int, 0>{}, SETS);
  barrier_tiles();
  for (int kt = 0; kt < nk; kt += SETS) for_each_set<SETS>([&](auto set) { step(set, kt + set); });
  static_assert(BM * 512 <= 2 * STAGE, "epilogue stage");
  store_tile_rows<WG, BM>(smem, acc, tid, [&](int r, int c, const f32x4& v) {
    const int64_t m = m0 + r, n = n0 + c;
    if (m >= p.M || n >= p.N) return;
    if (p.splits == 1) {
      grad_store4(p, m, n, v);
      return;
    }
    float* w = (float*)p.ws + ((int64_t)blockIdx.y * p.M + m) * p.N + n;
    if (p.N % 4 == 0) *(f32x4*)w = v;
    else
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) w[e] = v[e];
  });
}

// Operands of fewer than 16 bytes, which the general kernel's loads do not take, and
// empty sums: one output per thread, the values rounded as elsewhere.
template <class Op, int LA, bool TWO>
__global__ __launch_bounds__(256) void grad_tiny_kernel(GradArgs p) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= p.N) return;
  auto value = [](const i32x4 (&v)[2]) {
    const uint32_t b = (uint32_t)v[0][0] & 0xffffu;
    return std::is_same<Op, OpBF16>::value ? bit_cast<float>(b << 16) : f16_bits_to_f32(b);
  };
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    float acc = 0.0f;
    for (int64_t k = 0; k < p.K; ++k) {
      i32x4 hi[2], lo[2];
      widen16<Op, TWO>(i32x4{(int)(uint8_t)p.Q[k * p.ldq + n], 0, 0, 0}, p.sk[k], hi, lo);
      const i32x4 bits[2] = {i32x4{(int)((const uint16_t*)p.A)[LA == LAYOUT_K ? m * p.lda + k : k * p.lda + m], 0, 0, 0}, {}};
      acc = __builtin_fmaf(value(bits), value(hi), acc);
      if constexpr (TWO) acc = __builtin_fmaf(value(bits), value(lo), acc);
    }
    combine_store(p.C, p.D, m * p.ldd + n, acc, 1.0f, p.beta, p.use_c, p.out);
  }
}

// Adds the K ranges' sums in order (K ascending) and applies the epilogue.
__global__ __launch_bounds__(256) void grad_finish_kernel(GradArgs p) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= p.N) return;
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    const f32x4 acc = sum_ranges4<f32x4>((const float*)p.ws + m * p.N + n, p.M * p.N, p.splits, n, p.N);
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
  widen16<Op, TWO>(load_chunk(Q, Q + k * ldq + n0 + c, k < K ? (int)min(nc - c, (int64_t)16) : 0), s, h, l);
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
// K tiles of 64 values of the general kernel (fitted from 1 to 300 rows, 1000 to 8192
// columns and K 512 to 8192, K in 1 to 16 ranges)
TileCost general_cost(int rows, bool two) {
  if (two)
    return rows == 32   ? TileCost{1.0, 0.65, 2, 3.0}
           : rows == 64 ? TileCost{1.2, 0.8, 2, 4.0}
                        : TileCost{1.6, 1.6, 1, 8.0};
  return rows == 32   ? TileCost{0.75, 0.5, 4, 3.0}
         : rows == 64 ? TileCost{0.85, 0.6, 3, 4.0}
                      : TileCost{1.1, 0.78, 2, 8.0};
}
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
  a.pipe_tile = pp.tile;
  a.sk_tiles = d.sk_tiles;
  // the last panel is narrower, and may take a stream-K split where the others do not
  DenseArgs last = dense_args(la, a, a.N - (cdiv(a.N, a.panel_n) - 1) * a.panel_n);
  *used = panels + std::max(pp.ws, plan_pipe(dtA, last, num_cu, ws_bytes - panels).ws);
  const double widen = pass_us((double)a.ka * a.ldw * (1 + 2 * two));
  return (fixed > 0 ? pass_us(2.0 * fixed) : 0.0) + cdiv(a.N, a.panel_n) * (widen + two * pp.us);
}
}  // namespace

// Two ways: the general kernel widens Q's tiles on their way to LDS, once for every
// 128 rows of A, and takes any operands; panels widen Q once into the workspace (3 or
// 5 bytes an element: 8192 x 4096 bf16 in 23 us, 4.3 TB/s; 4000 x 2048 f16 in 11, half
// that rate) and multiply on the pipelined dense kernels, at about half the time per
// product.  The modelled times decide (bf16, in place against panels: 64 x 4096 x 4096
// 21.2 and 33.5 us, 100 x 4096 x 4096 28.1 and 31.4; 512^3 20.2 and 10.7, 4096^3 203 and
// 125, 8192^3 1480 and 873).
int64_t plan_grad(int dtA, int la, GradArgs& a, int num_cu, int64_t ws_bytes) {
  const int64_t nk = cdiv(a.K, KT_BYTES / 2);
  a.tile = general_rows(a.M);
  a.tiles_m = (int)cdiv(a.M, a.tile);
  a.tiles_n = (int)cdiv(a.N, 128);
  const int64_t slot = a.M * a.N * 4;
  const int64_t most = slot > 0 ? ws_bytes / slot : 1;
  double general_us;
  const int64_t s = plan_ranges((int64_t)a.tiles_m * a.tiles_n, nk, a.M * a.N, num_cu,
                                general_cost(a.tile, a.out == OUT_32), most < 64 ? most : 64, &general_us);
  a.kt_per_split = (int)(nk > 0 ? cdiv(nk, s) : 1);
  a.splits = (int)s;
  a.tiny = !any_operand_ok(2, la == LAYOUT_K ? a.M : a.K, la == LAYOUT_K ? a.K : a.M, a.lda) || !any_operand_ok(1, a.K, a.N, a.ldq);
  if (a.tiny) {
    a.panel_n = 0;
    a.splits = 1;
    return 0;
  }
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
    e = la == LAYOUT_K ? launch_align_rows({a.A, a.lda * 2, a.M, a.K * 2, (char*)a.ws, a.lda2 * 2, a.M}, s)
                       : launch_align_rows({a.A, a.lda * 2, a.K, a.M * 2, (char*)a.ws, a.lda2 * 2, a.K}, s);
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
static void launch_tiny(int la, const GradArgs& a, hipStream_t s) {
  const bool two = a.out == OUT_32;
  const dim3 grid((unsigned)cdiv(a.N, 256), (unsigned)std::min<int64_t>(a.M, 65535));
  if (la == LAYOUT_K) {
    if (two) hipLaunchKernelGGL((grad_tiny_kernel<Op, LAYOUT_K, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_tiny_kernel<Op, LAYOUT_K, false>), grid, dim3(256), 0, s, a);
  } else {
    if (two) hipLaunchKernelGGL((grad_tiny_kernel<Op, LAYOUT_MN, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_tiny_kernel<Op, LAYOUT_MN, false>), grid, dim3(256), 0, s, a);
  }
}
template <class Op, int BM>
static void launch_rows(int la, const GradArgs& a, dim3 grid, hipStream_t s) {
  const bool two = a.out == OUT_32;
  if (la == LAYOUT_K) {
    if (two) hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_K, true, BM>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_K, false, BM>), grid, dim3(256), 0, s, a);
  } else {
    if (two) hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_MN, true, BM>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grad_general_kernel<Op, LAYOUT_MN, false, BM>), grid, dim3(256), 0, s, a);
  }
}
template <class Op>
static void launch_general(int la, const GradArgs& a, dim3 grid, hipStream_t s) {
  if (a.tile == 32) launch_rows<Op, 32>(la, a, grid, s);
  else if (a.tile == 64) launch_rows<Op, 64>(la, a, grid, s);
  else launch_rows<Op, 128>(la, a, grid, s);
}

hipError_t launch_grad(int dtA, int layoutA, const GradArgs& a, int num_cu, hipStream_t s) {
  if (a.panel_n > 0) return launch_panels(dtA, layoutA, a, num_cu, s);
  if (a.tiny) {
    if (dtA == DT_BF16) launch_tiny<OpBF16>(layoutA, a, s);
    else launch_tiny<OpF16>(layoutA, a, s);
    return hipGetLastError();
  }
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
