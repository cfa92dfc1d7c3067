// dense.hip -- dense products with work in their epilogues (bias, activation, residual; the
// gated block) and their gradients: entry points, the choice of kernel, and the kernels
// around the matrix products (see include/bsg.h).
//
// The products themselves are instances of gemm_kernel (gemm_kernel.h) with an epilogue
// that finishes the fp32 accumulators in the kernel, or, for calls with too few tiles to
// fill the GPU, write fp32 sums of parts of the contraction that join_kernel finishes.
//
// Gradients.  dz = dD f'(z) is formed once, in one pass over dD and Z (and W in the gated
// form), rounded to bf16 for the matrix cores and read by two products: dA = dz B and
// dB = dz^T A.  Their contractions run over the rows of B, and of dz and A: neither
// operand is transposed in memory; the kernel copies rows as they lie and transposes when
// it reads them from LDS.  The bias's gradient is summed from the unrounded dz in the same
// pass, in an order fixed by the sizes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "act_math.h"
#include "gemm_kernel.h"
#include "internal.h"

namespace bsg {

static const int64_t kMaxTiles = int64_t(1) << 24;
static const int64_t kMaxRow = (int64_t(1) << 31) / 256 - 1;   // bytes of a row (32-bit offsets)
static const int64_t kMaxRows = (int64_t(1) << 29) - 1;        // a contraction's bytes stay in 31 bits

// What a form costs, in microseconds, fitted to sweeps of every form over 128 to 4096 rows
// (BF16 7168 x 2048, 2048 x 7168, the gated block and both strided products; FP8 4096 x
// 7168, 7168 x 2048; FP4 4096 x 7168): time per stage of one tile, rising from few tiles on
// the GPU to a full round of them, and a fixed part for launch, first stage and epilogue.
// The parts' fp32 sums pass through memory twice at about 5.5 TB/s, and the join is a
// launch of its own.
//   BF16 examples over K = 7168: 1024 x 2048: 256-row tiles 113 us, 128-row tiles 79, with the
//   deep ring 49, deep in 2 parts 40; 2048 x 2048: 112, 82, 61; 4096 x 2048: 123, 123, 141.
// Over 218 random sizes (64 .. 4096 rows, 256 .. 6800 columns, contractions of 128 .. 7900)
// the pick takes 2% more than the fastest form on average and 15% at most in BF16, 4% and
// 26% in FP8, 10% and 45% in FP4, whose short contractions it prices too low in 256-row
// tiles.  The costs are those of scale arrays that take 8-byte loads: with others, 256-row
// FP4 tiles take up to 8 us more (517 x 432 over 288: 20 us where parts take 9.4).
struct TileCost {
  int form;
  int64_t bm, bn, lo_tiles, cap;   // tile, tiles up to which `lo` holds, tiles of a full round
  double lo, hi, fixed;
  int round;                       // stages of a round of the ring; 0: no parts
  double fixed_part;               // a part's epilogue only stores its sums
};
static const TileCost kForms[3][3] = {
    {{DENSE_BIG, 256, 256, 128, 256, 0.50, 0.60, 8.0, 0, 0},
     {DENSE_SMALL, 128, 128, 256, 512, 0.33, 0.55, 5.5, 0, 0},
     {DENSE_DEEP, 128, 128, 128, 256, 0.20, 0.26, 7.0, 8, 4.6}},
    {{DENSE_BIG, 256, 256, 128, 256, 0.55, 0.58, 9.0, 0, 0},
     {DENSE_SMALL, 128, 256, 128, 256, 0.38, 0.43, 10.5, 6, 6.0},
     {}},
    {{DENSE_BIG, 256, 256, 128, 256, 0.55, 0.60, 9.0, 0, 0},
     {DENSE_SMALL, 128, 128, 256, 512, 0.49, 0.59, 9.5, 4, 5.5},
     {}}};

static double tiles_cost(const TileCost& c, int64_t tiles, int64_t stages, double fixed) {
  const int64_t full = tiles / c.cap, rest = tiles % c.cap;
  double t = full * (stages * c.hi + fixed);
  if (rest) {
    const double x = rest <= c.lo_tiles ? 0.0 : (double)(rest - c.lo_tiles) / (c.cap - c.lo_tiles);
    t += stages * (c.lo + x * (c.hi - c.lo)) + fixed;
  }
  return t;
}

DensePlan dense_plan(int kind, int64_t M, int64_t N, int64_t K, bool strided) {
  const int64_t bytes = kind == KIND_BF16 ? 2 * K : (kind == KIND_FP8 ? K : K / 2);
  const int64_t stages = (bytes + 63) / 64;
  // Few rows: the stream of B through registers.  Up to 32 rows at any K; up to 64 where a
  // row is at most 8 KiB (64 rows, BF16 7168 x 2048: 12.0 us against 14.6 in parts; 2048 x
  // 7168: 21.0 against 15.1: every workgroup reads all of A).
  // (one workgroup of up to 1024 threads to 16 columns, 2^32 threads to a launch)
  if (!strided && (M <= 32 || (M <= 64 && bytes <= 8192)) && N < (int64_t)1 << 25) return {DENSE_FEW, 1};
  DensePlan best = {DENSE_BIG, 1};
  double t_best = 1e30;
  for (const TileCost& c : kForms[kind]) {
    if (!c.bm) continue;
    const int64_t tiles = (M + c.bm - 1) / c.bm * ((N + c.bn - 1) / c.bn);
    const double t1 = tiles_cost(c, tiles, stages, c.fixed);
    if (t1 < t_best) {
      t_best = t1;
      best = {c.form, 1};
    }
    // Parts of whole rounds of the ring, all of them on the GPU at once.  (One part: the
    // epilogue moves to the join, whose threads are many; FP8 and FP4 tiles of few, tall
    // waves gain by it at small K: FP8 472 x 728 x 896 16.0 us in one kernel, 14.8 apart.  At most 16
    // parts: the costs were fitted up to there.)
    for (int64_t s = kind == KIND_BF16 ? 2 : 1; c.round && s <= 16 && s * tiles <= c.cap && c.round * (s - 1) < stages; ++s) {
      const int64_t per = ((stages + s - 1) / s + c.round - 1) / c.round * c.round;
      if ((stages + per - 1) / per != s) continue;
      const double t = tiles_cost(c, s * tiles, per, c.fixed_part) + 3.0 + 0.2 * s + (8.0 * s + 2.0) * M * N / 5.5e6;
      if (t < t_best) {
        t_best = t;
        best = {DENSE_PART, (int)s};
      }
    }
  }
  return best;
}

// Joins the parts of a split contraction: one thread finishes four consecutive columns of
// a row, 16 bytes of each part, four parts' loads at a time.  Bound by the parts' bytes,
// which mostly come from L2 and the cache behind it, where the product has just written
// them.
static __device__ __forceinline__ void sum_parts(const float* q, int64_t stride, int splits, float (&v)[4]) {
  typedef __attribute__((ext_vector_type(4))) float f32x4_t;
  f32x4_t t = {0, 0, 0, 0};
  int s = 0;
  for (; s + 4 <= splits; s += 4, q += 4 * stride) {
    const f32x4_t a = *(const f32x4_t*)q, c = *(const f32x4_t*)(q + stride), d = *(const f32x4_t*)(q + 2 * stride),
                  e = *(const f32x4_t*)(q + 3 * stride);
    t += (a + c) + (d + e);
  }
  for (; s < splits; ++s, q += stride) t += *(const f32x4_t*)q;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = t[e];
}

template <bool GLU>
__global__ __launch_bounds__(256) void join_kernel(const GemmArgs args) {
  const int cols = GLU ? args.inter : args.N, per = (cols + 3) / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = idx / per;
  const int n = 4 * (int)(idx - m * per);
  if (m >= args.M) return;
  const float* const p = args.P + m * args.ldp + n;
  const int cnt = cols - n < 4 ? cols - n : 4;
  Bf16s<4>::t r = {0, 0};
  float b[4] = {};
  if constexpr (!GLU) {
    if (args.R) r = load_bf16s<4>(args.R + m * args.ldr + n, cnt);
    if (args.bias) unpack<4>(load_bf16s<4>(args.bias + n, cnt), b);
  }
  float z[4];
  sum_parts(p, args.part_stride, args.splits, z);
  uint16_t* const Z = args.Z ? args.Z + m * args.ldz + n : nullptr;
  uint16_t* const D = args.D + m * args.ldd + n;
  if constexpr (GLU) {
    float u[4];
    sum_parts(p + args.inter, args.part_stride, args.splits, u);
    glu_row<4>(args.act, z, u, Z, args.inter, D, args.e_vec);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] += b[e];
    act_row<4>(args.act, z, Z, r, args.R != nullptr, D, args.e_vec, cnt);
  }
}

static int launched() { return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP; }

int dense_join(const GemmArgs& a, bool glu, void* stream) {
  const int64_t per = ((glu ? a.inter : a.N) + 3) / 4, blocks = (a.M * per + 255) / 256;
  if (blocks == 0) return BSG_OK;
  (void)hipGetLastError();
  if (glu)
    hipLaunchKernelGGL(join_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
  else
    hipLaunchKernelGGL(join_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
  return launched();
}

// dz of a block of 256 columns x `rows` rows (a multiple of 8): thread (x, y) takes columns
// 8x .. 8x+7 of rows y, y + 8, ...  Bound by memory: dD and Z read, dz written, each once.
// The columns' sums of dz stay in registers over the rows, then meet in LDS, one partial
// row a block.
//   GLU: columns are those of H; dz gets dg there and du inter columns further on.
//   ldq: leading dimension of dz, a multiple of 8; columns N .. ldq-1 are zeroed (the
//   products read whole 16-byte chunks).  dz or part may be null.
template <bool GLU>
__global__ __launch_bounds__(256) void dz_kernel(const uint16_t* __restrict__ dD, int64_t lddd,
                                                 const uint16_t* __restrict__ Z, int64_t ldz, uint16_t* __restrict__ dz,
                                                 int64_t ldq, float* __restrict__ part, int64_t M, int64_t N, int act,
                                                 int rows) {
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t per = (N + 255) / 256, by = blockIdx.x / per, bx = blockIdx.x - by * per;
  const int64_t n = bx * 256 + 8 * x, m0 = by * rows;
  const int cnt = N - n >= 8 ? 8 : (N > n ? (int)(N - n) : 0);
  float sum[8] = {};
  if (cnt > 0) {
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    Bf16s<8>::t vd, vz = {}, vw = {};
    auto load = [&](int64_t m) {
      vd = load_bf16s<8>(dD + m * lddd + n, cnt);
      if (act != BSG_ACT_NONE || GLU) vz = load_bf16s<8>(Z + m * ldz + n, cnt);
      if constexpr (GLU) vw = load_bf16s<8>(Z + m * ldz + N + n, cnt);
    };
    if (m0 + y < m1) load(m0 + y);
    for (int64_t m = m0 + y; m < m1; m += 8) {
      float d[8], z[8], w[8];
      unpack<8>(vd, d);
      unpack<8>(vz, z);
      unpack<8>(vw, w);
      if (m + 8 < m1) load(m + 8);   // the next row's loads run under this row's arithmetic
      with_act(act, [&](auto a) {
        constexpr int A = decltype(a)::value;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f;
          if constexpr (GLU) {
            const float df = act_df<A>(z[e], f);
            if constexpr (A == BSG_ACT_RELU)
              z[e] = z[e] <= 0.0f ? 0.0f : d[e] * w[e];   // (a select, as below)
            else
              z[e] = d[e] * w[e] * df;
            w[e] = d[e] * f;
          } else if constexpr (A == BSG_ACT_NONE) {
            z[e] = d[e];
          } else if constexpr (A == BSG_ACT_RELU) {
            z[e] = z[e] <= 0.0f ? 0.0f : d[e];   // (a select: an infinite dD meets no 0 * inf)
          } else {
            z[e] = d[e] * act_df<A>(z[e], f);
          }
        }
      });
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= cnt) z[e] = 0.0f;
        sum[e] += z[e];
      }
      if (dz) *(Bf16s<8>::t*)(dz + m * ldq + n) = pack<8>(z);
      if constexpr (GLU) *(Bf16s<8>::t*)(dz + m * ldq + N + n) = pack<8>(w);
    }
  }
  if constexpr (!GLU) {
    if (!part) return;
    __shared__ float s[8][256];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[y][8 * x + e] = sum[e];
    __syncthreads();
    const int64_t c = bx * 256 + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += s[k][threadIdx.x];
    if (c < N) part[by * N + c] = t;
  }
}

// Rows of a dz block: 64, or fewer where that leaves less than four blocks a CU.
static int dz_rows(int64_t M, int64_t N) {
  int rows = 64;
  while (rows > 8 && (M + rows - 1) / rows * ((N + 255) / 256) < 1024) rows /= 2;
  return rows;
}

// What is left after a backward pass's products, in one launch: the parts of either
// product joined, and dbias summed from the blocks' partial rows.
struct Joined {
  const float* P;
  uint16_t* D;
  int64_t ldd, ldp, part_stride, M;
  int32_t N, splits, vec, blocks;   // blocks: workgroups of this product (0: it was not split)
};

static __device__ __forceinline__ void join_rows(const Joined& a, int block) {
  const int per = (a.N + 3) / 4;
  const int64_t idx = (int64_t)block * 256 + threadIdx.x, m = idx / per;
  const int n = 4 * (int)(idx - m * per);
  if (m >= a.M) return;
  float z[4];
  sum_parts(a.P + m * a.ldp + n, a.part_stride, a.splits, z);
  store_bf16s<4>(a.D + m * a.ldd + n, z, a.vec, a.N - n < 4 ? a.N - n : 4);
}

// A dbias block sums 32 columns, eight rows at a time.
__global__ __launch_bounds__(256) void tail_kernel(const Joined a, const Joined b, const float* __restrict__ part,
                                                   int64_t rows, int64_t N, float* __restrict__ dbias) {
  int block = blockIdx.x;
  if (block < a.blocks) return join_rows(a, block);
  block -= a.blocks;
  if (block < b.blocks) return join_rows(b, block);
  block -= b.blocks;
  __shared__ float s[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t n = (int64_t)block * 32 + x;
  float t = 0.0f;
  if (n < N)
#pragma unroll 4
    for (int64_t r = y; r < rows; r += 8) t += part[r * N + n];
  s[y][x] = t;
  __syncthreads();
  if (y == 0 && n < N) {
#pragma unroll
    for (int k = 1; k < 8; ++k) t += s[k][x];
    dbias[n] = t;
  }
}

static bool al16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

static bool bad_act(int32_t act) { return act < BSG_ACT_NONE || act > BSG_ACT_GELU_TANH; }

// A row-major bf16 operand without alignment of its own: null, leading dimension, 2 bytes.
static int check_rows(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return BSG_OK;
  if (!p || ld < cols) return BSG_ERR_INVALID_ARG;
  if ((uintptr_t)p & 1) return BSG_ERR_MISALIGNED;
  return ld > (int64_t)1 << 30 ? BSG_ERR_UNSUPPORTED_SHAPE : BSG_OK;
}

// An operand of a product: 16-byte aligned rows, 32-bit row offsets.
static int check_operand(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return BSG_OK;
  if (!p || ld < cols) return BSG_ERR_INVALID_ARG;
  if (2 * ld > kMaxRow) return BSG_ERR_UNSUPPORTED_SHAPE;
  return al16(p, ld) ? BSG_OK : BSG_ERR_MISALIGNED;
}

static int check_tiles(int64_t M, int64_t N) {
  return (M + 127) / 128 * ((N + 127) / 128) >= kMaxTiles ? BSG_ERR_UNSUPPORTED_SHAPE : BSG_OK;
}

static int check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return BSG_OK;
  if (!ws || bytes < need) return BSG_ERR_INVALID_ARG;
  return ((uintptr_t)ws & 15) ? BSG_ERR_MISALIGNED : BSG_OK;
}

// Epilogue operands of an act call; sets the fields of a.
static int act_args(GemmArgs& a, int kind, const void* bias, int32_t act, const void* R, int64_t ldr, void* D,
                    int64_t ldd, void* Z, int64_t ldz, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes,
                    DensePlan& plan) {
  if (bad_act(act)) return BSG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BSG_OK;
  if ((uintptr_t)bias & 1) return BSG_ERR_MISALIGNED;
  int st = R ? check_rows(R, ldr, M, N) : BSG_OK;
  if (R && R == D && M > 1 && ldr != ldd) return BSG_ERR_INVALID_ARG;   // in place: the same rows
  if (st == BSG_OK && Z) st = check_rows(Z, ldz, M, N);
  if (st == BSG_OK) st = check_tiles(M, N);
  if (st != BSG_OK) return st;
  plan = dense_plan(kind, M, N, K);
  st = check_workspace(ws, ws_bytes, dense_part_bytes(plan, M, N));
  if (st != BSG_OK) return st;
  a.D = (uint16_t*)D;
  a.ldd = ldd;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.act = act;
  a.bias = (const uint16_t*)bias;
  a.R = (const uint16_t*)R;
  a.Z = (uint16_t*)Z;
  a.ldr = R ? ldr : 0;
  a.ldz = Z ? ldz : 0;
  a.P = (float*)ws;
  a.ldp = dense_ldp(N);
  a.part_stride = M * a.ldp;
  a.splits = plan.splits;
  a.e_vec = al16(D, ldd) && (!Z || al16(Z, ldz));
  return BSG_OK;
}

}  // namespace bsg

using namespace bsg;

extern "C" {

int64_t gemm_bf16_act_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0) return 0;
  return dense_part_bytes(dense_plan(KIND_BF16, M, N, K), M, N);
}
int64_t gemm_fp8_act_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0) return 0;
  return dense_part_bytes(dense_plan(KIND_FP8, M, N, K), M, N);
}
int64_t gemm_fp4_act_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0) return 0;
  return dense_part_bytes(dense_plan(KIND_FP4, M, N, K), M, N);
}
int64_t gemm_bf16_glu_workspace(int64_t M, int64_t inter, int64_t K) {
  return gemm_bf16_act_workspace(M, 2 * inter, K);
}

int gemm_bf16_act(const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias, int32_t act,
                  const void* R, int64_t ldr, void* D, int64_t ldd, void* Z, int64_t ldz, int64_t M, int64_t N,
                  int64_t K, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_dense(A, lda, B, ldb, D, ldd, M, N, K, 8, 2 * K, 2);
  if (st != BSG_OK) return st;
  GemmArgs a = {};
  DensePlan plan = {};
  st = act_args(a, KIND_BF16, bias, act, R, ldr, D, ldd, Z, ldz, M, N, K, workspace, workspace_bytes, plan);
  if (st != BSG_OK || M == 0 || N == 0) return st;
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.lda = K ? lda * 2 : 0;
  a.ldb = K ? ldb * 2 : 0;
  a.k_bytes = (int32_t)(2 * K);
  st = plan.form == DENSE_FEW ? dense_few(KIND_BF16, a, false, stream) : dense_bf16(a, plan.form, EPI_ACT, stream);
  return st == BSG_OK && plan.form == DENSE_PART ? dense_join(a, false, stream) : st;
}

int gemm_fp8_act(const void* A, int64_t lda, const int16_t* sfa, int64_t ld_sfa, const void* B, int64_t ldb,
                 const int16_t* sfb, int64_t ld_sfb, int32_t sfb_gran_mn, const void* bias, int32_t act,
                 const void* R, int64_t ldr, void* D, int64_t ldd, int64_t M, int64_t N, int64_t K,
                 void* workspace, int64_t workspace_bytes, void* stream) {
  if (sfb_gran_mn != 128 && sfb_gran_mn != 1) return BSG_ERR_UNSUPPORTED_SHAPE;
  int st = check_dense(A, lda, B, ldb, D, ldd, M, N, K, 128, K, 1);
  if (st != BSG_OK) return st;
  const int64_t sfb_rows = (N + sfb_gran_mn - 1) / sfb_gran_mn;
  if (M > 0 && N > 0) st = check_scales(sfa, ld_sfa, M, sfb, ld_sfb, sfb_rows, K, 128);
  if (st != BSG_OK) return st;
  GemmArgs a = {};
  DensePlan plan = {};
  st = act_args(a, KIND_FP8, bias, act, R, ldr, D, ldd, nullptr, 0, M, N, K, workspace, workspace_bytes, plan);
  if (st != BSG_OK || M == 0 || N == 0) return st;
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.sfa = sfa;
  a.sfb = sfb;
  a.lda = K ? lda : 0;
  a.ldb = K ? ldb : 0;
  a.ld_sfa = K ? ld_sfa : 0;
  a.ld_sfb = K ? ld_sfb : 0;
  a.k_bytes = (int32_t)K;
  a.kp_count = (int32_t)((K / 128 + 1) / 2);
  a.sfb_rows = (int32_t)sfb_rows;
  st = plan.form == DENSE_FEW ? dense_few(KIND_FP8, a, false, stream)
                              : dense_fp8(a, plan.form, (K && sv_ok(sfa, ld_sfa) ? 1 : 0) + (sfb_gran_mn == 1 ? 2 : 0), stream);
  return st == BSG_OK && plan.form == DENSE_PART ? dense_join(a, false, stream) : st;
}

int gemm_fp4_act(const void* A, int64_t lda, const int16_t* sfa, int64_t ld_sfa, const void* B, int64_t ldb,
                 const int16_t* sfb, int64_t ld_sfb, const void* bias, int32_t act, const void* R, int64_t ldr,
                 void* D, int64_t ldd, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                 void* stream) {
  int st = check_dense(A, lda, B, ldb, D, ldd, M, N, K, 32, K / 2, 1);
  if (st != BSG_OK) return st;
  if (M > 0 && N > 0) st = check_scales(sfa, ld_sfa, M, sfb, ld_sfb, N, K, 32);
  if (st != BSG_OK) return st;
  GemmArgs a = {};
  DensePlan plan = {};
  st = act_args(a, KIND_FP4, bias, act, R, ldr, D, ldd, nullptr, 0, M, N, K, workspace, workspace_bytes, plan);
  if (st != BSG_OK || M == 0 || N == 0) return st;
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.sfa = sfa;
  a.sfb = sfb;
  a.lda = K ? lda : 0;
  a.ldb = K ? ldb : 0;
  a.ld_sfa = K ? ld_sfa : 0;
  a.ld_sfb = K ? ld_sfb : 0;
  a.k_bytes = (int32_t)(K / 2);
  a.kp_count = (int32_t)((K / 32 + 1) / 2);
  a.sfb_rows = (int32_t)N;
  st = plan.form == DENSE_FEW ? dense_few(KIND_FP4, a, false, stream)
                              : dense_fp4(a, plan.form, K && sv_ok(sfa, ld_sfa) && sv_ok(sfb, ld_sfb) ? 1 : 0, stream);
  return st == BSG_OK && plan.form == DENSE_PART ? dense_join(a, false, stream) : st;
}

int gemm_bf16_glu(const void* X, int64_t ldx, const void* W13, int64_t ldw, int32_t act, void* H, int64_t ldh,
                  void* Z, int64_t ldz, int64_t M, int64_t inter, int64_t K, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  if (inter < 0 || inter > kMaxRows) return inter < 0 ? BSG_ERR_INVALID_ARG : BSG_ERR_UNSUPPORTED_SHAPE;
  if (inter % 8) return BSG_ERR_UNSUPPORTED_SHAPE;
  // (ldh holds inter columns: checked below)
  int st = check_dense(X, ldx, W13, ldw, H, ldh < inter ? ldh : 2 * inter, M, 2 * inter, K, 8, 2 * K, 2);
  if (st != BSG_OK) return st;
  if (bad_act(act)) return BSG_ERR_INVALID_ARG;
  if (M == 0 || inter == 0) return BSG_OK;
  st = check_rows(H, ldh, M, inter);
  if (st == BSG_OK && Z) st = check_rows(Z, ldz, M, 2 * inter);
  if (st == BSG_OK) st = check_tiles(M, 2 * inter);
  if (st != BSG_OK) return st;
  const DensePlan plan = dense_plan(KIND_BF16, M, 2 * inter, K);
  st = check_workspace(workspace, workspace_bytes, dense_part_bytes(plan, M, 2 * inter));
  if (st != BSG_OK) return st;
  GemmArgs a = {};
  a.A = (const uint8_t*)X;
  a.B = (const uint8_t*)W13;
  a.D = (uint16_t*)H;
  a.Z = (uint16_t*)Z;
  a.lda = K ? ldx * 2 : 0;
  a.ldb = K ? ldw * 2 : 0;
  a.ldd = ldh;
  a.ldz = Z ? ldz : 0;
  a.M = (int32_t)M;
  a.N = (int32_t)(2 * inter);
  a.K = (int32_t)K;
  a.k_bytes = (int32_t)(2 * K);
  a.inter = (int32_t)inter;
  a.act = act;
  a.P = (float*)workspace;
  a.ldp = dense_ldp(2 * inter);
  a.part_stride = M * a.ldp;
  a.splits = plan.splits;
  a.e_vec = al16(H, ldh) && (!Z || al16(Z, ldz));
  st = plan.form == DENSE_FEW ? dense_few(KIND_BF16, a, true, stream) : dense_bf16(a, plan.form, EPI_GLU, stream);
  return st == BSG_OK && plan.form == DENSE_PART ? dense_join(a, true, stream) : st;
}

}  // extern "C"

namespace bsg {

// D [M][N] = (A's rows or columns) x (B's columns), K long: tr 2 contracts B's rows with
// A's columns, tr 3 the rows of both; operands bf16 with leading dimensions in elements.  A
// split product leaves its parts in ws and says in `left` how to join them.
static int strided(int tr, const void* A, int64_t lda, const void* B, int64_t ldb, void* D, int64_t ldd, int64_t M,
                   int64_t N, int64_t K, void* ws, Joined& left, void* stream) {
  if (M == 0 || N == 0) return BSG_OK;
  const DensePlan plan = dense_plan(KIND_BF16, M, N, K, true);
  GemmArgs a = {};
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.D = (uint16_t*)D;
  a.lda = K ? lda * 2 : 0;
  a.ldb = K ? ldb * 2 : 0;
  a.ldd = ldd;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  // (a row of A holds whole 16-byte chunks: its columns past K are zeros, and rows of B
  // past K read zero)
  a.k_bytes = (int32_t)(2 * ((K + 7) / 8 * 8));
  a.P = (float*)ws;
  a.ldp = dense_ldp(N);
  a.part_stride = M * a.ldp;
  a.splits = plan.splits;
  if (plan.form == DENSE_PART)
    left = {a.P, a.D, ldd, a.ldp, a.part_stride, M, a.N, plan.splits, al16(D, ldd),
            (int32_t)((M * ((N + 3) / 4) + 255) / 256)};
  return dense_strided(a, plan.form, tr, stream);
}

static int64_t strided_bytes(int64_t M, int64_t N, int64_t K) {
  return M > 0 && N > 0 ? dense_part_bytes(dense_plan(KIND_BF16, M, N, K, true), M, N) : 0;
}

static int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

// Workspace of a backward pass: dz [M][ldq], the bias's partial rows, the parts of dA and of
// dB where they are split.
struct GradSpace {
  int64_t ldq, rows, blocks, part_at, da_at, db_at, bytes;
  GradSpace(int64_t M, int64_t cols, int64_t K, bool bias) {
    ldq = (cols + 7) / 8 * 8;
    part_at = 2 * M * ldq;
    rows = dz_rows(M, bias ? cols : cols / 2);
    blocks = (M + rows - 1) / rows;
    da_at = part_at + (bias ? up16(4 * blocks * cols) : 0);
    db_at = da_at + strided_bytes(M, K, cols);
    bytes = db_at + strided_bytes(cols, K, M);
  }
};

// Both products of a backward pass from dz [M][ldq], and the launch that finishes them and
// dbias (part: its partial rows).
static int grad_products(const void* dz, int64_t ldq, const void* A, int64_t lda, const void* B, int64_t ldb,
                         void* dA, int64_t ldda, void* dB, int64_t lddb, float* dbias, int64_t M, int64_t N, int64_t K,
                         uint8_t* ws, const GradSpace& w, void* stream) {
  Joined a = {}, b = {};
  int st = dA ? strided(2, dz, ldq, B, ldb, dA, ldda, M, K, N, ws + w.da_at, a, stream) : BSG_OK;
  if (st == BSG_OK && dB) st = strided(3, dz, ldq, A, lda, dB, lddb, N, K, M, ws + w.db_at, b, stream);
  const int64_t blocks = a.blocks + b.blocks + (dbias ? (N + 31) / 32 : 0);
  if (st != BSG_OK || blocks == 0) return st;
  (void)hipGetLastError();
  hipLaunchKernelGGL(tail_kernel, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a, b,
                     (const float*)(ws + w.part_at), w.blocks, N, dbias);
  return launched();
}

static int check_grad(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return BSG_ERR_INVALID_ARG;
  if (K % 8 || M > kMaxRows || 2 * (N + 7) > kMaxRow || 2 * K > kMaxRow) return BSG_ERR_UNSUPPORTED_SHAPE;
  if ((M + 63) / 64 * ((N + 255) / 256) >= kMaxTiles) return BSG_ERR_UNSUPPORTED_SHAPE;
  int st = check_tiles(M, N);
  if (st == BSG_OK) st = check_tiles(M, K);
  return st == BSG_OK ? check_tiles(N, K) : st;
}

}  // namespace bsg

extern "C" {

int64_t gemm_bf16_act_backward_workspace(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return 0;
  return GradSpace(M, N, K, true).bytes;
}
int64_t gemm_bf16_glu_backward_workspace(int64_t M, int64_t inter, int64_t K) {
  if (M < 0 || inter < 0 || K < 0) return 0;
  return GradSpace(M, 2 * inter, K, false).bytes;
}

int gemm_bf16_act_backward(const void* dD, int64_t lddd, const void* Z, int64_t ldz, const void* A, int64_t lda,
                           const void* B, int64_t ldb, int32_t act, void* dA, int64_t ldda, void* dB, int64_t lddb,
                           float* dbias, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  if (bad_act(act)) return BSG_ERR_INVALID_ARG;
  int st = check_grad(M, N, K);
  if (st == BSG_OK) st = check_rows(dD, lddd, M, N);
  if (st == BSG_OK && act != BSG_ACT_NONE) st = check_rows(Z, ldz, M, N);
  if (st == BSG_OK && dA) st = check_rows(dA, ldda, M, K);
  if (st == BSG_OK && dB) st = check_rows(dB, lddb, N, K);
  if (st == BSG_OK && dA && M > 0) st = check_operand(B, ldb, N, K);
  if (st == BSG_OK && dB && N > 0) st = check_operand(A, lda, M, K);
  if (st == BSG_OK && ((uintptr_t)dbias & 3)) st = BSG_ERR_MISALIGNED;
  if (st != BSG_OK) return st;
  const GradSpace w(M, N, K, true);
  st = check_workspace(workspace, workspace_bytes, w.bytes);
  if (st != BSG_OK) return st;
  uint8_t* const ws = (uint8_t*)workspace;
  // without an activation an aligned dD is dz itself
  const bool own = act == BSG_ACT_NONE && al16(dD, lddd) && N % 8 == 0 && 2 * lddd <= kMaxRow;
  const void* const dz = own ? dD : ws;
  const int64_t ldq = own ? lddd : w.ldq;
  float* const part = (float*)(ws + w.part_at);
  const bool products = dA || dB;
  (void)hipGetLastError();
  if (M > 0 && N > 0 && (dbias || (products && !own))) {
    hipLaunchKernelGGL(dz_kernel<false>, dim3((unsigned)((N + 255) / 256 * w.blocks)), dim3(256), 0,
                       (hipStream_t)stream, (const uint16_t*)dD, lddd, (const uint16_t*)Z, ldz,
                       products && !own ? (uint16_t*)ws : nullptr, w.ldq, dbias ? part : nullptr, M, N, act, (int)w.rows);
    st = launched();
    if (st != BSG_OK) return st;
  }
  return grad_products(dz, ldq, A, lda, B, ldb, K ? dA : nullptr, ldda, K ? dB : nullptr, lddb, dbias, M, N, K, ws, w,
                       stream);
}

int gemm_bf16_glu_backward(const void* dH, int64_t lddh, const void* Z, int64_t ldz, const void* X, int64_t ldx,
                           const void* W13, int64_t ldw, int32_t act, void* dX, int64_t lddx, void* dW13,
                           int64_t lddw, int64_t M, int64_t inter, int64_t K, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  if (bad_act(act)) return BSG_ERR_INVALID_ARG;
  if (inter < 0) return BSG_ERR_INVALID_ARG;
  if (inter % 8 || inter > kMaxRows) return BSG_ERR_UNSUPPORTED_SHAPE;
  const int64_t N = 2 * inter;
  int st = check_grad(M, N, K);
  if (st == BSG_OK) st = check_rows(dH, lddh, M, inter);
  if (st == BSG_OK) st = check_rows(Z, ldz, M, N);
  if (st == BSG_OK && dX) st = check_rows(dX, lddx, M, K);
  if (st == BSG_OK && dW13) st = check_rows(dW13, lddw, N, K);
  if (st == BSG_OK && dX && M > 0) st = check_operand(W13, ldw, N, K);
  if (st == BSG_OK && dW13 && N > 0) st = check_operand(X, ldx, M, K);
  if (st != BSG_OK) return st;
  const GradSpace w(M, N, K, false);
  st = check_workspace(workspace, workspace_bytes, w.bytes);
  if (st != BSG_OK || K == 0 || (!dX && !dW13)) return st;
  uint8_t* const ws = (uint8_t*)workspace;
  if (M > 0 && inter > 0) {
    (void)hipGetLastError();
    hipLaunchKernelGGL(dz_kernel<true>, dim3((unsigned)((inter + 255) / 256 * w.blocks)),
                       dim3(256), 0, (hipStream_t)stream, (const uint16_t*)dH, lddh, (const uint16_t*)Z, ldz,
                       (uint16_t*)ws, w.ldq, nullptr, M, inter, act, (int)w.rows);
    st = launched();
    if (st != BSG_OK) return st;
  }
  return grad_products(ws, w.ldq, X, ldx, W13, ldw, dX, lddx, dW13, lddw, nullptr, M, N, K, ws, w, stream);
}

}  // extern "C"
