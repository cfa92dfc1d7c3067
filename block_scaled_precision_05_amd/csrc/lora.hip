// lora.hip -- low-rank adapters of many requests at once, beside a shared projection:
//
//   out[t] = bf16( base[t] + s_g * B_g (A_g x_t) ),   g = the adapter of token t,
//
// for tokens sorted by adapter (sort_tokens with an alignment that is a multiple of
// 16), so that 16 consecutive rows of the plan, a tile, belong to one adapter.  The
// rows of X, base and out stay where they are: a tile gathers its 16 tokens.
//
// Two launches.  shrink: U[row][r] = A_g x in fp32, the long sum over K split over the
// waves of a workgroup and, when there are few tiles, over S workgroups whose partial
// sums go to S slabs of U.  expand: out = base + s_g B_g U, the S slabs added in order.
// Both are bound by memory (an adapter of rank r does r multiply-adds per element of
// X and of out, far under the matrix cores' rate), so operands go straight from global
// memory to MFMA fragments (v_mfma_f32_16x16x32_bf16: 16 rows of A_g or B_g against 16
// tokens) and the tiles are shaped to touch X, base and out once: several token tiles
// of one adapter share each fragment of A_g or B_g.
//
// U keeps fp32 precision through the second product: it enters as two bf16 terms, U =
// hi + lo with lo = bf16(U - hi), two MFMAs, a relative error of at most 2^-16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"

namespace bsg_lora {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 16;      // rows of the plan per MFMA tile

struct LoraArgs {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* A;      // [G][r][K]
  int64_t lda, stride_a;
  const uint16_t* B;      // [G][N][r]
  int64_t ldb, stride_b;
  const float* scale;     // [G] or null
  const int32_t* row_of;  // [T]
  const int32_t* pair_of;
  const int32_t* row_group;
  const uint16_t* base;   // or null
  int64_t ld_base;
  uint16_t* out;
  int64_t ldo;
  float* U;               // [S][tiles*16][r]
  int32_t T, G, K, N, r, rows, tiles, S;
  int32_t units;          // 64-element units of K
  int32_t plain;          // K, r or G is 0: no token has anything to add
  int32_t row_blocks;     // workgroups (x) that hold tiles; the rest copy tokens
};

// The adapter of a tile (that of its first row), or -1 when the tile holds no token.
__device__ __forceinline__ int tile_group(const LoraArgs& a, int tile) {
  if (tile >= a.tiles) return -1;
  const int g = a.row_group[tile * kTile];
  return (uint32_t)g < (uint32_t)a.G ? g : -1;
}

// The token of a row, or -1.
__device__ __forceinline__ int row_token(const LoraArgs& a, int row) {
  const int p = row < a.rows ? a.pair_of[row] : -1;
  return (uint32_t)p < (uint32_t)a.T ? p : -1;
}

// shrink.  A workgroup takes NT tiles and slice blockIdx.y of K; its four waves take the
// slice's 64-element units in turn (neighbouring waves read neighbouring lines) and their
// sums meet in LDS.  RF fragments of 16 rank rows.
template <int RF, int NT>
__global__ __launch_bounds__(kThreads) void shrink_kernel(const LoraArgs a) {
  __shared__ f32x4_t sums[kWaves - 1][RF][NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int per = (a.units + a.S - 1) / a.S;
  const int u0 = blockIdx.y * per, u1 = min(a.units, u0 + per);

  // tiles of this workgroup, taken together as long as they share the adapter
  for (int i = 0; i < NT;) {
    const int tile0 = blockIdx.x * NT + i;
    const int g = __builtin_amdgcn_readfirstlane(tile_group(a, tile0));
    if (g < 0) {
      ++i;
      continue;
    }
    int nt = 1;
    while (i + nt < NT && __builtin_amdgcn_readfirstlane(tile_group(a, tile0 + nt)) == g) ++nt;

    // rows past r repeat the last row: their sums are not stored
    const uint16_t* ap[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f)
      ap[f] = a.A + (int64_t)g * a.stride_a + (int64_t)min(16 * f + l16, a.r - 1) * a.lda;
    // rows without a token (and tiles past nt) read the first row's token: theirs are
    // columns of their own in the product, and not used
    const int t0 = row_token(a, tile0 * kTile);
    const uint16_t* xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n < nt ? row_token(a, (tile0 + n) * kTile + l16) : t0;
      xp[n] = a.X + (int64_t)max(t < 0 ? t0 : t, 0) * a.ldx;
    }
    f32x4_t acc[RF][NT];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[f][n] = (f32x4_t){0, 0, 0, 0};

    constexpr int UN = (RF + NT) <= 4 ? 4 : ((RF + NT) <= 8 ? 2 : 1);   // units in flight
    for (int u = u0 + wave; u < u1; u += kWaves * UN) {
      bf16x8_t xa[UN][2][NT], aa[UN][2][RF];
#pragma unroll
      for (int v = 0; v < UN; ++v)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = (u + v * kWaves) * 64 + 32 * h + 8 * lq;
          const bool in = u + v * kWaves < u1 && k < a.K;   // K % 8 == 0
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            u32x4_t w = {0, 0, 0, 0};
            if (in) w = *(const u32x4_t*)(xp[n] + k);
            xa[v][h][n] = __builtin_bit_cast(bf16x8_t, w);
          }
#pragma unroll
          for (int f = 0; f < RF; ++f) {
            u32x4_t w = {0, 0, 0, 0};
            if (in) w = *(const u32x4_t*)(ap[f] + k);
            aa[v][h][f] = __builtin_bit_cast(bf16x8_t, w);
          }
        }
#pragma unroll
      for (int v = 0; v < UN; ++v)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aa[v][h][f], xa[v][h][n], acc[f][n], 0, 0, 0);
    }
    __syncthreads();   // (the previous tiles' sums have been read)
    if (wave > 0) {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int n = 0; n < NT; ++n) sums[wave - 1][f][n][lane] = acc[f][n];
    }
    __syncthreads();
    if (wave == 0) {
      // lane (lq, l16) holds rank rows 16f + 4 lq .. +3 of token l16
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4_t v = acc[f][n];
#pragma unroll
          for (int w = 0; w < kWaves - 1; ++w) v += sums[w][f][n][lane];
          const int row = (tile0 + n) * kTile + l16, rr = 16 * f + 4 * lq;
          if (n < nt && rr < a.r)   // r % 8 == 0
            *(f32x4_t*)(a.U + ((int64_t)blockIdx.y * a.tiles * kTile + row) * a.r + rr) = v;
        }
    }
    i += nt;
  }
}

// expand.  A workgroup takes NT tiles and 256 columns, a wave 64 of them: four fragments
// of 16 rows of B_g.  Fragment f's row 4q + i is column 16q + 4f + i, so that a lane ends
// up with 16 consecutive columns of one token (32 bytes) and four lanes with 128 bytes.
// RK: k-steps of 32 rank elements.
__device__ __forceinline__ bool vec_ok(const void* p, int64_t ld) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0;
}

template <int RK, int NT>
__global__ __launch_bounds__(kThreads) void expand_kernel(const LoraArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.y * 256 + wave * 64;
  const bool vec = vec_ok(a.out, a.ldo) && (!a.base || vec_ok(a.base, a.ld_base));

  if ((int)blockIdx.x >= a.row_blocks) {
    // 16 tokens a workgroup: those without an adapter take base as it is, or zeros
    for (int i = 0; i < 16; ++i) {
      const int t = ((int)blockIdx.x - a.row_blocks) * 16 + i;
      if (t >= a.T || (!a.plain && a.row_of[t] >= 0)) continue;
      const int n = blockIdx.y * 256 + threadIdx.x;
      if (n < a.N) a.out[(int64_t)t * a.ldo + n] = a.base ? a.base[(int64_t)t * a.ld_base + n] : 0;
    }
    return;
  }
  if (n0 >= a.N) return;
  int g_have = -1;
  bf16x8_t b[RK][4];
  float s = 1.0f;
  for (int i = 0; i < NT; ++i) {
    const int tile = blockIdx.x * NT + i;
    const int g = __builtin_amdgcn_readfirstlane(tile_group(a, tile));
    if (g < 0) continue;
    if (g != g_have) {
      g_have = g;
      s = a.scale ? a.scale[g] : 1.0f;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = n0 + 16 * (l16 >> 2) + 4 * f + (l16 & 3);
        const uint16_t* bp = a.B + (int64_t)g * a.stride_b + (int64_t)min(n, a.N - 1) * a.ldb;
#pragma unroll
        for (int k = 0; k < RK; ++k) {
          u32x4_t w = {0, 0, 0, 0};
          if (32 * k + 8 * lq < a.r) w = *(const u32x4_t*)(bp + 32 * k + 8 * lq);
          b[k][f] = __builtin_bit_cast(bf16x8_t, w);
        }
      }
    }
    const int row = tile * kTile + l16, t = row_token(a, row);
    const int n = n0 + 16 * lq;
    // base first: the longest wait
    u32x4_t bv[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const bool whole = vec && n + 16 <= a.N;
    const uint16_t* bp = a.base + (int64_t)max(t, 0) * a.ld_base + n;
    if (a.base && t >= 0 && whole) {
      bv[0] = *(const u32x4_t*)bp;
      bv[1] = *(const u32x4_t*)(bp + 8);
    }
    f32x4_t acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = (f32x4_t){0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      float u[8] = {};
      if (32 * k + 8 * lq < a.r && t >= 0) {
        for (int sl = 0; sl < a.S; ++sl) {
          const float* up = a.U + ((int64_t)sl * a.tiles * kTile + row) * a.r + 32 * k + 8 * lq;
          const f32x4_t v0 = *(const f32x4_t*)up, v1 = *(const f32x4_t*)(up + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u[e] += v0[e];
            u[4 + e] += v1[e];
          }
        }
      }
      bf16x8_t hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = s * u[e];
        hi[e] = (__bf16)v;
        lo[e] = (__bf16)(v - (float)hi[e]);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[k][f], lo, acc[f], 0, 0, 0);
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[k][f], hi, acc[f], 0, 0, 0);
      }
    }
    if (t < 0) continue;
    uint16_t* op = a.out + (int64_t)t * a.ldo + n;
    if (whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // columns 8h + 2e, +1 of the lane's 16: register (2e) % 4 of fragment 2h + e/2
          const float x0 = acc[2 * h + e / 2][2 * (e % 2)] + __uint_as_float(bv[h][e] << 16);
          const float x1 = acc[2 * h + e / 2][2 * (e % 2) + 1] + __uint_as_float(bv[h][e] & 0xFFFF0000u);
          o[e] = __builtin_bit_cast(uint32_t, (bf16x2_t){(__bf16)x0, (__bf16)x1});
        }
        *(u32x4_t*)(op + 8 * h) = o;
      }
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + 4 * f + e < a.N) {
            const float x = a.base ? __uint_as_float((uint32_t)bp[4 * f + e] << 16) : 0.0f;
            op[4 * f + e] = __builtin_bit_cast(uint16_t, (__bf16)(acc[f][e] + x));
          }
    }
  }
}

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles that share a fragment of the adapter: all four while there are tiles to fill
// the chip, one when there are few.
static int tiles_per_wg(int64_t tiles) { return tiles >= 1024 ? 4 : (tiles >= 512 ? 2 : 1); }

// Slices of K: enough workgroups to fill the chip, at least 512 elements a slice.
static int slices(int64_t tiles, int64_t K) {
  const int64_t wgs = ceil_div(tiles, tiles_per_wg(tiles));
  int64_t s = ceil_div(1024, wgs > 0 ? wgs : 1);
  const int64_t most = K / 512 > 0 ? K / 512 : 1;
  return (int)(s < most ? s : most);
}

template <int NT>
static void launch_shrink(int rf, const LoraArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)ceil_div(a.tiles, NT), (unsigned)a.S);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, st, a); };
  if (rf == 1) go(shrink_kernel<1, NT>);
  else if (rf == 2) go(shrink_kernel<2, NT>);
  else if (rf <= 4) go(shrink_kernel<4, NT>);
  else go(shrink_kernel<8, NT>);
}

template <int NT>
static void launch_expand(int rk, const LoraArgs& a, unsigned x, hipStream_t st) {
  const dim3 grid(x, (unsigned)ceil_div(a.N, 256));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, st, a); };
  if (rk == 1) go(expand_kernel<1, NT>);
  else if (rk == 2) go(expand_kernel<2, NT>);
  else go(expand_kernel<4, NT>);
}

}  // namespace bsg_lora

using namespace bsg_lora;

extern "C" {

int64_t lora_add_workspace(int64_t rows, int64_t K, int32_t r) {
  if (rows <= 0 || K <= 0 || r <= 0) return 0;
  const int64_t tiles = ceil_div(rows, kTile);
  return 4 * (int64_t)slices(tiles, K) * tiles * kTile * r;
}

int lora_add_bf16(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t stride_a, const void* B,
                  int64_t ldb, int64_t stride_b, const float* scale, const int32_t* row_of,
                  const int32_t* pair_of, const int32_t* row_group, int64_t rows, const void* base,
                  int64_t ld_base, void* out, int64_t ldo, int64_t T, int32_t G, int64_t N, int64_t K,
                  int32_t r, void* workspace, int64_t workspace_bytes, void* stream) {
  if (T < 0 || G < 0 || N < 0 || K < 0 || r < 0 || rows < 0) return BSG_ERR_INVALID_ARG;
  if (r > 128 || r % 8 || K % 8) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T > kMaxDim / 2 || rows > kMaxDim / 2 || N > (int64_t(1) << 23) || K > kMaxDim / 2 || G > 1024)
    return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || N == 0) return BSG_OK;
  if (!out || ldo < N || !row_of || (base && ld_base < N)) return BSG_ERR_INVALID_ARG;
  if (((uintptr_t)out | (uintptr_t)base) & 1) return BSG_ERR_MISALIGNED;
  // in place only onto the same elements
  if (base == out && ld_base != ldo) return BSG_ERR_INVALID_ARG;
  const bool adapt = rows > 0 && G > 0 && K > 0 && r > 0;
  if (((uintptr_t)row_of | (uintptr_t)pair_of | (uintptr_t)row_group | (uintptr_t)scale) & 3)
    return BSG_ERR_MISALIGNED;
  if (rows > 0 && (!pair_of || !row_group)) return BSG_ERR_INVALID_ARG;
  const int64_t big = int64_t(1) << 40;
  if (adapt) {
    if (!X || !A || !B || ldx < K || lda < K || ldb < r || stride_a < 0 || stride_b < 0)
      return BSG_ERR_INVALID_ARG;
    if (G > 1 && (stride_a < (r - 1) * lda + K || stride_b < (N - 1) * ldb + r)) return BSG_ERR_INVALID_ARG;
    if (ldx > big || lda > big / 128 || ldb > big / N || stride_a > big || stride_b > big)
      return BSG_ERR_UNSUPPORTED_SHAPE;
    if (((uintptr_t)X | (uintptr_t)A | (uintptr_t)B) & 15) return BSG_ERR_MISALIGNED;
    if (ldx % 8 || lda % 8 || ldb % 8 || stride_a % 8 || stride_b % 8) return BSG_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < lora_add_workspace(rows, K, r)) return BSG_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 15) return BSG_ERR_MISALIGNED;
  }
  if (ldo > big || ld_base > big) return BSG_ERR_UNSUPPORTED_SHAPE;
  LoraArgs a = {};
  a.X = (const uint16_t*)X;
  a.ldx = ldx;
  a.A = (const uint16_t*)A;
  a.lda = lda;
  a.stride_a = stride_a;
  a.B = (const uint16_t*)B;
  a.ldb = ldb;
  a.stride_b = stride_b;
  a.scale = scale;
  a.row_of = row_of;
  a.pair_of = pair_of;
  a.row_group = row_group;
  a.base = (const uint16_t*)base;
  a.ld_base = ld_base;
  a.out = (uint16_t*)out;
  a.ldo = ldo;
  a.U = (float*)workspace;
  a.T = (int32_t)T;
  a.G = G;
  a.K = (int32_t)K;
  a.N = (int32_t)N;
  a.r = r;
  a.rows = (int32_t)rows;
  a.tiles = adapt ? (int32_t)ceil_div(rows, kTile) : 0;
  a.plain = !adapt;
  a.S = slices(a.tiles, K);
  a.units = (int32_t)ceil_div(K, 64);
  const hipStream_t st = (hipStream_t)stream;
  const int nt = tiles_per_wg(a.tiles);
  a.row_blocks = (int32_t)ceil_div(a.tiles, nt);
  // tokens without an adapter: nothing to do in place
  const int64_t rest = base == out ? 0 : ceil_div(T, 16);
  (void)hipGetLastError();
  if (a.tiles > 0) {
    const int rf = (r + 15) / 16;
    if (nt == 4) launch_shrink<4>(rf, a, st);
    else if (nt == 2) launch_shrink<2>(rf, a, st);
    else launch_shrink<1>(rf, a, st);
  }
  const int64_t x = a.row_blocks + rest;
  if (x > 0) {
    const int rk = (r + 31) / 32;
    if (nt == 4) launch_expand<4>(rk, a, (unsigned)x, st);
    else if (nt == 2) launch_expand<2>(rk, a, (unsigned)x, st);
    else launch_expand<1>(rk, a, (unsigned)x, st);
  }
  return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP;
}

}  // extern "C"
