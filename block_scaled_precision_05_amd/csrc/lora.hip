// lora.hip -- low-rank adapters of many requests at once, beside a shared projection:
//
//   out[t] = bf16( base[t] + s_g * B_g (A_g x_t) ),   g = the adapter of token t,
//
// for tokens sorted by adapter (sort_tokens with an alignment that is a multiple of
// 16), so that 16 consecutive rows of the plan, a tile, belong to one adapter.  The
// rows of X, base and out stay where they are: a tile gathers its 16 tokens.
//
// An adapter of rank r does r multiply-adds per element of X and of out, far under the
// matrix cores' rate (v_mfma_f32_16x16x32_bf16, 16 rows of A_g or B_g against 16 tokens):
// the work is bound by memory, and for few tokens by latency.  X, base and out should
// move once, at the rate of HBM, and the adapters come from L2.
//   Little work: whole_kernel.  1 token, rank 16, 1024 to 1024 wide: 4.1 us.
//   Few tokens: shrink_kernel (U in S slices of K), expand_kernel; operands go straight
//     from global memory to MFMA fragments.  64 tokens of 32 adapters, rank 16, 7168 to
//     2048 wide: 4.4 + 4.7 us; 1 token, rank 8: 3.4 + 5.2.
//   Many tokens: shrink_many_kernel, where U is large join_kernel, expand_many_kernel; 64
//     tokens share an adapter's rows through LDS.  8192 tokens of 16 adapters, rank 64,
//     7168 to 4096 wide: 31 + 5 + 24 us; the 263 MB take 54 us at the rate of a copy.
// A token without an adapter is copied by the first launch's last workgroups.
//
// U = s_g A_g x is summed in fp32 and keeps that precision through the second product:
// it enters as two bf16 terms, U = hi + lo with lo = bf16(U - hi), two MFMAs, a relative
// error of at most 2^-16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"

namespace bsg_lora {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any_t;   // at any element
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;

constexpr int kTile = 16;      // rows of the plan per MFMA tile

// Arguments, one struct a launch and each at most 112 bytes for few tokens: a launch whose
// arguments pass that size (gridDim and the like bring 256 bytes of their own) costs up to
// 1 us more on the host, which is what bounds those calls.  Strides of X, A and B count 8
// elements.
struct Rows {              // what a row of the plan is
  const int32_t* pair_of;
  const int32_t* row_group;
  const uint16_t* base;    // or null
  uint16_t* out;
  int32_t ld_base, ldo;
  int32_t T, N, rows, items;   // items: workgroups with tiles; those behind them copy tokens
  uint16_t G, r, S;        // S: slices of K ..
  uint16_t k_units;        // .. of that many times 128 elements
  __device__ __forceinline__ int tiles() const { return (rows + kTile - 1) / kTile; }
};
struct First : Rows {
  const uint16_t* X;
  const uint16_t* A;       // [G][r][K]
  const int32_t* row_of;   // [T]
  float* U;                // [slabs][tiles*16][r]
  int32_t ldx, lda, stride_a, K;
};
struct FirstMany : First {
  const int32_t* offsets;  // [G+1]
  int32_t cap;             // most items there can be
};
struct Second : Rows {
  const uint16_t* B;       // [G][N][r]
  const float* scale;      // [G] or null
  const float* U;
  int32_t ldb, stride_b;
  int32_t col_blocks, cols_per;   // workgroups that share a tile's columns, 64-column blocks of each
};
struct SecondMany : Rows {
  const uint16_t* B;
  const float* U;
  const __bf16* UW;        // [tiles*16][hi, lo][rank padded to 32], or null: U's slabs as they are
  const float* scale;
  const int32_t* offsets;
  int32_t ldb, stride_b;
  int32_t col_blocks, cap, K;
};
struct Join {
  const float* U;
  __bf16* UW;
  const float* scale;
  const int32_t* offsets;
  int32_t rows, G, r, S, K, ranks, cap;   // ranks: r padded to 32
};
struct Both {              // one launch for little work
  const int32_t *pair_of, *row_group, *row_of;
  const uint16_t *X, *A, *B, *base;
  const float* scale;
  uint16_t* out;
  int32_t ld_base, ldo, N, items, stride_a, stride_b;
  uint16_t T, rows, ldx, lda, ldb, K8, G, r;      // K8: K / 8
};
static_assert(sizeof(First) <= 112 && sizeof(Second) <= 112 && sizeof(Both) <= 112, "see above");

// The work item of workgroup b of n: workgroups are dealt round-robin to the 8 XCDs, so
// XCD x gets a contiguous chunk of the items.
__device__ __forceinline__ int xcd_item(int b, int n) {
  const int x = b & 7, q = n >> 3, rem = n & 7;
  return x * q + min(x, rem) + (b >> 3);
}

// The adapter of a tile (that of its first row), or -1 when the tile holds no token.
__device__ __forceinline__ int tile_group(const Rows& a, int tile) {
  const int g = a.row_group[tile * kTile];
  return (uint32_t)g < (uint32_t)a.G ? g : -1;
}

// The token of a row, or -1.
__device__ __forceinline__ int row_token(const Rows& a, int row) {
  const int p = row < a.rows ? a.pair_of[row] : -1;
  return (uint32_t)p < (uint32_t)a.T ? p : -1;
}

// One k-step of 32: acc += (16 RF rank rows) x (16 tokens), lane chunks from registers.
template <int RF>
__device__ __forceinline__ void mul_step(const u32x4_t& x, const u32x4_t (&av)[RF], f32x4_t (&acc)[RF]) {
#pragma unroll
  for (int f = 0; f < RF; ++f)
    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av[f]),
                                                     __builtin_bit_cast(bf16x8_t, x), acc[f], 0, 0, 0);
}

// The lane's row (l16) of RF fragments of A_g from f0 on, from its first chunk (lq) on.  Rows past r
// repeat the last row; their sums are not used.
template <int RF>
__device__ __forceinline__ void a_rows(const First& a, int g, int f0, const uint16_t* (&ap)[RF]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int f = 0; f < RF; ++f)
    ap[f] = a.A + 8 * ((int64_t)g * a.stride_a + (int64_t)min(16 * (f0 + f) + (lane & 15), a.r - 1) * a.lda + (lane >> 4));
}

// k-steps k, k + stride, ... below k_hi, the last one partial: K is a multiple of 8, so a
// lane's chunk is whole or empty.
template <int RF>
__device__ __forceinline__ void tail_steps(const uint16_t* x, const uint16_t* const (&ap)[RF], int k, int k_hi,
                                           int stride, f32x4_t (&acc)[RF]) {
  const int lq = (threadIdx.x & 63) >> 4;
  for (; k < k_hi; k += stride) {
    u32x4_t xv = {0, 0, 0, 0}, av[RF] = {};
    if (k + 8 * lq < k_hi) {
      xv = *(const u32x4_t*)(x + k);
#pragma unroll
      for (int f = 0; f < RF; ++f) av[f] = *(const u32x4_t*)(ap[f] + k);
    }
    mul_step<RF>(xv, av, acc);
  }
}

// ---------------------------------------------------------------------------
// First product for few tokens: the wave's share of A_g x for one tile, rank rows 16 f0 ..
// 16 (f0 + RF), columns [k_lo, k_hi) of K (k_lo a multiple of 32).  The wave takes units of 32*KS elements, every
// nw-th one, straight from global memory to fragments, with the next unit's loads in
// flight while this one's MFMAs run; the last, partial unit goes in k-steps.  The two
// halves of a 128-byte line are requested back to back.  Lane (lq, l16) ends up with
// rank rows 16f + 4lq .. +3 of token l16.
// ---------------------------------------------------------------------------
template <int RF, int KS>
__device__ __forceinline__ void low_rank_rows(const First& a, int g, int f0, const uint16_t* x, int k_lo, int k_hi,
                                              int w, int nw, f32x4_t (&acc)[RF]) {
  const uint16_t* ap[RF];
  a_rows<RF>(a, g, f0, ap);
  x += 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = (f32x4_t){0, 0, 0, 0};
  struct Unit {
    u32x4_t x[KS], a[KS][RF];
  };
  auto load = [&](Unit& v, int u) {
    const int k = k_lo + u * KS * 32;
#pragma unroll
    for (int s = 0; s < KS; ++s) v.x[s] = *(const u32x4_t*)(x + k + 32 * s);
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int s = 0; s < KS; ++s) v.a[s][f] = *(const u32x4_t*)(ap[f] + k + 32 * s);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul = [&](const Unit& v) {
#pragma unroll
    for (int s = 0; s < KS; ++s) mul_step<RF>(v.x[s], v.a[s], acc);
  };
  const int units = (k_hi - k_lo) / (32 * KS);
  Unit p, q;
  int u = w;
  if (u < units) load(p, u);
  for (; u < units; u += 2 * nw) {
    if (u + nw < units) load(q, u + nw);
    mul(p);
    if (u + nw >= units) break;
    if (u + 2 * nw < units) load(p, u + 2 * nw);
    mul(q);
  }
  tail_steps<RF>(x, ap, k_lo + (units * KS + w) * 32, k_hi, 32 * nw, acc);
}

// x = hi + lo to 2^-16 of x; an infinite or NaN x has no low term.
__device__ __forceinline__ void split_bf16(float x, __bf16& hi, __bf16& lo) {
  hi = (__bf16)x;
  const float d = x - (float)hi;
  lo = (__bf16)(__builtin_isfinite(d) ? d : 0.0f);
}

// U in LDS as the second product's operand: hi and lo bf16 terms, [token][rank], zeros
// past r.  The rows are 16 bytes longer than the rank so that 16 tokens' reads spread
// over the banks.
template <int RF>
struct URows {
  static constexpr int RK = (RF + 1) / 2;        // k-steps of 32 rank elements
  static constexpr int PITCH = 32 * RK + 8;
  static constexpr int QUADS = 8 * RK;           // groups of four ranks a token
  __bf16 hi[kTile][PITCH], lo[kTile][PITCH];
  __device__ __forceinline__ void put(int token, int rank, f32x4_t v, int r) {
    bf16x4_t h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __bf16 hh, ll;
      split_bf16(rank < r ? v[e] : 0.0f, hh, ll);    // r % 8 == 0
      h[e] = hh;
      l[e] = ll;
    }
    *(bf16x4_t*)&hi[token][rank] = h;
    *(bf16x4_t*)&lo[token][rank] = l;
  }
};

// ---------------------------------------------------------------------------
// Second product and the addition for one tile: columns 64*c .. for c = c0, c0 + step,
// ... below c1; one wave.  Fragment f of B_g is the columns 16f ..; the fp32 products of
// a tile go through the wave's own LDS scratch to a layout in which eight lanes hold the
// 64 columns of one token, so that base is read and out written by whole 128-byte lines
// (16 rows of 64 bytes an instruction reach 4.0 TB/s in a copy, 8 rows of 128 bytes 4.7).
// t[j]: the token of row 8j + lane/8, -1 for none.  The next block's B_g and
// base are in flight while this one is formed, the first block's while form_u puts U into
// LDS.  out is stored with the non-temporal hint: it is not read here, and left in L2 it
// would evict the adapters.  base and out may start at any element (8192 tokens, rank 64,
// 7168 to 4097 wide, with the products as they then were: 95 us, by single elements 149;
// 4096 wide 73; now 84 and 62).
// ---------------------------------------------------------------------------
// Four columns (quad) of a row sit at quad ^ row, so that 16 rows' writes of one quad, and
// two rows' reads of eight, cover the banks once.
struct Scratch {
  f32x4_t v[kTile][16];
  __device__ __forceinline__ f32x4_t& at(int row, int quad) { return v[row][quad ^ row]; }
};

// base of one tile's 64 columns from 64*c on, 16 bytes a lane of rows 8j + lane/8.
__device__ __forceinline__ void load_base(const Rows& a, const int (&t)[2], int c, u32x4_t (&base)[2]) {
  const int n0 = 64 * c + 8 * (threadIdx.x & 7);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    base[j] = (u32x4_t){0, 0, 0, 0};
    if (a.base && t[j] >= 0 && n0 + 8 <= a.N)
      base[j] = *(const u32x4_any_t*)(a.base + (int64_t)t[j] * a.ld_base + n0);
  }
}

// One tile's 64 columns: the products b x (hi + lo), through the scratch, base added,
// rounded and stored.
template <int RK>
__device__ __forceinline__ void add_block(const Rows& a, const int (&t)[2], int c, const u32x4_t (&b)[RK][4],
                                          const bf16x8_t (&uh)[RK], const bf16x8_t (&ul)[RK],
                                          const u32x4_t (&base)[2], Scratch& scratch) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, lq = lane >> 4;
  const int col8 = 8 * (lane & 7), n0 = 64 * c + col8;
  f32x4_t acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = (f32x4_t){0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < RK; ++k)
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b[k][f]), ul[k], acc[f], 0, 0, 0);
      acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b[k][f]), uh[k], acc[f], 0, 0, 0);
    }
  // (the wave's own scratch: its LDS accesses execute in order)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
  for (int f = 0; f < 4; ++f) scratch.at(l16, 4 * f + lq) = acc[f];
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x4_t d0 = scratch.at(8 * j + (lane >> 3), 2 * (lane & 7));
    const f32x4_t d1 = scratch.at(8 * j + (lane >> 3), 2 * (lane & 7) + 1);
    if (t[j] < 0) continue;
    uint16_t* orow = a.out + (int64_t)t[j] * a.ldo + n0;
    if (n0 + 8 <= a.N) {
      u32x4_t o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = (e < 2 ? d0[2 * e] : d1[2 * e - 4]) + __uint_as_float(base[j][e] << 16);
        const float x1 = (e < 2 ? d0[2 * e + 1] : d1[2 * e - 3]) + __uint_as_float(base[j][e] & 0xFFFF0000u);
        o[e] = __builtin_bit_cast(uint32_t, (bf16x2_t){(__bf16)x0, (__bf16)x1});
      }
      __builtin_nontemporal_store(o, (u32x4_any_t*)orow);
    } else {
      const uint16_t* brow = a.base + (int64_t)t[j] * a.ld_base + n0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n0 + e < a.N) {
          const float x = a.base ? __uint_as_float((uint32_t)brow[e] << 16) : 0.0f;
          orow[e] = __builtin_bit_cast(uint16_t, (__bf16)((e < 4 ? d0[e & 3] : d1[e & 3]) + x));
        }
    }
  }
}

template <int RF, class F>
__device__ __forceinline__ void add_columns(const Second& a, int g, const int (&t)[2], const URows<RF>& u,
                                            Scratch& scratch, int c0, int c1, int step, F&& form_u) {
  constexpr int RK = URows<RF>::RK;
  const int lane = threadIdx.x & 63, l16 = lane & 15, lq = lane >> 4;
  const uint16_t* bg = a.B + 8 * (int64_t)g * a.stride_b;
  struct Block {
    u32x4_t b[RK][4], base[2];
  };
  auto load = [&](Block& v, int c) {
    load_base(a, t, c, v.base);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const uint16_t* brow = bg + 8 * ((int64_t)min(64 * c + 16 * f + l16, a.N - 1) * a.ldb + lq);
#pragma unroll
      for (int k = 0; k < RK; ++k) {
        v.b[k][f] = (u32x4_t){0, 0, 0, 0};
        if (32 * k + 8 * lq < a.r) v.b[k][f] = *(const u32x4_t*)(brow + 32 * k);
      }
    }
  };
  bf16x8_t uh[RK], ul[RK];
  auto finish = [&](const Block& v, int c) { add_block<RK>(a, t, c, v.b, uh, ul, v.base, scratch); };
  Block p, q;
  int c = c0;
  if (c < c1) load(p, c);
  form_u();
#pragma unroll
  for (int k = 0; k < RK; ++k) {
    uh[k] = *(const bf16x8_t*)&u.hi[l16][32 * k + 8 * lq];
    ul[k] = *(const bf16x8_t*)&u.lo[l16][32 * k + 8 * lq];
  }
  for (; c < c1; c += 2 * step) {
    if (c + step < c1) load(q, c + step);
    finish(p, c);
    if (c + step >= c1) break;
    if (c + 2 * step < c1) load(p, c + 2 * step);
    finish(q, c + step);
  }
}

// Tokens without an adapter (all of them where nothing has tiles): base as it is, or zeros.  16 tokens a workgroup, whose waves
// share them out.
__device__ __forceinline__ void copy_tokens(const First& a, int block, int waves) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mine = block * 16 + lane;
  uint64_t rest = __ballot(lane < 16 && mine < a.T && (a.items == 0 || a.row_of[mine < a.T ? mine : 0] < 0));
  const int nv = a.N / 8;
  for (int i = 0; rest; ++i, rest &= rest - 1) {
    if (i % waves != wave) continue;
    const int64_t t = block * 16 + __builtin_ctzll(rest);
    const uint16_t* src = a.base + t * a.ld_base;
    uint16_t* dst = a.out + t * a.ldo;
#pragma unroll 4
    for (int v = lane; v < nv; v += 64)
      *(u32x4_any_t*)(dst + 8 * v) = a.base ? *(const u32x4_any_t*)(src + 8 * v) : (u32x4_t){0, 0, 0, 0};
    for (int n = 8 * nv + lane; n < a.N; n += 64) dst[n] = a.base ? src[n] : (uint16_t)0;
  }
}

// ---------------------------------------------------------------------------
// Few tokens: two launches.  What one CU can keep in flight bounds a workgroup to some 25
// bytes per ns (one launch in which a workgroup took its tile from X to out: one token of
// rank 8, 7168 to 2048 wide, 10 us against 4 + 4), so each tile's slices of K and parts of
// the rank, and then its blocks of columns, go to workgroups of their own.  The S slices'
// sums lie in slabs of U that every workgroup of the second launch adds in order.
// ---------------------------------------------------------------------------
constexpr int kSplitWaves = 4;

template <int RF>
__global__ __launch_bounds__(64 * kSplitWaves) void shrink_kernel(const First a) {
  __shared__ f32x4_t sums[kSplitWaves][RF][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x >= a.items) {
    copy_tokens(a, blockIdx.x - a.items, kSplitWaves);
    return;
  }
  const int item = xcd_item(blockIdx.x, a.items);
  // rank rows 16 f0 .. of one slice: the parts of a slice, which read the same X, side by side
  const int parts = (a.r + 16 * RF - 1) / (16 * RF);
  int f0 = 0, part = item;
  if (parts > 1) {
    part = item / parts;
    f0 = (item - part * parts) * RF;
  }
  const int tile = part / a.S, slice = part - tile * a.S;
  const int t = row_token(a, tile * kTile + (lane & 15));
  const int g = __builtin_amdgcn_readfirstlane(tile_group(a, tile));
  if (g < 0) return;
  const int k_per = 128 * a.k_units, k_lo = min(a.K, slice * k_per), k_hi = min(a.K, k_lo + k_per);
  const int t0 = max(__builtin_amdgcn_readfirstlane(t), 0);
  f32x4_t acc[RF];
  low_rank_rows<RF, RF <= 2 ? 4 / RF : 2>(a, g, f0, a.X + 8 * (int64_t)(t < 0 ? t0 : t) * a.ldx, k_lo, k_hi, wave, kSplitWaves, acc);
#pragma unroll
  for (int f = 0; f < RF; ++f) sums[wave][f][lane] = acc[f];
  __syncthreads();
  for (int j = threadIdx.x; j < 4 * RF * kTile; j += 64 * kSplitWaves) {
    const int r4 = j % (4 * RF), token = j / (4 * RF), rank = 16 * f0 + 4 * r4;
    f32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) v += sums[w][r4 >> 2][16 * (r4 & 3) + token];
    if (rank < a.r) *(f32x4_t*)(a.U + (((int64_t)slice * a.tiles() + tile) * kTile + token) * a.r + rank) = v;
  }
}

// First product for many tokens: NT tiles of an adapter against its whole rank, K in stages
// of KC elements (128 bytes a row).  Fragments straight from global memory would ask for 64
// bytes of each of 16 rows at a time, and what bounds the kernel is the number of requests
// a CU keeps in flight; here the stages of X and A_g are copied to LDS by whole lines,
// NS - 1 stages ahead, and each wave reads its 16 tokens' and A_g's fragments from there.
// 16-byte chunk c of row r sits at chunk c ^ (r * row bytes / 256 % chunks), so that 16
// rows' reads of one chunk cover the banks once.  8192 tokens, rank 64, 7168 wide: 31 us,
// 4.7 TB/s of X and U, and as much of the adapters from L2.
//
// Items: NT tiles of one adapter.  (Groups of NT tiles that ignore where an adapter ends
// need a pass per adapter in a group, and where everything runs at once the launch lasts
// as long as the workgroup with the most passes.)  They are found from the offsets by
// every wave, as only the device knows them; the items in use, not the plan's capacity,
// are dealt to the workgroups and XCDs.
template <int NT>
struct Items {
  const int32_t* offsets;
  int G, rows, incl, total;      // incl: items up to this lane's of the first 64 adapters
  int g, tile0, nt;              // find(): the item's adapter, first tile and tiles
  // tiles of adapter g, from tile `first`
  __device__ __forceinline__ int tiles_of(int g, int& first) const {
    const int lo = min(max(offsets[min(g, G)], 0), rows), hi = min(max(offsets[min(g + 1, G)], 0), rows);
    first = lo / kTile;
    return hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
  }
  // items of the 64 adapters from g0 on, summed up to this lane's
  __device__ __forceinline__ int scan(int g0) const {
    const int lane = threadIdx.x & 63;
    int first, v = (tiles_of(g0 + lane, first) + NT - 1) / NT;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d, 64);
      if (lane >= d) v += u;
    }
    return v;
  }
  __device__ __forceinline__ Items(const int32_t* offsets, int G, int rows, int cap) : offsets(offsets), G(G), rows(rows) {
    incl = scan(0);
    total = __builtin_amdgcn_readlane(incl, 63);
    for (int g0 = 64; g0 < G; g0 += 64) total += __builtin_amdgcn_readlane(scan(g0), 63);
    total = min(total, cap);     // (more only if offsets are broken)
  }
  __device__ __forceinline__ void find(int item) {
    int v = incl, before = 0, g0 = 0;
    for (int n; item >= before + (n = __builtin_amdgcn_readlane(v, 63)) && g0 + 64 < G;) {
      before += n;
      g0 += 64;
      v = scan(g0);
    }
    const uint64_t past = __ballot(before + v > item);
    const int lane = past ? __builtin_ctzll(past) : 63;
    g = __builtin_amdgcn_readfirstlane(min(g0 + lane, G - 1));
    const int at = NT * (item - before - (lane > 0 ? __builtin_amdgcn_readlane(v, max(lane, 1) - 1) : 0));
    int first;
    const int n = tiles_of(g, first);
    tile0 = __builtin_amdgcn_readfirstlane(first + max(at, 0));
    nt = __builtin_amdgcn_readfirstlane(min(n - at, NT));
  }
};

// The first product's work is cut evenly: stages of KC elements, item by item, in one
// sequence, quota() of them a workgroup, so a workgroup may end one item and begin the
// next.  A piece goes to the slab of U that counts the item's workgroups; at most S + 1.
// (Whole slices of groups of 64 rows, 492 workgroups at once, some with two passes: 36 us
// for 8192 tokens of 16 adapters, rank 64, 7168 wide, against 31.  Two workgroups a CU:
// the same there, 41 against 38 us in all for 8192 tokens, rank 128, 2048 to 1024 wide.)
constexpr int kStage = 64;                 // KC
constexpr int kFirstWorkgroups = 256;      // one a CU
__device__ __forceinline__ int quota(int total, int stages, int S) {
  return max((total * stages + kFirstWorkgroups - 1) / kFirstWorkgroups, (stages + S - 1) / S);
}
// Slabs of an item.
__device__ __forceinline__ int slabs_of(int item, int total, int K, int S) {
  const int stages = (K + kStage - 1) / kStage, share = quota(total, stages, S);
  return ((item + 1) * stages - 1) / share - item * stages / share + 1;
}

template <int AUX = 0>
__device__ __forceinline__ void lds_copy(const uint16_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, AUX);
}
constexpr int kNonTemporal = 2;     // cache policy bit of lines read once

// Waits until at most VM of the wave's loads are outstanding and its LDS reads are done,
// then for the workgroup; unlike __syncthreads() it leaves later copies in flight.
template <int VM>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

constexpr int kItemTiles = 4;       // tiles of an item, as many as waves

template <int RF, int NT, int KC, int NS>
__global__ __launch_bounds__(64 * NT) void shrink_many_kernel(const FirstMany a) {
  constexpr int ROW = 2 * KC, NC = KC / 8;      // bytes and 16-byte chunks of a row
  constexpr int RPC = 1024 / ROW;               // rows of one wave copy
  constexpr int X_BYTES = NT * kTile * ROW, STAGE = X_BYTES + 16 * RF * ROW;
  constexpr int XC = 16 / RPC;                  // copies of X per wave and stage: its own tile
  constexpr int AR = 16 * RF / NT;              // rows of A_g a wave copies
  constexpr int AC = AR >= RPC ? AR / RPC : 1;  // (fewer than a copy holds: part of its lanes)
  constexpr int COPIES = XC + AC;
  static_assert((NS - 1) * COPIES <= 63, "outstanding copies must fit the vmcnt counter");
  // Waves: each its own tile and the whole rank or, from four rank fragments on, two
  // tiles and half of the rank, which reads fewer fragments from LDS per MFMA.
  constexpr int TW = RF >= 4 ? 2 : 1, FW = RF / TW;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * STAGE];
  if ((int)blockIdx.x >= a.items) {
    copy_tokens(a, blockIdx.x - a.items, NT);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int tile_w = wave / TW * TW, frag_w = wave % TW * FW;
  const int all = (a.K + KC - 1) / KC;          // stages of an item, the last one perhaps partial
  Items<NT> items(a.offsets, a.G, a.rows, a.cap);
  const int share = quota(items.total, all, a.S), end = items.total * all;
  const int used = (end + share - 1) / share;
  if ((int)blockIdx.x >= used) return;
  const int me = xcd_item(blockIdx.x, used);

  for (int pos = me * share, next; pos < min(end, (me + 1) * share); pos = next) {
    const int item = pos / all, first = pos - item * all, last = min(all, first + (me + 1) * share - pos);
    next = pos + last - first;
    const int slab = me - item * all / share, k_lo = first * KC;
    const int stages = min(last, a.K / KC) - first;
    items.find(item);
    const int tile0 = items.tile0, nt = items.nt, g = items.g;
    // rows without a token read the item's first token (columns of their own, not used)
    const int t0 = max(__builtin_amdgcn_readfirstlane(row_token(a, tile0 * kTile)), 0);
    const uint16_t *xs[XC], *as[AC];
    const int cr = lane / NC;                   // row of a copy
#pragma unroll
    for (int c = 0; c < XC; ++c) {
      const int row = 16 * wave + RPC * c + cr;
      const int t = wave < nt ? row_token(a, tile0 * kTile + row) : -1;
      xs[c] = a.X + 8 * (int64_t)(t < 0 ? t0 : t) * a.ldx + k_lo + 8 * ((lane % NC) ^ (row * ROW / 256 % NC));
    }
#pragma unroll
    for (int c = 0; c < AC; ++c) {
      const int row = AR * wave + RPC * c + cr;
      as[c] = a.A + 8 * ((int64_t)g * a.stride_a + (int64_t)min(row, a.r - 1) * a.lda) + k_lo +
              8 * ((lane % NC) ^ (row * ROW / 256 % NC));
    }
    auto issue = [&](int s, int buf) {
      uint8_t* const b = ring + buf * STAGE;
#pragma unroll
      for (int c = 0; c < XC; ++c) lds_copy<kNonTemporal>(xs[c] + KC * s, b + (16 * wave + RPC * c) * ROW);
#pragma unroll
      for (int c = 0; c < AC; ++c)
        if (AR >= RPC || cr < AR) lds_copy(as[c] + KC * s, b + X_BYTES + (AR * wave + RPC * c) * ROW);
    };
    f32x4_t acc[TW][FW];
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int f = 0; f < FW; ++f) acc[j][f] = (f32x4_t){0, 0, 0, 0};
    auto compute = [&](int buf) {
      const uint8_t* const b = ring + buf * STAGE;
#pragma unroll
      for (int h = 0; h < KC / 32; ++h) {
        // (rows 16 apart share the swizzle)
        const int off = l16 * ROW + (((4 * h + lq) ^ (l16 * ROW / 256 % NC)) << 4);
        u32x4_t xv[TW], av[FW];
#pragma unroll
        for (int j = 0; j < TW; ++j) xv[j] = *(const u32x4_t*)(b + 16 * (tile_w + j) * ROW + off);
#pragma unroll
        for (int f = 0; f < FW; ++f) av[f] = *(const u32x4_t*)(b + X_BYTES + 16 * (frag_w + f) * ROW + off);
#pragma unroll
        for (int j = 0; j < TW; ++j) mul_step<FW>(xv[j], av, acc[j]);
      }
    };
    // (every wave has read the previous item's stages)
    stage_barrier<0>();
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      if (s < stages) issue(s, s);
    int s = 0, buf = 0;
    for (; s + NS - 1 < stages; ++s) {
      // stage s has landed; the buffer of stage s - 1 has been read by every wave
      stage_barrier<(NS - 2) * COPIES>();
      issue(s + NS - 1, buf == 0 ? NS - 1 : buf - 1);
      compute(buf);
      buf = buf + 1 == NS ? 0 : buf + 1;
    }
    stage_barrier<0>();
    for (; s < stages; ++s) {
      compute(buf);
      buf = buf + 1 == NS ? 0 : buf + 1;
    }
#pragma unroll
    for (int j = 0; j < TW; ++j) {
      const int tile = tile_w + j;
      if (tile >= nt) continue;
      const int row = (tile0 + tile) * kTile + l16;
      if (last == all && a.K % KC) {            // K's last elements
        const int t = row_token(a, row);
        const uint16_t* ap[FW];
        a_rows<FW>(a, g, frag_w, ap);
        tail_steps<FW>(a.X + 8 * ((int64_t)(t < 0 ? t0 : t) * a.ldx + lq), ap, a.K / KC * KC, a.K, 32, acc[j]);
      }
#pragma unroll
      for (int f = 0; f < FW; ++f)
        if (16 * (frag_w + f) + 4 * lq < a.r)   // r % 8 == 0
          *(f32x4_t*)(a.U + ((int64_t)slab * a.tiles() * kTile + row) * a.r + 16 * (frag_w + f) + 4 * lq) = acc[j][f];
    }
  }
}

template <int RF>
__global__ __launch_bounds__(64 * kSplitWaves) void expand_kernel(const Second a) {
  __shared__ URows<RF> u;
  __shared__ Scratch scratch[kSplitWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = xcd_item(blockIdx.x, a.items);
  const int tile = item / a.col_blocks, cb = item % a.col_blocks;
  const int blocks = (a.N + 63) / 64, c_lo = cb * a.cols_per, c_hi = min(blocks, c_lo + a.cols_per);
  const int t[2] = {row_token(a, tile * kTile + (lane >> 3)), row_token(a, tile * kTile + 8 + (lane >> 3))};
  const int g = __builtin_amdgcn_readfirstlane(tile_group(a, tile));
  if (g < 0) return;
  add_columns<RF>(a, g, t, u, scratch[wave], c_lo + wave, c_hi, kSplitWaves, [&] {
    const float s = a.scale ? a.scale[g] : 1.0f;
    constexpr int QUADS = URows<RF>::QUADS;
    for (int j = threadIdx.x; j < QUADS * kTile; j += 64 * kSplitWaves) {
      const int r4 = j % QUADS, row = j / QUADS;
      f32x4_t v = {0, 0, 0, 0};
      if (4 * r4 < a.r && row_token(a, tile * kTile + row) >= 0) {
        const float* up = a.U + ((int64_t)tile * kTile + row) * a.r + 4 * r4;
#pragma unroll 8
        for (int sl = 0; sl < a.S; ++sl) v += *(const f32x4_t*)(up + (int64_t)sl * a.tiles() * kTile * a.r);
      }
      u.put(row, 4 * r4, s * v, a.r);
    }
    __syncthreads();
  });
}

// Both products in one launch, for little work (whole_launch() below): every workgroup of a
// tile, which has 256 columns, forms the tile's U for itself.
template <int RF>
__global__ __launch_bounds__(64 * kSplitWaves) void whole_kernel(const Both b) {
  __shared__ f32x4_t sums[kSplitWaves][RF][64];
  __shared__ URows<RF> u;
  __shared__ Scratch scratch[kSplitWaves];
  First a;
  a.pair_of = b.pair_of;
  a.row_group = b.row_group;
  a.base = b.base;
  a.out = b.out;
  a.ld_base = b.ld_base;
  a.ldo = b.ldo;
  a.T = b.T;
  a.N = b.N;
  a.rows = b.rows;
  a.items = b.items;
  a.G = b.G;
  a.r = b.r;
  Second c;
  (Rows&)c = a;
  a.row_of = b.row_of;
  a.A = b.A;
  a.lda = b.lda;
  a.stride_a = b.stride_a;
  c.B = b.B;
  c.ldb = b.ldb;
  c.stride_b = b.stride_b;
  if ((int)blockIdx.x >= a.items) {
    copy_tokens(a, blockIdx.x - a.items, kSplitWaves);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (a.N + 63) / 64, col_blocks = (blocks + kSplitWaves - 1) / kSplitWaves;
  const int item = xcd_item(blockIdx.x, a.items), tile = item / col_blocks;
  const int c0 = (item - tile * col_blocks) * kSplitWaves + wave;
  const int tx = row_token(a, tile * kTile + (lane & 15));
  const int t[2] = {row_token(a, tile * kTile + (lane >> 3)), row_token(a, tile * kTile + 8 + (lane >> 3))};
  const int g = __builtin_amdgcn_readfirstlane(tile_group(a, tile));
  if (g < 0) return;
  const int t0 = max(__builtin_amdgcn_readfirstlane(tx), 0);
  add_columns<RF>(c, g, t, u, scratch[wave], c0, min(blocks, c0 + 1), 1, [&] {
    const float s = b.scale ? b.scale[g] : 1.0f;
    f32x4_t acc[RF];
    low_rank_rows<RF, 4 / RF>(a, g, 0, b.X + 8 * (int64_t)(tx < 0 ? t0 : tx) * b.ldx, 0, 8 * b.K8, wave, kSplitWaves, acc);
#pragma unroll
    for (int f = 0; f < RF; ++f) sums[wave][f][lane] = acc[f];
    __syncthreads();
    constexpr int QUADS = URows<RF>::QUADS;
    for (int j = threadIdx.x; j < QUADS * kTile; j += 64 * kSplitWaves) {
      const int r4 = j % QUADS, row = j / QUADS;
      f32x4_t v = {0, 0, 0, 0};
      if (4 * r4 < a.r)
#pragma unroll
        for (int w = 0; w < kSplitWaves; ++w) v += sums[w][r4 >> 2][16 * (r4 & 3) + row];
      u.put(row, 4 * r4, s * v, a.r);
    }
    __syncthreads();
  });
}

// Between the two for many tokens, where the slabs are large: a tile's slabs of U summed,
// scaled and split into the second product's two bf16 terms once, instead of by every
// workgroup that needs a row.  Row layout of UW: `ranks` hi terms, then `ranks` lo terms,
// zeros past r.
__global__ __launch_bounds__(256) void join_kernel(const Join a) {
  Items<kItemTiles> items(a.offsets, a.G, a.rows, a.cap);
  const int item = blockIdx.x / kItemTiles;
  if (item >= items.total) return;
  items.find(item);
  if ((int)(blockIdx.x % kItemTiles) >= items.nt) return;
  const int tile = items.tile0 + blockIdx.x % kItemTiles, quads = a.ranks / 4;
  const int slabs = slabs_of(item, items.total, a.K, a.S);
  const int64_t slab = (int64_t)((a.rows + kTile - 1) / kTile) * kTile * a.r;
  const float s = a.scale ? a.scale[items.g] : 1.0f;
  for (int j = threadIdx.x; j < kTile * quads; j += 256) {
    const int64_t row = tile * kTile + j / quads;
    const int r4 = j % quads;
    f32x4_t v = {0, 0, 0, 0};
    if (4 * r4 < a.r) {
      const float* up = a.U + row * a.r + 4 * r4;
#pragma unroll 4
      for (int sl = 0; sl < slabs; ++sl) v += *(const f32x4_t*)(up + sl * slab);
    }
    bf16x4_t h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __bf16 hh, ll;
      split_bf16(4 * r4 < a.r ? s * v[e] : 0.0f, hh, ll);    // (zero also where s is infinite)
      h[e] = hh;
      l[e] = ll;
    }
    *(bf16x4_t*)(a.UW + row * 2 * a.ranks + 4 * r4) = h;
    *(bf16x4_t*)(a.UW + row * 2 * a.ranks + a.ranks + 4 * r4) = l;
  }
}

// Second product for many tokens: a workgroup takes 64 rows, a tile a wave, and CB blocks
// of 64 columns, whose rows of B_g it copies to LDS once for its waves.  Everything a
// wave reads from memory (base, U, its share of B_g) is asked for at once; workgroups side
// by side on a CU cover the wait.  Chunk c of B_g row n sits at chunk c ^ (n * row bytes /
// 256 % chunks), as in the first product's ring.  8192 tokens, rank 64, 4096 wide: 24 us,
// 5.7 TB/s of base, out and U.
template <int RF, int CB, bool JOINED>
__global__ __launch_bounds__(64 * kSplitWaves) __attribute__((amdgpu_waves_per_eu(RF == 8 ? 2 : 3))) void expand_many_kernel(
    const SecondMany a) {
  constexpr int RK = URows<RF>::RK, NC = 4 * RK, ROW = 16 * NC;   // 16-byte chunks and bytes of a row
  constexpr int ROWS = 64 * CB, RPC = 1024 / ROW;                   // rows, and rows of one wave copy
  __shared__ __attribute__((aligned(1024))) uint8_t bl[ROWS * ROW];
  __shared__ Scratch scratch[kSplitWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  Items<kItemTiles> items(a.offsets, a.G, a.rows, a.cap);
  const int n = items.total * a.col_blocks;
  if ((int)blockIdx.x >= n) return;
  const int at = xcd_item(blockIdx.x, n), item = at / a.col_blocks, c0 = (at - item * a.col_blocks) * CB;
  items.find(item);
  const bool mine = wave < items.nt;
  const int tile = items.tile0 + (mine ? wave : 0);
  const int t[2] = {mine ? row_token(a, tile * kTile + (lane >> 3)) : -1,
                    mine ? row_token(a, tile * kTile + 8 + (lane >> 3)) : -1};
  const uint16_t* const bg = a.B + 8 * (int64_t)items.g * a.stride_b;
#pragma unroll
  for (int q = 0; q < ROWS / RPC / kSplitWaves; ++q) {
    const int row0 = (q * kSplitWaves + wave) * RPC, row = row0 + lane / NC;
    const int chunk = (lane % NC) ^ ((row * ROW / 256) % NC);
    // rows past N repeat the last one, chunks past r the first: neither is used
    lds_copy(bg + 8 * ((int64_t)min(64 * c0 + row, a.N - 1) * a.ldb + (8 * chunk < a.r ? chunk : 0)), bl + row0 * ROW);
  }
  u32x4_t base[CB][2];
  bf16x8_t uh[RK], ul[RK];
  f32x4_t u[JOINED ? 1 : 3][RK][2];
  int slabs = 0;
  const int64_t slab = (int64_t)a.tiles() * kTile * a.r;
  const float* const up = a.U + ((int64_t)tile * kTile + l16) * a.r + 8 * lq;
  if (JOINED) {
    const __bf16* wp = a.UW + ((int64_t)tile * kTile + l16) * (64 * RK) + 8 * lq;
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      uh[k] = *(const bf16x8_t*)(wp + 32 * k);
      ul[k] = *(const bf16x8_t*)(wp + 32 * RK + 32 * k);
    }
  } else {
    slabs = slabs_of(item, items.total, a.K, a.S);
#pragma unroll
    for (int x = 0; x < 3; ++x)      // (three at once; there are seldom more)
#pragma unroll
      for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u[x][k][e] = (f32x4_t){0, 0, 0, 0};
          if (x < slabs && 32 * k + 8 * lq < a.r) u[x][k][e] = *(const f32x4_t*)(up + x * slab + 32 * k + 4 * e);
        }
  }
#pragma unroll
  for (int c = 0; c < CB; ++c) load_base(a, t, c0 + c, base[c]);
  if (!JOINED) {
    const float s = a.scale ? a.scale[items.g] : 1.0f;
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      const bool in = 32 * k + 8 * lq < a.r;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f32x4_t v = u[0][k][e] + u[JOINED ? 0 : 1][k][e] + u[JOINED ? 0 : 2][k][e];
        for (int x = 3; x < slabs; ++x)
          if (in) v += *(const f32x4_t*)(up + x * slab + 32 * k + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __bf16 h, l;
          split_bf16(in ? s * v[i] : 0.0f, h, l);     // (zero also where s is infinite)
          uh[k][4 * e + i] = h;
          ul[k][4 * e + i] = l;
        }
      }
    }
  }
  stage_barrier<0>();
  if (!mine) return;
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    if (64 * (c0 + c) >= a.N) break;
    u32x4_t b[RK][4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int k = 0; k < RK; ++k) {
        const int row = 64 * c + 16 * f + l16;
        b[k][f] = *(const u32x4_t*)(bl + row * ROW + (((4 * k + lq) ^ ((row * ROW / 256) % NC)) << 4));
      }
    if (a.r % 32) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int k = 0; k < RK; ++k)
          if (32 * k + 8 * lq >= a.r) b[k][f] = (u32x4_t){0, 0, 0, 0};
    }
    add_block<RK>(a, t, c0 + c, b, uh, ul, base[c], scratch[wave]);
  }
}

constexpr int64_t kMaxRows = int64_t(1) << 26;          // with kMaxBlocks: work-items of a launch
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // (256 a workgroup) fit 32 bits
constexpr int kColBlocks = 4;                           // 64-column blocks a workgroup, many tokens
constexpr int64_t kMaxK = int64_t(1) << 22;             // 128-element units of K fit 16 bits
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Most items of kItemTiles tiles, each of one adapter, among the plan's tiles.
static int64_t most_items(int64_t tiles, int64_t G) {
  return ceil_div(tiles, kItemTiles) + (G < tiles ? G : tiles);
}

// Whether tiles are grouped (the forms for many tokens).  Tile by tile, every 16 tokens
// read a whole adapter from L2, T r (K + N) / 8 bytes; grouped, 64 tokens share it, for
// one more launch or two and workgroups that do more each.  Tokens, adapters (drawn evenly),
// K, N, rank, 2^20s of T r (K + N): us tile by tile / grouped, replayed:
//   2048, 8,  512,  512, 32:   64,  6.5 / 10.0;     1000, 8, 1000, 1000, 64: 122, 10.0 / 13.6;
//    600, 8, 2000, 2000, 96:  220, 12.3 / 18.5;      512, 8, 4096, 4096, 64: 256, 14.5 / 15.6;
//   8192, 8, 4096,  256,  8:  272, 24.4 / 18.2;     4000, 8, 4000,  512, 16: 275, 16.4 / 16.3;
//   2048, 8, 4096, 4096, 32:  512, 22.3 / 19.0;     512, 8, 4096, 4096, 128: 512, 25.8 / 21.0;
//   512, 64, 4096, 4096, 128: 512, 41.2 / 36.1;     8192, 8, 1024, 128, 64:  576, 20.7 / 14.9;
//   8192, 8, 512, 2048, 128: 2560, 68.1 / 33.5;     8192, 16, 7168, 4096, 64: 5632, 138 / 62.
// The product knows neither how many items there are nor how many columns they share, and
// decides these for the slower form:
//   1000, 8, 4000, 128, 128:  504, 19.3 / 23.0;     2000, 8, 2000, 256, 64:  275, 12.2 / 15.3;
//   2000, 8, 4000, 256, 64:   520, 17.2 / 18.6;     4096, 32, 1024, 512, 32: 192, 12.1 / 11.2.
// (Stages of the items, of kStage elements of K, are counted in 32 bits: a plan that can have
// more than 2^30, most of it padding, is taken tile by tile.)
static bool many_tokens(int64_t T, int64_t rows, int64_t G, int64_t N, int64_t K, int64_t r) {
  return T * r * (K + N) >= int64_t(270) << 20 &&
         most_items(ceil_div(rows, kTile), G) * ceil_div(K, kStage) <= int64_t(1) << 30;
}

// Rank fragments of a workgroup of the first product for few tokens: the whole rank, or
// parts of it, each of which reads X again, for about 1024 workgroups.  K = N = 4096, us of
// both products with 1 / 2 / 4 / 8 fragments of 16 a workgroup, replayed:
//      1 token, rank 128:                   9.2 / 10.1 / 12.2 / 16.6  (1 chosen);
//     16 tokens of 1, rank 128:            11.0 / 11.7 / 13.8 / 17.9  (1);
//    256 tokens of 1 or 8, rank 128:       16.7 / 16.5 / 16.0 / 20.2  (1);
//    256 tokens of 64, rank 128:           38.1 / 35.3 / 36.8 / 43.2  (4);
//   1024 tokens of 64, rank 64:            33.4 / 30.5 / 29.2         (2).
constexpr int kFewItems = 1024;
static int rank_fragments(int64_t tiles, int64_t S, int64_t r) {
  const int64_t all = r <= 16 ? 1 : (r <= 32 ? 2 : (r <= 64 ? 4 : 8)), frags = ceil_div(r, 16);
  int rf = 1;
  while (rf < all && tiles * S * ceil_div(frags, rf) > kFewItems) rf *= 2;
  return rf;
}

// The rank up to which the kernels' fragments reach.
static int64_t padded_rank(int64_t r) { return r <= 32 ? 32 : (r <= 64 ? 64 : 128); }

// Slices of K, workgroups for the whole chip: with few tokens at least 1024 elements (two
// units a wave), as every workgroup of the second launch adds the slabs; with many at
// least 512, and quota() may cut one slice more (256 elements: 1024 tokens, rank 128, 28
// against 24 us).
static int slices(bool many, int64_t tiles, int64_t K) {
  const int64_t s = many ? ceil_div(kFirstWorkgroups, ceil_div(tiles, kItemTiles)) : 512 / tiles;
  const int64_t most = ceil_div(K, many ? 512 : 1024);
  return (int)(s < 1 ? 1 : (s < most ? s : most));
}

// Whether the second product for many tokens adds U's slabs itself, once per 256 columns,
// or takes them joined by a launch of their own: itself while those reads are few and the
// slabs, which it takes one after the other past the third, few and narrow (tokens,
// adapters, K, N, rank: reads x slices, us joined / itself: 8192, 16, 7168, 4096, 16: 27 MB x 2, 50.5 / 47;
// 8192, 8, 4096, 4096, 32: 51 x 2, 43 / 40;  3000, 8, 4096, 2048, 32: 22 x 6, 19.4 / 18.1;
// 4096, 4, 2048, 2048, 64: 43 x 4, 22.7 / 23.2;  8192, 16, 7168, 4096, 64: 103 x 2, 62 /
// 63.5;  1024, 8, 4096, 4096, 64: 42 x 8, 18 / 21;  1000, 8, 4000, 128, 128: 5 x 8, 23 /
// 31;  2500, 8, 7168, 128, 24: 2 x 7, 18 / 16).
static bool adds_slabs(int64_t S, int64_t r, int64_t slab_bytes, int64_t col_blocks) {
  return S * r < 512 && (S + 1) * slab_bytes * col_blocks <= (int64_t(160) << 20) / S;
}

// Whether both products go into one launch: while what its workgroups read of K, which
// each of a tile's does again, takes less time than a second launch (3.3 us and up; two
// launches 5 and up, and twice the host's work).  us in one launch / in two, replayed:
//   K 256, N 1024, rank 8:  1 token 3.4 / 5.3, 512 tokens of 8 adapters 3.9 / 5.5;
//   K 2048, N 4096, rank 16:  16 tokens of 1 6.7 / 7.0, of 8 5.6 / 6.5, 256 of 8 10.6 / 7.4;
//   K 4096, N 4096, 1 token:  rank 8 6.3 / 6.8, rank 16 7.5 / 6.9;
//   N 1024, rank 32:  K 1024, 64 tokens of 8 5.8 / 6.7;   K 2048, 16 tokens of 8 7.5 / 6.6.
static bool whole_launch(int64_t T, int64_t workgroups, int64_t K, int64_t r) {
  return r <= 32 && 2 * K * (r + 8) + K * (T < 16 ? T : 16) <= 160000 * 128 / (workgroups < 128 ? 128 : workgroups);
}

struct Call {
  First first;
  Second second;
  const int32_t* offsets;
  bool many;
};

template <int RF>
static void launch(const Call& c, int copy_blocks, hipStream_t st) {
  First a = c.first;
  const int64_t tiles = ceil_div(a.rows, kTile), blocks = ceil_div(a.N, 64);
  const dim3 threads(64 * kSplitWaves);
  if (a.items > 0 && c.many) {
    constexpr int NS = RF == 1 ? 6 : (RF == 8 ? 3 : 4);       // (twice as many: no faster)
    constexpr int CB = kColBlocks, ranks = 32 * URows<RF>::RK;
    const int cap = (int)most_items(tiles, a.G);
    a.items = (int)(cap * (int64_t)a.S < kFirstWorkgroups ? cap * a.S : kFirstWorkgroups);
    hipLaunchKernelGGL((shrink_many_kernel<RF, kItemTiles, kStage, NS>), dim3((unsigned)(a.items + copy_blocks)),
                       dim3(64 * kItemTiles), 0, st, (FirstMany{a, c.offsets, cap}));
    SecondMany b = {c.second, c.second.B, a.U, nullptr, c.second.scale, c.offsets, c.second.ldb, c.second.stride_b};
    b.col_blocks = (int)ceil_div(blocks, CB);
    b.cap = cap;
    b.K = a.K;
    b.items = cap * b.col_blocks;
    const int64_t slab = 4 * tiles * kTile * a.r;
    if (adds_slabs(a.S, a.r, slab, b.col_blocks)) {
      hipLaunchKernelGGL((expand_many_kernel<RF, CB, false>), dim3((unsigned)b.items), threads, 0, st, b);
    } else {
      __bf16* const UW = (__bf16*)((uint8_t*)a.U + (a.S + 1) * slab);
      b.UW = UW;
      hipLaunchKernelGGL(join_kernel, dim3((unsigned)(cap * kItemTiles)), dim3(256), 0, st,
                         (Join{a.U, UW, c.second.scale, c.offsets, a.rows, a.G, a.r, a.S, a.K, ranks, cap}));
      hipLaunchKernelGGL((expand_many_kernel<RF, CB, true>), dim3((unsigned)b.items), threads, 0, st, b);
    }
    return;
  }
  if constexpr (RF <= 2) {
    const int64_t workgroups = tiles * ceil_div(blocks, kSplitWaves), most = (1 << 16) - 1;
    if (a.items > 0 && whole_launch(a.T, workgroups, a.K, a.r) && a.T <= most && a.rows <= most && a.ldx <= most &&
        a.lda <= most && c.second.ldb <= most) {
      const Both b = {a.pair_of, a.row_group, a.row_of, a.X, a.A, c.second.B, a.base, c.second.scale, a.out,
                      a.ld_base, a.ldo, a.N, (int)workgroups, a.stride_a, c.second.stride_b,
                      (uint16_t)a.T, (uint16_t)a.rows, (uint16_t)a.ldx, (uint16_t)a.lda, (uint16_t)c.second.ldb,
                      (uint16_t)(a.K / 8), a.G, a.r};
      hipLaunchKernelGGL(whole_kernel<RF>, dim3((unsigned)(workgroups + copy_blocks)), threads, 0, st, b);
      return;
    }
  }
  const int rf = rank_fragments(tiles, a.S, a.r);
  if (a.items > 0) a.items = (int)(tiles * a.S * ceil_div(a.r, 16 * rf));
  auto* const shrink = rf == 1 ? shrink_kernel<1> : (rf == 2 ? shrink_kernel<2> : (rf == 4 ? shrink_kernel<4> : shrink_kernel<8>));
  hipLaunchKernelGGL(shrink, dim3((unsigned)(a.items + copy_blocks)), threads, 0, st, a);
  if (a.items == 0) return;
  // columns: workgroups for the whole chip, at least one block of 64 a wave
  Second b = c.second;
  const int64_t want = ceil_div(1024, tiles), most = ceil_div(blocks, kSplitWaves);
  b.cols_per = (int)ceil_div(ceil_div(blocks, want < most ? want : most), kSplitWaves) * kSplitWaves;
  b.col_blocks = (int)ceil_div(blocks, b.cols_per);
  b.items = (int)(tiles * b.col_blocks);
  hipLaunchKernelGGL(expand_kernel<RF>, dim3((unsigned)b.items), threads, 0, st, b);
}

}  // namespace bsg_lora

using namespace bsg_lora;

extern "C" {

int64_t lora_add_workspace(int64_t T, int64_t rows, int32_t G, int64_t N, int64_t K, int32_t r) {
  if (T <= 0 || rows <= 0 || G <= 0 || N <= 0 || K <= 0 || r <= 0) return 0;
  const int64_t tiles = ceil_div(rows, kTile);
  const bool many = many_tokens(T, rows, G, N, K, r);
  const int64_t joined = many ? 4 * tiles * kTile * padded_rank(r) : 0;
  return 4 * ((int64_t)slices(many, tiles, K) + many) * tiles * kTile * r + joined;
}

int lora_add_bf16(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t stride_a, const void* B,
                  int64_t ldb, int64_t stride_b, const float* scale, const int32_t* offsets,
                  const int32_t* row_of, const int32_t* pair_of, const int32_t* row_group, int64_t rows,
                  const void* base, int64_t ld_base, void* out, int64_t ldo, int64_t T, int32_t G, int64_t N, int64_t K,
                  int32_t r, void* workspace, int64_t workspace_bytes, void* stream) {
  if (T < 0 || G < 0 || N < 0 || K < 0 || r < 0 || rows < 0) return BSG_ERR_INVALID_ARG;
  if (r > 128 || r % 8 || K % 8) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T > kMaxRows || rows > kMaxRows || N > (int64_t(1) << 23) || K > kMaxK || G > 1024) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || N == 0) return BSG_OK;
  if (!out || ldo < N || !row_of || (base && ld_base < N)) return BSG_ERR_INVALID_ARG;
  if (((uintptr_t)out | (uintptr_t)base) & 1) return BSG_ERR_MISALIGNED;
  // in place only onto the same elements
  if (base == out && ld_base != ldo) return BSG_ERR_INVALID_ARG;
  const bool adapt = rows > 0 && G > 0 && K > 0 && r > 0, many = many_tokens(T, rows, G, N, K, r);
  // (tile by tile a launch has some 1024 workgroups, or one a tile, and one per 16 tokens)
  if (adapt && many && most_items(ceil_div(rows, kTile), G) * ceil_div(N, 64 * kColBlocks) > kMaxBlocks)
    return BSG_ERR_UNSUPPORTED_SHAPE;
  if (((uintptr_t)offsets | (uintptr_t)row_of | (uintptr_t)pair_of | (uintptr_t)row_group | (uintptr_t)scale) & 3)
    return BSG_ERR_MISALIGNED;
  if (rows > 0 && (!pair_of || !row_group || !offsets)) return BSG_ERR_INVALID_ARG;
  const int64_t kMaxLd = (int64_t(1) << 31) - 1, kMaxStride = 8 * kMaxLd;     // 32 bits, of X, A and B in eights
  if (adapt) {
    if (!X || !A || !B || ldx < K || lda < K || ldb < r || stride_a < 0 || stride_b < 0)
      return BSG_ERR_INVALID_ARG;
    if (ldx > kMaxStride || lda > kMaxStride || ldb > kMaxStride || stride_a > kMaxStride || stride_b > kMaxStride)
      return BSG_ERR_UNSUPPORTED_SHAPE;
    if (G > 1 && (stride_a < (r - 1) * lda + K || stride_b < (N - 1) * ldb + r)) return BSG_ERR_INVALID_ARG;
    if (((uintptr_t)X | (uintptr_t)A | (uintptr_t)B) & 15) return BSG_ERR_MISALIGNED;
    if (ldx % 8 || lda % 8 || ldb % 8 || stride_a % 8 || stride_b % 8) return BSG_ERR_MISALIGNED;
    const int64_t need = lora_add_workspace(T, rows, G, N, K, r);
    if (workspace_bytes < need || (need > 0 && !workspace)) return BSG_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 15) return BSG_ERR_MISALIGNED;
  }
  if (ldo > kMaxLd || ld_base > kMaxLd) return BSG_ERR_UNSUPPORTED_SHAPE;
  Call c = {};
  Rows rw = {};
  rw.pair_of = pair_of;
  rw.row_group = row_group;
  rw.base = (const uint16_t*)base;
  rw.out = (uint16_t*)out;
  rw.ld_base = (int32_t)ld_base;
  rw.ldo = (int32_t)ldo;
  rw.T = (int32_t)T;
  rw.N = (int32_t)N;
  rw.rows = (int32_t)rows;
  rw.items = adapt;      // (until the launch is laid out: whether there are any)
  rw.G = (uint16_t)G;
  rw.r = (uint16_t)r;
  const int S = adapt ? slices(many, ceil_div(rows, kTile), K) : 1;
  rw.S = (uint16_t)S;
  (Rows&)c.first = rw;
  c.first.k_units = (uint16_t)ceil_div(ceil_div(K, S), 128);
  c.first.K = (int32_t)K;
  c.first.X = (const uint16_t*)X;
  c.first.A = (const uint16_t*)A;
  c.first.row_of = row_of;
  c.first.U = (float*)workspace;
  c.first.ldx = (int32_t)(ldx / 8);
  c.first.lda = (int32_t)(lda / 8);
  c.first.stride_a = (int32_t)(stride_a / 8);
  (Rows&)c.second = rw;
  c.second.B = (const uint16_t*)B;
  c.second.scale = scale;
  c.second.U = (const float*)workspace;
  c.second.ldb = (int32_t)(ldb / 8);
  c.second.stride_b = (int32_t)(stride_b / 8);
  c.offsets = offsets;
  c.many = many;
  const hipStream_t st = (hipStream_t)stream;
  // tokens without an adapter: nothing to do in place
  const int copy_blocks = base == out ? 0 : (int)ceil_div(T, 16);
  if (!adapt && copy_blocks == 0) return BSG_OK;      // in place and nothing to add
  (void)hipGetLastError();
  if (r <= 16) launch<1>(c, copy_blocks, st);
  else if (r <= 32) launch<2>(c, copy_blocks, st);
  else if (r <= 64) launch<4>(c, copy_blocks, st);
  else launch<8>(c, copy_blocks, st);
  return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP;
}

}  // extern "C"
