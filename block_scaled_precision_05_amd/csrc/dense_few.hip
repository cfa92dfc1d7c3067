// dense_few.hip -- the dense products with epilogues for few rows (a decode step): up to 64
// rows of A, where the product is a stream of B from memory.  (Times here: us a call in graphs
// of six calls over three sets of operands.)
//
// One workgroup of W waves owns 16 NF rows of B (16 NF columns of D; in the gated block 16
// gate rows and their 16 up rows) and shares out the contraction: wave w takes the
// 128-byte steps w, w + W, ... of every row.  A wave loads a step into registers, four
// lanes to 64 consecutive bytes of a row, while the step before it goes through the wave's own LDS pieces into fragments and the matrix cores; no barrier until
// the end.  (Loaded straight into the fragments' layout, neighbouring lanes hold different
// rows, and the CU's address unit takes 64 cycles for a load instead of 16: one row, 512 x
// 7168: 10.7 us against 7.9; 32 rows: 27 against 13.)  The waves' sums meet in LDS in the
// order of the waves (the same bits on every run), and the epilogue finishes four
// consecutive columns a lane.
//
// Bound by the stream of B once that is long (one row, gated 2 x 2048 x 7168: 58.7 MB in
// 12.2 us, 4.8 TB/s), by launch and first access when short (7.3 MB: 7.8 us), and from
// some 32 rows on by A, which every workgroup reads whole.
//
// Fragments (16x16x32 BF16, 16x16x128 FP8 and FP4): lane l holds row l % 16, bytes
// 64 h + 16 (l / 16) .. +15 of the step (piece h = 0, 1).  For BF16 and FP4 each piece
// feeds one instruction, for FP8 both feed one; the order of K inside an instruction is the same
// for both operands and does not matter otherwise.  Scales: an FP8 step is one 128-wide
// K-block, an FP4 lane's 16 bytes one 32-wide block, so each lane loads the scale byte of
// its row and block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "act_math.h"
#include "gemm_kernel.h"
#include "internal.h"

namespace bsg {

typedef __attribute__((ext_vector_type(4))) float few_f32x4_t;

// GLU: 0 no gate, 1 a gate and an up fragment, 2 one fragment of eight gate and eight up rows.
template <int KIND, int MF, int NF, int GLU, int W>
__global__ __launch_bounds__(W * 64) void few_kernel(const GemmArgs args) {
  static_assert(!GLU || (KIND == KIND_BF16 && NF == (GLU == 1 ? 2 : 1)), "gate and up rows");
  constexpr int NO = GLU ? 1 : NF;            // output fragments along N
  constexpr int NC = GLU == 2 ? 8 : 16 * NO;  // output columns
  // a wave's step on its way to the fragments; at the end its sums
  constexpr int PIECES = 2 * (MF + NF);
  static_assert(MF * NF <= PIECES, "the sums take the step's place");
  __shared__ __attribute__((aligned(16))) i32x4_t smem[W][PIECES][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int n_lim = GLU ? args.inter : args.N;
  const int n0 = blockIdx.x * NC;
  const int rows_n = n_lim - n0 < NC ? n_lim - n0 : NC;

  // The epilogue's part of this thread: output fragments wave, wave + W, ...; in each row m,
  // columns n .. n+3.  What it reads is loaded ahead of the product.
  constexpr int Q = (MF * NO + W - 1) / W;
  auto row_of = [&](int q) { return 16 * ((wave + q * W) / NO) + r16; };
  auto col_of = [&](int q) { return n0 + 16 * ((wave + q * W) % NO) + 4 * lg; };
  auto mine = [&](int q) {
    return wave + q * W < MF * NO && row_of(q) < args.M && col_of(q) < n_lim && (GLU != 2 || lg < 2);
  };
  Bf16s<4>::t res[Q] = {};
  float bias[Q][4] = {};
  if constexpr (!GLU) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (!mine(q)) continue;
      const int n = col_of(q), cnt = n_lim - n < 4 ? n_lim - n : 4;
      if (args.R) res[q] = load_bf16s<4>(args.R + (int64_t)row_of(q) * args.ldr + n, cnt);
      if (args.bias) unpack<4>(load_bf16s<4>(args.bias + n, cnt), bias[q]);
    }
  }

  // records end with the operands' last byte: rows past M or N read zero
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(args.A, (uint32_t)((args.M - 1) * args.lda + args.k_bytes));
  const uint8_t* const B0 = args.B + (int64_t)n0 * args.ldb;
  // (both kinds of rows through one resource: the launcher keeps its record below 2^31)
  const uint32_t rec_b = (uint32_t)((rows_n - 1 + (GLU == 2 ? (int64_t)args.inter : 0)) * args.ldb + args.k_bytes);
  const __amdgpu_buffer_rsrc_t rb0 = make_rsrc(B0, rec_b);
  const __amdgpu_buffer_rsrc_t rb1 = make_rsrc(GLU == 1 ? B0 + (int64_t)args.inter * args.ldb : B0, rec_b);
  uint32_t va[MF], vb[NF];
#pragma unroll
  for (int f = 0; f < MF; ++f) va[f] = (uint32_t)((16 * f + (lane >> 2)) * args.lda) + 16 * (lane & 3);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = lane >> 2;
    const int64_t row = GLU == 2 ? (r & 7) + (r >> 3) * args.inter : (GLU ? 0 : 16 * f) + r;
    vb[f] = (uint32_t)(row * args.ldb) + 16 * (lane & 3);
  }
  // piece (16 rows x 64 bytes): row r's chunk c at 4r + (c ^ (r >> 2)), so that both the
  // stores (4 rows of 4 chunks) and the fragment reads (one chunk of 16 rows) of 16 lanes
  // cover all banks once
  const int put = (lane & ~3) | ((lane & 3) ^ ((lane >> 4) & 3)), get = 4 * r16 + (lg ^ (r16 >> 2));

  // scale bytes: packed word of (K-block pair, row), the block's byte of it
  const __amdgpu_buffer_rsrc_t rsa = make_rsrc(args.sfa, scale_record(args.kp_count, args.ld_sfa, args.M));
  const __amdgpu_buffer_rsrc_t rsb = make_rsrc(args.sfb, scale_record(args.kp_count, args.ld_sfb, args.sfb_rows));
  const bool b_row = KIND == KIND_FP4 || args.sfb_rows == args.N;
  const int kblocks = KIND == KIND_FP8 ? args.k_bytes / 128 : args.k_bytes / 16;
  auto scale = [&](const __amdgpu_buffer_rsrc_t& rs, int64_t ld, int row, int kb) {
    const uint32_t off = 2u * ((uint32_t)(kb >> 1) * (uint32_t)ld + (uint32_t)row) + (kb & 1);
    const uint32_t b = (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, off, 0, 0);
    return kb < kblocks ? b : 127u;   // (past K: the data are zeros, the scale must be finite)
  };

  few_f32x4_t acc[MF][NF] = {};
  const int steps = (args.k_bytes + 127) / 128;
  constexpr int NSC = KIND == KIND_BF16 ? 0 : (KIND == KIND_FP8 ? 1 : 2);   // scale bytes a fragment and step
  // Two steps a wave: one is multiplied while the other's loads are in flight.
  struct Step {
    i32x4_t a[2][MF], b[2][NF];
    uint32_t sa[NSC ? NSC : 1][MF], sb[NSC ? NSC : 1][NF];
  };
  auto load = [&](Step& t, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = 128u * s + 64 * h;
      // past K (and past the last step) the offset leaves every record
      const uint32_t oob = (int)(k + 16 * (lane & 3)) < args.k_bytes ? 0u : kOOB;
#pragma unroll
      for (int f = 0; f < NF; ++f)
        t.b[h][f] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(GLU == 1 && f ? rb1 : rb0, (vb[f] + k) | oob, 0, 0));
#pragma unroll
      for (int f = 0; f < MF; ++f)
        t.a[h][f] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, (va[f] + k) | oob, 0, 0));
    }
#pragma unroll
    for (int h = 0; h < NSC; ++h) {
      const int kb = KIND == KIND_FP8 ? s : 8 * s + 4 * h + lg;
#pragma unroll
      for (int f = 0; f < MF; ++f) t.sa[h][f] = scale(rsa, args.ld_sfa, 16 * f + r16, kb);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int row = n0 + 16 * f + r16;
        t.sb[h][f] = scale(rsb, args.ld_sfb, b_row ? row : row / 128, kb);
      }
    }
  };
  auto multiply = [&](const Step& t) __attribute__((always_inline)) {
    i32x4_t(*const mine_)[64] = smem[wave];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int f = 0; f < NF; ++f) mine_[h * (MF + NF) + f][put] = t.b[h][f];
#pragma unroll
      for (int f = 0; f < MF; ++f) mine_[h * (MF + NF) + NF + f][put] = t.a[h][f];
    }
    // (only this wave uses its pieces, and its LDS accesses execute in order)
    __builtin_amdgcn_wave_barrier();
    i32x4_t a[2][MF], b[2][NF];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int f = 0; f < NF; ++f) b[h][f] = mine_[h * (MF + NF) + f][get];
#pragma unroll
      for (int f = 0; f < MF; ++f) a[h][f] = mine_[h * (MF + NF) + NF + f][get];
    }
#pragma unroll
    for (int fa = 0; fa < MF; ++fa)
#pragma unroll
      for (int fb = 0; fb < NF; ++fb) {
        if constexpr (KIND == KIND_FP8) {
          const i32x4_t bl = b[0][fb], bh = b[1][fb], al = a[0][fa], ah = a[1][fa];
          acc[fa][fb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              (i32x8_t){bl[0], bl[1], bl[2], bl[3], bh[0], bh[1], bh[2], bh[3]},
              (i32x8_t){al[0], al[1], al[2], al[3], ah[0], ah[1], ah[2], ah[3]}, acc[fa][fb], 0, 0, 0,
              (int)t.sb[0][fb], 0, (int)t.sa[0][fa]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const i32x4_t bv = b[h][fb], av = a[h][fa];
            if constexpr (KIND == KIND_BF16)
              acc[fa][fb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, bv), __builtin_bit_cast(bf16x8_t, av), acc[fa][fb], 0, 0, 0);
            else
              acc[fa][fb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  (i32x8_t){bv[0], bv[1], bv[2], bv[3], 0, 0, 0, 0},
                  (i32x8_t){av[0], av[1], av[2], av[3], 0, 0, 0, 0}, acc[fa][fb], 4, 4, 0, (int)t.sb[h][fb], 0,
                  (int)t.sa[h][fa]);
          }
        }
      }
    __builtin_amdgcn_wave_barrier();
  };
  Step t0, t1;
  if (wave < steps) load(t0, wave);
  for (int s = wave; s < steps; s += 2 * W) {
    load(t1, s + W);
    __builtin_amdgcn_sched_barrier(0);
    multiply(t0);
    __builtin_amdgcn_sched_barrier(0);
    load(t0, s + 2 * W);
    __builtin_amdgcn_sched_barrier(0);
    multiply(t1);
    __builtin_amdgcn_sched_barrier(0);
  }

  // lane l's register r: column 4 (l / 16) + r, row l % 16 of the fragment
#pragma unroll
  for (int fa = 0; fa < MF; ++fa)
#pragma unroll
    for (int fb = 0; fb < NF; ++fb) smem[wave][fa * NF + fb][lane] = __builtin_bit_cast(i32x4_t, acc[fa][fb]);
  __syncthreads();
  auto sum = [&](int f, float (&v)[4], int ln) {
    few_f32x4_t t = __builtin_bit_cast(few_f32x4_t, smem[0][f][ln]);
#pragma unroll
    for (int w = 1; w < W; ++w) t += __builtin_bit_cast(few_f32x4_t, smem[w][f][ln]);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  };
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (!mine(q)) continue;
    const int fm = (wave + q * W) / NO, fn = (wave + q * W) % NO, n = col_of(q);
    const int64_t m = row_of(q);
    uint16_t* const Z = args.Z ? args.Z + m * args.ldz + n : nullptr;
    uint16_t* const D = args.D + m * args.ldd + n;
    float z[4];
    if constexpr (GLU) {
      float u[4];
      sum(fm * NF, z, lane);
      sum(fm * NF + (GLU == 1 ? 1 : 0), u, GLU == 1 ? lane : lane + 32);   // (up rows: 8 .. 15 of the fragment)
      glu_row<4>(args.act, z, u, Z, args.inter, D, args.e_vec);
    } else {
      sum(fm * NF + fn, z, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += bias[q][e];
      act_row<4>(args.act, z, Z, res[q], args.R != nullptr, D, args.e_vec, n_lim - n < 4 ? n_lim - n : 4);
    }
  }
}

template <int KIND, int MF, int NF, int GLU, int W>
static int go(const GemmArgs& a, hipStream_t st) {
  const int per = GLU == 2 ? 8 : (GLU ? 16 : 16 * NF), n = GLU ? a.inter : a.N;
  (void)hipGetLastError();
  hipLaunchKernelGGL((few_kernel<KIND, MF, NF, GLU, W>), dim3((unsigned)((n + per - 1) / per)), dim3(W * 64), 0, st,
                     a);
  return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP;
}

// Waves and columns of a workgroup.  Up to 16 rows: 16 waves of 16 columns (BF16 7168 x 2048,
// one row: 7.8 us; 8 waves 8.7; 32 columns no faster).  More rows: 32 columns halve what is
// read of A (32 rows, 7168 x 2048: 9.5 us against 10.3) where that leaves most CUs a
// workgroup, 16 otherwise (2048 x 7168: 13.7 against 18.1); 64 rows: 4 waves of 32 columns
// 12.0 us against 13.3 with 8.
template <int KIND>
static int go_rows(const GemmArgs& a, hipStream_t st) {
  if (a.M <= 16) return go<KIND, 1, 1, 0, 16>(a, st);
  const bool wide = a.N >= 32 * 192;
  if (a.M <= 32) return wide ? go<KIND, 2, 2, 0, 8>(a, st) : go<KIND, 2, 1, 0, 8>(a, st);
  return wide ? go<KIND, 4, 2, 0, 4>(a, st) : go<KIND, 4, 1, 0, 8>(a, st);
}

int dense_few(int kind, const GemmArgs& a, bool glu, void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  if (glu) {
    const bool narrow = a.inter < 16 * 192 && (a.inter + 8) * a.ldb < (int64_t)1 << 31;
    if (a.M <= 16) return narrow ? go<KIND_BF16, 1, 1, 2, 16>(a, st) : go<KIND_BF16, 1, 2, 1, 16>(a, st);
    if (a.M <= 32) return narrow ? go<KIND_BF16, 2, 1, 2, 8>(a, st) : go<KIND_BF16, 2, 2, 1, 8>(a, st);
    return narrow ? go<KIND_BF16, 4, 1, 2, 8>(a, st) : go<KIND_BF16, 4, 2, 1, 8>(a, st);
  }
  switch (kind) {
    case KIND_BF16: return go_rows<KIND_BF16>(a, st);
    case KIND_FP8: return go_rows<KIND_FP8>(a, st);
    default: return go_rows<KIND_FP4>(a, st);
  }
}

}  // namespace bsg
