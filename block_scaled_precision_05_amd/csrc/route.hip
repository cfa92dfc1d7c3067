// route.hip -- rows grouped by a device-side id: tokens sorted by expert (or by
// adapter), their rows dispatched to the groups (bf16 copies, or quantised on the way
// to FP8 / FP4 with packed UE8M0 scales, the operands of the grouped GEMMs), the
// experts' output rows combined with the router's weights, and the gradient of that.
//
// A pair p = t*k + j is token t's j-th choice.  Four index arrays connect the steps
// (include/bsg.h): offsets, row_of[p], pair_of[row], row_group[row].  Every kernel
// checks an index it reads from them against its arrays' sizes, so broken indices give
// wrong rows but no access outside the operands.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/bsg.h"
#include "quant_math.h"

namespace bsg_route {

using namespace bsg_qm;

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(2))) short short2_t;
typedef __attribute__((ext_vector_type(2))) unsigned short ushort2_t;

constexpr int kNone = -1;      // row_of: no row; pair_of: a padding row; row_group: no pair
constexpr int kOutside = -2;   // pair_of: a row that belongs to no group
constexpr int kMaxGroups = 1024;

static int launch_status() { return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP; }

// ---------------------------------------------------------------------------
// Stable counting sort of the pairs by group.
//
// Only a few bytes per pair move (4 read, 12 written), so the cost is latency: launches,
// dependent steps, and the scattered 4-byte writes, of which one CU finishes some two a
// ns.  Up to kSingle pairs there is one launch, in which every workgroup sorts all the
// pairs for itself, in LDS, and writes a share of the results (replayed from a graph, us
// shared / where one workgroup writes everything: 4096 pairs, 256 groups 7.2 / 8.2, and 8.0
// in two launches; 2048 pairs, 256 groups 4.9 / 6.0; 768 pairs, 384 groups 3.8 / 3.7).  More
// pairs are cut into chunks, counted by a first launch (hist[chunk][g]); in a second one
// every workgroup sums the counts of all chunks itself (coalesced reads from L2, under which
// it forms the first ranks) instead of waiting for a scan launch, and places its chunk, or a
// share of it where chunks are few (98304 pairs, 384 groups: 11.1 us with the gap between the
// launches, at 256 groups 2.5 + 8.2 in the kernels; 24576 pairs in shares 8.5, half a us
// less than unshared; masked, 24576 pairs, 48 groups of 1024 7.7).
//
// Ranks, in pair order: a wave takes 64 pairs; a lane's peers, the lanes with its id,
// come from one ballot per id bit; its rank in the wave is the number of peers below it,
// and the first peer stores the wave's count of that id in LDS.  A scan over the waves
// per group then gives every wave its base, and the groups' sizes.  No atomic decides an
// order, so the result is the same on every run.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxSteps = 4;
constexpr int kSingle = kMaxSteps * kSortThreads;   // most pairs a workgroup sorts alone
constexpr int kMaxChunks = 256;                     // workgroups of the two-launch form
constexpr int64_t kMaxPairs = int64_t(1) << 23;      // a chunk's counts fit 16 bits
// Rows are stepped through in 32 bits by at most kMaxChunks workgroups: the step past the last must fit.
constexpr int64_t kMaxSortRows = (int64_t(1) << 31) - kMaxChunks * kSortThreads;
constexpr int kSharePairs = 64, kFillRows = 2048;   // pairs and rows that a workgroup of the one-launch form writes
static_assert(kMaxGroups == kSortThreads && kMaxPairs / kMaxChunks < 65536, "one thread a group, 16-bit counts");

struct SortArgs {
  const int32_t* ids;
  int64_t ld_ids;
  int32_t k;
  int32_t flat;      // ids are contiguous: pair p's id is ids[p]
  int32_t n;         // pairs, T*k
  int32_t G;
  int32_t align;
  int32_t cap;       // > 0: masked layout
  int32_t chunk;     // pairs per workgroup, a multiple of kSortThreads
  int32_t nchunks;
  int32_t share;     // workgroups that share the placing of a chunk
  int32_t blocks;    // workgroups (gridDim would bring 256 bytes of arguments along, and 1 us a launch)
  int32_t* offsets;
  int32_t* row_of;
  int32_t* pair_of;
  int32_t* row_group;
  int32_t rows;
  uint32_t* hist;    // [nchunks][ceil(G/2)], two 16-bit counts a word; unused with one chunk
};

// Group of pair p, or -1 (an id outside [0, G), or p past the end).
__device__ __forceinline__ int pair_group(const SortArgs& a, int p) {
  if (p >= a.n) return -1;
  int id;
  if (a.flat) {
    id = a.ids[p];
  } else {
    const int t = p / a.k;
    id = a.ids[(int64_t)t * a.ld_ids + (p - t * a.k)];
  }
  return (uint32_t)id < (uint32_t)a.G ? id : -1;
}

// Lanes of the wave whose g equals this lane's (g >= 0; for g = -1 the result is not used).
__device__ __forceinline__ uint64_t same_group(int g, int G) {
  uint64_t peers = __ballot(g >= 0);
  const int bits = G > 1 ? 32 - __builtin_clz((unsigned)(G - 1)) : 0;      // of the largest id
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((g >> b) & 1);
    peers &= (g >> b) & 1 ? set : ~set;
  }
  return peers;
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(const SortArgs a) {
  __shared__ int32_t cnt[kMaxGroups];
  const int words = (a.G + 1) / 2;
  for (int g = threadIdx.x; g < 2 * words; g += kSortThreads) cnt[g] = 0;
  __syncthreads();
  const int p0 = blockIdx.x * a.chunk;
  for (int i = threadIdx.x; i < a.chunk; i += kSortThreads) {
    const int g = pair_group(a, p0 + i);
    if (g >= 0) atomicAdd(&cnt[g], 1);   // a sum: the order does not matter
  }
  __syncthreads();
  for (int w = threadIdx.x; w < words; w += kSortThreads)
    a.hist[blockIdx.x * words + w] = (uint32_t)cnt[2 * w] | (uint32_t)cnt[2 * w + 1] << 16;
}

// Inclusive scan over the workgroup, one value per thread (wave_sum is free on entry).
__device__ __forceinline__ int block_incl_scan(int v, int32_t* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  if (lane == 63) wave_sum[wave] = v;
  __syncthreads();
  // the waves before this one: lanes 0 .. wave-1 hold their sums
  int before = lane < wave ? wave_sum[lane & (kSortWaves - 1)] : 0;
#pragma unroll
  for (int d = 1; d < kSortWaves; d <<= 1) before += __shfl_xor(before, d, 64);
  return v + __shfl(before, 0, 64);
}

// First rows of the groups from their sizes (cnt: thread g's group; 0 for g >= G), into
// start[0 .. G]; workgroup 0 writes offsets.  Ends with a barrier.
__device__ __forceinline__ void group_starts(const SortArgs& a, int cnt, int32_t* start, int32_t* wave_sum) {
  const int tid = threadIdx.x;
  if (a.cap > 0) {
    if (tid <= a.G) start[tid] = tid * a.cap;
    if (tid == 0) start[a.G] = a.G * a.cap;      // (G may be the number of threads)
    if (blockIdx.x == 0 && tid < a.G) a.offsets[tid] = cnt < a.cap ? cnt : a.cap;
  } else {
    const int incl = block_incl_scan((cnt + a.align - 1) / a.align * a.align, wave_sum);
    if (tid < a.G) start[tid + 1] = incl;
    if (tid == 0) start[0] = 0;
    if (blockIdx.x == 0) {
      if (tid < a.G) a.offsets[tid + 1] = incl;
      if (tid == 0) a.offsets[0] = 0;
    }
  }
  __syncthreads();
}

// Places pair p of group g at position `at` of its group.
__device__ __forceinline__ void place(const SortArgs& a, int p, int g, int at, const int32_t* start) {
  if (p >= a.n) return;
  int row = kNone;
  if (g >= 0) {
    if (a.cap == 0 || at < a.cap) row = start[g] + at;
    if (row >= a.rows) row = kNone;   // the host's capacity check makes this unreachable
  }
  a.row_of[p] = row;
  if (row >= 0) {
    a.pair_of[row] = p;
    a.row_group[row] = g;
  }
}

// Rows without a pair: each group's from start + size on, and those behind the last group.
// size(g): group g's pairs.  One thread per group for short paddings, a wave for long.
template <class F>
__device__ __forceinline__ void fill_rest(const SortArgs& a, const int32_t* start, F&& size) {
  const int tid = blockIdx.x * kSortThreads + threadIdx.x, threads = a.blocks * kSortThreads;
  if (a.align > 1 || a.cap > 0) {
    const int tpg = a.cap > 0 || a.align > 32 ? 64 : 1;
    for (int g = tid / tpg; g < a.G; g += threads / tpg)
      for (int r = start[g] + size(g) + tid % tpg; r < start[g + 1]; r += tpg) {
        a.pair_of[r] = a.cap > 0 ? kOutside : kNone;
        a.row_group[r] = kNone;
      }
  }
  for (int r = start[a.G] + tid; r < a.rows; r += threads) {
    a.pair_of[r] = kOutside;
    a.row_group[r] = kNone;
  }
}

// At most STEPS * kSortThreads pairs.  Every workgroup sorts them all; wave w's pairs are
// written by workgroup w % workgroups, and the rows without a pair are shared out too.
template <int STEPS>
__global__ __launch_bounds__(kSortThreads) void sort_single_kernel(const SortArgs a) {
  constexpr int W = STEPS * kSortWaves;
  __shared__ uint16_t wcnt[W][kMaxGroups];
  __shared__ int32_t total[kMaxGroups], start[kMaxGroups + 1], wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int g[STEPS], rank[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) g[s] = pair_group(a, s * kSortThreads + tid);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    uint16_t* const mine = wcnt[s * kSortWaves + wave];
    for (int x = lane; x < (a.G + 1) / 2; x += 64) ((uint32_t*)mine)[x] = 0;
    // (a wave's own row: its LDS accesses execute in order)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    const uint64_t peers = same_group(g[s], a.G);
    rank[s] = __popcll(peers & ((1ull << lane) - 1));
    if (g[s] >= 0 && rank[s] == 0) mine[g[s]] = (uint16_t)__popcll(peers);
  }
  __syncthreads();
  int cnt = 0;
  if (tid < a.G) {
#pragma unroll 1
    for (int w0 = 0; w0 < W; w0 += 16) {
      int c[16];      // read together: a store between two reads would make each wait
#pragma unroll
      for (int w = 0; w < 16; ++w) c[w] = wcnt[w0 + w][tid];
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        wcnt[w0 + w][tid] = (uint16_t)cnt;
        cnt += c[w];
      }
    }
    total[tid] = cnt;
  }
  group_starts(a, cnt, start, wave_sum);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int w = s * kSortWaves + wave;
    if (w % a.blocks == (int)blockIdx.x)
      place(a, s * kSortThreads + tid, g[s], g[s] >= 0 ? wcnt[w][g[s]] + rank[s] : 0, start);
  }
  fill_rest(a, start, [&](int gg) { return total[gg]; });
}

__global__ __launch_bounds__(kSortThreads) void no_rows_kernel(int32_t* row_of, int n) {
  const int p = blockIdx.x * kSortThreads + threadIdx.x;
  if (p < n) row_of[p] = kNone;
}

// One chunk of several, after sort_hist_kernel.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(const SortArgs a) {
  __shared__ int32_t total[kMaxGroups];      // pairs of each group
  __shared__ int32_t next[kMaxGroups];       // pairs of each group in earlier chunks / steps
  __shared__ int32_t start[kMaxGroups + 1];  // first row of each group
  __shared__ uint16_t wcnt[kSortWaves][kMaxGroups];
  __shared__ int32_t wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x / a.share, part = blockIdx.x % a.share;
  const int p0 = chunk * a.chunk;
  int g = pair_group(a, p0 + tid), rank = 0, run = 0;

  // The chunks' counts: 2^s threads share a word (two groups) and take every 2^s-th chunk,
  // 16 loads in flight together, which the first pairs' ranks are formed under.
  const int words = (a.G + 1) / 2;
  int s = 0;
  while ((words << (s + 1)) <= kSortThreads) ++s;
  const int parts = 1 << s, w = tid % words, first = tid / words;
  uint32_t v[16];
  auto load_counts = [&](int c0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = c0 + i * parts;
      v[i] = a.hist[min(c, a.nchunks - 1) * words + w];
      if (c >= a.nchunks) v[i] = 0;
    }
  };
  if (first < parts) load_counts(first);
  total[tid] = next[tid] = 0;      // kSortThreads == kMaxGroups

  // a pair's rank in its wave, and the wave's counts
  auto rank_wave = [&] {
    for (int x = lane; x < words; x += 64) ((uint32_t*)&wcnt[wave][0])[x] = 0;
    // (a wave's own row: its LDS accesses execute in order)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    const uint64_t peers = same_group(g, a.G);
    rank = __popcll(peers & ((1ull << lane) - 1));
    if (g >= 0 && rank == 0) wcnt[wave][g] = (uint16_t)__popcll(peers);
  };
  // counts to the waves' bases in their groups; run: the workgroup's pairs of group tid
  auto wave_bases = [&] {
    run = 0;
    if (tid < a.G) {
      int c[kSortWaves];
#pragma unroll
      for (int x = 0; x < kSortWaves; ++x) c[x] = wcnt[x][tid];
#pragma unroll
      for (int x = 0; x < kSortWaves; ++x) {
        wcnt[x][tid] = (uint16_t)run;
        run += c[x];
      }
    }
  };
  rank_wave();
  __syncthreads();
  if (first < parts) {
    int sum0 = 0, sum1 = 0, mine0 = 0, mine1 = 0;
    for (int c0 = first; c0 < a.nchunks; c0 += 16 * parts) {
      if (c0 > first) load_counts(c0);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool before = c0 + i * parts < chunk;
        sum0 += v[i] & 0xFFFF;
        sum1 += v[i] >> 16;
        mine0 += before ? v[i] & 0xFFFF : 0;
        mine1 += before ? v[i] >> 16 : 0;
      }
    }
    // (integer sums: any order gives the same result)
    atomicAdd(&total[2 * w], sum0);
    atomicAdd(&total[2 * w + 1], sum1);
    atomicAdd(&next[2 * w], mine0);
    atomicAdd(&next[2 * w + 1], mine1);
  }
  wave_bases();
  __syncthreads();
  group_starts(a, tid < a.G ? total[tid] : 0, start, wave_sum);

  for (int i0 = 0;; i0 += kSortThreads) {   // uniform over the workgroup
    if (i0 > 0) {
      if (tid < a.G) next[tid] += run;
      g = pair_group(a, p0 + i0 + tid);
      rank_wave();
      __syncthreads();
      wave_bases();
      __syncthreads();
    }
    if (wave % a.share == part) place(a, p0 + i0 + tid, g, g >= 0 ? next[g] + wcnt[wave][g] + rank : 0, start);
    if (i0 + kSortThreads >= a.chunk || p0 + i0 + kSortThreads >= a.n) break;
    __syncthreads();      // (every wave has read next and wcnt)
  }
  fill_rest(a, start, [&](int gg) { return total[gg]; });
}

// ---------------------------------------------------------------------------
// The copying kernels move each byte once, and rows scattered over the matrices, so they
// are bound by HBM; what helps is many requests in flight (a wave's loads are issued
// together, 16 bytes a lane, 1 KiB an instruction) and, for matrices beyond the L2s (32
// MiB in all), the non-temporal hint on what is read or written once and not shared:
// rows that will not be read again then evict nothing (16384 tokens, 6 choices, 7168
// wide: combine 273 against 320 us, FP8 dispatch 215 against 232; the gradient at 8192
// tokens 353 against 378).  Smaller matrices keep the plain policy, so that the next
// kernel finds them in L2.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kStreamAux = 2;                        // the non-temporal hint
constexpr int64_t kStreamBytes = int64_t(32) << 20;  // matrices from this size on take it
constexpr int kChunk = 8;                            // rows of a token in flight together

// Padding rows (pair_of == -1) are zeroed by the kernels' first workgroups, each of which
// looks at kPadRows rows (few: padding comes in runs, which many workgroups then share).
// fill(row, lane) is called by one whole wave for every padding row of this block.
constexpr int kPadRows = 16;

template <class F>
__device__ __forceinline__ void padding_rows(const int32_t* pair_of, int rows, int block, F&& fill) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = block * kPadRows + lane;
  uint64_t pads = __ballot(lane < kPadRows && r < rows && pair_of[r < rows ? r : rows - 1] == kNone);
  for (int i = 0; pads; ++i, pads &= pads - 1)
    if (i % kWaves == wave) fill(block * kPadRows + __builtin_ctzll(pads), lane);
}

// Buffer over one row: `bytes` long, or empty when the row index is not in [0, rows),
// so that loads give zeros and stores are dropped.  The index is wave-uniform.
constexpr int kRsrcWord3 = 0x00020000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, int64_t row, int64_t rows,
                                                           int64_t stride_bytes, uint32_t bytes) {
  const bool in = row >= 0 && row < rows;
  const uint64_t at = (uint64_t)base + (in ? row * stride_bytes : 0);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(lo | (hi << 32)), (short)0,
                                           __builtin_amdgcn_readfirstlane(in ? (int)bytes : 0), kRsrcWord3);
}

// Loads and stores of VEC bf16 elements a lane: 8 (one 16-byte access) or 1, where a width, a
// leading dimension or an address is not a multiple of 8 elements (4095 tokens, 8 choices,
// 2048 against 2047 wide, us: dispatch 25 / 74, combine 27 / 69, gradient 52 / 73).
template <int VEC>
struct Vec;
template <>
struct Vec<8> {
  u32x4_t w;
  template <int AUX>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    w = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, AUX);
  }
  template <int AUX>
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
    __builtin_amdgcn_raw_buffer_store_b128(w, r, off, 0, AUX);
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(uint32_t, (bf16x2_t){(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
  }
};
template <>
struct Vec<1> {
  uint16_t w;
  template <int AUX>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    w = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, AUX);
  }
  template <int AUX>
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
    __builtin_amdgcn_raw_buffer_store_b16(w, r, off, 0, AUX);
  }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)w << 16); }
  __device__ __forceinline__ void set(const float (&v)[1]) {
    w = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
  }
};

// Zeroes one row; one wave.
template <int VEC, int AUX>
__device__ __forceinline__ void zero_row(__amdgpu_buffer_rsrc_t row, uint32_t row_bytes, int lane) {
  Vec<VEC> z;
  const float zero[VEC] = {};
  z.set(zero);
  for (uint32_t off = 2u * VEC * lane; off < row_bytes; off += 128u * VEC) z.template store<AUX>(row, off);
}

// Rows of choices j .. j + KC - 1 of a token (n of them exist), -1 past the last; whether
// any is a row.
template <int KC>
__device__ __forceinline__ bool choice_rows(const int32_t* row_of, int n, int (&r)[KC]) {
  int all = kNone;      // the sign bit stays set unless a row clears it
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    r[j] = j < n ? row_of[j] : kNone;
    all &= r[j];
  }
  return all >= 0;
}

// Whether token t has a row at all.  With experts spread over GPUs many tokens have none
// here, and are not read.
__device__ __forceinline__ bool has_rows(const int32_t* row_of, int k) {
  for (int j0 = 0; j0 < k; j0 += kChunk) {
    int r[kChunk];
    if (choice_rows(row_of + j0, k - j0, r)) return true;
  }
  return false;
}

// ---------------------------------------------------------------------------
// Dispatch, bf16: row row_of[t][j] of the output is token t's row.  A wave owns one
// segment of 64*VEC elements of one token, reads it once and writes it k times (4095
// tokens, 8 choices, 2048 wide: 26 us, 5.9 TB/s).
// ---------------------------------------------------------------------------
template <int VEC, int AUX>
__global__ __launch_bounds__(kThreads) void dispatch_bf16_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, const int32_t* __restrict__ row_of,
    const int32_t* __restrict__ pair_of, int T, int k, int rows, int H, uint16_t* __restrict__ out,
    int64_t ldo, int segs, int pad_blocks) {
  const int lane = threadIdx.x & 63;
  const uint32_t row_bytes = 2u * (uint32_t)H;
  if ((int)blockIdx.x < pad_blocks) {
    padding_rows(pair_of, rows, blockIdx.x, [&](int r, int ln) {
      zero_row<VEC, AUX>(row_rsrc(out, r, rows, 2 * ldo, row_bytes), row_bytes, ln);
    });
    return;
  }
  const int64_t task =
      (int64_t)(blockIdx.x - pad_blocks) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(task / segs), s = (int)(task - (int64_t)t * segs);
  if (t >= T) return;
  const uint32_t off = 2u * VEC * (uint32_t)(s * 64 + lane);
  const int32_t* ro = row_of + (int64_t)t * k;
  if (!has_rows(ro, k)) return;
  Vec<VEC> v;
  v.template load<0>(row_rsrc(X, t, T, 2 * ldx, row_bytes), off);
  for (int j0 = 0; j0 < k; j0 += kChunk) {
    int r[kChunk];
    choice_rows(ro + j0, k - j0, r);
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (j0 + j < k) v.template store<AUX>(row_rsrc(out, r[j], rows, 2 * ldo, row_bytes), off);
  }
}

// ---------------------------------------------------------------------------
// Dispatch with quantisation: token t's row is quantised once (the codes and scale
// bytes of the per-token quantisers, bit for bit) and its codes and packed scale words
// written to its k rows.  A wave owns 1024 elements of one token, 16 a lane, so a
// row's codes leave in 16-byte (e4m3) or 8-byte (e2m1) stores.  A scale word is two bytes
// of a line that 32 rows of a group share; with many tokens each XCD takes a contiguous
// part of them, so that most lines fill up in one L2 (835 MB written in place of 872, 212
// us in place of 214, 5.1 TB/s for 16384 tokens, 6 choices, 7168 wide; 512 tokens on an
// eighth of the experts 4.7 us).  FP4 of the same sizes, either rule: 253 us, 238 MB read and
// 656 written at 3.5 TB/s (a row has 112 scale words of 2 bytes in as many lines, FP8 has
// 28); 4.7 us for the 512 tokens.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a),
                                                                __builtin_bit_cast(ushort2_t, b)));
}
__device__ __forceinline__ uint32_t pk_min_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(ushort2_t, a),
                                                                __builtin_bit_cast(ushort2_t, b)));
}

constexpr int kQElems = 1024;   // elements of a wave's segment

// Sixteen bf16 values of one row a lane (two per word): their codes in q (4 words e4m3,
// 2 words e2m1) and their block's scale byte.
template <int FMT, int RULE>
__device__ __forceinline__ int quantize16(uint32_t (&w)[8], uint32_t (&q)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = pk_max_u16(m, w[i] & 0x7FFF7FFFu);
  uint32_t h = max(m & 0xFFFFu, m >> 16);
  // the block's lanes: 2 (e2m1) or 8 (e4m3), by DPP moves (quad_perm [1,0,3,2] and
  // [2,3,0,1], then row_half_mirror, which pairs the two quads of eight lanes)
  h = max(h, (uint32_t)__builtin_amdgcn_mov_dpp((int)h, 0xB1, 0xF, 0xF, false));
  if (FMT == FMT_E4M3) {
    h = max(h, (uint32_t)__builtin_amdgcn_mov_dpp((int)h, 0x4E, 0xF, 0xF, false));
    h = max(h, (uint32_t)__builtin_amdgcn_mov_dpp((int)h, 0x141, 0xF, 0xF, false));
  }
  const int byte = scale_byte<FMT, RULE>(h << 16);
  const float sc = scale_f32(byte);
  if (FMT == FMT_E4M3) {
    if (RULE == BSG_SCALE_OCP_MX) {
      // saturate at 448 * sc first, where the conversion would give NaN
      const uint32_t lim = 0x43E0u + (uint32_t)((byte - 127) << 7);
      const uint32_t lim2 = lim | (lim << 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pk_min_u16(w[i] & 0x7FFF7FFFu, lim2) | (w[i] & 0x80008000u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      short2_t c = {0, 0};
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2_t, w[2 * i]), sc, false);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2_t, w[2 * i + 1]), sc, true);
      q[i] = __builtin_bit_cast(uint32_t, c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[4 * i]), sc, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[4 * i + 1]), sc, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[4 * i + 2]), sc, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[4 * i + 3]), sc, 3);
      q[i] = c;
    }
  }
  return byte;
}

// The work item of workgroup b of n: workgroups are dealt round-robin to the 8 XCDs, so
// XCD x gets a contiguous chunk of the items.
__device__ __forceinline__ int xcd_item(int b, int n) {
  const int x = b & 7, q = n >> 3, rem = n & 7;
  return x * q + min(x, rem) + (b >> 3);
}

template <int FMT, int RULE, int AUX>
__global__ __launch_bounds__(kThreads) void dispatch_quant_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, const int32_t* __restrict__ row_of,
    const int32_t* __restrict__ pair_of, int T, int k, int rows, int H, uint8_t* __restrict__ Q,
    int64_t ldq, int16_t* __restrict__ sf, int64_t ld_sf, int segs, int pad_blocks,
    int blocks) {
  constexpr int GK = Fmt<FMT>::GK;
  constexpr int LPB = GK / 16;               // lanes per block
  constexpr int WPS = kQElems / GK / 2;      // packed words per segment: 4 (e4m3), 16 (e2m1)
  const int lane = threadIdx.x & 63;
  const uint32_t q_bytes = FMT == FMT_E4M3 ? (uint32_t)H : (uint32_t)H / 2;
  const int kb = H / GK, kp = (kb + 1) / 2;
  if ((int)blockIdx.x < pad_blocks) {
    // a padding row is a quantised zero row: codes 0, scale bytes 0 (the filler 0x7F)
    padding_rows(pair_of, rows, blockIdx.x, [&](int r, int ln) {
      const __amdgpu_buffer_rsrc_t o = row_rsrc(Q, r, rows, ldq, q_bytes);
      for (uint32_t off = 16u * ln; off < q_bytes; off += 1024u)
        __builtin_amdgcn_raw_buffer_store_b128((u32x4_t){0, 0, 0, 0}, o, off, 0, AUX);
      for (int i = ln; i < kp; i += 64)
        sf[(int64_t)i * ld_sf + r] = (int16_t)(2 * i + 1 < kb ? 0 : 0x7F00);
    });
    return;
  }
  const int64_t task =
      (int64_t)(AUX ? xcd_item(blockIdx.x - pad_blocks, blocks) : blockIdx.x - pad_blocks) * kWaves +
      __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(task / segs), s = (int)(task - (int64_t)t * segs);
  if (t >= T || !has_rows(row_of + (int64_t)t * k, k)) return;
  const __amdgpu_buffer_rsrc_t xr = row_rsrc(X, t, T, 2 * ldx, 2u * (uint32_t)H);
  const uint32_t e0 = (uint32_t)(s * kQElems + 16 * lane);   // lane's first element
  const u32x4_t x0 = __builtin_amdgcn_raw_buffer_load_b128(xr, 2 * e0, 0, 0);
  const u32x4_t x1 = __builtin_amdgcn_raw_buffer_load_b128(xr, 2 * e0 + 16, 0, 0);
  uint32_t w[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
  uint32_t q[4] = {};
  const int byte = quantize16<FMT, RULE>(w, q);
  // packed words of the segment: lane 2*LPB*i holds word i's low byte, lane
  // 2*LPB*i + LPB its high byte; spread so that lane i (mod WPS) holds word i
  const int wi = lane % WPS;
  const int lo = __shfl(byte, 2 * LPB * wi), hi = __shfl(byte, 2 * LPB * wi + LPB);
  const int pair = s * WPS + wi;
  const int word = lo | ((2 * pair + 1 < kb ? hi : 0x7F) << 8);
  for (int j0 = 0; j0 < k; j0 += kChunk) {
    int r[kChunk];
    choice_rows(row_of + (int64_t)t * k + j0, k - j0, r);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      if (j0 + j >= k) break;
      const __amdgpu_buffer_rsrc_t o = row_rsrc(Q, r[j], rows, ldq, q_bytes);
      if (FMT == FMT_E4M3)
        __builtin_amdgcn_raw_buffer_store_b128((u32x4_t){q[0], q[1], q[2], q[3]}, o, e0, 0, AUX);
      else
        __builtin_amdgcn_raw_buffer_store_b64((u32x2_t){q[0], q[1]}, o, e0 / 2, 0, AUX);
    }
  }
  // lanes WPS*j .. WPS*j + WPS-1 store row j's words
  for (int j0 = 0; j0 < k; j0 += 64 / WPS) {
    const int j = j0 + lane / WPS;
    if (j < k && pair < kp) {
      const int r = row_of[(int64_t)t * k + j];
      if ((uint32_t)r < (uint32_t)rows) sf[(int64_t)pair * ld_sf + r] = (int16_t)word;
    }
  }
}

// ---------------------------------------------------------------------------
// Combine: out[t] = bf16( sum_j w[t][j] * Y[row_of[t][j]] ), fp32 sums in the order of
// j, rounded once.  A wave owns 64*VEC elements of one token; the loads of KC rows (all
// of them up to eight choices) are in flight together.  A pair without a row reads zeros
// through an empty buffer and its weight counts as zero.  16384 tokens, 6 choices, 7168
// wide: 271 us, 6.1 TB/s, while the output is one 235 MB buffer, which the memory-side
// cache (256 MB) holds; 296 where two outputs alternate.  33 tokens, 8 choices: 3.3 us.
// ---------------------------------------------------------------------------
template <int VEC, int KC, int AUX>
__global__ __launch_bounds__(kThreads) void combine_kernel(
    const uint16_t* __restrict__ Y, int64_t ldy, const int32_t* __restrict__ row_of,
    const float* __restrict__ W, int64_t ldw, int T, int k, int rows, int H,
    uint16_t* __restrict__ out, int64_t ldo, int segs) {
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(task / segs), s = (int)(task - (int64_t)t * segs);
  if (t >= T) return;
  const uint32_t off = 2u * VEC * (uint32_t)(s * 64 + lane);
  float acc[VEC] = {};
  for (int j0 = 0; j0 < k; j0 += KC) {
    int r[KC];
    float w[KC];
    Vec<VEC> v[KC];
    choice_rows(row_of + (int64_t)t * k + j0, k - j0, r);
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      v[j].template load<AUX>(row_rsrc(Y, r[j], rows, 2 * ldy, 2u * (uint32_t)H), off);
      w[j] = (uint32_t)r[j] < (uint32_t)rows ? (W ? W[(int64_t)t * ldw + j0 + j] : 1.0f) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = __builtin_fmaf(w[j], v[j].get(i), acc[i]);
  }
  Vec<VEC> o;
  o.set(acc);
  o.template store<0>(row_rsrc(out, t, T, 2 * ldo, 2u * (uint32_t)H), off);
}

// ---------------------------------------------------------------------------
// Gradient of combine: dY[row_of[t][j]] = bf16( w[t][j] * dO[t] ) and dW[t][j] =
// <dO[t], Y[row_of[t][j]]> in fp32.  A workgroup owns KC of a token's choices (all of them
// up to eight; fewer where tokens are fewer than CUs, of which one moves some 25 bytes a
// ns): its waves take the token's segments in turn, keep one partial dot product per
// choice and lane, and add them over lanes and waves in a fixed order.  Where rows are
// short a wave does that alone (WPT 1).  dO is read once per KC choices, Y once, dY written
// once.  8192 tokens, 6 choices, 7168 wide, groups of 128 rows: 347 us, 5.2 TB/s with the
// padding rows (370 where three dO of 117 MB take turns, more than the memory-side cache
// holds);  257 tokens, 2 choices, 2056 wide: 3.9 us;  1 token, 8 choices, 7168 wide:
// 3.4 us (7.1 in one workgroup);  8192 tokens, 8 choices, 128 wide: 14 us (31 with a
// workgroup a token;  1024 wide, past the L2s: 55, and 52 with a workgroup).
// ---------------------------------------------------------------------------
template <int VEC, int KC, int AUX, int WPT>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dO, int64_t ldo, const uint16_t* __restrict__ Y, int64_t ldy,
    const int32_t* __restrict__ row_of, const int32_t* __restrict__ pair_of,
    const float* __restrict__ W, int64_t ldw, int T, int k, int rows, int H,
    uint16_t* __restrict__ dY, int64_t lddy, float* __restrict__ dW, int64_t lddw) {
  static_assert(WPT == 1 || WPT == kWaves, "a wave or a workgroup");
  __shared__ float part[WPT > 1 ? kWaves : 1][KC];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t row_bytes = 2u * (uint32_t)H;
  // (from the sizes: more than 112 bytes of arguments cost 1 us a launch)
  const int segs = (H + 64 * VEC - 1) / (64 * VEC), pad_blocks = (rows + kPadRows - 1) / kPadRows;
  if ((int)blockIdx.x < pad_blocks) {
    padding_rows(pair_of, rows, blockIdx.x, [&](int r, int ln) {
      zero_row<VEC, AUX>(row_rsrc(dY, r, rows, 2 * lddy, row_bytes), row_bytes, ln);
    });
    return;
  }
  const int parts = (k + KC - 1) / KC;
  const int at = ((int)blockIdx.x - pad_blocks) * (kWaves / WPT) + wave / WPT, t = at / parts;
  if (t >= T) return;
  const int j0 = (at - t * parts) * KC, n = k - j0;      // choices from j0 on, n or KC of them
  const __amdgpu_buffer_rsrc_t g = row_rsrc(dO, t, T, 2 * ldo, row_bytes);
  int r[KC];
  float w[KC], dot[KC] = {};
  // (a token without rows among these choices reads nothing; its gradients are zeros)
  const int my_segs = choice_rows(row_of + (int64_t)t * k + j0, n, r) ? segs : 0;
#pragma unroll
  for (int j = 0; j < KC; ++j) w[j] = j < n ? (W ? W[(int64_t)t * ldw + j0 + j] : 1.0f) : 0.0f;
  for (int s = wave % WPT; s < my_segs; s += WPT) {
    const uint32_t off = 2u * VEC * (uint32_t)(s * 64 + lane);
    Vec<VEC> d, y[KC];
    d.template load<0>(g, off);
    if (dW) {
#pragma unroll
      for (int j = 0; j < KC; ++j) y[j].template load<AUX>(row_rsrc(Y, r[j], rows, 2 * ldy, row_bytes), off);
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = w[j] * d.get(i);
      Vec<VEC> o;
      o.set(v);
      // (choices past the last have no row: the store is dropped)
      o.template store<AUX>(row_rsrc(dY, r[j], rows, 2 * lddy, row_bytes), off);
    }
    if (dW) {
#pragma unroll
      for (int j = 0; j < KC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dot[j] = __builtin_fmaf(d.get(i), y[j].get(i), dot[j]);
    }
  }
  if (!dW) return;
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    float v = dot[j];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
    if (WPT == 1) {
      if (lane == j) dot[0] = v;
    } else if (lane == 0) {
      part[wave][j] = v;
    }
  }
  const int j = WPT == 1 ? lane : (int)threadIdx.x;
  if (WPT > 1) __syncthreads();
  if (j < (n < KC ? n : KC)) {
    float v = dot[0];
    if (WPT > 1) {
      v = 0.0f;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) v += part[x][j];
    }
    // (a pair without a row has read zeros; an infinity in dO must not turn its
    // gradient into NaN)
    const int rr = row_of[(int64_t)t * k + j0 + j];
    dW[(int64_t)t * lddw + j0 + j] = (uint32_t)rr < (uint32_t)rows ? v : 0.0f;
  }
}

// f(KC, AUX) as compile-time constants: rows in flight (k up to kChunk), and the stream
// hint or not.
template <class F>
static void with_chunk(int k, bool stream, F&& f) {
  auto go = [&](auto kc) {
    if (stream) f(kc, std::integral_constant<int, kStreamAux>{});
    else f(kc, std::integral_constant<int, 0>{});
  };
  switch (k) {
    case 0: case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 5: go(std::integral_constant<int, 5>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    case 7: go(std::integral_constant<int, 7>{}); break;
    default: go(std::integral_constant<int, kChunk>{}); break;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;   // of kThreads: work-items of a launch fit 32 bits
constexpr int kMaxK = 64;
constexpr int64_t kCUs = 256;
constexpr int64_t kShortRow = 1024;                      // elements, two segments; one past the L2s
static_assert(kMaxBlocks * kThreads <= 0xFFFFFFFFll, "work-items of a launch");

// Checks shared by the operators that use a sorted plan.  need_pairs: pair_of is read or
// written.
static int plan_check(const int32_t* row_of, const int32_t* pair_of, bool need_pairs, int64_t T,
                      int32_t k, int64_t rows, int64_t H) {
  if (T < 0 || k < 0 || rows < 0 || H < 0) return BSG_ERR_INVALID_ARG;
  if (k > kMaxK || rows > kMaxDim - kSortThreads || (k > 0 && T > (kMaxDim - kSortThreads) / k) ||
      T > kMaxDim - kSortThreads || H > (int64_t(1) << 28))
    return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T * k > 0 && !row_of) return BSG_ERR_INVALID_ARG;
  if (need_pairs && rows > 0 && !pair_of) return BSG_ERR_INVALID_ARG;
  if (((uintptr_t)row_of | (uintptr_t)pair_of) & 3) return BSG_ERR_MISALIGNED;
  return BSG_OK;
}

// A bf16 matrix operand: present, rows of at least H elements, 2-byte aligned.
static int mat_check(const void* p, int64_t ld, int64_t H) {
  if (!p || ld < H) return BSG_ERR_INVALID_ARG;
  if (ld > (int64_t(1) << 40)) return BSG_ERR_UNSUPPORTED_SHAPE;
  return ((uintptr_t)p & 1) ? BSG_ERR_MISALIGNED : BSG_OK;
}
static bool vec8(const void* p, int64_t ld, int64_t H) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && H % 8 == 0;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace bsg_route

using namespace bsg_route;

extern "C" {

int64_t sort_tokens_workspace(int64_t pairs, int32_t G) {
  if (pairs <= kSingle || G <= 0) return 0;
  return int64_t(4) * kMaxChunks * (((G < kMaxGroups ? G : kMaxGroups) + 1) / 2);
}

int sort_tokens(const int32_t* ids, int64_t ld_ids, int64_t T, int32_t k, int32_t G, int32_t align,
                int32_t cap, int32_t* offsets, int32_t* row_of, int32_t* pair_of, int32_t* row_group,
                int64_t rows, void* workspace, int64_t workspace_bytes, void* stream) {
  if (T < 0 || k < 0 || G < 0 || align < 1 || cap < 0 || rows < 0) return BSG_ERR_INVALID_ARG;
  if (cap > 0 && align != 1) return BSG_ERR_INVALID_ARG;
  if (G > kMaxGroups || (k > 0 && T > kMaxPairs / k)) return BSG_ERR_UNSUPPORTED_SHAPE;
  const int st = plan_check(row_of, pair_of, true, T, k, rows, 0);
  if (st != BSG_OK) return st;
  const int64_t n = T * k;
  if (n > 0 && (!ids || ld_ids < k)) return BSG_ERR_INVALID_ARG;
  if (!offsets && !(cap > 0 && G == 0)) return BSG_ERR_INVALID_ARG;
  if (rows > 0 && !row_group) return BSG_ERR_INVALID_ARG;
  if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)row_group | (uintptr_t)workspace) & 3)
    return BSG_ERR_MISALIGNED;
  // every possible outcome must fit: all pairs in the groups that pad most
  if (align > kMaxDim / (2 * kMaxGroups) || (cap > 0 && G > 0 && cap > kMaxDim / (2 * G)))
    return BSG_ERR_UNSUPPORTED_SHAPE;
  const int64_t need = cap > 0 ? (int64_t)G * cap
                               : (G > 0 ? n + (G < n ? G : n) * (int64_t)(align - 1) : 0);
  if (rows < need) return BSG_ERR_INVALID_ARG;
  if (rows > kMaxSortRows) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < sort_tokens_workspace(n, G) || (sort_tokens_workspace(n, G) > 0 && !workspace))
    return BSG_ERR_INVALID_ARG;
  SortArgs a = {};
  a.ids = ids;
  a.ld_ids = ld_ids;
  a.k = k > 0 ? k : 1;
  a.n = (int32_t)n;
  a.G = G;
  a.align = align;
  a.cap = cap;
  a.offsets = offsets;
  a.row_of = row_of;
  a.pair_of = pair_of;
  a.row_group = row_group;
  a.rows = (int32_t)rows;
  a.hist = (uint32_t*)workspace;
  a.flat = ld_ids == k || T <= 1;
  const int64_t steps = ceil_div(n > 0 ? n : 1, kSortThreads);
  const hipStream_t st_ = (hipStream_t)stream;
  (void)hipGetLastError();
  if (G == 0 && n > 0) {      // no pair has a row
    hipLaunchKernelGGL(no_rows_kernel, dim3((unsigned)ceil_div(n, kSortThreads)), dim3(kSortThreads), 0, st_, row_of,
                       (int)n);
    a.n = 0;
  }
  if (n <= kSingle || G == 0) {
    int64_t blocks = ceil_div(n, kSharePairs);
    blocks = blocks > ceil_div(rows, kFillRows) ? blocks : ceil_div(rows, kFillRows);
    blocks = blocks < 1 ? 1 : (blocks < kMaxChunks ? blocks : kMaxChunks);
    a.blocks = (int32_t)blocks;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kSortThreads), 0, st_, a); };
    if (steps <= 1 || G == 0) go(sort_single_kernel<1>);
    else if (steps <= 2) go(sort_single_kernel<2>);
    else go(sort_single_kernel<4>);
  } else {
    a.chunk = (int32_t)(ceil_div(steps, kMaxChunks) * kSortThreads);
    a.nchunks = (int32_t)ceil_div(n, a.chunk);
    hipLaunchKernelGGL(sort_hist_kernel, dim3(a.nchunks), dim3(kSortThreads), 0, st_, a);
    a.share = kMaxChunks / a.nchunks < kSortWaves ? kMaxChunks / a.nchunks : kSortWaves;
    a.blocks = a.nchunks * a.share;
    hipLaunchKernelGGL(sort_scatter_kernel, dim3((unsigned)a.blocks), dim3(kSortThreads), 0, st_, a);
  }
  return launch_status();
}

int moe_dispatch_bf16(const void* X, int64_t ldx, const int32_t* row_of, const int32_t* pair_of,
                      int64_t T, int32_t k, int64_t rows, int64_t H, void* out, int64_t ldo,
                      void* stream) {
  int st = plan_check(row_of, pair_of, true, T, k, rows, H);
  if (st != BSG_OK || rows == 0 || H == 0) return st;
  if (T > 0 && (st = mat_check(X, ldx, H)) != BSG_OK) return st;
  if ((st = mat_check(out, ldo, H)) != BSG_OK) return st;
  const bool v = vec8(X, ldx, H) && vec8(out, ldo, H);
  const int64_t segs = ceil_div(H, v ? 512 : 64);
  const int64_t pads = ceil_div(rows, kPadRows), blocks = pads + (k > 0 ? ceil_div(T * segs, kWaves) : 0);
  if (blocks > kMaxBlocks) return BSG_ERR_UNSUPPORTED_SHAPE;
  const bool big = 2 * T * k * H >= kStreamBytes;
  (void)hipGetLastError();
  hipLaunchKernelGGL((v ? (big ? dispatch_bf16_kernel<8, kStreamAux> : dispatch_bf16_kernel<8, 0>)
                        : dispatch_bf16_kernel<1, 0>),
                     dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, (const uint16_t*)X, ldx,
                     row_of, pair_of, (int)T, k, (int)rows, (int)H, (uint16_t*)out, ldo, (int)segs, (int)pads);
  return launch_status();
}

}  // extern "C"

namespace bsg_route {

template <int FMT>
static int dispatch_quant(const void* X, int64_t ldx, const int32_t* row_of, const int32_t* pair_of,
                          int64_t T, int32_t k, int64_t rows, int64_t H, void* Q, int64_t ldq,
                          int16_t* sf, int64_t ld_sf, int32_t rule, void* stream) {
  constexpr int64_t GK = Fmt<FMT>::GK, per = FMT == FMT_E4M3 ? 1 : 2, qa = FMT == FMT_E4M3 ? 16 : 8;
  int st = plan_check(row_of, pair_of, true, T, k, rows, H);
  if (st != BSG_OK) return st;
  if (rule != BSG_SCALE_CEIL && rule != BSG_SCALE_OCP_MX) return BSG_ERR_INVALID_ARG;
  if (H % GK) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || H == 0) return BSG_OK;
  if (T > 0 && (st = mat_check(X, ldx, H)) != BSG_OK) return st;
  if (!Q || !sf || ldq < H / per || ld_sf < rows) return BSG_ERR_INVALID_ARG;
  if (ldq > (int64_t(1) << 40) || ld_sf > (int64_t(1) << 40)) return BSG_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (((uintptr_t)X & 15) || ldx % 8)) return BSG_ERR_MISALIGNED;
  if (((uintptr_t)Q & (qa - 1)) || ldq % qa || ((uintptr_t)sf & 1)) return BSG_ERR_MISALIGNED;
  const int64_t segs = ceil_div(H, kQElems);
  const int64_t pads = ceil_div(rows, kPadRows), blocks = pads + (k > 0 ? ceil_div(T * segs, kWaves) : 0);
  if (blocks > kMaxBlocks) return BSG_ERR_UNSUPPORTED_SHAPE;
  const bool big = T * k * H / per >= kStreamBytes;
  (void)hipGetLastError();
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, (const uint16_t*)X,
                       ldx, row_of, pair_of, (int)T, k, (int)rows, (int)H, (uint8_t*)Q, ldq, sf, ld_sf,
                       (int)segs, (int)pads, (int)(blocks - pads));
  };
  if (rule == BSG_SCALE_CEIL)
    big ? go(dispatch_quant_kernel<FMT, BSG_SCALE_CEIL, kStreamAux>) : go(dispatch_quant_kernel<FMT, BSG_SCALE_CEIL, 0>);
  else
    big ? go(dispatch_quant_kernel<FMT, BSG_SCALE_OCP_MX, kStreamAux>) : go(dispatch_quant_kernel<FMT, BSG_SCALE_OCP_MX, 0>);
  return launch_status();
}

}  // namespace bsg_route

extern "C" {

int moe_dispatch_fp8(const void* X, int64_t ldx, const int32_t* row_of, const int32_t* pair_of,
                     int64_t T, int32_t k, int64_t rows, int64_t H, void* Q, int64_t ldq, int16_t* sf,
                     int64_t ld_sf, int32_t rule, void* stream) {
  return dispatch_quant<FMT_E4M3>(X, ldx, row_of, pair_of, T, k, rows, H, Q, ldq, sf, ld_sf, rule, stream);
}

int moe_dispatch_fp4(const void* X, int64_t ldx, const int32_t* row_of, const int32_t* pair_of,
                     int64_t T, int32_t k, int64_t rows, int64_t H, void* Q, int64_t ldq, int16_t* sf,
                     int64_t ld_sf, int32_t rule, void* stream) {
  return dispatch_quant<FMT_E2M1>(X, ldx, row_of, pair_of, T, k, rows, H, Q, ldq, sf, ld_sf, rule, stream);
}

int moe_combine(const void* Y, int64_t ldy, const int32_t* row_of, const float* W, int64_t ldw,
                int64_t T, int32_t k, int64_t rows, int64_t H, void* out, int64_t ldo, void* stream) {
  int st = plan_check(row_of, nullptr, false, T, k, rows, H);
  if (st != BSG_OK || T == 0 || H == 0) return st;
  if (rows > 0 && (st = mat_check(Y, ldy, H)) != BSG_OK) return st;
  if ((st = mat_check(out, ldo, H)) != BSG_OK) return st;
  if (W && ldw < k) return BSG_ERR_INVALID_ARG;
  if ((uintptr_t)W & 3) return BSG_ERR_MISALIGNED;
  const bool v = (rows == 0 || vec8(Y, ldy, H)) && vec8(out, ldo, H);
  const int64_t segs = ceil_div(H, v ? 512 : 64), blocks = ceil_div(T * segs, kWaves);
  if (blocks > kMaxBlocks) return BSG_ERR_UNSUPPORTED_SHAPE;
  (void)hipGetLastError();
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, (const uint16_t*)Y,
                       ldy, row_of, W, ldw, (int)T, k, (int)rows, (int)H, (uint16_t*)out, ldo, (int)segs);
  };
  if (v)
    with_chunk(k, 2 * T * k * H >= kStreamBytes, [&](auto kc, auto aux) { go(combine_kernel<8, kc.value, aux.value>); });
  else
    go(combine_kernel<1, kChunk, 0>);
  return launch_status();
}

int moe_combine_backward(const void* dO, int64_t ldo, const void* Y, int64_t ldy, const int32_t* row_of,
                         const int32_t* pair_of, const float* W, int64_t ldw, int64_t T, int32_t k,
                         int64_t rows, int64_t H, void* dY, int64_t lddy, float* dW, int64_t lddw,
                         void* stream) {
  int st = plan_check(row_of, pair_of, true, T, k, rows, H);
  if (st != BSG_OK) return st;
  if ((W && ldw < k) || (dW && lddw < k)) return BSG_ERR_INVALID_ARG;
  if (((uintptr_t)W | (uintptr_t)dW) & 3) return BSG_ERR_MISALIGNED;
  if (H > 0 && T > 0 && (st = mat_check(dO, ldo, H)) != BSG_OK) return st;
  if (H > 0 && rows > 0) {
    if ((st = mat_check(dY, lddy, H)) != BSG_OK) return st;
    if (dW && (st = mat_check(Y, ldy, H)) != BSG_OK) return st;
  }
  const bool v = (T == 0 || vec8(dO, ldo, H)) && (rows == 0 || vec8(dY, lddy, H)) &&
                 (!dW || rows == 0 || vec8(Y, ldy, H));
  const int64_t pads = ceil_div(rows, kPadRows);
  const bool big = 2 * T * k * H >= kStreamBytes;
  int64_t kc = v && k < kChunk ? k : kChunk, tasks = k > 0 ? T * ceil_div(k, kc) : 0;
  if (v && tasks > 0 && tasks < kCUs) {
    kc = ceil_div(kc, ceil_div(kCUs, tasks));
    tasks = T * ceil_div(k, kc);
  }
  const bool waves = v && H <= (big ? kShortRow / 2 : kShortRow) && tasks >= kCUs;
  if (pads + tasks == 0) return BSG_OK;
  if (pads + tasks > kMaxBlocks) return BSG_ERR_UNSUPPORTED_SHAPE;
  const int64_t blocks = pads + (waves ? ceil_div(tasks, kWaves) : tasks);
  (void)hipGetLastError();
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, (const uint16_t*)dO,
                       ldo, (const uint16_t*)Y, ldy, row_of, pair_of, W, ldw, (int)T, k, (int)rows, (int)H,
                       (uint16_t*)dY, lddy, dW, lddw);
  };
  if (v)
    with_chunk((int)kc, big, [&](auto c, auto aux) {
      if (waves) go(combine_backward_kernel<8, c.value, aux.value, 1>);
      else go(combine_backward_kernel<8, c.value, aux.value, kWaves>);
    });
  else
    go(combine_backward_kernel<1, kChunk, 0, kWaves>);
  return launch_status();
}

}  // extern "C"
