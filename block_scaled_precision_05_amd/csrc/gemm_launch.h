// gemm_launch.h -- launch of one gemm_kernel instance: tile counts, grid and the leading dead
// stages of the first round (see gemm_kernel.h), shared by the translation units that hold
// instances.
#pragma once

#include "gemm_kernel.h"

namespace bsg {

inline int g_num_cus[64];

inline int num_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (g_num_cus[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    g_num_cus[dev] = n;
  }
  return g_num_cus[dev];
}

template <int KIND, int BM, int BN, int WM, int WN, int SB, int NS, int PR, bool GROUPED, int SV = 0,
          int EPI = 0>
int launch(GemmArgs a, hipStream_t stream) {
  using T = GemmTile<KIND, BM, BN, WM, WN, SB, NS, PR, SV, GROUPED>;
  a.d_vec = (((uintptr_t)a.D & 15) == 0 && (a.ldd % 8) == 0) ? 2
            : (((uintptr_t)a.D & 7) == 0 && (a.ldd % 4) == 0) ? 1 : 0;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.nk = (a.k_bytes + SB - 1) / SB;
  constexpr bool PART = (EPI & 7) == EPI_PART;
  if (PART) a.nk = ((a.nk + a.splits - 1) / a.splits + T::U - 1) / T::U * T::U;
  int grid;
  if (GROUPED) {
    grid = num_cus();
  } else {
    // As many tiles per workgroup as the CUs require, then as few workgroups as give
    // every one that many: 448 tiles run as 224 workgroups of two rather than 256 of
    // one or two.  The idle CUs leave power to the busy ones (1-1.4% faster at
    // 4096x7168x16384 in an alternating A/B).  A multiple of 8, so a workgroup's later
    // tiles stay on its XCD (tile i runs on XCD i % 8; see xcd_remap).
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n * (PART ? a.splits : 1);
    const int64_t cus = num_cus() * T::WGS;
    const int64_t per = (tiles + cus - 1) / cus;
    int64_t g = (tiles + per - 1) / per;
    if (per > 1) g = (g + 7) / 8 * 8;
    grid = (int)(g < cus ? g : cus);
  }
  // Leading dead stages of the first round: nk padded up to whole rounds of U
  // stages, the padding rounded down to an even count (paired stages).  BF16 and FP4
  // peel it at any size (at K = 16384, 8 of 520 and 2 of 130 stages: 0.7% and 0.4%
  // faster than the same padding at the end, in an alternating A/B).  FP8 keeps a
  // padding under 2% of the loop at the end, where it multiplies zeros: its 8-register
  // fragments leave the peeled round no registers to spare (the dense kernel spills
  // there, 2% slower at K = 16384).
  constexpr int U = T::U;
  int koff = a.nk % U ? (U - a.nk % U) & ~1 : 0;
  if (KIND == KIND_FP8 && koff * 50 <= a.nk + koff) koff = 0;
  // Only the dense 256-row tiles peel it; of the products with epilogues only those whose
  // scales take wide loads (an instance for each length costs the build five seconds).
  // A part of a contraction is a whole number of rounds, but for the last.
  constexpr bool PEEL = (EPI & 7) < 3 ? BM == 256 || GROUPED
                                      : BM == 256 && !PART && (KIND == KIND_BF16 || (SV & 1));
  if (!PEEL) koff = 0;
  (void)hipGetLastError();
  int st = BSG_OK;
  auto go = [&](auto kc) {
    constexpr int KO = decltype(kc)::value;
    if constexpr (KO < U && (KO == 0 || PEEL))
      hipLaunchKernelGGL((gemm_kernel<KIND, BM, BN, WM, WN, SB, NS, PR, GROUPED, SV, KO, EPI>), dim3(grid),
                         dim3(T::NT), 0, stream, a);
    else
      st = BSG_ERR_UNSUPPORTED_SHAPE;   // not reached: koff < U by construction
  };
  static_assert(U <= 16, "leading dead stages are instantiated up to 14");
  switch (koff) {
    case 0: go(std::integral_constant<int, 0>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    case 8: go(std::integral_constant<int, 8>{}); break;
    case 10: go(std::integral_constant<int, 10>{}); break;
    case 12: go(std::integral_constant<int, 12>{}); break;
    case 14: go(std::integral_constant<int, 14>{}); break;
    default: return BSG_ERR_UNSUPPORTED_SHAPE;
  }
  if (st != BSG_OK) return st;
  return hipGetLastError() == hipSuccess ? BSG_OK : BSG_ERR_HIP;
}

}  // namespace bsg
