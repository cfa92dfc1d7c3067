// dense_fp8.hip -- the FP8 instances of the dense product with an epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "configs.h"
#include "gemm_launch.h"
#include "internal.h"

namespace bsg {

template <int SV>
static int go(const GemmArgs& a, int form, hipStream_t st) {
  if (form == DENSE_PART) return launch<KIND_FP8, BSG_FP8_SMALL_CFG, false, SV, EPI_PART>(a, st);
  return form == DENSE_BIG ? launch<KIND_FP8, BSG_FP8_CFG, false, SV, EPI_ACT>(a, st)
                           : launch<KIND_FP8, BSG_FP8_SMALL_CFG, false, SV, EPI_ACT>(a, st);
}

int dense_fp8(const GemmArgs& a, int form, int sv, void* stream) {
  switch (sv) {
    case 0: return go<0>(a, form, (hipStream_t)stream);
    case 1: return go<1>(a, form, (hipStream_t)stream);
    case 2: return go<2>(a, form, (hipStream_t)stream);
    default: return go<3>(a, form, (hipStream_t)stream);
  }
}

}  // namespace bsg
