// dense_fp4.hip -- the FP4 instances of the dense product with an epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "configs.h"
#include "gemm_launch.h"
#include "internal.h"

namespace bsg {

template <int SV>
static int go(const GemmArgs& a, int form, hipStream_t st) {
  if (form == DENSE_PART) return launch<KIND_FP4, BSG_FP4_SMALL_CFG, false, SV, EPI_PART>(a, st);
  return form == DENSE_BIG ? launch<KIND_FP4, BSG_FP4_CFG, false, SV, EPI_ACT>(a, st)
                           : launch<KIND_FP4, BSG_FP4_SMALL_CFG, false, SV, EPI_ACT>(a, st);
}

int dense_fp4(const GemmArgs& a, int form, int sv, void* stream) {
  return sv ? go<1>(a, form, (hipStream_t)stream) : go<0>(a, form, (hipStream_t)stream);
}

}  // namespace bsg
