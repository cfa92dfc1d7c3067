// dense_bf16.hip -- the BF16 instances of the dense products with epilogues.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "configs.h"
#include "gemm_launch.h"
#include "internal.h"

namespace bsg {

template <int EPI>
static int go(const GemmArgs& a, int form, hipStream_t st) {
  if (form == DENSE_DEEP) return launch<KIND_BF16, BSG_BF16_DEEP_CFG, false, 0, EPI>(a, st);
  return form == DENSE_BIG ? launch<KIND_BF16, BSG_BF16_CFG, false, 0, EPI>(a, st)
                           : launch<KIND_BF16, BSG_BF16_SMALL_CFG, false, 0, EPI>(a, st);
}

int dense_bf16(const GemmArgs& a, int form, int epi, void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  if (form == DENSE_PART) return launch<KIND_BF16, BSG_BF16_DEEP_CFG, false, 0, EPI_PART>(a, st);
  return epi == EPI_GLU ? go<EPI_GLU>(a, form, st) : go<EPI_ACT>(a, form, st);
}

}  // namespace bsg
