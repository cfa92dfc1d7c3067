// dense_bf16.hip -- the BF16 instances of the dense products with epilogues.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "configs.h"
#include "gemm_launch.h"
#include "internal.h"

namespace bsg {

int dense_bf16(const GemmArgs& a, int form, int epi, void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  if (form == DENSE_SMALL_PART) return launch<KIND_BF16, BSG_BF16_SMALL_CFG, false, 0, EPI_PART>(a, st);
  if (form == DENSE_BIG_PART) return launch<KIND_BF16, BSG_BF16_PART_CFG, false, 0, EPI_PART>(a, st);
  if (epi == EPI_GLU)
    return form == DENSE_BIG ? launch<KIND_BF16, BSG_BF16_CFG, false, 0, EPI_GLU>(a, st)
                             : launch<KIND_BF16, BSG_BF16_SMALL_CFG, false, 0, EPI_GLU>(a, st);
  return form == DENSE_BIG ? launch<KIND_BF16, BSG_BF16_CFG, false, 0, EPI_ACT>(a, st)
                           : launch<KIND_BF16, BSG_BF16_SMALL_CFG, false, 0, EPI_ACT>(a, st);
}

}  // namespace bsg
