// dense_strided.hip -- products whose contraction strides through memory (the gradients of
// D = A B^T: dA = dZ B contracts B's rows, dB = dZ^T A the rows of both), BF16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"
#include "configs.h"
#include "gemm_launch.h"
#include "internal.h"

namespace bsg {

template <int TR>
static int go(const GemmArgs& a, int form, hipStream_t st) {
  if (form == DENSE_PART) return launch<KIND_BF16, BSG_BF16_DEEP_CFG, false, 0, TR + EPI_PART>(a, st);
  if (form == DENSE_DEEP) return launch<KIND_BF16, BSG_BF16_DEEP_CFG, false, 0, TR>(a, st);
  return form == DENSE_BIG ? launch<KIND_BF16, BSG_BF16_CFG, false, 0, TR>(a, st)
                           : launch<KIND_BF16, BSG_BF16_SMALL_CFG, false, 0, TR>(a, st);
}

int dense_strided(const GemmArgs& a, int form, int tr, void* stream) {
  return tr == 3 ? go<EPI_TRA + EPI_TRB>(a, form, (hipStream_t)stream) : go<EPI_TRB>(a, form, (hipStream_t)stream);
}

}  // namespace bsg
