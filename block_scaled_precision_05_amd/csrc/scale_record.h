// scale_record.h -- how many bytes of a packed scale array the kernels' buffer records cover
// (plain C++: the formula is also checked on the host).
#pragma once

#include <stdint.h>

namespace bsg {

// Record of a packed scale array of kp_count rows, `ld` int16 apart, from its start to the
// end of `rows` words of the last row.  With no K-blocks (K == 0) there is no array and the
// pointer may be null: the record is empty whatever ld and rows are, so the scale loads
// that the kernels issue ahead of their stage loops read zero and touch no memory.
constexpr uint32_t scale_record(int32_t kp_count, int64_t ld, int32_t rows) {
  return kp_count > 0 ? (uint32_t)(2 * ((int64_t)(kp_count - 1) * ld + rows)) : 0u;
}

}  // namespace bsg
