// internal.h -- host-side helpers shared between the library's translation units
// (not part of the C ABI).
#pragma once

#include <stdint.h>

namespace bsg {

// Argument checks of the dense GEMMs and of packed scale arrays (see api.hip), and whether
// a packed scale array takes 8-byte loads.
int check_dense(const void* A, int64_t lda, const void* B, int64_t ldb, const void* D, int64_t ldd, int64_t M,
                int64_t N, int64_t K, int64_t kgran, int64_t k_bytes, int64_t elem_bytes);
int check_scales(const int16_t* sfa, int64_t ld_sfa, int64_t rows_a, const int16_t* sfb, int64_t ld_sfb,
                 int64_t rows_b, int64_t K, int64_t kgran);
bool sv_ok(const int16_t* sf, int64_t ld);

// Argument checks of the M-grouped GEMMs without the launch (kind 0 BF16, 1 FP8,
// 2 FP4): BSG_OK or the status the entry point would return.
int grouped_check(int kind, const void* A, int64_t lda, const int16_t* sfa, int64_t ld_sfa,
                  const void* B, int64_t ldb, int64_t stride_b, const int16_t* sfb,
                  int64_t ld_sfb, int64_t stride_sfb, const void* D, int64_t ldd,
                  const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N, int64_t K);

// Argument checks of m_grouped_gemm_fp8 without the launch: BSG_OK or the status
// the entry point would return.
int grouped_fp8_check(const void* A, int64_t lda, const int16_t* sfa, int64_t ld_sfa,
                      const void* B, int64_t ldb, int64_t stride_b, const int16_t* sfb,
                      int64_t ld_sfb, int64_t stride_sfb, const void* D, int64_t ldd,
                      const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N,
                      int64_t K);

// The FFN core's up-projection with the SwiGLU epilogue (Y codes and packed 1x128
// scales instead of H); arguments already checked.
int grouped_fp8_swiglu(const void* A, int64_t lda, const int16_t* sfa, int64_t ld_sfa, const void* W13,
                       int64_t ldw, int64_t stride_w, const int16_t* sfw, int64_t ld_sfw,
                       int64_t stride_sfw, const int32_t* group_offsets, int32_t G, int64_t M_total,
                       int64_t hidden, int64_t inter, void* Y, int64_t ldy, int16_t* sfy, int64_t ld_sfy,
                       int32_t rule, void* stream);

struct GemmArgs;

// Dense products with epilogues and with strided contractions: how a call is carried out.
//   DENSE_BIG    256x256 tiles, the epilogue in the kernel
//   DENSE_SMALL  smaller tiles (128 rows), the epilogue in the kernel
//   DENSE_DEEP   the same with a deeper ring, for at most one workgroup a CU (BF16)
//   DENSE_PART   smaller tiles over `splits` parts of the contraction, fp32 sums in a
//                workspace [splits][M][ldp], joined by a second kernel with the epilogue
//   DENSE_FEW    up to 64 rows of A: B streamed through registers
enum DenseForm { DENSE_BIG, DENSE_SMALL, DENSE_DEEP, DENSE_PART, DENSE_FEW };
struct DensePlan {
  int form;
  int splits;
};

// The plan of a product of M x N outputs over K elements (kind 0 BF16, 1 FP8, 2 FP4);
// strided: one of the gradients' products.
DensePlan dense_plan(int kind, int64_t M, int64_t N, int64_t K, bool strided = false);
inline int64_t dense_ldp(int64_t N) { return (N + 7) / 8 * 8; }
inline int64_t dense_part_bytes(const DensePlan& p, int64_t M, int64_t N) {
  return p.form == DENSE_PART ? 4 * p.splits * M * dense_ldp(N) : 0;
}

// Launches of the kernel instances, one function a translation unit.  epi: EPI_ACT or
// EPI_GLU for the forms with the epilogue in the kernel; sv: the kernels' scale-form flags.
int dense_bf16(const GemmArgs& a, int form, int epi, void* stream);
int dense_fp8(const GemmArgs& a, int form, int sv, void* stream);
int dense_fp4(const GemmArgs& a, int form, int sv, void* stream);
int dense_few(int kind, const GemmArgs& a, bool glu, void* stream);
// The gradients' products: tr = 2 (B strided) or 3 (both); plain bf16 D or partial sums.
int dense_strided(const GemmArgs& a, int form, int tr, void* stream);

// Joins the parts of a split call in a.P: D = R + f(sum + bias), or with inter > 0 the
// gated block over [gate, up] columns.
int dense_join(const GemmArgs& a, bool glu, void* stream);

}  // namespace bsg
