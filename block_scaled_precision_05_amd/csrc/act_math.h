// act_math.h -- activations of the dense products' epilogues, their derivatives, and the
// finishing of eight consecutive outputs of a row (bias, activation, residual, gate),
// shared by the matrix kernels' epilogues, the few-row kernel and the kernels that join a
// split contraction, so that all of them round and evaluate alike.
//
// Everything is formed in fp32 from fp32 sums and rounded to bf16 once at the store.  The
// exponential is the hardware's (v_exp_f32 of x log2 e), the reciprocal v_rcp_f32: a few
// 2^-23 relative, plus |x| 2^-24 from the rounded exponent, far below the 2^-9 of the bf16
// store and, for the fp32 sums of the bias gradient, averaged over the rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"

namespace bsg {

typedef __attribute__((ext_vector_type(4))) int am_i32x4_t;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __bf16 a = (__bf16)lo;   // v_cvt_pk_bf16_f32: round to nearest even
  __bf16 b = (__bf16)hi;
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

__device__ __forceinline__ uint16_t bf16_of(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// The eight bf16 of a 16-byte vector.
__device__ __forceinline__ void unpack8(const am_i32x4_t& v, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float((uint32_t)v[j] << 16);
    x[2 * j + 1] = __uint_as_float((uint32_t)v[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ am_i32x4_t pack8(const float (&x)[8]) {
  return (am_i32x4_t){(int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3]), (int)pack_bf16x2(x[4], x[5]),
                      (int)pack_bf16x2(x[6], x[7])};
}

// e^x through the hardware's 2^x; inf and 0 past the range.
__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }

// The normal distribution's upper tail Q(x) = erfc(x / sqrt 2) / 2 for x >= 0, and
// e^(-x^2/2) beside it.  Q(x) = e^(-x^2/2) t P(t) with t = 1 / (1 + 0.3 x): P, of degree 7,
// fitted here to Q e^(x^2/2) / t for 0 <= x <= 15 by reweighted least squares (largest
// relative error 1.8e-7, 3.2e-7 evaluated in fp32); beyond 13.5 both factors underflow.
// The relative form keeps the tail's digits, which 1 + erf would cancel.
__device__ __forceinline__ float normal_tail(float x, float& e) {
  e = exp_f32(-0.5f * x * x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, x, 1.0f));
  float p = 0.035178739577531815f;
  p = __builtin_fmaf(p, t, -0.15514235198497772f);
  p = __builtin_fmaf(p, t, 0.20281627774238586f);
  p = __builtin_fmaf(p, t, -0.050444018095731735f);
  p = __builtin_fmaf(p, t, 0.12685854732990265f);
  p = __builtin_fmaf(p, t, 0.10042543709278107f);
  p = __builtin_fmaf(p, t, 0.12067275494337082f);
  p = __builtin_fmaf(p, t, 0.11963453143835068f);
  return e * t * p;
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// f(z).  NaN stays NaN in each.
template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == BSG_ACT_RELU) {
    return z <= 0.0f ? 0.0f : z;
  } else if constexpr (ACT == BSG_ACT_SILU) {
    return z * sigmoid_f32(z);
  } else if constexpr (ACT == BSG_ACT_GELU) {
    float e;
    const float q = normal_tail(fabsf(z), e);   // z Phi(z): z q below zero, z - z q above
    return z < 0.0f ? z * q : __builtin_fmaf(-z, q, z);
  } else if constexpr (ACT == BSG_ACT_GELU_TANH) {
    // 1 + tanh(u) = 2 sigmoid(2u)
    return z * sigmoid_f32(2.0f * kGeluC * z * __builtin_fmaf(kGeluA * z, z, 1.0f));
  } else {
    return z;
  }
}

// f(z) and f'(z).  Where f' has a product of a growing and a vanishing factor, the growing
// one is held within +-100, where the other is already 0 (an infinite z then gives the
// limit, not NaN).
template <int ACT>
__device__ __forceinline__ float act_df(float z, float& f) {
  const float zc = z > 100.0f ? 100.0f : (z < -100.0f ? -100.0f : z);
  if constexpr (ACT == BSG_ACT_RELU) {
    f = z <= 0.0f ? 0.0f : z;
    return z <= 0.0f ? 0.0f : 1.0f;
  } else if constexpr (ACT == BSG_ACT_SILU) {
    const float s = sigmoid_f32(z);
    f = z * s;
    return __builtin_fmaf(zc * s, 1.0f - s, s);
  } else if constexpr (ACT == BSG_ACT_GELU) {
    float e;
    const float q = normal_tail(fabsf(zc), e);
    f = z < 0.0f ? z * q : __builtin_fmaf(-z, q, z);
    return (z < 0.0f ? q : 1.0f - q) + zc * e * 0.3989422804014327f;
  } else if constexpr (ACT == BSG_ACT_GELU_TANH) {
    const float s = sigmoid_f32(2.0f * kGeluC * z * __builtin_fmaf(kGeluA * z, z, 1.0f));
    f = z * s;
    return __builtin_fmaf(zc * s * (1.0f - s), 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluA * zc, zc, 1.0f), s);
  } else {
    f = z;
    return 1.0f;
  }
}

// body(std::integral_constant<int, ACT>) for a run-time activation (uniform over the wave).
template <class F>
__device__ __forceinline__ void with_act(int act, F body) {
  switch (act) {
    case BSG_ACT_RELU: body(std::integral_constant<int, BSG_ACT_RELU>{}); break;
    case BSG_ACT_SILU: body(std::integral_constant<int, BSG_ACT_SILU>{}); break;
    case BSG_ACT_GELU: body(std::integral_constant<int, BSG_ACT_GELU>{}); break;
    case BSG_ACT_GELU_TANH: body(std::integral_constant<int, BSG_ACT_GELU_TANH>{}); break;
    default: body(std::integral_constant<int, BSG_ACT_NONE>{}); break;
  }
}

// Eight consecutive outputs of a row: z (bias already added) -> Z, D = R + f(z).  Z and R
// may be null.  vec: all eight exist and every given row takes 16-byte accesses; r16 then
// holds the residual's eight values.  Otherwise cnt of the eight exist, accessed one by
// one.  Z and D carry the non-temporal hint: they are written once here and read, if at
// all, by another kernel.
__device__ __forceinline__ void act_row8(int act, float (&z)[8], uint16_t* Z, const uint16_t* R,
                                         const am_i32x4_t& r16, uint16_t* D, bool vec, int cnt) {
  if (Z) {
    if (vec)
      __builtin_nontemporal_store(pack8(z), (am_i32x4_t*)Z);
    else
      for (int e = 0; e < 8; ++e)
        if (e < cnt) Z[e] = bf16_of(z[e]);
  }
  with_act(act, [&](auto a) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = act_f<decltype(a)::value>(z[e]);
  });
  if (vec) {
    if (R) {
      float r[8];
      unpack8(r16, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] += r[e];
    }
    __builtin_nontemporal_store(pack8(z), (am_i32x4_t*)D);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cnt) D[e] = bf16_of(R ? z[e] + bf16_f32(R[e]) : z[e]);
  }
}

// Eight consecutive outputs of the gated block: D = f(g) u, Z = [g .. | inter further on: u ..].
__device__ __forceinline__ void glu_row8(int act, float (&g)[8], const float (&u)[8], uint16_t* Z, int64_t inter,
                                         uint16_t* D, bool vec) {
  if (Z) {
    if (vec) {
      __builtin_nontemporal_store(pack8(g), (am_i32x4_t*)Z);
      __builtin_nontemporal_store(pack8(u), (am_i32x4_t*)(Z + inter));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        Z[e] = bf16_of(g[e]);
        Z[inter + e] = bf16_of(u[e]);
      }
    }
  }
  with_act(act, [&](auto a) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = act_f<decltype(a)::value>(g[e]) * u[e];
  });
  if (vec) {
    __builtin_nontemporal_store(pack8(g), (am_i32x4_t*)D);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) D[e] = bf16_of(g[e]);
  }
}

}  // namespace bsg
