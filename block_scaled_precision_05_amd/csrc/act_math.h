// act_math.h -- activations of the dense products' epilogues, their derivatives, and the
// finishing of consecutive outputs of a row (bias, activation, residual, gate),
// shared by the matrix kernels' epilogues, the few-row kernel and the kernels that join a
// split contraction, so that all of them round and evaluate alike.
//
// Everything is formed in fp32 from fp32 sums and rounded to bf16 once at the store.  The
// exponential is the hardware's (v_exp_f32 of x log2 e), the reciprocal v_rcp_f32: a few
// 2^-23 relative, plus |x| 2^-24 from the rounded exponent, far below the 2^-9 of the bf16
// store and, for the fp32 sums of the bias gradient, averaged over the rows.  What sinks
// below the exponential's range is lost: at most 2^-120 of a result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsg.h"

namespace bsg {

// V consecutive bf16 as one access: 16 bytes (V = 8) or 8 (V = 4).
template <int V>
struct Bf16s {
  typedef __attribute__((ext_vector_type(V / 2))) int t;
  typedef t any __attribute__((aligned(2)));   // the same at any element of a row
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __bf16 a = (__bf16)lo;   // v_cvt_pk_bf16_f32: round to nearest even
  __bf16 b = (__bf16)hi;
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

__device__ __forceinline__ uint16_t bf16_of(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

template <int V>
__device__ __forceinline__ void unpack(const typename Bf16s<V>::t& v, float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    x[2 * j] = __uint_as_float((uint32_t)v[j] << 16);
    x[2 * j + 1] = __uint_as_float((uint32_t)v[j] & 0xFFFF0000u);
  }
}

template <int V>
__device__ __forceinline__ typename Bf16s<V>::t pack(const float (&x)[V]) {
  typename Bf16s<V>::t v;
#pragma unroll
  for (int j = 0; j < V / 2; ++j) v[j] = (int)pack_bf16x2(x[2 * j], x[2 * j + 1]);
  return v;
}

// V consecutive bf16 at any element of a row: where all V exist one access, which the
// hardware takes at any even address, else the cnt that do, one by one (the rest read 0).
template <int V>
__device__ __forceinline__ typename Bf16s<V>::t load_bf16s(const uint16_t* p, int cnt) {
  typename Bf16s<V>::t v;
  if (cnt >= V) {
    v = *(const typename Bf16s<V>::any*)p;
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      v[j] = (2 * j < cnt ? p[2 * j] : 0) | (uint32_t)(2 * j + 1 < cnt ? p[2 * j + 1] : 0) << 16;
  }
  return v;
}

// Stores carry the non-temporal hint where every row is aligned (vec): outputs are written
// once here and read, if at all, by another kernel.
template <int V>
__device__ __forceinline__ void store_bf16s(uint16_t* p, const float (&x)[V], bool vec, int cnt) {
  if (cnt >= V) {
    if (vec)
      __builtin_nontemporal_store(pack<V>(x), (typename Bf16s<V>::t*)p);
    else
      *(typename Bf16s<V>::any*)p = pack<V>(x);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < cnt) p[e] = bf16_of(x[e]);
  }
}

// e^x through the hardware's 2^x; inf and 0 past the range.
__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// 1 / (1 + e^-x).  v_rcp_f32 gives 0 for a result below 2^-126 (x < -87.3), the multiply
// keeps it: the reciprocal is taken of 2^-8 (1 + e^-x).  0 from x = -88.7 on, where e^-x
// overflows (the value is below 2^-128).
__device__ __forceinline__ float sigmoid_f32(float x) {
  return 0x1p-8f * __builtin_amdgcn_rcpf(__builtin_fmaf(exp_f32(-x), 0x1p-8f, 0x1p-8f));
}

// The normal distribution's upper tail Q(x) = erfc(x / sqrt 2) / 2 for x >= 0, and
// e^(-x^2/2) beside it.  Q(x) = e^(-x^2/2) t P(t) with t = 1 / (1 + 0.3 x): P, of degree 7,
// fitted here to Q e^(x^2/2) / t for 0 <= x <= 15 by reweighted least squares (largest
// relative error 1.8e-7, 4.8e-7 evaluated in fp32); beyond 13.5 both factors underflow.
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
    // z Phi(z): z q below zero, z - z q above (past 20, where q is 0, an infinite z has to
    // stay one)
    float e;
    const float zc = z > 20.0f ? 20.0f : z, q = normal_tail(fabsf(zc), e);
    return z < 0.0f ? z * q : __builtin_fmaf(-zc, q, z);
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
    f = z < 0.0f ? z * q : __builtin_fmaf(-zc, q, z);
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

template <int V>
__device__ __forceinline__ void act_all(int act, float (&z)[V]) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = act_f<decltype(a)::value>(z[e]);
  });
}

// V consecutive outputs of a row, cnt of which exist: z (bias already added) -> Z,
// D = r + f(z).  Z may be null; r holds the residual (zeros without one).
template <int V>
__device__ __forceinline__ void act_row(int act, float (&z)[V], uint16_t* Z, const typename Bf16s<V>::t& r, bool add,
                                        uint16_t* D, bool vec, int cnt) {
  if (Z) store_bf16s<V>(Z, z, vec, cnt);
  act_all<V>(act, z);
  if (add) {
    float x[V];
    unpack<V>(r, x);
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] += x[e];
  }
  store_bf16s<V>(D, z, vec, cnt);
}

// V consecutive outputs of the gated block (inter is a multiple of 8: all of them exist):
// D = f(g) u, Z = [g .. | inter further on: u ..].
template <int V>
__device__ __forceinline__ void glu_row(int act, float (&g)[V], const float (&u)[V], uint16_t* Z, int64_t inter,
                                        uint16_t* D, bool vec) {
  if (Z) {
    store_bf16s<V>(Z, g, vec, V);
    store_bf16s<V>(Z + inter, u, vec, V);
  }
  with_act(act, [&](auto a) {
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = act_f<decltype(a)::value>(g[e]) * u[e];
  });
  store_bf16s<V>(D, g, vec, V);
}

}  // namespace bsg
