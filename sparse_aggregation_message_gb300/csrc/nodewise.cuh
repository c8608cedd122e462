// Element types, 16-byte row accesses and activations shared by the node-wise
// operators (group norm, gated projections, AdamW).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gnnagg.h"

namespace gnn {

inline bool is_type(int t) { return t == GNN_F32 || t == GNN_BF16 || t == GNN_F16; }
inline bool is_act(int a) { return a >= GNN_ACT_NONE && a <= GNN_ACT_SIGMOID; }
inline int type_size(int t) { return t == GNN_F32 ? 4 : 2; }

template <class T>
struct Pack2;
template <>
struct Pack2<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 from(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Pack2<__half> {
  static __device__ __forceinline__ uint32_t to(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 from(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
};

// N consecutive elements to or from fp32 registers in one access of up to 16
// bytes (two for eight fp32 values).  `p` is aligned to the access.
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(p + i);
    v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
  }
}
template <int N, class T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[N]) {
  uint32_t w[N / 2];
  if constexpr (N == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
    static_assert(N == 4, "4 or 8 elements");
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 f = Pack2<T>::from(w[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N, class T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(Pack2<T>::to(v[0], v[1]), Pack2<T>::to(v[2], v[3]),
                                              Pack2<T>::to(v[4], v[5]), Pack2<T>::to(v[6], v[7]));
  } else {
    static_assert(N == 4, "4 or 8 elements");
    *reinterpret_cast<uint2*>(p) = make_uint2(Pack2<T>::to(v[0], v[1]), Pack2<T>::to(v[2], v[3]));
  }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// 2^x and 1/x in one instruction each, subnormals taken as zero: all that is
// formed from them below is compared with one.
__device__ __forceinline__ float ex2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-z)): exp(-z) may reach infinity, whose reciprocal is zero.
__device__ __forceinline__ float sigmoid_f(float z) { return rcp_f(1.f + ex2_f(-kLog2e * z)); }

// The normal distribution's Phi(z) and exp(-z^2/2).  With x = |z|/sqrt 2,
// erfc(x) = t P(t) exp(-x^2), t = 1/(1 + 0.3275911 x): Abramowitz and Stegun
// 7.1.26, absolute error at most 1.5e-7, so at most 7.5e-8 in Phi.  It shares
// its exponential with the derivative of gelu.
__device__ __forceinline__ float phi_f(float z, float& e) {
  const float x = fabsf(z);
  e = ex2_f((-0.5f * kLog2e) * z * z);
  const float t = rcp_f(fmaf(0.3275911f * 0.70710678118654752f, x, 1.f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * t * q * e;
  return z >= 0.f ? 1.f - q : q;
}

// act(z); `act` is the same for a whole launch, so the branch is uniform.
__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case GNN_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case GNN_ACT_SILU: return z * sigmoid_f(z);
    case GNN_ACT_GELU: {
      float e;
      return z * phi_f(z, e);
    }
    case GNN_ACT_SIGMOID: return sigmoid_f(z);
    default: return z;
  }
}

// act(z) and act'(z).
__device__ __forceinline__ void act_grad_f(float z, int act, float& a, float& d) {
  switch (act) {
    case GNN_ACT_RELU:
      d = z > 0.f ? 1.f : 0.f;
      a = z > 0.f ? z : (z != z ? z : 0.f);
      break;
    case GNN_ACT_SILU: {
      const float s = sigmoid_f(z);
      a = z * s;
      d = fmaf(a, 1.f - s, s);
      break;
    }
    case GNN_ACT_GELU: {
      float e;
      const float c = phi_f(z, e);
      a = z * c;
      d = fmaf(z * 0.39894228040143268f, e, c);
      break;
    }
    case GNN_ACT_SIGMOID:
      a = sigmoid_f(z);
      d = a * (1.f - a);
      break;
    default:
      a = z;
      d = 1.f;
  }
}

// Runs f with the activation as a compile-time value.
template <class Fn>
__device__ __forceinline__ void with_act(int act, Fn f) {
  switch (act) {
    case GNN_ACT_RELU: f(std::integral_constant<int, GNN_ACT_RELU>()); break;
    case GNN_ACT_SILU: f(std::integral_constant<int, GNN_ACT_SILU>()); break;
    case GNN_ACT_GELU: f(std::integral_constant<int, GNN_ACT_GELU>()); break;
    case GNN_ACT_SIGMOID: f(std::integral_constant<int, GNN_ACT_SIGMOID>()); break;
    default: f(std::integral_constant<int, GNN_ACT_NONE>());
  }
}

}  // namespace gnn
