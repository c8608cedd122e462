// Element types, 16-byte row accesses and activations shared by the node-wise
// operators (group norm, gated projections, AdamW).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.cuh"
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
// formed from them below is compared with one.  In fp32 the backward is off by
// 2e-7 to 7e-7 of a gradient's norm with them (7e-8 to 1e-7 with full-length ones).
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

__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2_f(x.x), ex2_f(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp_f(x.x), rcp_f(x.y)); }

// The activations work on pairs, two operations to an instruction: the kernels
// that use them run short of instructions before bandwidth.

// 1 / (1 + exp(-z)): exp(-z) may reach infinity, whose reciprocal is zero.
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  return rcp_2(add2_rn(ex2_2(mul2_rn(z, dup2(-kLog2e))), dup2(1.f)));
}

// The normal distribution's Phi(z) and e = exp(-z^2/2).  With x = |z|/sqrt 2,
// erfc(x) = t P(t) exp(-x^2), t = 1/(1 + 0.3275911 x): Abramowitz and Stegun
// 7.1.26, absolute error at most 1.5e-7, so at most 7.5e-8 in q = erfc(x)/2;
// Phi = 1/2 + sign(z) (1/2 - q).  It shares its exponential with the derivative
// of gelu.
__device__ __forceinline__ float2 phi2(float2 z, float2& e) {
  e = ex2_2(mul2_rn(mul2_rn(z, dup2(-0.5f * kLog2e)), z));
  const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 t = rcp_2(fma2_rn(dup2(0.3275911f * 0.70710678118654752f), x, dup2(1.f)));
  float2 q = fma2_rn(dup2(0.5f * 1.061405429f), t, dup2(0.5f * -1.453152027f));
  q = fma2_rn(q, t, dup2(0.5f * 1.421413741f));
  q = fma2_rn(q, t, dup2(0.5f * -0.284496736f));
  q = fma2_rn(q, t, dup2(0.5f * 0.254829592f));
  const float2 r = fma2_rn(neg2(mul2_rn(t, q)), e, dup2(0.5f));
  return add2_rn(make_float2(copysignf(r.x, z.x), copysignf(r.y, z.y)), dup2(0.5f));
}

// act(z); `act` is the same for a whole launch, so the branch is uniform.
__device__ __forceinline__ float2 act2(float2 z, int act) {
  switch (act) {
    case GNN_ACT_RELU: return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);  // keeps a NaN
    case GNN_ACT_SILU: return mul2_rn(z, sigmoid2(z));
    case GNN_ACT_GELU: {
      float2 e;
      return mul2_rn(z, phi2(z, e));
    }
    case GNN_ACT_SIGMOID: return sigmoid2(z);
    default: return z;
  }
}
__device__ __forceinline__ float act_f(float z, int act) { return act2(make_float2(z, z), act).x; }

// act(z) and act'(z).
__device__ __forceinline__ void act_grad2(float2 z, int act, float2& a, float2& d) {
  switch (act) {
    case GNN_ACT_RELU:
      d = make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
      a = act2(z, GNN_ACT_RELU);
      break;
    case GNN_ACT_SILU: {
      const float2 s = sigmoid2(z);
      a = mul2_rn(z, s);
      d = fma2_rn(a, fma2_rn(s, dup2(-1.f), dup2(1.f)), s);
      break;
    }
    case GNN_ACT_GELU: {
      float2 e;
      const float2 c = phi2(z, e);
      a = mul2_rn(z, c);
      d = fma2_rn(mul2_rn(z, dup2(0.39894228040143268f)), e, c);
      break;
    }
    case GNN_ACT_SIGMOID:
      a = sigmoid2(z);
      d = fma2_rn(neg2(a), a, a);
      break;
    default:
      a = z;
      d = dup2(1.f);
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
