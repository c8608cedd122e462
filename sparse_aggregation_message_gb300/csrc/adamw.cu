// One AdamW step over many tensors, states in fp32 or in 8 bits, with clipping
// by the global gradient norm.
//
// Three launches at most: the norm's partial sums (only with clipping), one
// block that advances the step count and forms the scalars of this step, and
// the update.  The tensors' descriptors are launch parameters, so nothing is
// copied to the device and nothing about a tensor is kept between calls.
// A warp takes 256 elements at a time, eight a lane: that is one block of an
// 8-bit state, so its largest magnitude is one warp reduction.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "device.cuh"
#include "internal.h"
#include "nodewise.cuh"

namespace gnn {

namespace {

constexpr int BLOCK = 256;      // elements that share a scale, and of one warp step
constexpr int MAX_UNITS = 8;    // blocks a warp takes in a row, at most
constexpr int NORM_UNITS = 4;
constexpr int THREADS = 256;
constexpr int MAX_TENSORS = 56;  // of one launch: the descriptors stay below 4 KB
constexpr int NORM_BLOCKS = 152 * 4;
constexpr float F8_INV = 1.f / 448.f;  // 448: the largest e4m3 value

struct Table {
  int count;
  int units;  // blocks of a chunk, which one warp takes
  int64_t first[MAX_TENSORS + 1];  // first chunk of tensor i
  gnn_adamw_tensor t[MAX_TENSORS];
  uint64_t aligned;  // bit i: every pointer of tensor i suits eight elements a lane
};

struct Hyper {
  float b1, c1, b2, c2, decay, eps;
  bool paired;  // eps <= 2^60: denominators stay in the paired quotient's range
};

// The scalars of a step, formed by begin_kernel.
struct Control {
  float grad;  // what gradients are multiplied by
  float step;  // lr / (1 - beta1^t)
  float fix;   // 1 / sqrt(1 - beta2^t)
  int skip;
};

// The tensor that holds chunk c.
__device__ __forceinline__ int tensor_of(const Table& tab, int64_t c) {
  int lo = 0, hi = tab.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The eight elements of a lane in a 256-element step, as they lie in memory
// (two words a byte of the type).  VEC: consecutive ones, in 16-byte accesses
// where they fit; else every 32nd, one by one, of which `live` exist (the others
// read as zero and are not written).  `p` points at the first.
template <class T, bool VEC>
struct Raw {
  static constexpr int W = 2 * sizeof(T);
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p, int live) {
    if constexpr (VEC) {
      if constexpr (W == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x, w[1] = a.y;
      } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          const uint4 a = reinterpret_cast<const uint4*>(p)[i / 4];
          w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < live) {
          if constexpr (sizeof(T) == 4)
            w[j] = reinterpret_cast<const uint32_t*>(p)[j * 32];
          else if constexpr (sizeof(T) == 2)
            w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j * 32] << (16 * (j & 1));
          else
            w[j >> 2] |= (uint32_t)reinterpret_cast<const uint8_t*>(p)[j * 32] << (8 * (j & 3));
        }
      }
    }
  }
  // From a lane's slot of a ring: parts of 16 bytes (8 for a one-byte type), each
  // for every thread of the block side by side.
  __device__ __forceinline__ void from_ring(const char* part) {
    if constexpr (W == 2) {
      const uint2 a = reinterpret_cast<const uint2*>(part)[threadIdx.x];
      w[0] = a.x, w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 a = reinterpret_cast<const uint4*>(part)[threadIdx.x + i / 4 * THREADS];
        w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
      }
    }
  }
  static __device__ __forceinline__ void to_ring(uint32_t part, const T* p) {
    if constexpr (W == 2) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(part + threadIdx.x * 8), "l"(p) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        // through L1: a lane's two halves of eight fp32 values share a sector (past
        // L1 each half fetched it: 664 against 572 us at 242M elements)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(part + (threadIdx.x + i / 4 * THREADS) * 16),
                     "l"(reinterpret_cast<const char*>(p) + 4 * i)
                     : "memory");
    }
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if constexpr (sizeof(T) == 4) {
        v[j] = __uint_as_float(w[j]), v[j + 1] = __uint_as_float(w[j + 1]);
      } else if constexpr (sizeof(T) == 2) {
        const float2 f = Pack2<T>::from(w[j >> 1]);
        v[j] = f.x, v[j + 1] = f.y;
      } else {  // e4m3 codes
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 2] >> (8 * (j & 3))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[j] = f.x, v[j + 1] = f.y;
      }
    }
  }
};

template <bool VEC, class T>
__device__ __forceinline__ void store8(T* p, int live, const float (&v)[8]) {
  if constexpr (VEC && sizeof(T) == 4) {
    // a whole sector a lane
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else if constexpr (VEC) {
    store_vec<8>(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < live) p[j * 32] = from_f32<T>(v[j]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, int live, const uint32_t (&w)[2]) {
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < live) p[j * 32] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// Codes of a warp's 256 values and their scale, which lane 0 writes; top: the
// largest magnitude of this lane's.  LOW: values above zero keep at least the
// smallest code; `usual`: all of them are above zero, and far from subnormal,
// so what would round to zero is lifted just over half of that code first.
template <bool VEC, bool LOW>
__device__ __forceinline__ void quantise8(const float (&x)[8], float top, bool usual, int live, uint8_t* codes,
                                          float* scale_out) {
  // magnitudes are ordered as their bit patterns are, NaN above all
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  float scale = __fmul_rn(top, F8_INV);
  if (scale < 1.17549435e-38f) scale = 0.f;
  const float inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float2 y = mul2_rn(make_float2(x[j], x[j + 1]), dup2(inv));
    if (LOW && usual) y = make_float2(fmaxf(y.x, 0x1.000002p-10f), fmaxf(y.y, 0x1.000002p-10f));
    uint32_t q = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    if (LOW && !usual && scale > 0.f) {
      if (x[j] > 0.f && (q & 0xffu) == 0) q |= 1u;
      if (x[j + 1] > 0.f && (q & 0xff00u) == 0) q |= 0x100u;
    }
    w[j >> 2] |= q << (8 * (j & 3));
  }
  store8<VEC>(codes, live, w);
  if ((threadIdx.x & 31) == 0) *scale_out = scale;
}

// Smallest and largest of three; a NaN is the largest of any.
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min8(const float (&v)[8]) {
  return min3(min3(min3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])), fabsf(v[3]), fabsf(v[4])),
              min3(fabsf(v[5]), fabsf(v[6]), fabsf(v[7])), __int_as_float(0x7f800000));
}
__device__ __forceinline__ float max8(const float (&v)[8]) {
  return max3_nan(max3_nan(max3_nan(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])), fabsf(v[3]), fabsf(v[4])),
                  max3_nan(fabsf(v[5]), fabsf(v[6]), fabsf(v[7])), 0.f);
}

// Square roots and quotients of pairs, rounded to nearest, for operands whose
// every step below stays normal (the caller checks).  The root is Goldschmidt's
// iteration from an approximate reciprocal root, with h -> 1/(2 sqrt v), and a
// final residual correction (Markstein, "Software division and square root using
// Goldschmidt's algorithms", RNC6, 2004); the quotient is Markstein's method (IBM J. Res.
// Dev. 34(1), 1990): the reciprocal to the last bit by one Newton step, a
// quotient made faithful by one fused residual and rounded correctly by the
// next.  Two operations to an instruction: the update had 70 instructions an
// element with the scalar root and quotient and issue was as scarce as
// bandwidth in the 8-bit form.
__device__ __forceinline__ float2 sqrt2_rn(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  float2 g = mul2_rn(v, y), h = mul2_rn(dup2(0.5f), y);
  const float2 e = fma2_rn(make_float2(-h.x, -h.y), g, dup2(0.5f));
  g = fma2_rn(g, e, g);
  h = fma2_rn(h, e, h);
  return fma2_rn(fma2_rn(make_float2(-g.x, -g.y), g, v), h, g);
}
__device__ __forceinline__ float2 quot2_rn(float2 a, float2 b) {
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(b.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(b.y));
  const float2 nb = make_float2(-b.x, -b.y);
  y = fma2_rn(fma2_rn(nb, y, dup2(1.f)), y, y);
  float2 q = mul2_rn(a, y);
  q = fma2_rn(fma2_rn(nb, q, a), y, q);
  return fma2_rn(fma2_rn(nb, q, a), y, q);
}

// One tensor's arrays at a lane's first element of a step, and what the step
// reads of them.
template <class TP, class TG, bool Q8, bool VEC>
struct Step {
  using TS = typename std::conditional<Q8, uint8_t, float>::type;
  Raw<TP, VEC> p;
  Raw<TG, VEC> g;
  Raw<TS, VEC> m, v;
  float ms, vs;
  // bytes of the parts of a ring slot
  static constexpr int P = THREADS * 8 * sizeof(TP), G = THREADS * 8 * sizeof(TG), S = THREADS * 8 * sizeof(TS);
  static constexpr int SLOT = P + G + 2 * S;
  __device__ __forceinline__ void from_ring(const char* slot) {
    p.from_ring(slot), g.from_ring(slot + P), m.from_ring(slot + P + G), v.from_ring(slot + P + G + S);
  }
};
template <class TP, class TG, bool Q8>
struct At {
  using TS = typename std::conditional<Q8, uint8_t, float>::type;
  TP* p;
  const TG* g;
  TS *m, *v;
  float *ms, *vs;
  __nv_bfloat16* copy;
  __device__ __forceinline__ At(const gnn_adamw_tensor& t, int64_t base, int64_t at)
      : p(static_cast<TP*>(t.param) + at), g(static_cast<const TG*>(t.grad) + at), m(static_cast<TS*>(t.m) + at),
        v(static_cast<TS*>(t.v) + at), ms(Q8 ? t.m_scale + base / BLOCK : nullptr),
        vs(Q8 ? t.v_scale + base / BLOCK : nullptr),
        copy(t.copy ? reinterpret_cast<__nv_bfloat16*>(t.copy) + at : nullptr) {}
  // step u of a chunk
  template <bool VEC>
  __device__ __forceinline__ void load(Step<TP, TG, Q8, VEC>& s, int u, int live) const {
    s.p.load(p + u * BLOCK, live);
    s.g.load(g + u * BLOCK, live);
    s.m.load(m + u * BLOCK, live);
    s.v.load(v + u * BLOCK, live);
    if (Q8) s.ms = ms[u], s.vs = vs[u];
  }
  __device__ __forceinline__ void to_ring(uint32_t slot, int u) const {
    using S = Step<TP, TG, Q8, true>;
    Raw<TP, true>::to_ring(slot, p + u * BLOCK);
    Raw<TG, true>::to_ring(slot + S::P, g + u * BLOCK);
    Raw<TS, true>::to_ring(slot + S::P + S::G, m + u * BLOCK);
    Raw<TS, true>::to_ring(slot + S::P + S::G + S::S, v + u * BLOCK);
  }
};

template <class TP, class TG, bool Q8, bool VEC>
__device__ __forceinline__ void update(const Step<TP, TG, Q8, VEC>& now, const At<TP, TG, Q8>& at, int u, int live,
                                       const Hyper& h, const Control& c) {
  float p[8], g[8], m[8], v[8];
  now.p.to(p), now.g.to(g), now.m.to(m), now.v.to(v);
  // A product that feeds a sum stays scalar: in paired form the two may be
  // contracted into one fused operation.
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    if (Q8) {
      const float2 a = mul2_rn(make_float2(m[j], m[j + 1]), dup2(now.ms));
      float2 b = mul2_rn(make_float2(v[j], v[j + 1]), dup2(now.vs));
      b = mul2_rn(b, b);
      m[j] = a.x, m[j + 1] = a.y, v[j] = b.x, v[j + 1] = b.y;
    }
    const float2 gs = mul2_rn(make_float2(g[j], g[j + 1]), dup2(c.grad));
    const float2 gc = mul2_rn(gs, dup2(h.c2));
    m[j] = __fadd_rn(__fmul_rn(m[j], h.b1), __fmul_rn(gs.x, h.c1));
    m[j + 1] = __fadd_rn(__fmul_rn(m[j + 1], h.b1), __fmul_rn(gs.y, h.c1));
    v[j] = __fadd_rn(__fmul_rn(v[j], h.b2), __fmul_rn(gc.x, gs.x));
    v[j + 1] = __fadd_rn(__fmul_rn(v[j + 1], h.b2), __fmul_rn(gc.y, gs.y));
  }
  // v in [2^-80, 2^80] and |m| in [2^-50, 2^50] leave every step of the paired
  // root and quotient normal (sqrt(v)/sqrt(1 - beta2^t) + eps lies in
  // [2^-40, 2^68]); where a lane has zeros, NaN or what is outside, its warp
  // takes the scalar ones
  const float mtop = max8(m), vtop = max8(v);
  const bool usual = __all_sync(0xffffffffu, h.paired && mtop <= 0x1p50f && vtop <= 0x1p80f &&
                                                 min8(m) >= 0x1p-50f && min8(v) >= 0x1p-80f);
  if (usual) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 s = sqrt2_rn(make_float2(v[j], v[j + 1]));
      const float2 q = quot2_rn(make_float2(m[j], m[j + 1]), make_float2(__fadd_rn(__fmul_rn(s.x, c.fix), h.eps),
                                                                         __fadd_rn(__fmul_rn(s.y, c.fix), h.eps)));
      const float2 d = mul2_rn(dup2(c.step), q);
      p[j] = __fsub_rn(__fmul_rn(p[j], h.decay), d.x);
      p[j + 1] = __fsub_rn(__fmul_rn(p[j + 1], h.decay), d.y);
      if (Q8) v[j] = s.x, v[j + 1] = s.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = __fsqrt_rn(v[j]);
      const float q = __fdiv_rn(m[j], __fadd_rn(__fmul_rn(s, c.fix), h.eps));
      p[j] = __fsub_rn(__fmul_rn(p[j], h.decay), __fmul_rn(c.step, q));
      if (Q8) v[j] = s;
    }
  }
  store8<VEC>(at.p + u * BLOCK, live, p);
  if (at.copy) store8<VEC>(at.copy + u * BLOCK, live, p);
  if constexpr (Q8) {
    quantise8<VEC, false>(m, mtop, usual, live, at.m + u * BLOCK, at.ms + u);
    quantise8<VEC, true>(v, __fsqrt_rn(vtop), usual, live, at.v + u * BLOCK, at.vs + u);
  } else {
    store8<VEC>(at.m + u * BLOCK, live, m);
    store8<VEC>(at.v + u * BLOCK, live, v);
  }
}

// With 8-bit states a lane's next steps are copied into its own slots of shared
// memory AHEAD steps before their use (no barrier: each lane reads what it
// copied); registers alone could hold one step ahead.  242M elements take 572 us,
// 6.8 TB/s.  With fp32 states 24 warps of plain loads reach the bandwidth (184M
// elements in 736 us, 7.0 TB/s), and holding a step ahead in registers spilt and
// lost 7%.
constexpr int AHEAD = 2;
template <class TP, class TG, bool Q8>
constexpr int ring_bytes() {
  return Q8 ? (AHEAD + 1) * Step<TP, TG, Q8, true>::SLOT : 0;
}

template <class TP, class TG, bool Q8>
__global__ void __launch_bounds__(THREADS, 3)
    adamw_kernel(const __grid_constant__ Table tab, const Hyper h, const Control* ctl) {
  extern __shared__ __align__(16) char slots[];
  cudaGridDependencySynchronize();
  const Control c = *ctl;
  if (c.skip) return;
  const int lane = threadIdx.x & 31;
  const int64_t chunks = tab.first[tab.count];
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  for (int64_t k = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); k < chunks; k += warps) {
    const int i = tensor_of(tab, k);
    const gnn_adamw_tensor& t = tab.t[i];
    const int64_t base = (k - tab.first[i]) * (tab.units * BLOCK), left = t.n - base;
    // whole steps of an aligned tensor, then what remains
    const int whole = (tab.aligned >> i & 1) ? (int)min(left / BLOCK, (int64_t)tab.units) : 0;
    if (whole) {
      const At<TP, TG, Q8> at(t, base, base + lane * 8);
      Step<TP, TG, Q8, true> now;
      if constexpr (Q8) {
        // lanes 0-15 hold the chunk's scales of m, 16-31 those of v
        static_assert(MAX_UNITS <= 16, "a scale to a lane");
        float scale = 0.f;
        if ((lane & 15) < whole) scale = lane < 16 ? at.ms[lane] : at.vs[lane - 16];
        const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
        constexpr int SLOT = Step<TP, TG, Q8, true>::SLOT;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (u < whole) at.to_ring(ring + u * SLOT, u);
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int use = 0, fill = AHEAD * SLOT;
#pragma unroll 1
        for (int u = 0; u < whole; ++u) {
          asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
          now.from_ring(slots + use);
          now.ms = __shfl_sync(0xffffffffu, scale, u);
          now.vs = __shfl_sync(0xffffffffu, scale, 16 + u);
          if (u + AHEAD < whole) at.to_ring(ring + fill, u + AHEAD);
          asm volatile("cp.async.commit_group;" ::: "memory");
          fill = use;  // used up before the next step's copies go there
          use = use == AHEAD * SLOT ? 0 : use + SLOT;
          update(now, at, u, 8, h, c);
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < whole; ++u) {
          at.load(now, u, 8);
          update(now, at, u, 8, h, c);
        }
      }
    }
    if (whole < tab.units && left > whole * BLOCK) {
      const At<TP, TG, Q8> at(t, base, base + lane);
#pragma unroll 1
      for (int u = whole; u < tab.units && left > u * BLOCK; ++u) {
        const int64_t mine = left - u * BLOCK - lane;  // elements from this lane's first one on
        const int live = mine <= 0 ? 0 : (int)min((mine + 31) / 32, (int64_t)8);
        Step<TP, TG, Q8, false> now;
        at.load(now, u, live);
        update(now, at, u, live, h, c);
      }
    }
  }
}

__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < THREADS / 32; ++w) s += sm[w];
  return s;
}

// A lane's 32 squares of a chunk are added in fp32, chunks in fp64 (with eight
// squares to an fp64 addition the fp64 pipe was 73% busy); where the 32 leave
// the range that fp32 holds well, they are formed again in fp64.
template <class TG, bool VEC>
__device__ __forceinline__ double squares(const Raw<TG, VEC> (&raw)[NORM_UNITS]) {
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < NORM_UNITS; ++u) {
    float g[8];
    raw[u].to(g);
    s += ((g[0] * g[0] + g[1] * g[1]) + (g[2] * g[2] + g[3] * g[3])) +
         ((g[4] * g[4] + g[5] * g[5]) + (g[6] * g[6] + g[7] * g[7]));
  }
  if (s > 1e-28f && s < 1e38f) return (double)s;
  double d = 0;
#pragma unroll
  for (int u = 0; u < NORM_UNITS; ++u) {
    float g[8];
    raw[u].to(g);
#pragma unroll
    for (int j = 0; j < 8; ++j) d += (double)g[j] * (double)g[j];
  }
  return d;
}

// Partial sums of g^2, one per block; the first `have` of them hold those of
// earlier launches.
template <class TG>
__global__ void __launch_bounds__(THREADS) norm_kernel(const __grid_constant__ Table tab, double* partial,
                                                       int have) {
  __shared__ double sm[THREADS / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31;
  const int64_t chunks = tab.first[tab.count];
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  double sum = 0;
  for (int64_t k = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); k < chunks; k += warps) {
    const int i = tensor_of(tab, k);
    const gnn_adamw_tensor& t = tab.t[i];
    const int64_t base = (k - tab.first[i]) * (NORM_UNITS * BLOCK), left = t.n - base;
    const TG* g = static_cast<const TG*>(t.grad) + base;
    if ((tab.aligned >> i & 1) && left >= NORM_UNITS * BLOCK) {
      Raw<TG, true> raw[NORM_UNITS];
#pragma unroll
      for (int u = 0; u < NORM_UNITS; ++u) raw[u].load(g + u * BLOCK + lane * 8, 8);
      sum += squares(raw);
    } else {
      Raw<TG, false> raw[NORM_UNITS];
#pragma unroll
      for (int u = 0; u < NORM_UNITS; ++u) {
        const int64_t mine = left - u * BLOCK - lane;
        raw[u].load(g + u * BLOCK + lane, mine <= 0 ? 0 : (int)min((mine + 31) / 32, (int64_t)8));
      }
      sum += squares(raw);
    }
  }
  const double total = block_sum(sum, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = total + ((int)blockIdx.x < have ? partial[blockIdx.x] : 0.0);
}

// The scalars of this step, and the step count's advance.
__global__ void __launch_bounds__(THREADS)
    begin_kernel(const double* partial, int n_partial, gnn_adamw_state* state, double lr, double beta1,
                 double beta2, double grad_scale, double max_norm, float* grad_norm, Control* ctl) {
  // max_norm 0: there are no partials, and no norm
  __shared__ double sm[THREADS / 32];
  __shared__ float scalars[2];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  // what the norm has no part in, one thread each
  double power = 0;
  if (threadIdx.x == 32) {
    power = state->beta1_pow * beta1;
    scalars[0] = (float)(lr / (1.0 - power));
  } else if (threadIdx.x == 64) {
    power = state->beta2_pow * beta2;
    scalars[1] = (float)(1.0 / sqrt(1.0 - power));
  }
  double sum = 0;
  for (int i = threadIdx.x; i < n_partial; i += THREADS) sum += partial[i];
  sum = block_sum(sum, sm);
  __shared__ int skip;
  if (threadIdx.x == 0) {
    Control c{(float)grad_scale, scalars[0], scalars[1], 0};
    if (max_norm > 0) {
      const double norm = fabs(grad_scale) * sqrt(sum);
      if (grad_norm) *grad_norm = (float)norm;
      if (!isfinite(norm))
        c.skip = 1;
      else if (isfinite(max_norm))
        c.grad = (float)(grad_scale * (max_norm / fmax(norm + 1e-6, max_norm)));
    }
    *ctl = c;
    if (c.skip)
      state->skipped += 1.0;
    else
      state->steps += 1.0;
    skip = c.skip;
  }
  __syncthreads();
  if (skip) return;
  if (threadIdx.x == 32) state->beta1_pow = power;
  if (threadIdx.x == 64) state->beta2_pow = power;
}

bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Every launch may start while the kernel before it ends, and waits for that
// before it touches memory.
template <class... P, class... A>
gnn_status launch(cudaStream_t st, int64_t grid, size_t smem, void (*k)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launch();
  GNN_CUDA(cudaLaunchKernelEx(&cfg, k, args...));
  return GNN_OK;
}

using Update = gnn_status (*)(cudaStream_t, int64_t, const Table&, const Hyper&, const Control*);

template <class TP, class TG, bool Q8>
gnn_status launch_update(cudaStream_t st, int64_t grid, const Table& tab, const Hyper& h,
                         const Control* ctl) {
  constexpr int smem = ring_bytes<TP, TG, Q8>();
  static PerDevice done;
  const gnn_status s = allow_smem(adamw_kernel<TP, TG, Q8>, smem, done);
  if (s != GNN_OK) return s;
  return launch(st, grid, smem, adamw_kernel<TP, TG, Q8>, tab, h, ctl);
}
template <class TP, class TG>
Update update_for(bool q8) {
  return q8 ? launch_update<TP, TG, true> : launch_update<TP, TG, false>;
}
template <class TP>
Update update_for(int gt, bool q8) {
  if (gt == GNN_BF16) return update_for<TP, __nv_bfloat16>(q8);
  if (gt == GNN_F16) return update_for<TP, __half>(q8);
  return update_for<TP, float>(q8);
}

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_adamw_workspace(size_t* ws_bytes) {
  GNN_REQUIRE(ws_bytes, "gnn_adamw_workspace: NULL ws_bytes");
  *ws_bytes = 256 + sizeof(double) * NORM_BLOCKS;
  return GNN_OK;
}

extern "C" gnn_status gnn_adamw_step(const gnn_adamw_tensor* tensors, int32_t n_tensors,
                                     int32_t param_type, int32_t grad_type, int32_t state_bits,
                                     gnn_adamw_state* state, double lr, double beta1, double beta2,
                                     double eps, double weight_decay, double grad_scale,
                                     double max_norm, float* grad_norm, void* ws, size_t ws_bytes,
                                     gnn_stream_t stream) {
  GNN_REQUIRE(n_tensors >= 0 && (tensors || n_tensors == 0), "gnn_adamw_step: bad tensor list");
  GNN_REQUIRE(is_type(grad_type), "gnn_adamw_step: unknown grad_type");
  if (param_type != GNN_F32 && param_type != GNN_BF16)
    return fail(GNN_ERR_UNSUPPORTED, "gnn_adamw_step: parameters are fp32 or bf16");
  GNN_REQUIRE(state_bits == 8 || state_bits == 32, "gnn_adamw_step: state_bits is 8 or 32");
  GNN_REQUIRE(state && aligned_to(state, 8), "gnn_adamw_step: bad state");
  GNN_REQUIRE(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1, "gnn_adamw_step: betas lie in [0, 1)");
  GNN_REQUIRE(std::isfinite(lr) && std::isfinite(weight_decay) && std::isfinite(grad_scale) && eps >= 0 &&
                  std::isfinite(eps), "gnn_adamw_step: lr, eps, weight_decay or grad_scale out of range");
  GNN_REQUIRE(max_norm >= 0, "gnn_adamw_step: max_norm is 0 (no clipping) or positive");
  GNN_REQUIRE(aligned_to(grad_norm, 4), "gnn_adamw_step: misaligned grad_norm");
  size_t need;
  gnn_adamw_workspace(&need);
  GNN_REQUIRE(ws && aligned_to(ws, 8) && ws_bytes >= need, "gnn_adamw_step: workspace too small (%zu < %zu)",
              ws_bytes, need);
  const bool q8 = state_bits == 8;
  const uintptr_t ps = type_size(param_type), gs = type_size(grad_type);
  for (int i = 0; i < n_tensors; ++i) {
    const gnn_adamw_tensor& t = tensors[i];
    GNN_REQUIRE(t.n >= 0, "gnn_adamw_step: tensor %d has a negative size", i);
    if (t.n == 0) continue;
    GNN_REQUIRE(t.param && t.grad && t.m && t.v && (!q8 || (t.m_scale && t.v_scale)),
                "gnn_adamw_step: tensor %d has a NULL array", i);
    GNN_REQUIRE(aligned_to(t.param, ps) && aligned_to(t.grad, gs) && aligned_to(t.copy, 2) &&
                    (q8 || (aligned_to(t.m, 4) && aligned_to(t.v, 4))) && aligned_to(t.m_scale, 4) &&
                    aligned_to(t.v_scale, 4), "gnn_adamw_step: tensor %d has a misaligned array", i);
  }
  cudaStream_t st = as_stream(stream);
  Control* ctl = static_cast<Control*>(ws);
  double* partial = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  const Hyper h{(float)beta1, (float)(1.0 - beta1), (float)beta2, (float)(1.0 - beta2),
                (float)(1.0 - lr * weight_decay), (float)eps, eps <= 0x1p60};
  const Update update = param_type == GNN_F32 ? update_for<float>(grad_type, q8)
                                              : update_for<__nv_bfloat16>(grad_type, q8);
  auto* norm = grad_type == GNN_BF16 ? norm_kernel<__nv_bfloat16>
               : grad_type == GNN_F16 ? norm_kernel<__half> : norm_kernel<float>;
  // the launches a pass over all tensors takes: tables of up to MAX_TENSORS
  auto each = [&](int units, auto&& run) -> gnn_status {
    Table tab;
    tab.units = units;
    const int64_t chunk = (int64_t)units * BLOCK;
    int i = 0;
    while (i < n_tensors) {
      tab.count = 0;
      tab.aligned = 0;
      tab.first[0] = 0;
      for (; i < n_tensors && tab.count < MAX_TENSORS; ++i) {
        const gnn_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        const int k = tab.count++;
        tab.t[k] = t;
        tab.first[k + 1] = tab.first[k] + (t.n + chunk - 1) / chunk;
        if (aligned_to(t.param, 8 * ps) && aligned_to(t.grad, 16) && aligned_to(t.m, q8 ? 8 : 32) &&
            aligned_to(t.v, q8 ? 8 : 32) && aligned_to(t.copy, 16))
          tab.aligned |= 1ull << k;
      }
      if (tab.count == 0) break;
      const gnn_status s = run(tab);
      if (s != GNN_OK) return s;
    }
    return GNN_OK;
  };
  auto grid_for = [](const Table& tab, int64_t most) {
    const int64_t blocks = (tab.first[tab.count] + THREADS / 32 - 1) / (THREADS / 32);
    return blocks < most ? blocks : most;
  };
  int n_partial = 0;
  if (max_norm > 0) {
    const gnn_status s = each(NORM_UNITS, [&](const Table& tab) -> gnn_status {
      // each launch has the blocks that its own tensors need (on the first's, sixty
      // of 64 elements before one of 30M made a step of 171 us take 598)
      const int64_t grid = grid_for(tab, NORM_BLOCKS);
      const gnn_status r = launch(st, grid, 0, norm, tab, partial, n_partial);
      n_partial = grid > n_partial ? (int)grid : n_partial;
      return r;
    });
    if (s != GNN_OK) return s;
  }
  gnn_status s = launch(st, 1, 0, begin_kernel, (const double*)partial, n_partial, state, lr,
                        beta1, beta2, grad_scale, max_norm, grad_norm, ctl);
  if (s != GNN_OK) return s;
  // A chunk is what a warp takes in a row: long enough to fill its ring, short
  // enough that every warp of the card has a few.
  int64_t blocks = 0;
  for (int i = 0; i < n_tensors; ++i) blocks += (tensors[i].n + BLOCK - 1) / BLOCK;
  const int64_t share = blocks / (152 * 3 * (THREADS / 32) * 4);
  const int units = share < 1 ? 1 : share > MAX_UNITS ? MAX_UNITS : (int)share;
  return each(units, [&](const Table& tab) { return update(st, grid_for(tab, 152 * 3 * 16), tab, h, ctl); });
}
