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

#include "internal.h"
#include "nodewise.cuh"

namespace gnn {

namespace {

constexpr int BLOCK = 256;      // elements that share a scale, and of one warp step
constexpr int CHUNK = 4 * BLOCK;  // elements a warp takes at a time
constexpr int THREADS = 256;
constexpr int MAX_TENSORS = 56;  // of one launch: the descriptors stay below 4 KB
constexpr int NORM_BLOCKS = 152 * 4;
constexpr float F8_MAX = 448.f;

struct Table {
  int count;
  int64_t first[MAX_TENSORS + 1];  // first chunk of tensor i
  gnn_adamw_tensor t[MAX_TENSORS];
  uint64_t aligned;  // bit i: every pointer of tensor i suits eight elements a lane
};

struct Hyper {
  float b1, c1, b2, c2, decay, eps;
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

// Eight elements of a 256-element step: consecutive ones where the tensor is
// aligned and the step is full, else every 32nd, one by one (elements past the
// end read as zero and are not written).
struct Lane {
  int64_t at;  // element of j = 0
  int stride;  // to the next j
  int live;    // how many of the eight exist
  bool vec;
  __device__ __forceinline__ Lane(int64_t base, int64_t n, bool aligned) {
    const int lane = threadIdx.x & 31;
    vec = aligned && base + BLOCK <= n;
    at = base + (vec ? lane * 8 : lane);
    stride = vec ? 1 : 32;
    live = vec ? 8 : at < n ? (int)min((int64_t)8, (n - at + 31) / 32) : 0;
  }
};

template <class T>
__device__ __forceinline__ void load8(const T* p, const Lane& l, float (&v)[8]) {
  if (l.vec) {
    load_vec<8>(p + l.at, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < l.live ? to_f32(p[l.at + j * 32]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const Lane& l, const float (&v)[8]) {
  if (l.vec) {
    store_vec<8>(p + l.at, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < l.live) p[l.at + j * 32] = from_f32<T>(v[j]);
  }
}
// e4m3 codes
__device__ __forceinline__ void load8(const uint8_t* p, const Lane& l, float (&v)[8]) {
  uint32_t w[2] = {0, 0};
  if (l.vec) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + l.at);
    w[0] = a.x, w[1] = a.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < l.live) w[j >> 2] |= (uint32_t)p[l.at + j * 32] << (8 * (j & 3));
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 2] >> (8 * (j & 3))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[j] = f.x, v[j + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(uint8_t* p, const Lane& l, const uint32_t (&w)[2]) {
  if (l.vec) {
    *reinterpret_cast<uint2*>(p + l.at) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < l.live) p[l.at + j * 32] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// Codes of a warp's 256 values and their scale, which lane 0 writes.  `low`:
// values above zero keep at least the smallest code.
template <bool LOW>
__device__ __forceinline__ void quantise8(const float (&x)[8], const Lane& l, uint8_t* codes, float* scale_out) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = fabsf(x[j]);
    top = m > top || m != m ? m : top;
  }
  // magnitudes are ordered as their bit patterns are, NaN above all
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  float scale = __fdiv_rn(top, F8_MAX);
  if (scale < 1.17549435e-38f) scale = 0.f;
  const float inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[j], inv), __fmul_rn(x[j + 1], inv)),
                                          __NV_SATFINITE, __NV_E4M3);
    if (LOW && scale > 0.f) {
      if (x[j] > 0.f && (q & 0xffu) == 0) q |= 1u;
      if (x[j + 1] > 0.f && (q & 0xff00u) == 0) q |= 0x100u;
    }
    w[j >> 2] |= q << (8 * (j & 3));
  }
  store8(codes, l, w);
  if ((threadIdx.x & 31) == 0) *scale_out = scale;
}

template <class TP, class TG, bool Q8>
__global__ void __launch_bounds__(THREADS, 3)
    adamw_kernel(const __grid_constant__ Table tab, const Hyper h, const Control* ctl) {
  cudaGridDependencySynchronize();
  const Control c = *ctl;
  if (c.skip) return;
  const int64_t chunks = tab.first[tab.count];
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  for (int64_t k = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); k < chunks; k += warps) {
    const int i = tensor_of(tab, k);
    const gnn_adamw_tensor& t = tab.t[i];
    const bool aligned = tab.aligned >> i & 1;
    const int64_t b0 = (k - tab.first[i]) * CHUNK;
    for (int64_t base = b0; base < min(b0 + CHUNK, t.n); base += BLOCK) {
      const Lane l(base, t.n, aligned);
      float p[8], g[8], m[8], v[8];
      load8(static_cast<const TP*>(t.param), l, p);
      load8(static_cast<const TG*>(t.grad), l, g);
      if constexpr (Q8) {
        load8(static_cast<const uint8_t*>(t.m), l, m);
        load8(static_cast<const uint8_t*>(t.v), l, v);
        const float ms = t.m_scale[base / BLOCK], vs = t.v_scale[base / BLOCK];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = __fmul_rn(m[j], ms);
          v[j] = __fmul_rn(v[j], vs);
          v[j] = __fmul_rn(v[j], v[j]);
        }
      } else {
        load8(static_cast<const float*>(t.m), l, m);
        load8(static_cast<const float*>(t.v), l, v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gs = __fmul_rn(g[j], c.grad);
        m[j] = __fadd_rn(__fmul_rn(m[j], h.b1), __fmul_rn(gs, h.c1));
        v[j] = __fadd_rn(__fmul_rn(v[j], h.b2), __fmul_rn(__fmul_rn(gs, h.c2), gs));
        const float root = __fsqrt_rn(v[j]);
        const float den = __fadd_rn(__fmul_rn(root, c.fix), h.eps);
        p[j] = __fsub_rn(__fmul_rn(p[j], h.decay), __fmul_rn(c.step, __fdiv_rn(m[j], den)));
        if (Q8) v[j] = root;
      }
      store8(static_cast<TP*>(t.param), l, p);
      if (t.copy) store8(reinterpret_cast<__nv_bfloat16*>(t.copy), l, p);
      if constexpr (Q8) {
        quantise8<false>(m, l, static_cast<uint8_t*>(t.m), t.m_scale + base / BLOCK);
        quantise8<true>(v, l, static_cast<uint8_t*>(t.v), t.v_scale + base / BLOCK);
      } else {
        store8(static_cast<float*>(t.m), l, m);
        store8(static_cast<float*>(t.v), l, v);
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

// Partial sums of g^2, one per block.  Eight squares are added in fp32 and the
// eights in fp64 (fp64 rates are low); where eight squares leave the range
// that fp32 holds well, they are formed again in fp64.
template <class TG>
__global__ void __launch_bounds__(THREADS) norm_kernel(const __grid_constant__ Table tab, double* partial,
                                                       int add) {
  __shared__ double sm[THREADS / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t chunks = tab.first[tab.count];
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  double sum = 0;
  for (int64_t k = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); k < chunks; k += warps) {
    const int i = tensor_of(tab, k);
    const gnn_adamw_tensor& t = tab.t[i];
    const bool aligned = tab.aligned >> i & 1;
    const int64_t b0 = (k - tab.first[i]) * CHUNK;
    for (int64_t base = b0; base < min(b0 + CHUNK, t.n); base += BLOCK) {
      const Lane l(base, t.n, aligned);
      float g[8];
      load8(static_cast<const TG*>(t.grad), l, g);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += g[j] * g[j];
      if (s > 1e-30f && s < 1e38f) {
        sum += (double)s;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += (double)g[j] * (double)g[j];
      }
    }
  }
  const double total = block_sum(sum, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = total + (add ? partial[blockIdx.x] : 0.0);
}

// The scalars of this step, and the step count's advance.
__global__ void __launch_bounds__(THREADS)
    begin_kernel(const double* partial, int n_partial, gnn_adamw_state* state, double lr, double beta1,
                 double beta2, double grad_scale, double max_norm, float* grad_norm, Control* ctl) {
  // max_norm 0: there are no partials, and no norm
  __shared__ double sm[THREADS / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  double sum = 0;
  for (int i = threadIdx.x; i < n_partial; i += THREADS) sum += partial[i];
  sum = block_sum(sum, sm);
  if (threadIdx.x != 0) return;
  Control c{(float)grad_scale, 0.f, 0.f, 0};
  if (max_norm > 0) {
    const double norm = fabs(grad_scale) * sqrt(sum);
    if (grad_norm) *grad_norm = (float)norm;
    if (!isfinite(norm)) {
      c.skip = 1;
      state->skipped += 1.0;
    } else if (isfinite(max_norm)) {
      c.grad = (float)(grad_scale * (max_norm / fmax(norm + 1e-6, max_norm)));
    }
  }
  if (!c.skip) {
    const double p1 = state->beta1_pow * beta1, p2 = state->beta2_pow * beta2;
    c.step = (float)(lr / (1.0 - p1));
    c.fix = (float)(1.0 / sqrt(1.0 - p2));
    state->steps += 1.0;
    state->beta1_pow = p1;
    state->beta2_pow = p2;
  }
  *ctl = c;
}

bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <class TP, class TG, bool Q8>
void (*update_kernel())(const Table, const Hyper, const Control*) {
  return adamw_kernel<TP, TG, Q8>;
}
template <class TP, class TG>
void (*update_kernel(bool q8))(const Table, const Hyper, const Control*) {
  return q8 ? update_kernel<TP, TG, true>() : update_kernel<TP, TG, false>();
}
template <class TP>
void (*update_kernel(int gt, bool q8))(const Table, const Hyper, const Control*) {
  if (gt == GNN_BF16) return update_kernel<TP, __nv_bfloat16>(q8);
  if (gt == GNN_F16) return update_kernel<TP, __half>(q8);
  return update_kernel<TP, float>(q8);
}

template <class... P, class... A>
gnn_status launch(cudaStream_t st, bool after, int64_t grid, void (*k)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 1 : 0;
  count_launch();
  GNN_CUDA(cudaLaunchKernelEx(&cfg, k, args...));
  return GNN_OK;
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
                (float)(1.0 - lr * weight_decay), (float)eps};
  auto* update = param_type == GNN_F32 ? update_kernel<float>(grad_type, q8)
                                       : update_kernel<__nv_bfloat16>(grad_type, q8);
  auto* norm = grad_type == GNN_BF16 ? norm_kernel<__nv_bfloat16>
               : grad_type == GNN_F16 ? norm_kernel<__half> : norm_kernel<float>;
  // the launches a pass over all tensors takes: tables of up to MAX_TENSORS
  auto each = [&](auto&& run) -> gnn_status {
    Table tab;
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
        tab.first[k + 1] = tab.first[k] + (t.n + CHUNK - 1) / CHUNK;
        if (aligned_to(t.param, 16) && aligned_to(t.grad, 16) && aligned_to(t.m, q8 ? 8 : 16) &&
            aligned_to(t.v, q8 ? 8 : 16) && aligned_to(t.copy, 16))
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
    const gnn_status s = each([&](const Table& tab) -> gnn_status {
      // every launch writes or adds to all partials of the first's grid
      const int64_t grid = n_partial ? n_partial : grid_for(tab, NORM_BLOCKS);
      const gnn_status r = launch(st, false, grid, norm, tab, partial, n_partial ? 1 : 0);
      n_partial = (int)grid;
      return r;
    });
    if (s != GNN_OK) return s;
  }
  gnn_status s = launch(st, n_partial > 0, 1, begin_kernel, (const double*)partial, n_partial, state, lr,
                        beta1, beta2, grad_scale, max_norm, grad_norm, ctl);
  if (s != GNN_OK) return s;
  bool first = true;
  return each([&](const Table& tab) -> gnn_status {
    const gnn_status r = launch(st, first, grid_for(tab, 152 * 3 * 4), update, tab, h, (const Control*)ctl);
    first = false;
    return r;
  });
}
