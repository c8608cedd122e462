// The residual sum between two blocks, with the norms around it:
//   H = R + s act(G) z,  z = w_post norm_post(B) + b_post
//   Y = w_pre norm_pre(H) + b_pre
// and its backward, row by row.  Every matrix is read once and written once; what
// bounds both passes is DRAM.
//
// A row belongs to a group of L lanes with K times eight channels each in registers,
// so that a row's statistics, its sum and the second norm need one read: 4 to 32
// lanes of a warp (several rows to a warp when rows are short) and K of 1 to 4, or
// several warps that add through shared memory (shape_for says when).  The rows ahead
// arrive in a ring in shared memory by asynchronous copies; each lane copies and reads
// its own pieces, so the ring has no barriers.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "internal.h"
#include "nodewise.cuh"

namespace gnn {

namespace {

constexpr int THREADS = 256;  // of a block; rows of more than 256 lanes: one row's
constexpr int FEW = 128;      // where a lane has more than one vector
constexpr int MAX_LANES = 512;
constexpr int MAX_C = 8 * MAX_LANES;

struct Args {
  const void *B, *R, *G;  // branch, stream, gate
  const void *dH, *dY;
  void *H, *Y;            // forward: outputs; backward: H is read
  void *dR, *dB, *dG;
  int64_t ldb, ldr, ldg, ldh, ldy, lddh, lddr, lddb, lddg;
  int64_t n;
  int C, lanes;
  int gate;               // 0: none, 1: one value a row, 2: a matrix
  int act, post, pre;
  const float *w_post, *b_post, *scale, *w_pre, *b_pre;
  int scale_cols;         // 0, 1 or C
  float eps, inv_c;
  float4* stats;
  float* part;            // backward: [blocks][4][8 lanes K]
  float* part_lo;         // where a lane has more than CHAIN rows: what the sums over its chains lost, else NULL
  double* part_s;         // backward, one learned scale: every block's share of its gradient, or NULL
  int want_q, want_p;     // backward: which sums over all rows are kept
  int64_t rounds, rest;   // backward: whole rounds of a row for every group of the grid, and rows left
  // the ring: stages, 16-byte pieces of a lane in one, and where each matrix's begin
  int stages, pieces, at[5];
};

// ------------------------------------------------------- eight channels a lane
// Two fours of channels: side by side where every matrix is of a 2-byte type (one
// 16-byte access each), else 4 lanes apart (SPLIT), so that a warp's 16 bytes of fp32
// a lane lie side by side as well (in pairs 32 bytes apart 200,000 x 602 forward in
// fp32 took 763 us).
using Eight = float2[4];

// Channels of the row from each of the two fours' first on.
struct Left {
  int a, b;
};

__device__ __forceinline__ void mask(Eight& x, Left m) {
  if (m.a < 4 || m.b < 4) {
    x[0] = make_float2(m.a > 0 ? x[0].x : 0.f, m.a > 1 ? x[0].y : 0.f);
    x[1] = make_float2(m.a > 2 ? x[1].x : 0.f, m.a > 3 ? x[1].y : 0.f);
    x[2] = make_float2(m.b > 0 ? x[2].x : 0.f, m.b > 1 ? x[2].y : 0.f);
    x[3] = make_float2(m.b > 2 ? x[3].x : 0.f, m.b > 3 ? x[3].y : 0.f);
  }
}

__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy8(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(there ? 8 : 0)
               : "memory");
}

// A lane's pieces of one stage of the ring, `threads` apart: row `at`, from channel c
// and `apart` channels further on.  What is past the row comes as zero.
template <class T, bool SPLIT>
__device__ __forceinline__ void fetch(uint4* to, int threads, const void* base, int64_t at, int c, int apart, Left m) {
  const T* row = static_cast<const T*>(base) + (m.a > 0 ? at + c : 0);
  if constexpr (std::is_same<T, float>::value) {
    copy16(to, row, m.a > 0);
    copy16(to + threads, m.b > 0 ? row + apart : row, m.b > 0);
  } else if constexpr (SPLIT) {
    copy8(to, row, m.a > 0);
    copy8(reinterpret_cast<char*>(to) + 8, m.b > 0 ? row + apart : row, m.b > 0);
  } else {
    copy16(to, row, m.a > 0);
  }
}
// Channels past the row's last are zero.
template <class T>
__device__ __forceinline__ void take(const uint4* from, int threads, Left m, Eight& x) {
  const uint4 a = *from;
  if constexpr (std::is_same<T, float>::value) {
    const uint4 b = from[threads];
    x[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y)), x[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    x[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y)), x[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
  } else {
    x[0] = Pack2<T>::from(a.x), x[1] = Pack2<T>::from(a.y), x[2] = Pack2<T>::from(a.z), x[3] = Pack2<T>::from(a.w);
  }
  mask(x, m);
}

// Writes the lane's channels and the zeros that pad a row (to a multiple of 16
// channels in a 2-byte type, of 4 in fp32).
template <class T, bool SPLIT>
__device__ __forceinline__ void put(void* base, int64_t at, int c, int apart, Eight& x, Left m) {
  T* p = static_cast<T*>(base) + at + c;
  mask(x, m);
  if constexpr (std::is_same<T, float>::value) {
    if (m.a > 0) *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    if (m.b > 0) *reinterpret_cast<float4*>(p + apart) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  } else {
    const uint2 a = make_uint2(Pack2<T>::to(x[0].x, x[0].y), Pack2<T>::to(x[1].x, x[1].y)),
                b = make_uint2(Pack2<T>::to(x[2].x, x[2].y), Pack2<T>::to(x[3].x, x[3].y));
    // a four is written where its sixteen channels begin inside of the row
    if constexpr (SPLIT) {
      if (m.a > -(c & 15)) *reinterpret_cast<uint2*>(p) = a;
      if (m.b > -((c + apart) & 15)) *reinterpret_cast<uint2*>(p + apart) = b;
    } else {
      if (m.a > -(c & 15)) *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// 1 / sqrt(x) by one Newton step on the approximate root.
__device__ __forceinline__ float inv_root(float x) {
  const float y = rsqrtf(x);
  return x < 1e37f && x > 1e-37f ? fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y) : y;
}

__device__ __forceinline__ float add_up(const Eight& x) {
  const float2 s = add2_rn(add2_rn(x[0], x[1]), add2_rn(x[2], x[3]));
  return s.x + s.y;
}
__device__ __forceinline__ float dot(const Eight& x, const Eight& y) {
  float2 s = mul2_rn(x[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2_rn(x[i], y[i], s);
  return s.x + s.y;
}

// Sums over the lanes of a row, the same bits in each of them.
template <bool MULTI>
struct Row {
  int lanes, lane, group;
  float* buf;  // MULTI: two turns of 4 values for each warp of the block
  int turn;
  __device__ Row(int lanes_, float* sm) : lanes(lanes_), buf(sm), turn(0) {
    group = threadIdx.x / lanes;
    lane = threadIdx.x - group * lanes;
  }
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      if (MULTI || o < lanes) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
    }
    if (MULTI) {
      const int warps = lanes >> 5;
      float* mine = buf + (turn * (MAX_LANES / 32) + group * warps) * 4;
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) mine[(lane >> 5) * 4 + i] = v[i];
      }
      // a row's warps only; a warp that writes a turn again has passed the other
      // turn's barrier, which every reader of this turn has reached
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
      for (int w = 0; w < warps; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += mine[w * 4 + i];
      }
      turn ^= 1;
    }
  }
};

// Mean and 1/deviation of a row; the variance about the mean.  `left`: of the lane's
// first vector, `span`: channels from one of its vectors to the next.
template <int K, bool MULTI>
__device__ __forceinline__ void statistics(const Eight (&x)[K], Left left, int span, int kind, float eps, float inv_c,
                                           Row<MULTI>& row, float& mean, float& rstd) {
  mean = 0.f, rstd = 1.f;
  if (kind == GNN_NORM_NONE) return;
  float s[1] = {0.f};
  if (kind == GNN_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[0] += add_up(x[k]);
    row.sum(s);
    mean = s[0] * inv_c;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Eight d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = add2_rn(x[k][i], dup2(-mean));
      mask(d, {left.a - k * span, left.b - k * span});
      s[0] += dot(d, d);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) s[0] += dot(x[k], x[k]);
  }
  row.sum(s);
  rstd = inv_root(fmaf(s[0], inv_c, eps));
}

// (x - mean) rstd, zero past the row's end.
__device__ __forceinline__ void normalise(Eight& x, Left m, float mean, float rstd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2_rn(add2_rn(x[i], dup2(-mean)), dup2(rstd));
  mask(x, m);
}

// Where channel c's weight lies in the block's copy of a vector: the first fours of
// every lane, then the second ones, so that a warp's accesses lie side by side.
template <bool SPLIT>
__device__ __forceinline__ int weight_at(int c, int width) {
  return SPLIT ? c : (c & 4 ? width / 2 : 0) + c / 8 * 4 + (c & 3);
}
// Eight weights of this lane, from channel c on.
template <bool SPLIT>
__device__ __forceinline__ void from_shared(const float* p, int c, int apart, int width, Eight& w) {
  const float4 a = *reinterpret_cast<const float4*>(p + weight_at<SPLIT>(c, width)),
               b = *reinterpret_cast<const float4*>(p + weight_at<SPLIT>(c + apart, width));
  w[0] = make_float2(a.x, a.y), w[1] = make_float2(a.z, a.w), w[2] = make_float2(b.x, b.y), w[3] = make_float2(b.z, b.w);
}

// s w_post, s b_post, w_pre and (forward) b_pre of the block's `width` channels, zero
// past the row's end.  Where the gradient of one scale of all channels is wanted, that is
// kept apart: the gradient is a sum of z without it.
template <bool FWD, bool SPLIT>
__device__ __forceinline__ void share_weights(const Args& g, float* to, int width) {
  for (int c = threadIdx.x; c < width; c += blockDim.x) {
    const bool there = c < g.C;
    const int at = weight_at<SPLIT>(c, width);
    const float s = !there ? 0.f : g.scale_cols == 0 || (!FWD && g.part_s) ? 1.f : __ldg(g.scale + (g.scale_cols == 1 ? 0 : c));
    to[at] = s * (there && g.w_post ? __ldg(g.w_post + c) : 1.f);
    to[width + at] = there && g.b_post ? s * __ldg(g.b_post + c) : 0.f;
    to[2 * width + at] = there ? (g.w_pre ? __ldg(g.w_pre + c) : 1.f) : 0.f;
    if (FWD) to[3 * width + at] = there && g.b_pre ? __ldg(g.b_pre + c) : 0.f;
  }
  __syncthreads();
}

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// All but the newest stages - 1 rows have arrived.
__device__ __forceinline__ void wait_row(int stages) {
  if (stages == 4)
    wait_copies<3>();
  else if (stages == 3)
    wait_copies<2>();
  else
    wait_copies<1>();
}

// Bound by DRAM: 716,847 x 256 with a bf16 branch and an fp32 stream 418 us, 6.2 TB/s of
// 6.8 that a copy reaches; with layer norms 200,000 x 1024 bf16 433 us (4.7).  Rows of
// several warps wait for each other's sums: 30,000 x 4096 bf16 506 us (2.4).
template <class TB, class TR, class TY, bool MULTI, int K>
__global__ void __launch_bounds__(MULTI ? MAX_LANES : K == 1 ? THREADS : FEW)
    residual_fwd_kernel(const __grid_constant__ Args g) {
  extern __shared__ uint4 smem[];
  __shared__ float sm[MULTI ? 2 * 4 * (MAX_LANES / 32) : 1];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  Row<MULTI> row(g.lanes, sm);
  const int threads = blockDim.x, groups = threads / g.lanes, span = 8 * g.lanes, width = K * span;
  const int64_t step = (int64_t)gridDim.x * groups;
  // the warp's first row: its groups leave the loop together
  const int ahead = MULTI ? 0 : row.group & (32 / g.lanes - 1);
  constexpr bool SPLIT = std::is_same<TB, float>::value || std::is_same<TR, float>::value || std::is_same<TY, float>::value;
  const int c = (SPLIT ? 4 : 8) * row.lane, apart = SPLIT ? 4 * g.lanes : 4;
  const Left left{g.C - c, g.C - c - apart};
  float* const w_at = reinterpret_cast<float*>(smem);
  uint4* const mine = smem + width + threadIdx.x;
  const int stage_size = K * g.pieces * threads;
  auto request = [&](int st, int64_t i) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint4* to = mine + st * stage_size + k * g.pieces * threads;
      const int ck = c + k * span;
      const Left m = i < g.n ? Left{left.a - k * span, left.b - k * span} : Left{0, 0};
      fetch<TR, SPLIT>(to + g.at[0] * threads, threads, g.R, i * g.ldr, ck, apart, m);
      if (g.B) fetch<TB, SPLIT>(to + g.at[1] * threads, threads, g.B, i * g.ldb, ck, apart, m);
      if (g.gate == 2) fetch<TB, SPLIT>(to + g.at[2] * threads, threads, g.G, i * g.ldg, ck, apart, m);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto row_gate = [&](int64_t i) { return g.gate == 1 && i < g.n ? to_f32(static_cast<const TB*>(g.G)[i * g.ldg]) : 0.f; };
  int64_t i = (int64_t)blockIdx.x * groups + row.group;
  for (int k = 0; k < g.stages - 1; ++k) request(k, i + k * step);
  float t_next = row_gate(i);
  share_weights<true, SPLIT>(g, w_at, width);
  int st = 0, into = g.stages - 1;
  for (; i - ahead < g.n; i += step) {
    request(into, i + (g.stages - 1) * step);
    const float t_row = t_next;
    t_next = row_gate(i + step);
    wait_row(g.stages);
    const bool live = i < g.n;
    const uint4* from = mine + st * stage_size;
    auto piece = [&](int which, int k) { return from + (k * g.pieces + g.at[which]) * threads; };
    if (++st == g.stages) st = 0;
    if (++into == g.stages) into = 0;
    float4 stat = make_float4(0.f, 1.f, 0.f, 1.f);
    Eight h[K];
    if (g.B) {
#pragma unroll
      for (int k = 0; k < K; ++k) take<TB>(piece(1, k), threads, Left{left.a - k * span, left.b - k * span}, h[k]);
      statistics<K>(h, left, span, g.post, g.eps, g.inv_c, row, stat.x, stat.y);
      const float t1 = g.gate == 1 ? act_f(t_row, g.act) : 1.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Left m{left.a - k * span, left.b - k * span};
        Eight t, w, b, r;
        if (g.gate == 2) {
          take<TB>(piece(2, k), threads, m, t);
          with_act(g.act, [&](auto A) {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = act2(t[j], A);
          });
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = dup2(t1);
        }
        normalise(h[k], m, stat.x, stat.y);
        from_shared<SPLIT>(w_at, c + k * span, apart, width, w);
        from_shared<SPLIT>(w_at + width, c + k * span, apart, width, b);
        take<TR>(piece(0, k), threads, m, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = fma2_rn(t[j], fma2_rn(w[j], h[k][j], b[j]), r[j]);
        mask(h[k], m);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) take<TR>(piece(0, k), threads, Left{left.a - k * span, left.b - k * span}, h[k]);
    }
    if (g.H && live) {
#pragma unroll
      for (int k = 0; k < K; ++k) put<TR, SPLIT>(g.H, i * g.ldh, c + k * span, apart, h[k], Left{left.a - k * span, left.b - k * span});
    }
    if (g.pre != GNN_NORM_NONE) {
      statistics<K>(h, left, span, g.pre, g.eps, g.inv_c, row, stat.z, stat.w);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Left m{left.a - k * span, left.b - k * span};
        Eight w, b;
        normalise(h[k], m, stat.z, stat.w);
        from_shared<SPLIT>(w_at + 2 * width, c + k * span, apart, width, w);
        from_shared<SPLIT>(w_at + 3 * width, c + k * span, apart, width, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = fma2_rn(w[j], h[k][j], b[j]);
        if (live) put<TY, SPLIT>(g.Y, i * g.ldy, c + k * span, apart, h[k], m);
      }
    }
    if (g.stats && live && row.lane == 0) g.stats[i] = stat;
  }
}

// The channels' sums stay in registers over CHAIN rows of a group, so its registers leave
// 16 warps to an SM: 716,847 x 256 bf16 534 us, 5.5 TB/s, issue slots
// 60% taken beside DRAM; 232,965 x 602 in fp32, three warps a row, 687 us, 4.9 TB/s.
//
// An addition to a lane's running sum errs by up to 2^-24 of the sum so far, equal terms
// all to one side: a chain of 88 by 44.5 units at most, and with what follows (a warp's
// groups, a block's warps, its share of 304 in the join, the join's lanes) by 64; a chain of
// 1,028 equal terms measured 189.  So a block adds its lanes' sums up every CHAIN rows, in
// two terms (716,847 x 256 bf16: 534 us, one chain 536).
constexpr int CHAIN = 88;

template <class TB, class TR, class TY, bool MULTI, int K>
__global__ void __launch_bounds__(MULTI ? MAX_LANES : K == 1 ? THREADS : FEW, MULTI ? 1 : 2)
    residual_bwd_kernel(const __grid_constant__ Args g) {
  extern __shared__ uint4 smem[];
  __shared__ float sm[MULTI ? 2 * 4 * (MAX_LANES / 32) : 1];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  Row<MULTI> row(g.lanes, sm);
  const int threads = blockDim.x, groups = threads / g.lanes, span = 8 * g.lanes, width = K * span;
  const int64_t step = (int64_t)gridDim.x * groups;
  constexpr bool SPLIT = std::is_same<TB, float>::value || std::is_same<TR, float>::value || std::is_same<TY, float>::value;
  const int c = (SPLIT ? 4 : 8) * row.lane, apart = SPLIT ? 4 * g.lanes : 4;
  const Left left{g.C - c, g.C - c - apart};
  float* const w_at = reinterpret_cast<float*>(smem);
  uint4* const ring = smem + 3 * width / 4;
  uint4* const mine = ring + threadIdx.x;
  const int stage_size = K * g.pieces * threads;
  auto request = [&](int st, int64_t i) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint4* to = mine + st * stage_size + k * g.pieces * threads;
      const int ck = c + k * span;
      const Left m = i < g.n ? Left{left.a - k * span, left.b - k * span} : Left{0, 0};
      if (g.dY) {
        fetch<TY, SPLIT>(to + g.at[0] * threads, threads, g.dY, i * g.ldy, ck, apart, m);
        fetch<TR, SPLIT>(to + g.at[1] * threads, threads, g.H, i * g.ldh, ck, apart, m);
      }
      if (g.dH) fetch<TR, SPLIT>(to + g.at[2] * threads, threads, g.dH, i * g.lddh, ck, apart, m);
      if (g.B) fetch<TB, SPLIT>(to + g.at[3] * threads, threads, g.B, i * g.ldb, ck, apart, m);
      if (g.gate == 2) fetch<TB, SPLIT>(to + g.at[4] * threads, threads, g.G, i * g.ldg, ck, apart, m);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto row_gate = [&](int64_t i) { return g.gate == 1 && i < g.n ? to_f32(static_cast<const TB*>(g.G)[i * g.ldg]) : 0.f; };
  auto row_stats = [&](int64_t i) { return i < g.n ? __ldg(g.stats + i) : make_float4(0.f, 0.f, 0.f, 0.f); };
  int64_t i = (int64_t)blockIdx.x * groups + row.group;
  for (int k = 0; k < g.stages - 1; ++k) request(k, i + k * step);
  float t_next = row_gate(i);
  float4 s_next = row_stats(i);
  share_weights<false, SPLIT>(g, w_at, width);
  const float2 one_scale = dup2(g.part_s ? __ldg(g.scale) : 1.f);
  float ds_hi = 0.f, ds_lo = 0.f;  // D t z over this lane's channels and rows, and what the sum lost
  // a sum of millions of terms of either sign: Knuth's two-term sum keeps its tail
  auto add_ds = [&](float x) {
    const float sum = ds_hi + x, part = sum - ds_hi;
    ds_lo += (ds_hi - (sum - part)) + (x - part);
    ds_hi = sum;
  };
  auto one_scale_sum = [&] {
    if (!g.part_s) return;
    __shared__ double share[MAX_LANES / 32];
    double t = (double)ds_hi + (double)ds_lo;
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
      t = 0;
      for (int k = 0; k < threads / 32; ++k) t += share[k];
      g.part_s[blockIdx.x] = t;
    }
  };
  int st = 0, into = g.stages - 1;
  // the block's rounds of one row a group; with several chains the first ends sooner in some
  // blocks, so that not all of the card adds up at the same time
  int64_t rounds = g.rounds + ((int64_t)blockIdx.x * groups < g.rest);
  int chain = !g.part_lo ? 0x7fffffff : CHAIN - (blockIdx.x + 2 * (blockIdx.x / 152)) % 4 * (CHAIN / 4);
  bool first = true;
  do {
    Eight acc[4][K];  // sums of dY yh, dY, D t bh, D t
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[a][k][j] = dup2(0.f);
    int left_here = (int)min(rounds, (int64_t)chain);
    rounds -= left_here;
    chain = CHAIN;
    for (; left_here > 0; --left_here, i += step) {
      request(into, i + (g.stages - 1) * step);
      const float t_row = t_next;
      const float4 stat = s_next;
      t_next = row_gate(i + step), s_next = row_stats(i + step);
      wait_row(g.stages);
      const bool live = i < g.n;
      const uint4* from = mine + st * stage_size;
      auto piece = [&](int which, int k) { return from + (k * g.pieces + g.at[which]) * threads; };
      if (++st == g.stages) st = 0;
      if (++into == g.stages) into = 0;
      Eight d[K];
      if (g.dY) {
        // q = w dY; D = dH + rstd (q - mean q - yh mean(q yh)); K > 1 reads yh again after
        // the sums instead of keeping it
        float s[2] = {0.f, 0.f};
        Eight kept;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Left m{left.a - k * span, left.b - k * span};
          Eight yh, w;
          take<TY>(piece(0, k), threads, m, d[k]);
          take<TR>(piece(1, k), threads, m, yh);
          normalise(yh, m, stat.z, stat.w);
          from_shared<SPLIT>(w_at + 2 * width, c + k * span, apart, width, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0][k][j] = fma2_rn(d[k][j], yh[j], acc[0][k][j]);
            acc[1][k][j] = add2_rn(d[k][j], acc[1][k][j]);
            d[k][j] = mul2_rn(d[k][j], w[j]);
            if (K == 1) kept[j] = yh[j];
          }
          s[0] += dot(d[k], yh), s[1] += add_up(d[k]);
        }
        if (g.pre == GNN_NORM_LAYER) {
          row.sum(s);
        } else {
          float one[1] = {s[0]};
          row.sum(one);
          s[0] = one[0], s[1] = 0.f;
        }
        const float2 along = dup2(-s[0] * g.inv_c), mean = dup2(-s[1] * g.inv_c), r = dup2(stat.w);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Left m{left.a - k * span, left.b - k * span};
          Eight dh;
          if (K > 1) {
            take<TR>(piece(1, k), threads, m, kept);
            normalise(kept, m, stat.z, stat.w);
          }
          if (g.dH) {
            take<TR>(piece(2, k), threads, m, dh);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) dh[j] = dup2(0.f);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) d[k][j] = fma2_rn(r, fma2_rn(kept[j], along, add2_rn(d[k][j], mean)), dh[j]);
          mask(d[k], m);
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) take<TR>(piece(2, k), threads, Left{left.a - k * span, left.b - k * span}, d[k]);
      }
      if (g.dR && live) {
#pragma unroll
        for (int k = 0; k < K; ++k) put<TR, SPLIT>(g.dR, i * g.lddr, c + k * span, apart, d[k], Left{left.a - k * span, left.b - k * span});
      }
      if (g.B) {
        float s[3] = {0.f, 0.f, 0.f};
        float2 t1 = dup2(1.f), slope1 = dup2(0.f);
        if (g.gate == 1) act_grad2(dup2(t_row), g.act, t1, slope1);
        Eight kept;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Left m{left.a - k * span, left.b - k * span};
          Eight bh, w, b;
          take<TB>(piece(3, k), threads, m, bh);
          normalise(bh, m, stat.x, stat.y);
          from_shared<SPLIT>(w_at, c + k * span, apart, width, w);
          from_shared<SPLIT>(w_at + width, c + k * span, apart, width, b);
          if (g.gate == 2) {
            Eight t, slope;
            take<TB>(piece(4, k), threads, m, t);
            with_act(g.act, [&](auto A) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 z = t[j];
                act_grad2(z, A, t[j], slope[j]);
              }
            });
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 z = fma2_rn(w[j], bh[j], b[j]);
              slope[j] = mul2_rn(slope[j], mul2_rn(d[k][j], z));
              d[k][j] = mul2_rn(d[k][j], t[j]);
              t[j] = z;
            }
            if (g.part_s) {
              add_ds(dot(d[k], t));
#pragma unroll
              for (int j = 0; j < 4; ++j) slope[j] = mul2_rn(slope[j], one_scale);
            }
            if (g.dG && live) put<TB, SPLIT>(g.dG, i * g.lddg, c + k * span, apart, slope, m);
          } else if (g.gate == 1 || g.part_s) {
            float2 z = dup2(0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z = fma2_rn(d[k][j], fma2_rn(w[j], bh[j], b[j]), z);
              d[k][j] = mul2_rn(d[k][j], t1);
            }
            s[2] += z.x + z.y;
            if (g.part_s) add_ds(t1.x * (z.x + z.y));
          }
          if (g.part_s) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul2_rn(w[j], one_scale);
          }
          // d: D t here, and times s w_post from here on
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[2][k][j] = fma2_rn(d[k][j], bh[j], acc[2][k][j]);
            acc[3][k][j] = add2_rn(d[k][j], acc[3][k][j]);
            d[k][j] = mul2_rn(d[k][j], w[j]);
            if (K == 1) kept[j] = bh[j];
          }
          s[0] += dot(d[k], bh), s[1] += add_up(d[k]);
        }
        const bool norm = g.post != GNN_NORM_NONE;
        if (g.gate == 1) {
          row.sum(s);
          if (g.dG && live && row.lane == 0)
            static_cast<TB*>(g.dG)[i * g.lddg] = from_f32<TB>(s[2] * one_scale.x * slope1.x);
        } else if (g.post == GNN_NORM_LAYER) {
          float two[2] = {s[0], s[1]};
          row.sum(two);
          s[0] = two[0], s[1] = two[1];
        } else if (norm) {
          float one[1] = {s[0]};
          row.sum(one);
          s[0] = one[0];
        }
        if (g.dB && live) {
          const float2 along = dup2(-s[0] * g.inv_c), mean = dup2(g.post == GNN_NORM_LAYER ? -s[1] * g.inv_c : 0.f),
                       r = dup2(stat.y);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const Left m{left.a - k * span, left.b - k * span};
            if (norm) {
              if (K > 1) {
                take<TB>(piece(3, k), threads, m, kept);
                normalise(kept, m, stat.x, stat.y);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) d[k][j] = mul2_rn(r, fma2_rn(kept[j], along, add2_rn(d[k][j], mean)));
            }
            put<TB, SPLIT>(g.dB, i * g.lddb, c + k * span, apart, d[k], m);
          }
        }
      }
    }
    if (!g.want_q && !g.want_p) continue;
    // over the groups of a warp, then over the block's warps or groups in order: one of the
    // four sums at a time beside the ring, or, behind a block's only chain, all of them in
    // the ring's memory (every copy has landed: the last rows' are waited for)
    if (!MULTI) {
      for (int o = g.lanes; o < 32; o <<= 1) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[a][k][j] = add2_rn(acc[a][k][j], make_float2(__shfl_xor_sync(0xffffffffu, acc[a][k][j].x, o),
                                                               __shfl_xor_sync(0xffffffffu, acc[a][k][j].y, o)));
      }
    }
    const int turns = MULTI ? groups : threads / 32, turn = MULTI ? row.group : threadIdx.x >> 5;
    float* const out = g.part + (int64_t)blockIdx.x * 4 * width;
    auto pass_on = [&](float* to, int a) {
      if (MULTI || (threadIdx.x & 31) < g.lanes) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float* at = to + c + k * span;
          *reinterpret_cast<float4*>(at) = make_float4(acc[a][k][0].x, acc[a][k][0].y, acc[a][k][1].x, acc[a][k][1].y);
          *reinterpret_cast<float4*>(at + apart) = make_float4(acc[a][k][2].x, acc[a][k][2].y, acc[a][k][3].x, acc[a][k][3].y);
        }
      }
    };
    if (!g.part_lo) {  // [turns][4][width]
      wait_copies<0>();
      __syncthreads();
      float* const all = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int a = 0; a < 4; ++a) pass_on(all + (turn * 4 + a) * width, a);
      __syncthreads();
      for (int at = threadIdx.x; at < 4 * width; at += threads) {
        float s = all[at];
        for (int k = 1; k < turns; ++k) s += all[k * 4 * width + at];
        out[at] = s;
      }
      return one_scale_sum();
    }
    // [turns][width]; every column of the running sums is one thread's, which asks for them
    // early: where registers allow it for the next kind's while it adds this one's
    constexpr int COLS = MULTI ? 8 : K == 1 ? 1 : 2 * K;  // of a thread, at most
    constexpr int AHEAD = MULTI ? 0 : 1;
    float* const all = reinterpret_cast<float*>(ring + g.stages * stage_size);
    float hi[AHEAD + 1][COLS], lo[AHEAD + 1][COLS];
    auto ask = [&](int a) {
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const int at = threadIdx.x + j * threads;
        const bool there = !first && at < width;
        hi[a & AHEAD][j] = there ? out[a * width + at] : 0.f;
        lo[a & AHEAD][j] = there ? out[a * width + at + (g.part_lo - g.part)] : 0.f;
      }
    };
    if (AHEAD) ask(0);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a + AHEAD < 4) ask(a + AHEAD);
      pass_on(all + turn * width, a);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const int at = threadIdx.x + j * threads;
        if (at >= width) break;
        float s = all[at];
        for (int k = 1; k < turns; ++k) s += all[k * width + at];
        const float before = hi[a & AHEAD][j], sum = before + s, part = sum - before;  // two terms (Knuth)
        const float lost = lo[a & AHEAD][j] + ((before - (sum - part)) + (s - part));
        out[a * width + at] = rounds > 0 ? sum : sum + lost;
        if (rounds > 0) out[a * width + at + (g.part_lo - g.part)] = lost;
      }
      __syncthreads();
    }
    first = false;
  } while (rounds > 0);
  one_scale_sum();
}

// The blocks' sums, in order, and the weights' gradients from them.  In fp32: an
// SM adds two fp64 numbers a clock, and with those this kernel took 27 us of 39 for
// 2,500 x 300 (6 now).  A block takes 32 channels of the pre norm's two sums or of the
// post norm's; with one learned scale a block more adds its gradient.
constexpr int JOIN_ROWS = 32;
struct Join {
  const float* part;
  const double* part_s;
  int blocks, width, C, scale_cols;
  const float *w_post, *b_post, *scale;
  float *dw_post, *db_post, *dscale, *dw_pre, *db_pre;
  int want_q, want_p;
};
__global__ void __launch_bounds__(32 * JOIN_ROWS) residual_join_kernel(const Join g) {
  __shared__ float sm[2][JOIN_ROWS][33];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int pieces = (g.C + 31) / 32, of = (int)blockIdx.x / pieces, c = ((int)blockIdx.x - of * pieces) * 32 + lane;
  if (of == 2) {
    if (r) return;
    double s = 0;
    for (int b = lane; b < g.blocks; b += 32) s += g.part_s[b];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) g.dscale[0] = (float)s;
    return;
  }
  if (!(of ? g.want_p : g.want_q)) return;
  float s[2] = {0.f, 0.f};
  if (c < g.C) {
    const float* p = g.part + 2 * of * g.width + c;
#pragma unroll 10
    for (int b = r; b < g.blocks; b += JOIN_ROWS) {
      const int64_t at = (int64_t)b * 4 * g.width;
      s[0] += p[at], s[1] += p[at + g.width];
    }
  }
  sm[0][r][lane] = s[0], sm[1][r][lane] = s[1];
  __syncthreads();
  // a warp for each channel: its lanes are the rows
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    s[a] = sm[a][lane][r];
#pragma unroll
    for (int o = 16; o; o >>= 1) s[a] += __shfl_xor_sync(0xffffffffu, s[a], o);
  }
  __syncthreads();
  if (lane < 2) sm[lane][0][r] = lane ? s[1] : s[0];
  __syncthreads();
  if (r || c >= g.C) return;
  const float s1 = sm[0][0][lane], s2 = sm[1][0][lane];
  if (of == 0) {
    if (g.dw_pre) g.dw_pre[c] = s1;
    if (g.db_pre) g.db_pre[c] = s2;
    return;
  }
  const float sc = g.scale_cols == 0 ? 1.f : g.scale_cols == 1 ? g.scale[0] : g.scale[c];
  if (g.dw_post) g.dw_post[c] = sc * s1;
  if (g.db_post) g.db_post[c] = sc * s2;
  if (g.dscale && g.scale_cols > 1) g.dscale[c] = fmaf(g.w_post ? g.w_post[c] : 1.f, s1, (g.b_post ? g.b_post[c] : 0.f) * s2);
}

// ---------------------------------------------------------------- host side
// Lanes and vectors of a row of C channels, padding to 16 included.  One warp's lanes
// with up to four vectors in the forward; in the backward, whose channel sums fill the
// registers, three where that leaves fewer lanes idle than several warps would
// (300,000 x 300 bf16: 548 us against 651; 1024 channels with four: 1,213 against 747).
struct Shape {
  int lanes, vecs, threads;
  bool multi;
};
constexpr Shape shape_for(int C, bool bwd) {
  const int v = (C + 15) / 16 * 2;
  Shape s{0, 0, 0, false};
  for (int k = 1; k <= (bwd ? 3 : 4); k += bwd ? 2 : 1)
    for (int l = 4; l <= 32; l *= 2)
      if (l * k >= v && (!s.lanes || l * k < s.lanes * s.vecs)) s = {l, k, k == 1 ? THREADS : FEW, false};
  const int lanes = (v + 31) / 32 * 32;
  if (s.lanes && (s.vecs == 1 || s.lanes * s.vecs < lanes + (bwd ? 0 : 1))) return s;
  // 64 lanes at least here, so at most eight rows and their barriers to a block; few
  // blocks: each takes sixteen barriers, and an SM has them for four
  return {lanes, 1, MAX_LANES / lanes * lanes, true};
}

// What the kernels take for granted of a width's shape: the row fits, rows of one warp are a
// power of two of lanes and have a kernel, and those of several are whole warps, each row
// with a named barrier of its own (a block has fifteen beside its common one).
constexpr bool fits(const Shape& s, int C, bool bwd) {
  if (s.lanes < 1 || s.threads % s.lanes || s.threads > MAX_LANES || 8 * s.lanes * s.vecs < (C + 15) / 16 * 16) return false;
  if (s.multi) return s.vecs == 1 && s.lanes % 32 == 0 && s.threads / s.lanes <= 15;
  return 32 % s.lanes == 0 && s.threads == (s.vecs == 1 ? THREADS : FEW) && s.vecs >= 1 && s.vecs <= 4 &&
         (!bwd || s.vecs == 1 || s.vecs == 3);
}
constexpr bool every_width_fits() {
  for (int C = 1; C <= MAX_C; ++C)
    if (!fits(shape_for(C, false), C, false) || !fits(shape_for(C, true), C, true)) return false;
  return true;
}
static_assert(every_width_fits(), "a width whose rows have no kernel, or more than fifteen to a block of barriers");

// What one of the four sums of every warp or group takes on its way through shared memory.
int one_sum(const Shape& s) { return (s.multi ? s.threads / s.lanes : s.threads / 32) * 8 * s.lanes * s.vecs * (int)sizeof(float); }

// Blocks that an SM holds at once, by the kernels' registers and with two stages of the ring
// at least; up to four stages in what that leaves of shared memory.  The 4 KB are for static
// shared memory, what the system takes of it (2 KB together at most) and, where lanes have
// several chains of sums, a sum of up to 2 KB on its way.
struct Fit {
  int blocks, stages;
};
Fit fit_of(const Shape& s, bool bwd, int pieces, bool chains = false) {
  const int regs = bwd ? (s.vecs == 1 ? 128 : 256) : s.vecs == 1 ? 104 : 128;
  const int stage = s.vecs * pieces * s.threads * 16;
  const int weights = (bwd ? 12 : 16) * 8 * s.lanes * s.vecs + (chains ? std::max(0, one_sum(s) - 2048) : 0) + 4096;
  const int most = 227 << 10;
  Fit f{std::max(1, 65536 / (regs * s.threads)), 4};
  while (f.blocks > 1 && f.blocks * (weights + 2 * stage) > most) --f.blocks;
  f.stages = std::max(2, std::min(4, (most / f.blocks - weights) / std::max(stage, 1)));
  return f;
}
// The backward's join reads a piece of each block's, so their number does not depend on
// which matrices there are.
int64_t blocks_for(int64_t n, const Shape& s, bool bwd) {
  const int64_t rows = s.threads / s.lanes;
  return std::max<int64_t>(1, std::min<int64_t>((n + rows - 1) / rows, 152 * fit_of(s, bwd, bwd ? 5 : 3).blocks));
}

// Whether some lane has more rows than one chain of sums takes.
bool chained(int64_t n, const Shape& s) { return n > CHAIN * blocks_for(n, s, true) * (s.threads / s.lanes); }

struct ResidualWs {
  float *part, *part_lo;
  double* part_s;
  size_t bytes;
};
ResidualWs residual_ws(void* base, size_t cap, int64_t n, int C, bool* ok) {
  Arena ar(base, cap);
  ResidualWs w{};
  const Shape s = shape_for(C, true);
  const size_t sums = (size_t)blocks_for(n, s, true) * 4 * s.lanes * s.vecs * 8;
  w.part = ar.take<float>(sums);
  w.part_lo = chained(n, s) ? ar.take<float>(sums) : nullptr;
  w.part_s = ar.take<double>((size_t)blocks_for(n, s, true));
  w.bytes = ar.used;
  *ok = ar.ok();
  return w;
}

// A launch may start while the kernel before it ends; each waits for that before
// it touches memory.
template <class... P, class... A>
gnn_status launch(int64_t grid, int block, size_t smem, cudaStream_t st, void (*k)(P...), const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
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

constexpr int SMEM_MOST = 224 << 10;  // of 227 KB; less than one is static, and fit_of leaves 4 out

template <bool BWD, class TB, class TR, class TY, bool MULTI, int K>
gnn_status run_shape(Args& g, const Shape& s, cudaStream_t st) {
  static PerDevice done;
  auto* k = [] {
    if constexpr (BWD)
      return residual_bwd_kernel<TB, TR, TY, MULTI, K>;
    else
      return residual_fwd_kernel<TB, TR, TY, MULTI, K>;
  }();
  const gnn_status r = allow_smem(k, SMEM_MOST, done);
  if (r != GNN_OK) return r;
  const int width = 8 * s.lanes * K * (int)sizeof(float), weights = (BWD ? 3 : 4) * width;
  g.stages = fit_of(s, BWD, g.pieces, g.part_lo != nullptr).stages;
  int ring = g.stages * K * g.pieces * s.threads * 16;
  // the backward's sums pass beside the ring, or all at once through it
  if (BWD) ring = g.part_lo ? ring + one_sum(s) : std::max(ring, 4 * one_sum(s));
  // No more blocks to an SM than the grid counts on: a launch that starts while the
  // last one ends would crowd SMs that are free first (716,847 x 256 forward, one
  // call behind another: 541 us against 423 alone).
  const int smem = std::max(weights + ring, (227 << 10) / (fit_of(s, BWD, BWD ? 5 : 3).blocks + 1));
  const int64_t blocks = blocks_for(g.n, s, BWD), round = blocks * (s.threads / s.lanes);
  g.rounds = g.n / round, g.rest = g.n % round;
  return launch(blocks, s.threads, smem, st, k, g);
}
template <bool BWD, class TB, class TR, class TY>
gnn_status run(Args& g, cudaStream_t st) {
  const Shape s = shape_for(g.C, BWD);
  g.lanes = s.lanes;
  // pieces of 16 bytes of a lane's eight channels
  auto add = [&](int k, const void* p, int elem) {
    g.at[k] = g.pieces;
    if (p) g.pieces += elem / 2;
  };
  g.pieces = 0;
  if (BWD) {
    add(0, g.dY, sizeof(TY)), add(1, g.dY, sizeof(TR)), add(2, g.dH, sizeof(TR)), add(3, g.B, sizeof(TB));
    add(4, g.gate == 2 ? g.G : nullptr, sizeof(TB));
  } else {
    add(0, g.R, sizeof(TR)), add(1, g.B, sizeof(TB)), add(2, g.gate == 2 ? g.G : nullptr, sizeof(TB));
  }
  if (s.multi) return run_shape<BWD, TB, TR, TY, true, 1>(g, s, st);
  if (s.vecs == 1) return run_shape<BWD, TB, TR, TY, false, 1>(g, s, st);
  if (s.vecs == 3) return run_shape<BWD, TB, TR, TY, false, 3>(g, s, st);
  if constexpr (BWD) return GNN_ERR_UNSUPPORTED;  // shape_for has no such row
  else return s.vecs == 2 ? run_shape<false, TB, TR, TY, false, 2>(g, s, st) : run_shape<false, TB, TR, TY, false, 4>(g, s, st);
}

// Types of branch, stream and next operand (one type, or an fp32 stream with a
// 2-byte rest, or fp32 with a 2-byte operand).
template <class Fn>
gnn_status with_types(int bt, int rt, int yt, Fn f) {
  using B16 = __nv_bfloat16;
  if (bt == GNN_F32 && rt == GNN_F32 && yt == GNN_F32) return f(float(), float(), float());
  if (bt == GNN_F32 && rt == GNN_F32 && yt == GNN_BF16) return f(float(), float(), B16());
  if (bt == GNN_F32 && rt == GNN_F32 && yt == GNN_F16) return f(float(), float(), __half());
  if (bt == GNN_BF16 && rt == GNN_BF16 && yt == GNN_BF16) return f(B16(), B16(), B16());
  if (bt == GNN_F16 && rt == GNN_F16 && yt == GNN_F16) return f(__half(), __half(), __half());
  if (bt == GNN_BF16 && rt == GNN_F32 && yt == GNN_BF16) return f(B16(), float(), B16());
  if (bt == GNN_F16 && rt == GNN_F32 && yt == GNN_F16) return f(__half(), float(), __half());
  return GNN_ERR_UNSUPPORTED;
}
bool good_types(int bt, int rt, int yt) {
  return with_types(bt, rt, yt, [](auto, auto, auto) { return GNN_OK; }) == GNN_OK;
}

// What an output's row has to hold: the padding is written too.
int64_t out_cols(int C, int t) { return t == GNN_F32 ? (C + 3) / 4 * 4 : (C + 15) / 16 * 16; }
constexpr int64_t LD_MOST = (int64_t)1 << 36;
bool bad_mat(const void* p, int64_t ld, int64_t cols, int t) {
  const int64_t e = type_size(t);
  return !p || ((uintptr_t)p & 15) || (ld * e) % 16 || ld < cols || ld > LD_MOST;
}
bool bad_vec(const void* p) { return ((uintptr_t)p & 3) != 0; }
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int t) {
  return {p, rows, ld * type_size(t), cols * type_size(t)};
}
Span flat(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

bool is_norm(int k) { return k == GNN_NORM_NONE || k == GNN_NORM_RMS || k == GNN_NORM_LAYER; }

// What both directions ask of a call.
gnn_status check(const char* who, const void* B, int64_t ldb, int bt, const void* G, int64_t ldg, int gate_cols, int act,
                 int64_t n, int C, int rt, int yt, int post, const float* w_post, const float* b_post, const float* scale,
                 int scale_cols, int pre, const float* w_pre) {
  if (n < 0 || n > ((int64_t)1 << 40)) return fail(GNN_ERR_INVALID_ARG, "%s: bad row count", who);
  if (C < 1) return fail(GNN_ERR_INVALID_ARG, "%s: C must be >= 1", who);
  if (C > MAX_C) return fail(GNN_ERR_UNSUPPORTED, "%s: C > %d", who, MAX_C);
  if (!is_type(bt) || !is_type(rt) || !is_type(yt)) return fail(GNN_ERR_INVALID_ARG, "%s: unknown type", who);
  if (!good_types(bt, rt, yt))
    return fail(GNN_ERR_UNSUPPORTED, "%s: types are (t, t, t), (t, fp32, t), (fp32, fp32, t) or fp32 for branch, stream and Y", who);
  if (!is_norm(post) || !is_norm(pre)) return fail(GNN_ERR_INVALID_ARG, "%s: post and pre are GNN_NORM_*", who);
  if (!is_act(act)) return fail(GNN_ERR_INVALID_ARG, "%s: gate_act is GNN_ACT_*", who);
  if (gate_cols != 0 && gate_cols != 1 && gate_cols != C)
    return fail(GNN_ERR_INVALID_ARG, "%s: gate_cols is 0, 1 or C", who);
  if (scale_cols != 0 && scale_cols != 1 && scale_cols != C)
    return fail(GNN_ERR_INVALID_ARG, "%s: scale_cols is 0, 1 or C", who);
  if ((scale_cols != 0) != (scale != nullptr)) return fail(GNN_ERR_INVALID_ARG, "%s: scale and scale_cols disagree", who);
  if (bad_vec(w_post) || bad_vec(b_post) || bad_vec(scale) || bad_vec(w_pre))
    return fail(GNN_ERR_INVALID_ARG, "%s: misaligned weights", who);
  if (n == 0) return GNN_OK;
  if (!B && (gate_cols || scale || w_post || b_post || post != GNN_NORM_NONE))
    return fail(GNN_ERR_INVALID_ARG, "%s: without a branch there is no post norm, gate or scale", who);
  if (B && bad_mat(B, ldb, C, bt)) return fail(GNN_ERR_INVALID_ARG, "%s: B needs 16-byte aligned rows and ldb >= C", who);
  if (gate_cols > 1 && bad_mat(G, ldg, C, bt))
    return fail(GNN_ERR_INVALID_ARG, "%s: gate needs 16-byte aligned rows and ldg >= C", who);
  if (gate_cols == 1 && (!G || ((uintptr_t)G & (type_size(bt) - 1)) || ldg < 1 || ldg > LD_MOST))
    return fail(GNN_ERR_INVALID_ARG, "%s: gate of one value a row is NULL, misaligned or has no stride", who);
  return GNN_OK;
}

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_residual_norm_workspace(int64_t n, int32_t C, size_t* bwd_bytes) {
  GNN_REQUIRE(n >= 0 && C >= 1, "gnn_residual_norm_workspace: bad sizes");
  GNN_REQUIRE(bwd_bytes, "gnn_residual_norm_workspace: NULL result");
  if (C > MAX_C) return fail(GNN_ERR_UNSUPPORTED, "gnn_residual_norm_workspace: C > %d", MAX_C);
  bool ok;
  *bwd_bytes = residual_ws(nullptr, 0, n, C, &ok).bytes;
  return GNN_OK;
}

extern "C" gnn_status gnn_residual_norm_fwd(const void* B, int64_t ldb, int32_t b_type, const void* R, int64_t ldr,
                                            int32_t r_type, const void* gate, int64_t ldg, int32_t gate_cols,
                                            int32_t gate_act, int64_t n, int32_t C, int32_t post, const float* w_post,
                                            const float* b_post, const float* scale, int32_t scale_cols, int32_t pre,
                                            const float* w_pre, const float* b_pre, double eps, void* H, int64_t ldh,
                                            void* Y, int64_t ldy, int32_t y_type, float* stats, gnn_stream_t stream) {
  static const char* who = "gnn_residual_norm_fwd";
  gnn_status s = check(who, B, ldb, b_type, gate, ldg, gate_cols, gate_act, n, C, r_type, y_type, post, w_post, b_post, scale,
                       scale_cols, pre, w_pre);
  if (s != GNN_OK) return s;
  GNN_REQUIRE((float)eps > 0.f && std::isfinite((float)eps), "%s: eps must be positive in fp32", who);
  GNN_REQUIRE(!bad_vec(b_pre), "%s: misaligned weights", who);
  GNN_REQUIRE(pre != GNN_NORM_NONE || (!w_pre && !b_pre), "%s: w_pre and b_pre come with a pre norm", who);
  if (n == 0) return GNN_OK;
  GNN_REQUIRE((pre == GNN_NORM_NONE) == (Y == nullptr), "%s: Y comes with a pre norm, and only then", who);
  GNN_REQUIRE(!bad_mat(R, ldr, C, r_type), "%s: R needs 16-byte aligned rows and ldr >= C", who);
  GNN_REQUIRE(H || !B, "%s: H is NULL", who);
  GNN_REQUIRE(H || Y, "%s: nothing to write", who);
  GNN_REQUIRE(!H || !bad_mat(H, ldh, out_cols(C, r_type), r_type),
              "%s: H needs 16-byte aligned rows and ldh >= C with its padding", who);
  GNN_REQUIRE(!Y || !bad_mat(Y, ldy, out_cols(C, y_type), y_type),
              "%s: Y needs 16-byte aligned rows and ldy >= C with its padding", who);
  GNN_REQUIRE(((uintptr_t)stats & 15) == 0, "%s: misaligned stats", who);
  const Span hs = span(H, n, out_cols(C, r_type), ldh, r_type), ys = span(Y, n, out_cols(C, y_type), ldy, y_type),
             ss = flat(stats, n * 16);
  const Span bs = span(B, n, C, ldb, b_type), rs = span(R, n, C, ldr, r_type),
             gs = span(gate_cols ? gate : nullptr, n, gate_cols, ldg, b_type);
  const Span vecs[5] = {flat(w_post, 4ll * C), flat(b_post, 4ll * C), flat(scale, 4ll * scale_cols), flat(w_pre, 4ll * C),
                        flat(b_pre, 4ll * C)};
  GNN_REQUIRE(!overlap(hs, bs) && !overlap(hs, gs) && ((H == R && ldh == ldr) || !overlap(hs, rs)),
              "%s: H overlaps an input (it may be R)", who);
  GNN_REQUIRE(!overlap(ys, bs) && !overlap(ys, gs) && !overlap(ys, rs) && !overlap(ys, hs), "%s: Y overlaps", who);
  GNN_REQUIRE(!overlap(ss, bs) && !overlap(ss, gs) && !overlap(ss, rs) && !overlap(ss, hs) && !overlap(ss, ys),
              "%s: stats overlaps", who);
  for (const Span& v : vecs)
    GNN_REQUIRE(!overlap(hs, v) && !overlap(ys, v) && !overlap(ss, v), "%s: an output overlaps a weight", who);
  Args g{};
  g.B = B, g.R = R, g.G = gate, g.H = H, g.Y = Y;
  g.ldb = ldb, g.ldr = ldr, g.ldg = ldg, g.ldh = ldh, g.ldy = ldy;
  g.n = n, g.C = C, g.gate = gate_cols == 1 ? 1 : gate_cols ? 2 : 0, g.act = gate_act, g.post = post, g.pre = pre;
  g.w_post = w_post, g.b_post = b_post, g.scale = scale, g.w_pre = w_pre, g.b_pre = b_pre;
  g.scale_cols = scale_cols, g.eps = (float)eps, g.inv_c = 1.f / (float)C, g.stats = reinterpret_cast<float4*>(stats);
  return with_types(b_type, r_type, y_type, [&](auto b, auto r, auto y) {
    return run<false, decltype(b), decltype(r), decltype(y)>(g, as_stream(stream));
  });
}

extern "C" gnn_status gnn_residual_norm_bwd(const void* dH, int64_t lddh, const void* dY, int64_t lddy, int32_t y_type,
                                            const void* B, int64_t ldb, int32_t b_type, const void* H, int64_t ldh,
                                            int32_t r_type, const void* gate, int64_t ldg, int32_t gate_cols,
                                            int32_t gate_act, int64_t n, int32_t C, int32_t post, const float* w_post,
                                            const float* b_post, const float* scale, int32_t scale_cols, int32_t pre,
                                            const float* w_pre, const float* stats, void* dR, int64_t lddr, void* dB,
                                            int64_t lddb, void* dgate, int64_t lddg, float* dw_post, float* db_post,
                                            float* dscale, float* dw_pre, float* db_pre, void* ws, size_t ws_bytes,
                                            gnn_stream_t stream) {
  static const char* who = "gnn_residual_norm_bwd";
  gnn_status s = check(who, B, ldb, b_type, gate, ldg, gate_cols, gate_act, n, C, r_type, y_type, post, w_post, b_post, scale,
                       scale_cols, pre, w_pre);
  if (s != GNN_OK) return s;
  GNN_REQUIRE(!bad_vec(dw_post) && !bad_vec(db_post) && !bad_vec(dscale) && !bad_vec(dw_pre) && !bad_vec(db_pre),
              "%s: misaligned gradients", who);
  GNN_REQUIRE(pre != GNN_NORM_NONE || (!w_pre && !dw_pre && !db_pre), "%s: w_pre and its gradients come with a pre norm", who);
  GNN_REQUIRE(!dscale || scale, "%s: dscale without a scale", who);
  if (n > 0) {
    GNN_REQUIRE(B || (!dB && !dgate && !dw_post && !db_post && !dscale), "%s: gradients of a branch that is not there", who);
    GNN_REQUIRE(gate_cols || !dgate, "%s: dgate without a gate", who);
    GNN_REQUIRE(pre != GNN_NORM_NONE || !dY, "%s: dY comes with a pre norm", who);
    GNN_REQUIRE(dH || dY, "%s: neither dH nor dY", who);
    GNN_REQUIRE(!dH || !bad_mat(dH, lddh, C, r_type), "%s: dH needs 16-byte aligned rows and lddh >= C", who);
    GNN_REQUIRE(!dY || !bad_mat(dY, lddy, C, y_type), "%s: dY needs 16-byte aligned rows and lddy >= C", who);
    GNN_REQUIRE(!dY || !bad_mat(H, ldh, C, r_type), "%s: H needs 16-byte aligned rows and ldh >= C", who);
    GNN_REQUIRE(stats && ((uintptr_t)stats & 15) == 0, "%s: stats is NULL or misaligned", who);
    GNN_REQUIRE(!dR || !bad_mat(dR, lddr, out_cols(C, r_type), r_type),
                "%s: dR needs 16-byte aligned rows and lddr >= C with its padding", who);
    GNN_REQUIRE(!dB || !bad_mat(dB, lddb, out_cols(C, b_type), b_type),
                "%s: dB needs 16-byte aligned rows and lddb >= C with its padding", who);
    GNN_REQUIRE(gate_cols <= 1 || !dgate || !bad_mat(dgate, lddg, out_cols(C, b_type), b_type),
                "%s: dgate needs 16-byte aligned rows and lddg >= C with its padding", who);
    GNN_REQUIRE(gate_cols != 1 || !dgate || (((uintptr_t)dgate & (type_size(b_type) - 1)) == 0 && lddg >= 1 && lddg <= LD_MOST),
                "%s: dgate of one value a row is misaligned or has no stride", who);
  }
  const int want_q = dw_pre || db_pre, want_p = dw_post || db_post || (dscale && scale_cols > 1), want_s = dscale && scale_cols == 1;
  const Shape sh = shape_for(C, true);
  bool ok;
  const ResidualWs w = residual_ws(ws, ws_bytes, n, C, &ok);
  GNN_REQUIRE((!want_q && !want_p && !want_s) || (ws && ok && ((uintptr_t)ws & 7) == 0),
              "%s: workspace too small (%zu < %zu) or misaligned", who, ws_bytes, w.bytes);
  if (n > 0) {
    const Span outs[9] = {span(dR, n, out_cols(C, r_type), lddr, r_type), span(dB, n, out_cols(C, b_type), lddb, b_type),
                          span(dgate, n, gate_cols > 1 ? out_cols(C, b_type) : 1, lddg, b_type), flat(dw_post, 4ll * C),
                          flat(db_post, 4ll * C), flat(dscale, 4ll * scale_cols), flat(dw_pre, 4ll * C), flat(db_pre, 4ll * C),
                          flat(want_q || want_p || want_s ? ws : nullptr, (int64_t)w.bytes)};
    const Span ins[10] = {span(dH, n, C, lddh, r_type), span(dY, n, C, lddy, y_type), span(B, n, C, ldb, b_type),
                          span(dY ? H : nullptr, n, C, ldh, r_type), span(gate_cols ? gate : nullptr, n, gate_cols, ldg, b_type),
                          flat(stats, n * 16), flat(w_post, 4ll * C), flat(b_post, 4ll * C), flat(scale, 4ll * scale_cols),
                          flat(w_pre, 4ll * C)};
    for (int o = 0; o < 9; ++o) {
      for (int i = 0; i < 10; ++i)
        GNN_REQUIRE((o == 0 && i == 0 && dR == dH && lddr == lddh) || !overlap(outs[o], ins[i]),
                    "%s: an output overlaps an input (dR may be dH)", who);
      for (int i = 0; i < o; ++i) GNN_REQUIRE(!overlap(outs[o], outs[i]), "%s: outputs overlap", who);
    }
    Args g{};
    g.B = B, g.G = gate, g.dH = dH, g.dY = dY, g.H = const_cast<void*>(H), g.dR = dR, g.dB = dB, g.dG = dgate;
    g.ldb = ldb, g.ldg = ldg, g.ldh = ldh, g.ldy = lddy, g.lddh = lddh, g.lddr = lddr, g.lddb = lddb, g.lddg = lddg;
    g.n = n, g.C = C, g.gate = gate_cols == 1 ? 1 : gate_cols ? 2 : 0, g.act = gate_act, g.post = post, g.pre = pre;
    g.w_post = w_post, g.b_post = b_post, g.scale = scale, g.w_pre = w_pre;
    g.scale_cols = scale_cols, g.inv_c = 1.f / (float)C;
    g.stats = reinterpret_cast<float4*>(const_cast<float*>(stats)), g.part = w.part;
    g.want_q = want_q, g.want_p = want_p, g.part_s = want_s ? w.part_s : nullptr;
    g.part_lo = want_q || want_p ? w.part_lo : nullptr;
    s = with_types(b_type, r_type, y_type, [&](auto b, auto r, auto y) {
      return run<true, decltype(b), decltype(r), decltype(y)>(g, as_stream(stream));
    });
    if (s != GNN_OK) return s;
  }
  if (!want_q && !want_p && !want_s) return GNN_OK;
  const int blocks = (C + 31) / 32;
  const Join j{w.part, w.part_s, n > 0 ? (int)blocks_for(n, sh, true) : 0, sh.lanes * sh.vecs * 8, C, scale_cols, w_post, b_post,
               scale, dw_post, db_post, dscale, dw_pre, db_pre, want_q, want_p};
  return launch(2 * blocks + want_s, 32 * JOIN_ROWS, 0, as_stream(stream), residual_join_kernel, j);
}

// A struct's numbers that the calls take in 32 bits.
static bool narrow(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x != (int32_t)x) return false;
  return true;
}

extern "C" gnn_status gnn_residual_norm_fwd_struct(const gnn_residual_norm_fwd_args* a) {
  GNN_REQUIRE(a, "gnn_residual_norm_fwd: NULL arguments");
  GNN_REQUIRE(narrow({a->b_type, a->r_type, a->gate_cols, a->gate_act, a->C, a->post, a->scale_cols, a->pre, a->y_type}),
              "gnn_residual_norm_fwd: a number of more than 32 bits");
  return gnn_residual_norm_fwd(a->B, a->ldb, (int32_t)a->b_type, a->R, a->ldr, (int32_t)a->r_type, a->gate, a->ldg,
                               (int32_t)a->gate_cols, (int32_t)a->gate_act, a->n, (int32_t)a->C, (int32_t)a->post, a->w_post,
                               a->b_post, a->scale, (int32_t)a->scale_cols, (int32_t)a->pre, a->w_pre, a->b_pre, a->eps, a->H,
                               a->ldh, a->Y, a->ldy, (int32_t)a->y_type, a->stats, a->stream);
}

extern "C" gnn_status gnn_residual_norm_bwd_struct(const gnn_residual_norm_bwd_args* a) {
  GNN_REQUIRE(a, "gnn_residual_norm_bwd: NULL arguments");
  GNN_REQUIRE(narrow({a->y_type, a->b_type, a->r_type, a->gate_cols, a->gate_act, a->C, a->post, a->scale_cols, a->pre}) &&
                  a->ws_bytes >= 0, "gnn_residual_norm_bwd: a number of more than 32 bits");
  return gnn_residual_norm_bwd(a->dH, a->lddh, a->dY, a->lddy, (int32_t)a->y_type, a->B, a->ldb, (int32_t)a->b_type, a->H,
                               a->ldh, (int32_t)a->r_type, a->gate, a->ldg, (int32_t)a->gate_cols, (int32_t)a->gate_act, a->n,
                               (int32_t)a->C, (int32_t)a->post, a->w_post, a->b_post, a->scale, (int32_t)a->scale_cols,
                               (int32_t)a->pre, a->w_pre, a->stats, a->dR, a->lddr, a->dB, a->lddb, a->dgate, a->lddg,
                               a->dw_post, a->db_post, a->dscale, a->dw_pre, a->db_pre, a->ws, (size_t)a->ws_bytes, a->stream);
}
