// Group norm with an activation, channels last, over contiguous row ranges
// ("segments": graphs of a batch, or partitions), forward and backward.
//
// The rows are cut into tiles of R.  A segment of at most max(2R, 256) rows is
// "short": the block of the tile it starts in takes it whole, statistics and
// output in one launch (the second read of its rows comes from shared memory, L1
// or L2).  A longer segment is cut at the tile borders: the first launch leaves
// per (piece, group) partials, the second joins them in piece order, the third
// forms the output.  The piece of segment s in tile t has index t + s, which is
// unique because both only grow along the rows; so no plan has to be built from
// seg_start.
//
// Bound by memory where segments are long: X (backward: X and dY) is read twice,
// since a segment of a partition does not stay on the chip.  716847 x 300 fp32 to
// bf16 in 8 segments: 330 us on the GPU, 6.5 TB/s with the second read; 232965 x
// 602 backward: 366 us, 6.1 TB/s.  Many short segments (65537 x 256 in 2800,
// backward with gelu: 73 us for 0.2 GB) are bound by what a block does once per
// segment.  The backward on 2-byte rows spills (eight channels a thread, about 1 KB
// of reloads): 716847 x 256 bf16 in 8 segments takes 316 us, 5.8 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "internal.h"
#include "nodewise.cuh"

namespace gnn {

namespace {

// A block holds as many rows of CH chunks side by side as fit its threads, at
// least one: few threads are idle whatever a row's width (256 threads left 41% of
// them idle at 602 fp32 channels).  Where segments are short a block is 128
// threads: it takes them one at a time, and most of what a warp does for a
// segment does not depend on its rows.
constexpr int block_threads(int V, bool small = false) { return small ? 128 : V == 4 ? 384 : 192; }
constexpr int fwd_blocks(int V, bool small) { return small ? 6 : V == 4 ? 2 : 4; }  // per SM at least
constexpr int bwd_blocks(int V, bool small) { return small ? 5 : V == 4 ? 2 : 3; }
constexpr int FIN_THREADS = 512;

struct NormArgs {
  const void* X;
  const void* dY;
  void* out;  // Y or dX
  int64_t ldx, ldy, ldo;
  int n;
  int C, groups, cg, n_seg, act;
  int CH;  // chunks of V channels a row has, padding columns of the output included
  int RP;  // rows a block holds side by side: RP * CH threads take part
  int R;
  int longest;  // rows of a short segment
  int keep;     // rows of a thread that stay in shared memory
  int q;        // chunks of a group where groups are whole chunks, else 0
  int L;        // lanes that share a group in its sums
  int join_width;  // segments of a block of the join launch, up to 32
  int tiles;
  const int64_t* seg;  // may be NULL: one segment
  const float* gamma;
  const float* beta;
  float eps;
  float* mean;
  float* rstd;
  float2* part;  // forward: (mean, M2) of a piece's group; backward: the two sums
  float2* joined;  // backward: the two sums over a long segment's group, / m
  float* dpart;    // backward: [tiles][2][C] sums of dz and dz xh
  int* has_long;   // [tiles]: whether pieces of long segments are left for the last launch
  float* dgamma;
  float* dbeta;
  unsigned* flags;
};

// A border, brought into [0, n] whatever seg_start holds.
__device__ __forceinline__ int seg_at(const NormArgs& a, int s) {
  if (!a.seg) return s ? a.n : 0;
  return (int)min(max(a.seg[s], (int64_t)0), (int64_t)a.n);
}
// The segment that holds row r: the last one that starts at or before it.  A
// whole warp searches, 32 borders to a step: a step is a trip to L2, and a
// bisection's dozen of them took longer than a small batch's rows.
__device__ __forceinline__ int seg_of(const NormArgs& a, int r) {
  if (!a.seg) return 0;
  int lo = 0, hi = a.n_seg;  // seg[lo] <= r < seg[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 31) / 32, probe = lo + 1 + (int)(threadIdx.x & 31) * step;
    const int below = __popc(__ballot_sync(0xffffffffu, probe < hi && a.seg[probe < hi ? probe : lo] <= r));
    const int first = lo + 1 + below * step;  // the first probe past r
    hi = min(hi, first);
    if (below) lo = first - step;
  }
  return lo;
}

__device__ __forceinline__ float* align16(float* p) {
  return reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The pieces of tile t in row order: calls f(s, first row, end row, whole),
// `whole` true for a short segment taken from its first row to its last.
template <class Fn>
__device__ __forceinline__ void for_pieces(const NormArgs& a, int t, Fn f) {
  const int r0 = t * a.R, r1 = min((int64_t)a.n, (int64_t)r0 + a.R);
  int s = seg_of(a, r0);
  int row = r0;
  while (row < r1 && s < a.n_seg) {
    const int sb = seg_at(a, s), se = seg_at(a, s + 1);
    if (se <= row) {  // empty, perhaps one of many (or not ascending, which the join launch flags)
      s = max(s + 1, seg_of(a, row));
      continue;
    }
    if (sb > row) break;
    if (se - sb <= a.longest) {
      if (sb >= r0) f(s, sb, se, true);
    } else {
      f(s, row, min(se, r1), false);
    }
    row = se;
    ++s;
  }
}

// A thread's place: V channels of every RP-th row of a piece.
template <int V>
struct Place {
  int ro, c0;
  bool on, in;  // takes part; has channels below C
  int g[V];
  __device__ __forceinline__ Place(const NormArgs& a) {
    ro = threadIdx.x / a.CH;
    c0 = (threadIdx.x % a.CH) * V;
    on = ro < a.RP;
    in = on && c0 < a.C;
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = min(c0 + k, a.C - 1) / a.cg;
  }
  // how many rows of [ra, rb) are this thread's
  __device__ __forceinline__ int rows(const NormArgs& a, int ra, int rb) const {
    return on ? (unsigned)(rb - ra - ro + a.RP - 1) / (unsigned)a.RP : 0;
  }
};

// A thread's own ring in shared memory: pairs of rows are requested with
// asynchronous copies DEPTH pairs ahead of their use, so 2 DEPTH rows a thread
// are in flight at no cost in registers.  Every thread reads only what it
// copied itself, so there is no barrier; the slot that is filled is the one
// that was used up an iteration earlier.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// V elements from a shared-memory address, as fp32.
template <int V, class T>
__device__ __forceinline__ void load_shared(uint32_t at, float (&v)[V]) {
  constexpr int W = V * sizeof(T) / 4;
  uint32_t w[W];
  if constexpr (W == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(at + 4 * i)
                   : "memory");
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = Pack2<T>::from(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_shared(uint32_t at, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 4 * i), "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]),
                 "f"(v[i + 3])
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One or two matrices (pb NULL: one) walked row by row in steps of da, db
// elements from pa, pb, V elements a row and thread; f(a, b) for every row.
template <int V, int DEPTH, bool TWO, class TA, class TB, class Fn>
__device__ __forceinline__ void stream_rows(char* ring, int rows, const TA* pa, int64_t da, const TB* pb,
                                            int64_t db, Fn f) {
  constexpr int SA = V * sizeof(TA), SB = V * sizeof(TB);
  const uint32_t row_a = blockDim.x * SA, row_b = blockDim.x * SB;  // bytes between a slot's two rows
  const uint32_t end = 2 * row_a * (DEPTH + 1);
  const uint32_t sa = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * SA;
  const uint32_t sb = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + end + threadIdx.x * SB;
  int ahead = rows;  // rows not yet requested
  auto request = [&](uint32_t slot) {
    if (ahead > 0) {
      copy_async<SA>(sa + slot, pa);
      if (TWO) copy_async<SB>(sb + slot * SB / SA, pb);
    }
    if (ahead > 1) {
      copy_async<SA>(sa + slot + row_a, pa + da);
      if (TWO) copy_async<SB>(sb + slot * SB / SA + row_b, pb + db);
    }
    ahead -= 2;
    pa += 2 * da;
    if (TWO) pb += 2 * db;
    copy_commit();
  };
  auto read = [&](uint32_t slot, int second, float (&a)[V], float (&b)[V]) {
    load_shared<V, TA>(sa + slot + second * row_a, a);
    if (TWO) load_shared<V, TB>(sb + slot * SB / SA + second * row_b, b);
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) request(i * 2 * row_a);
  uint32_t use = 0, fill = DEPTH * 2 * row_a;
  for (int i = rows; i > 0; i -= 2) {
    copy_wait<DEPTH - 1>();
    float a0[V], b0[V], a1[V], b1[V];
    read(use, 0, a0, b0);
    read(use, 1, a1, b1);  // without a second row: what the slot held, not used
    request(fill);
    fill = use;
    use += 2 * row_a;
    if (use == end) use = 0;
    f(a0, b0);
    if (i > 1) f(a1, b1);
  }
  copy_wait<0>();
}
constexpr int FWD_DEPTH = 4, BWD_DEPTH = 2;

// Zero in the columns of the thread that are past C.
template <int V>
__device__ __forceinline__ void clear_padding(const Place<V>& p, int C, float (&v)[V]) {
  if (p.c0 + V > C) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (p.c0 + k >= C) v[k] = 0.f;
  }
}

// One fp32 value per channel of the thread (the fill where src is NULL).
template <int V>
__device__ __forceinline__ void load_channels(const float* src, const Place<V>& p, int C, float fill,
                                              float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = src && p.c0 + k < C ? src[p.c0 + k] : fill;
}

// Sums over the row places, then over each group's channels: red1/red2 hold
// [RP][CH * V] partials; ch1/ch2 [C] get the channel sums and f(g, s1, s2) runs
// in one lane per group with the group's sums, each channel times w[c] (NULL:
// 1).  L lanes (a power of two) share a group, so narrow groups do not leave
// most of a warp idle.  A barrier of the caller's ends it.
template <class Fn>
__device__ __forceinline__ void block_sums(const NormArgs& a, int width, const float* red1,
                                           const float* red2, float* ch1, float* ch2, const float* w,
                                           Fn f) {
  const int L = a.L;
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
    float s1 = 0.f, s2 = 0.f;
    for (int r = 0; r < a.RP; ++r) {
      s1 += red1[r * width + c];
      s2 += red2[r * width + c];
    }
    ch1[c] = s1;
    ch2[c] = s2;
  }
  __syncthreads();
  const int per = blockDim.x / L, l = threadIdx.x & (L - 1);
  for (int g0 = 0; g0 < a.groups; g0 += per) {
    const int g = g0 + threadIdx.x / L;
    float s1 = 0.f, s2 = 0.f;
    if (g < a.groups) {
      for (int j = l; j < a.cg; j += L) {
        const int c = g * a.cg + j;
        const float wc = w ? w[c] : 1.f;
        s1 += wc * ch1[c];
        s2 += wc * ch2[c];
      }
    }
    for (int o = L >> 1; o; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (g < a.groups && l == 0) f(g, s1, s2);
  }
}

// The same where a group is whole chunks, for small blocks (65537 x 256 in 2800
// segments backward 79.4 -> 77.0 us, in bf16 forward 46 -> 41 us; in large blocks
// its registers cost more than it saves): a thread brings one pair of sums over
// its channels, which lands beside the others of its group; half the barriers and
// a quarter of the traffic of the way over channels.  part: [groups][RP q].
template <class Fn>
__device__ __forceinline__ void chunk_sums(const NormArgs& a, float2* part, int at, bool in, float s1, float s2, Fn f) {
  if (in) part[at] = make_float2(s1, s2);
  __syncthreads();
  const int per = blockDim.x / a.L, l = threadIdx.x & (a.L - 1), count = a.RP * a.q;
  for (int g0 = 0; g0 < a.groups; g0 += per) {
    const int g = g0 + threadIdx.x / a.L;
    s1 = s2 = 0.f;
    if (g < a.groups) {
      for (int e = l; e < count; e += a.L) {
        const float2 v = part[g * count + e];
        s1 += v.x;
        s2 += v.y;
      }
    }
    for (int o = a.L >> 1; o; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (g < a.groups && l == 0) f(g, s1, s2);
  }
}
// A thread's place in them.
template <int V>
__device__ __forceinline__ int chunk_place(const NormArgs& a, const Place<V>& p) {
  return p.g[0] * (a.RP * a.q) + p.ro * a.q + (p.c0 - p.g[0] * a.cg) / V;
}

// Mean, gamma rstd and beta of a thread's channels.
template <int V>
__device__ __forceinline__ void fwd_channels(const NormArgs& a, const Place<V>& p, const float* gmean,
                                             const float* grstd, float (&mu)[V], float (&sc)[V], float (&bt)[V]) {
  load_channels<V>(a.gamma, p, a.C, 1.f, sc);
  load_channels<V>(a.beta, p, a.C, 0.f, bt);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    mu[k] = gmean[p.g[k]];
    sc[k] *= grstd[p.g[k]];
  }
}
// act((x - mean) gamma rstd + beta)
template <int V, class Act>
__device__ __forceinline__ void fwd_output(const float (&x)[V], const float (&mu)[V], const float (&sc)[V],
                                           const float (&bt)[V], float (&y)[V], Act act) {
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    const float2 d = add2_rn(make_float2(x[k], x[k + 1]), make_float2(-mu[k], -mu[k + 1]));
    const float2 v = act2(fma2_rn(d, make_float2(sc[k], sc[k + 1]), make_float2(bt[k], bt[k + 1])), act);
    y[k] = v.x, y[k + 1] = v.y;
  }
}

// Y of the rows [ra, rb) from per-group (mean, rstd), last rows first: those
// are the ones the statistics pass read last and the caches still hold.
template <class TX, class TY, int V>
__device__ __forceinline__ void fwd_rows(const NormArgs& a, const Place<V>& p, int ra, int rb,
                                         const float* gmean, const float* grstd, char* ring) {
  const int rows = p.rows(a, ra, rb);
  float mu[V], sc[V], bt[V];
  fwd_channels<V>(a, p, gmean, grstd, mu, sc, bt);
  const int64_t last = ra + p.ro + (rows - 1) * a.RP;
  const TX* X = static_cast<const TX*>(a.X) + last * a.ldx + p.c0;
  TY* Y = static_cast<TY*>(a.out) + last * a.ldo + p.c0;
  const int64_t dx = (int64_t)a.RP * a.ldx, dy = (int64_t)a.RP * a.ldo;
  if (!p.in) {  // padding columns only
    const float zero[V] = {};
    for (int i = 0; i < rows; ++i, Y -= dy) store_vec<V>(Y, zero);
    return;
  }
  with_act(a.act, [&](auto act) {
    stream_rows<V, FWD_DEPTH, false>(ring, rows, X, -dx, X, 0, [&](float (&x)[V], float (&)[V]) {
      float y[V];
      fwd_output<V>(x, mu, sc, bt, y, act);
      clear_padding<V>(p, a.C, y);
      store_vec<V>(Y, y);
      Y -= dy;
    });
  });
}

// Statistics of every piece of a tile; short segments end here with their
// output.  A group's sums S, Q of d = x - pivot and d^2 are formed about its value
// in the piece's first row, so a mean far from zero does not cancel in
// M2 = Q - S^2/m.  The pivot has to be a typical value for that: the difference
// loses 1 + (mean - pivot)^2/var of the sums' precision.  Where that is more than
// 1 + kFar in any group, the sums are formed once more about the mean that the
// first ones gave, which is off by a few 2^-24 of |mean - pivot| and so by less
// than the deviation (that is at least |mean - pivot|/sqrt(m)).  Of normally
// distributed pieces one group in 16,000 takes the second turn; where every piece
// of 716847 x 300 takes it, the forward takes 410 us instead of 333.
constexpr float kFar = 16.f;
// Also where Q has left fp32's range, but not where the rows hold what is not finite.
__device__ __forceinline__ bool is_far(float d, float var, float mean) {
  return !(d * d <= kFar * var) && fabsf(mean) < __int_as_float(0x7f800000);
}
template <class TX, class TY, int V, bool SMALL>
__global__ void __launch_bounds__(block_threads(V, SMALL), fwd_blocks(V, SMALL)) norm_fwd_stats_kernel(NormArgs a) {
  extern __shared__ float sm[];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const Place<V> p(a);
  const int width = a.CH * V;
  float* red1 = sm;
  float* red2 = red1 + a.RP * width;
  float* ch1 = red2 + a.RP * width;
  float* ch2 = ch1 + a.C;
  float* gm = ch2 + a.C;
  float* gr = gm + a.groups;
  float2* part = reinterpret_cast<float2*>(align16(gr + a.groups));
  char* ring = reinterpret_cast<char*>(align16(reinterpret_cast<float*>(part + a.RP * a.CH)));
  const bool chunks = SMALL && a.q;  // the sums go over chunks
  const int at_part = chunks ? chunk_place<V>(a, p) : 0;
  const TX* X = static_cast<const TX*>(a.X);
  const int t = blockIdx.x;
  int left = 0;  // pieces of long segments
  // slot i of this thread: its i-th row of a short segment, kept for the output
  const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16;
  const uint32_t next = blockDim.x * 16;
  for_pieces(a, t, [&](int s, int ra, int rb, bool whole) {
    left |= !whole;
    const bool keep = whole && rb - ra <= a.keep * a.RP;
    const int rows = p.rows(a, ra, rb);
    const float inv = rcp_f((float)(rb - ra) * (float)a.cg);  // 1 / values of a group
    // AGAIN: the turn about the mean, in code of its own (one loop for both turns spilt:
    // 716847 x 256 bf16 215 us against 201); true where another one is due
    const auto sums = [&](auto AGAIN) -> bool {
      constexpr bool again = decltype(AGAIN)::value;
      bool far = false;  // in a group whose sums this thread finished
      float s1 = 0.f, s2 = 0.f;  // over this thread's channels
      if (p.on) {
        constexpr int U = 32 / V;
        float piv[V], S[V], Q[V];
        const TX* at = X + (ra + p.ro) * a.ldx + p.c0;
        const int64_t dx = (int64_t)a.RP * a.ldx;
        if (keep && p.in && !again) {
          for (int i = 0; i < rows; ++i, at += dx) copy_async<16>(slots + i * next, at);
          copy_commit();
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
          piv[k] = again ? gm[p.g[k]] : to_f32(X[ra * a.ldx + (int64_t)p.g[k] * a.cg]);
          S[k] = 0.f;
          Q[k] = 0.f;
        }
        const auto add = [&](const float (&x)[V]) {
#pragma unroll
          for (int k = 0; k < V; k += 2) {
            const float2 d = add2_rn(make_float2(x[k], x[k + 1]), make_float2(-piv[k], -piv[k + 1]));
            const float2 s2 = add2_rn(make_float2(S[k], S[k + 1]), d);
            const float2 q2 = fma2_rn(d, d, make_float2(Q[k], Q[k + 1]));
            S[k] = s2.x, S[k + 1] = s2.y, Q[k] = q2.x, Q[k + 1] = q2.y;
          }
        };
        if (keep) {
          copy_wait<0>();
          int i = 0;
          for (; p.in && i + 4 <= rows; i += 4) {
            float x[4][V];
#pragma unroll
            for (int u = 0; u < 4; ++u) load_shared<V, TX>(slots + (i + u) * next, x[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) add(x[u]);
          }
          for (; p.in && i < rows; ++i) {
            float x[V];
            load_shared<V, TX>(slots + i * next, x);
            add(x);
          }
        }
        for (int i = p.in && !keep ? rows : 0; i > 0; i -= U) {
          float x[U][V];
#pragma unroll
          for (int u = 0; u < U; ++u, at += dx) {
            if (u < i) {
              load_vec<V>(at, x[u]);
            } else {
#pragma unroll
              for (int k = 0; k < V; ++k) x[u][k] = piv[k];
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) add(x[u]);
        }
        if (chunks) {
#pragma unroll
          for (int k = 0; k < V; ++k) s1 += S[k], s2 += Q[k];
        } else {
          store_vec<V>(red1 + p.ro * width + p.c0, S);
          store_vec<V>(red2 + p.ro * width + p.c0, Q);
        }
      }
      const auto finish = [&](int g, float S, float Q) {
        const float d = S * inv;
        const float mean = (again ? gm[g] : to_f32(X[ra * a.ldx + (int64_t)g * a.cg])) + d;
        const float m2 = fmaxf(Q - S * d, 0.f) + 0.f * Q;  // the product keeps a NaN
        gm[g] = mean;
        if (is_far(d, m2 * inv, mean)) far = true;
        if (whole) {
          const float rstd = rsqrtf(m2 * inv + a.eps);
          gr[g] = rstd;
          a.mean[(int64_t)s * a.groups + g] = mean;
          a.rstd[(int64_t)s * a.groups + g] = rstd;
        } else {
          a.part[((int64_t)t + s) * a.groups + g] = make_float2(mean, m2);
        }
      };
      if (chunks)
        chunk_sums(a, part, at_part, p.in, s1, s2, finish);
      else
        block_sums(a, width, red1, red2, ch1, ch2, nullptr, finish);
      if constexpr (again) {
        __syncthreads();
        return false;
      } else {
        return __syncthreads_or(far);  // ends the sums, and decides for the whole block
      }
    };
    if (sums(std::false_type())) sums(std::true_type());
    if (keep) {
      float mu[V], sc[V], bt[V];
      fwd_channels<V>(a, p, gm, gr, mu, sc, bt);
      TY* Y = static_cast<TY*>(a.out) + (ra + p.ro) * a.ldo + p.c0;
      const int64_t dy = (int64_t)a.RP * a.ldo;
      with_act(a.act, [&](auto act) {
        for (int i = 0; i < rows; ++i, Y += dy) {
          float x[V] = {}, y[V];
          if (p.in) load_shared<V, TX>(slots + i * next, x);
          fwd_output<V>(x, mu, sc, bt, y, act);
          clear_padding<V>(p, a.C, y);
          store_vec<V>(Y, y);
        }
      });
    } else if (whole) {
      fwd_rows<TX, TY, V>(a, p, ra, rb, gm, gr, ring);
    }
    if (whole) __syncthreads();  // gm, gr, the partials and the slots are written again
  });
  if (threadIdx.x == 0) a.has_long[t] = left;
}

// Segments without rows, and what seg_start has to be.
__device__ __forceinline__ void check_segments(const NormArgs& a, int blocks, bool fill) {
  const int64_t stride = (int64_t)blocks * blockDim.x;
  for (int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; s < a.n_seg; s += stride) {
    const int64_t sb = a.seg ? a.seg[s] : 0, se = a.seg ? a.seg[s + 1] : a.n;
    if (sb > se || (s == 0 && sb != 0) || (s == a.n_seg - 1 && se != a.n)) atomicOr(a.flags, 1u);
    if (fill && se <= sb) {
      for (int g = 0; g < a.groups; ++g) {
        a.mean[s * a.groups + g] = 0.f;
        a.rstd[s * a.groups + g] = rsqrtf(a.eps);
      }
    }
  }
}

// Calls f(s, first row, end row, first piece's tile, last one's, group) in every
// warp for the long segments and groups of this block: up to 32 segments, which a
// warp looks over at once, and 16 groups to a block.  Few segments get a block each
// (eight in one block's turn: 367 against 327 us at 716847 x 300 forward).
constexpr int JOIN_GROUPS = FIN_THREADS / 32;
template <class Fn>
__device__ __forceinline__ void for_long(const NormArgs& a, int blocks, Fn f) {
  const int parts = (a.groups + JOIN_GROUPS - 1) / JOIN_GROUPS, lane = threadIdx.x & 31;
  const int g = (int)(blockIdx.x % parts) * JOIN_GROUPS + (threadIdx.x >> 5);
  const int64_t w = a.join_width;
  for (int64_t b = blockIdx.x / parts * w; b < a.n_seg; b += blocks / parts * w) {
    int sb = 0, se = 0;
    if (lane < w && b + lane < a.n_seg) sb = seg_at(a, (int)b + lane), se = seg_at(a, (int)b + lane + 1);
    unsigned some = __ballot_sync(0xffffffffu, se - sb > a.longest);
    if (g >= a.groups) some = 0;
    for (; some; some &= some - 1) {
      const int k = __ffs(some) - 1;
      const int first = __shfl_sync(0xffffffffu, sb, k), end = __shfl_sync(0xffffffffu, se, k);
      f((int)b + k, first, end, first / a.R, (end - 1) / a.R, g);
    }
  }
}

// Joins the pieces of long segments about the first one's mean: with
// d_i = mean_i - mean_0 and D = sum m_i d_i / M, mean = mean_0 + D and
// M2 = sum (M2_i + m_i d_i^2) - M D^2.  Where the first piece lies far from the
// others, once more about the mean, as above (always both: 47 -> 52 us at one
// segment of 65537 x 256).
__global__ void __launch_bounds__(FIN_THREADS) norm_fwd_join_kernel(NormArgs a) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  check_segments(a, gridDim.x, true);
  const int lane = threadIdx.x & 31;
  for_long(a, gridDim.x, [&](int s, int sb, int se, int t0, int t1, int g) {
    const float2* part = a.part + (int64_t)s * a.groups + g;
    float about = part[(int64_t)t0 * a.groups].x;
    for (int turn = 0; turn < 2; ++turn) {
      float M = 0.f, S = 0.f, Q = 0.f;
#pragma unroll 8
      for (int i = t0 + lane; i <= t1; i += 32) {
        const float2 v = part[(int64_t)i * a.groups];
        const float m = (float)((int)min((int64_t)se, (i + 1) * (int64_t)a.R) - max(sb, i * a.R)) * (float)a.cg;
        const float d = v.x - about;
        M += m;
        S += m * d;
        Q += v.y + m * d * d;
      }
      M = warp_sum(M), S = warp_sum(S), Q = warp_sum(Q);
      const float D = S / M, var = fmaxf(Q - S * D, 0.f) / M + 0.f * Q;
      about += D;
      if (lane == 0) {
        a.mean[(int64_t)s * a.groups + g] = about;
        a.rstd[(int64_t)s * a.groups + g] = rsqrtf(var + a.eps);
      }
      if (!is_far(D, var, about)) break;  // the same in every lane
    }
  });
}

template <class TX, class TY, int V>
__global__ void __launch_bounds__(block_threads(V), fwd_blocks(V, false)) norm_fwd_apply_kernel(NormArgs a) {
  extern __shared__ float sm[];
  cudaGridDependencySynchronize();
  // last tiles first, as within a tile
  const int t = a.tiles - 1 - (int)blockIdx.x;
  if (!a.has_long[t]) return;
  const Place<V> p(a);
  for_pieces(a, t, [&](int s, int ra, int rb, bool whole) {
    if (!whole)
      fwd_rows<TX, TY, V>(a, p, ra, rb, a.mean + (int64_t)s * a.groups, a.rstd + (int64_t)s * a.groups,
                             reinterpret_cast<char*>(sm));
  });
}

// ------------------------------------------------------------------ backward
// gamma and beta of a thread's channels, and one segment's statistics of them.
template <int V>
struct BwdChannels {
  float mu[V], rs[V], ga[V], be[V];
  __device__ __forceinline__ BwdChannels(const NormArgs& a, const Place<V>& p) {
    load_channels<V>(a.gamma, p, a.C, 1.f, ga);
    load_channels<V>(a.beta, p, a.C, 0.f, be);
  }
  __device__ __forceinline__ void segment(const NormArgs& a, const Place<V>& p, int s) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      mu[k] = a.mean[(int64_t)s * a.groups + p.g[k]];
      rs[k] = a.rstd[(int64_t)s * a.groups + p.g[k]];
    }
  }
  // x becomes xh and dy becomes dz
  template <class Act>
  __device__ __forceinline__ void derive(float (&x)[V], float (&dy)[V], Act act) const {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 xh = mul2_rn(add2_rn(make_float2(x[k], x[k + 1]), make_float2(-mu[k], -mu[k + 1])),
                                make_float2(rs[k], rs[k + 1]));
      float2 av, d;
      act_grad2(fma2_rn(make_float2(ga[k], ga[k + 1]), xh, make_float2(be[k], be[k + 1])), act, av, d);
      d = mul2_rn(make_float2(dy[k], dy[k + 1]), d);
      x[k] = xh.x, x[k + 1] = xh.y, dy[k] = d.x, dy[k + 1] = d.y;
    }
  }
  // rs (gamma dz - A - xh B)
  __device__ __forceinline__ void output(const float (&xh)[V], const float (&dz)[V], const float (&A)[V],
                                         const float (&B)[V], float (&o)[V]) const {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      float2 v = fma2_rn(make_float2(ga[k], ga[k + 1]), make_float2(dz[k], dz[k + 1]), make_float2(-A[k], -A[k + 1]));
      v = fma2_rn(make_float2(-xh[k], -xh[k + 1]), make_float2(B[k], B[k + 1]), v);
      v = mul2_rn(v, make_float2(rs[k], rs[k + 1]));
      o[k] = v.x, o[k + 1] = v.y;
    }
  }
};

// P1 += dz, P2 += dz xh
template <int V>
__device__ __forceinline__ void add_sums(const float (&xh)[V], const float (&dz)[V], float (&P1)[V], float (&P2)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    const float2 z = make_float2(dz[k], dz[k + 1]);
    const float2 s = add2_rn(make_float2(P1[k], P1[k + 1]), z);
    const float2 q = fma2_rn(z, make_float2(xh[k], xh[k + 1]), make_float2(P2[k], P2[k + 1]));
    P1[k] = s.x, P1[k + 1] = s.y, P2[k] = q.x, P2[k + 1] = q.y;
  }
}

// dX of the rows [ra, rb); gA, gB: the segment's two sums over each group, / m.
template <class TX, class TY, int V>
__device__ __forceinline__ void bwd_rows(const NormArgs& a, const Place<V>& p, const BwdChannels<V>& b,
                                         int ra, int rb, const float* gA, const float* gB, int gstride,
                                         char* ring) {
  const int rows = p.rows(a, ra, rb);
  float A[V], B[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    A[k] = gA[p.g[k] * gstride];
    B[k] = gB[p.g[k] * gstride];
  }
  const int64_t last = ra + p.ro + (rows - 1) * a.RP;
  const TX* X = static_cast<const TX*>(a.X) + last * a.ldx + p.c0;
  const TY* dY = static_cast<const TY*>(a.dY) + last * a.ldy + p.c0;
  TX* dX = static_cast<TX*>(a.out) + last * a.ldo + p.c0;
  const int64_t sx = (int64_t)a.RP * a.ldx, sy = (int64_t)a.RP * a.ldy, so = (int64_t)a.RP * a.ldo;
  if (!p.in) {
    const float zero[V] = {};
    for (int i = 0; i < rows; ++i, dX -= so) store_vec<V>(dX, zero);
    return;
  }
  with_act(a.act, [&](auto act) {
    stream_rows<V, BWD_DEPTH, true>(ring, rows, X, -sx, dY, -sy, [&](float (&x)[V], float (&dy)[V]) {
      float o[V];
      b.derive(x, dy, act);
      b.output(x, dy, A, B, o);
      clear_padding<V>(p, a.C, o);
      store_vec<V>(dX, o);
      dX -= so;
    });
  });
}

// A short segment of at most a.keep rows a thread stays in shared memory between
// its sums and its output, as xh and dz in fp32: nothing is read or derived
// twice then.
template <class TX, class TY, int V, bool SMALL>
__global__ void __launch_bounds__(block_threads(V, SMALL), bwd_blocks(V, SMALL)) norm_bwd_sums_kernel(NormArgs a) {
  extern __shared__ float sm[];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const Place<V> p(a);
  const int width = a.CH * V;
  float* red1 = sm;
  float* red2 = red1 + a.RP * width;
  float* ch1 = red2 + a.RP * width;
  float* ch2 = ch1 + a.C;
  float* acc1 = ch2 + a.C;  // this block's share of dbeta, dgamma
  float* acc2 = acc1 + a.C;
  float* gA = acc2 + a.C;
  float* gB = gA + a.groups;
  float2* part = reinterpret_cast<float2*>(align16(gB + a.groups));
  char* ring = reinterpret_cast<char*>(align16(reinterpret_cast<float*>(part + a.RP * a.CH)));
  const bool chunks = SMALL && a.q;  // the sums go over chunks
  const int at_part = chunks ? chunk_place<V>(a, p) : 0;
  const TX* X = static_cast<const TX*>(a.X);
  const TY* dY = static_cast<const TY*>(a.dY);
  constexpr int SLOT = V * 4;
  // slot i of this thread: xh (first x) and, `keep` slots on, dz (first dY)
  const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * SLOT;
  const uint32_t next = blockDim.x * SLOT, dz_at = a.keep * next;
  BwdChannels<V> b(a, p);
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) acc1[c] = acc2[c] = 0.f;
  // where groups are whole chunks, red1 and red2 hold each thread's own shares of
  // dbeta and dgamma over the tile
  float* own1 = red1 + p.ro * width + p.c0;
  float* own2 = red2 + p.ro * width + p.c0;
  if (chunks && p.on) {
    const float zero[V] = {};
    store_vec<V>(own1, zero);
    store_vec<V>(own2, zero);
  }
  const int t = blockIdx.x;
  int left = 0;
  for_pieces(a, t, [&](int s, int ra, int rb, bool whole) {
    left |= !whole;
    const bool keep = whole && rb - ra <= a.keep * a.RP;
    const int rows = p.rows(a, ra, rb);
    float s1 = 0.f, s2 = 0.f;  // over this thread's channels
    if (p.on) {
      const TX* px = X + (ra + p.ro) * a.ldx + p.c0;
      const TY* py = dY + (ra + p.ro) * a.ldy + p.c0;
      const int64_t sx = (int64_t)a.RP * a.ldx, sy = (int64_t)a.RP * a.ldy;
      float P1[V], P2[V];
#pragma unroll
      for (int k = 0; k < V; ++k) P1[k] = P2[k] = 0.f;
      if (keep && p.in) {
        for (int i = 0; i < rows; ++i, px += sx, py += sy) {
          copy_async<V * sizeof(TX)>(slots + i * next, px);
          copy_async<V * sizeof(TY)>(slots + dz_at + i * next, py);
        }
        copy_commit();
      }
      b.segment(a, p, s);
      with_act(a.act, [&](auto act) {
        if (keep) {
          copy_wait<0>();
          // two rows at a time, for their independent chains
          for (int i = 0; i < (p.in ? rows : 0); i += 2) {
            const uint32_t at = slots + i * next;
            const bool two = i + 1 < rows;
            float x[V], dy[V], x1[V], dy1[V];
            load_shared<V, TX>(at, x);
            load_shared<V, TY>(at + dz_at, dy);
            if (two) {
              load_shared<V, TX>(at + next, x1);
              load_shared<V, TY>(at + next + dz_at, dy1);
              b.derive(x1, dy1, act);
              add_sums<V>(x1, dy1, P1, P2);
              store_shared<V>(at + next, x1);
              store_shared<V>(at + next + dz_at, dy1);
            }
            b.derive(x, dy, act);
            add_sums<V>(x, dy, P1, P2);
            store_shared<V>(at, x);
            store_shared<V>(at + dz_at, dy);
          }
        } else {
          stream_rows<V, BWD_DEPTH, true>(ring, p.in ? rows : 0, px, sx, py, sy, [&](float (&x)[V], float (&dy)[V]) {
            b.derive(x, dy, act);
            add_sums<V>(x, dy, P1, P2);
          });
        }
      });
      if (chunks) {
        float o1[V], o2[V];
        load_vec<V>(own1, o1);
        load_vec<V>(own2, o2);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          s1 += b.ga[k] * P1[k], s2 += b.ga[k] * P2[k];
          o1[k] += P1[k], o2[k] += P2[k];
        }
        store_vec<V>(own1, o1);
        store_vec<V>(own2, o2);
      } else {
        store_vec<V>(own1, P1);
        store_vec<V>(own2, P2);
      }
    }
    const float inv = rcp_f((float)(rb - ra) * (float)a.cg);  // 1 / values of a group
    const auto finish = [&](int g, float A, float B) {
      if (whole) {
        gA[g] = A * inv;
        gB[g] = B * inv;
      } else {
        a.part[((int64_t)t + s) * a.groups + g] = make_float2(A, B);
      }
    };
    if (chunks) {
      chunk_sums(a, part, at_part, p.in, s1, s2, finish);
      __syncthreads();
    } else {
      block_sums(a, width, red1, red2, ch1, ch2, a.gamma, finish);
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        acc1[c] += ch1[c];
        acc2[c] += ch2[c];
      }
    }
    if (keep) {
      TX* dX = static_cast<TX*>(a.out) + (ra + p.ro) * a.ldo + p.c0;
      const int64_t so = (int64_t)a.RP * a.ldo;
      float A[V], B[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        A[k] = gA[p.g[k]];
        B[k] = gB[p.g[k]];
      }
      for (int i = 0; i < rows; ++i, dX += so) {
        float xh[V] = {}, dz[V] = {}, o[V];
        if (p.in) {
          load_shared<V, float>(slots + i * next, xh);
          load_shared<V, float>(slots + dz_at + i * next, dz);
        }
        b.output(xh, dz, A, B, o);
        clear_padding<V>(p, a.C, o);
        store_vec<V>(dX, o);
      }
    } else if (whole) {
      bwd_rows<TX, TY, V>(a, p, b, ra, rb, gA, gB, 1, ring);
    }
    __syncthreads();
  });
  if (threadIdx.x == 0) a.has_long[t] = left;
  if (a.dpart) {
    float* d = a.dpart + (int64_t)t * 2 * a.C;
    if (chunks) __syncthreads();
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
      float v1 = acc1[c], v2 = acc2[c];
      for (int i = 0; chunks && i < a.RP; ++i) {
        v1 += red1[i * width + c];
        v2 += red2[i * width + c];
      }
      d[c] = v1;
      d[a.C + c] = v2;
    }
  }
}

// The first `joiners` blocks join long segments; the others add the blocks'
// shares of dbeta and dgamma, 8 columns each, in a fixed order.
__global__ void __launch_bounds__(FIN_THREADS) norm_bwd_join_kernel(NormArgs a, int joiners) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= joiners) {
    // 8 columns to a block: 64 threads share each
    __shared__ float red[FIN_THREADS / 8][8];
    const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int col = ((int)blockIdx.x - joiners) * 8 + c;
    float sum = 0.f;
    if (col < 2 * a.C) {
#pragma unroll 8
      for (int i = r; i < a.tiles; i += FIN_THREADS / 8) sum += a.dpart[(int64_t)i * 2 * a.C + col];
    }
    red[r][c] = sum;
    __syncthreads();
    if (r < 4) {
      sum = 0.f;
      for (int w = r; w < FIN_THREADS / 8; w += 4) sum += red[w][c];
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (r == 0 && col < 2 * a.C) {
        if (col < a.C) {
          if (a.dbeta) a.dbeta[col] = sum;
        } else if (a.dgamma) {
          a.dgamma[col - a.C] = sum;
        }
      }
    }
    return;
  }
  check_segments(a, joiners, false);
  for_long(a, joiners, [&](int s, int sb, int se, int t0, int t1, int g) {
    const float m = (float)(se - sb) * (float)a.cg;
    const float2* part = a.part + (int64_t)s * a.groups + g;
    float A = 0.f, B = 0.f;
#pragma unroll 8
    for (int i = t0 + lane; i <= t1; i += 32) {
      const float2 v = part[(int64_t)i * a.groups];
      A += v.x;
      B += v.y;
    }
    A = warp_sum(A), B = warp_sum(B);
    if (lane == 0) a.joined[(int64_t)s * a.groups + g] = make_float2(A / m, B / m);
  });
}

template <class TX, class TY, int V>
__global__ void __launch_bounds__(block_threads(V), bwd_blocks(V, false)) norm_bwd_apply_kernel(NormArgs a) {
  extern __shared__ float sm[];
  cudaGridDependencySynchronize();
  // last tiles first, as within a tile
  const int t = a.tiles - 1 - (int)blockIdx.x;
  if (!a.has_long[t]) return;
  const Place<V> p(a);
  for_pieces(a, t, [&](int s, int ra, int rb, bool whole) {
    if (!whole) {
      const float* j = &a.joined[(int64_t)s * a.groups].x;
      BwdChannels<V> b(a, p);
      b.segment(a, p, s);
      bwd_rows<TX, TY, V>(a, p, b, ra, rb, j, j + 1, 2, reinterpret_cast<char*>(sm));
    }
  });
}

// ---------------------------------------------------------------- host side
// Tiles per SM: a long segment's balance better when there are more of them, up
// to what their partials cost (measured with 4, 8, 16: 716847 x 300 in 8 segments
// forward 365, 342, 326 us; 232965 x 602 in 8 backward 365, 368, 387 us; 65537 x
// 256 in 2800 backward, with 10 kept rows a thread, -, 78, 94 us).  A tile has at
// least 16 rows, and 16 a thread while that leaves two tiles an SM.
//
// Blocks are small where the segments have kShortMean rows or fewer in the mean
// (65537 x 256, small against large blocks, forward and backward: 51, 78 against
// 76, 81 us at 23 rows; 56, 98 against 61, 83 us at 55; one long segment behind
// 2,000 to 20,000 of one row each, whose mean is below kShortMean too: 139 to 144
// against 282 to 339).  A segment of kShortRows or fewer is one block's in any case.
constexpr int kShortRows = 256, kShortMean = 40;

int tile_rows(int64_t n, int RP, bool backward, bool small) {
  const auto per = [&](int64_t tiles) { return (int)((n + tiles - 1) / tiles); };
  int R = per(small || backward ? 152 * 8 : 152 * 16);
  // whole turns of two blocks an SM, 16 rows a thread where they allow it
  if (!small) R = std::max(R, per(152 * 2 * std::max<int64_t>(n / (16 * RP) / (152 * 2), 1)));
  return std::max(R, std::max(RP, 16));
}
int64_t most_tiles(int64_t n) {
  const int64_t R = std::max<int64_t>((n + 152 * 16 - 1) / (152 * 16), 16);
  return (n + R - 1) / R;
}

struct NormWs {
  float2* part;
  float2* joined;
  float* dpart;
  int* has_long;
  size_t bytes;
};
NormWs norm_ws(void* base, size_t cap, int64_t n, int C, int groups, int n_seg, bool* ok) {
  Arena ar(base, cap);
  NormWs w{};
  w.part = ar.take<float2>((size_t)(most_tiles(n) + n_seg) * groups);
  w.joined = ar.take<float2>((size_t)n_seg * groups);
  w.dpart = ar.take<float>((size_t)most_tiles(n) * 2 * C);
  w.has_long = ar.take<int>((size_t)most_tiles(n));
  w.bytes = ar.used;
  *ok = ar.ok();
  return w;
}

gnn_status check_norm(const char* who, int64_t n, int C, int groups, int n_seg) {
  if (n < 0 || n > (int64_t)0x7fffffff) return fail(GNN_ERR_INVALID_ARG, "%s: bad row count", who);
  if (C < 1 || groups < 1 || C % groups || n_seg < 1 || n_seg > 0x3fffffff)
    return fail(GNN_ERR_INVALID_ARG, "%s: needs groups >= 1 that divide C >= 1, and 1 <= n_seg < 2^30", who);
  if (C > kMaxF) return fail(GNN_ERR_UNSUPPORTED, "%s: C=%d > %d", who, C, kMaxF);
  return GNN_OK;
}

// One matrix operand: type size, row stride, alignment.
bool bad_rows(const void* p, int64_t ld, int type, int C, bool output) {
  const int64_t unit = type == GNN_F32 ? 4 : 8, pad = type == GNN_F32 ? 4 : output ? 16 : 8;
  return !p || ((uintptr_t)p & 15) || ld % unit || ld < (C + pad - 1) / pad * pad;
}

// Whether an output may be written while an input is read: apart from it, or in its
// place (each element is then read by the thread that writes it, before it does).
bool clashes(const void* out, int64_t ldo, int otype, const void* in, int64_t ldi, int itype, int64_t n, int C) {
  if (out == in && ldo == ldi && otype == itype) return false;
  const int64_t so = type_size(otype), si = type_size(itype), pad = otype == GNN_F32 ? 4 : 16;
  return overlap({out, n, ldo * so, (C + pad - 1) / pad * pad * so}, {in, n, ldi * si, C * si});
}

struct Launch {
  cudaStream_t st;
  template <class... P, class... A>
  gnn_status run(int64_t grid, int block, size_t smem, void (*k)(P...), A... args) const {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;  // may start while the kernel before it ends: each waits for that first
    count_launch();
    GNN_CUDA(cudaLaunchKernelEx(&cfg, k, args...));
    return GNN_OK;
  }
};

int lanes_for(int cg) {
  int l = 1;
  while (l < cg && l < 32) l <<= 1;
  return l;
}

// Threads, rows and tiles of a launch; returns the block size.
int plan(NormArgs& a, int pad, int V, bool backward, bool* small) {
  a.CH = (a.C + pad - 1) / pad * pad / V;
  *small = a.n / a.n_seg <= kShortMean && a.CH <= block_threads(V, true);
  a.RP = block_threads(V, *small) / a.CH;
  a.R = tile_rows(a.n, a.RP, backward, *small);
  a.longest = 2 * a.R > kShortRows ? 2 * a.R : kShortRows;
  a.q = *small && a.cg % V == 0 ? a.cg / V : 0;
  a.L = lanes_for(a.q ? a.RP * a.q : a.cg);
  a.keep = backward ? (*small ? 40 / V : 28 / V) : (*small ? 12 : 10);
  a.tiles = (int)(((int64_t)a.n + a.R - 1) / a.R);
  return (a.RP * a.CH + 31) / 32 * 32;
}
// Blocks of a join launch: a multiple of the group parts.
int joiners(NormArgs& a) {
  const int64_t parts = (a.groups + JOIN_GROUPS - 1) / JOIN_GROUPS, most = std::max<int64_t>(152 / parts, 1);
  a.join_width = (int)std::min<int64_t>((a.n_seg + most - 1) / most, 32);
  return (int)(parts * std::min<int64_t>((a.n_seg + a.join_width - 1) / a.join_width, most));
}

constexpr int kSmemMost = 160 * 1024;  // of a block, its ring included

template <class TX, class TY, int V, bool SMALL>
gnn_status norm_fwd(NormArgs a, int threads, cudaStream_t st) {
  static PerDevice stats_done, apply_done;
  const size_t ring = (size_t)2 * (FWD_DEPTH + 1) * threads * V * sizeof(TX);
  const size_t kept = (size_t)a.keep * threads * V * sizeof(TX);
  const size_t smem = sizeof(float) * (size_t)(2 * a.RP * (a.CH * V + a.CH) + 2 * a.C + 2 * a.groups) + 48 + std::max(ring, kept);
  const Launch l{st};
  gnn_status s = allow_smem(norm_fwd_stats_kernel<TX, TY, V, SMALL>, kSmemMost, stats_done);
  if (s == GNN_OK) s = allow_smem(norm_fwd_apply_kernel<TX, TY, V>, kSmemMost, apply_done);
  if (s == GNN_OK && a.tiles)
    s = l.run(a.tiles, threads, smem, norm_fwd_stats_kernel<TX, TY, V, SMALL>, a);
  const int blocks = joiners(a);
  if (s == GNN_OK) s = l.run(blocks, FIN_THREADS, 0, norm_fwd_join_kernel, a);
  if (s == GNN_OK && a.tiles) s = l.run(a.tiles, threads, ring, norm_fwd_apply_kernel<TX, TY, V>, a);
  return s;
}
template <class TX, class TY, int V>
gnn_status norm_fwd(NormArgs a, cudaStream_t st) {
  bool small;
  const int threads = plan(a, sizeof(TY) == 4 ? 4 : 16, V, false, &small);
  return small ? norm_fwd<TX, TY, V, true>(a, threads, st) : norm_fwd<TX, TY, V, false>(a, threads, st);
}

template <class TX, class TY, int V, bool SMALL>
gnn_status norm_bwd(NormArgs a, int threads, cudaStream_t st) {
  static PerDevice stats_done, apply_done;
  const size_t stream = (size_t)2 * (BWD_DEPTH + 1) * threads * V * (sizeof(TX) + sizeof(TY));
  const size_t kept = (size_t)2 * a.keep * threads * V * 4, ring = stream > kept ? stream : kept;
  const size_t smem = sizeof(float) * (size_t)(2 * a.RP * (a.CH * V + a.CH) + 4 * a.C + 2 * a.groups) + 48 + ring;
  const Launch l{st};
  gnn_status s = allow_smem(norm_bwd_sums_kernel<TX, TY, V, SMALL>, kSmemMost, stats_done);
  if (s == GNN_OK) s = allow_smem(norm_bwd_apply_kernel<TX, TY, V>, kSmemMost, apply_done);
  if (s == GNN_OK && a.tiles)
    s = l.run(a.tiles, threads, smem, norm_bwd_sums_kernel<TX, TY, V, SMALL>, a);
  const int cols = a.dpart ? (2 * a.C + 7) / 8 : 0;
  const int blocks = joiners(a);
  if (s == GNN_OK) s = l.run(blocks + cols, FIN_THREADS, 0, norm_bwd_join_kernel, a, blocks);
  if (s == GNN_OK && a.tiles) s = l.run(a.tiles, threads, stream, norm_bwd_apply_kernel<TX, TY, V>, a);
  return s;
}
template <class TX, class TY, int V>
gnn_status norm_bwd(NormArgs a, cudaStream_t st) {
  bool small;
  const int threads = plan(a, sizeof(TX) == 4 ? 4 : 16, V, true, &small);
  return small ? norm_bwd<TX, TY, V, true>(a, threads, st) : norm_bwd<TX, TY, V, false>(a, threads, st);
}

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_group_norm_workspace(int64_t n, int32_t C, int32_t groups, int32_t n_seg,
                                               size_t* ws_bytes) {
  gnn_status s = check_norm("gnn_group_norm_workspace", n, C, groups, n_seg);
  if (s != GNN_OK) return s;
  GNN_REQUIRE(ws_bytes, "gnn_group_norm_workspace: NULL ws_bytes");
  bool ok;
  *ws_bytes = norm_ws(nullptr, 0, n, C, groups, n_seg, &ok).bytes;
  return GNN_OK;
}

static gnn_status check_norm_args(const char* who, int x_type, int y_type, int act, const int64_t* seg, int n_seg,
                                  std::initializer_list<const void*> fp32, const void* ws) {
  if (!is_type(x_type) || !is_type(y_type) || !is_act(act))
    return fail(GNN_ERR_INVALID_ARG, "%s: unknown type or activation", who);
  if (x_type != GNN_F32 && x_type != y_type)
    return fail(GNN_ERR_UNSUPPORTED, "%s: a 2-byte x_type needs the same y_type", who);
  if (!seg && n_seg != 1) return fail(GNN_ERR_INVALID_ARG, "%s: seg_start NULL needs n_seg = 1", who);
  uintptr_t low = 0;
  for (const void* p : fp32) low |= (uintptr_t)p;
  if (((uintptr_t)seg & 7) || (low & 3))
    return fail(GNN_ERR_INVALID_ARG, "%s: misaligned seg_start or fp32 vector", who);
  if ((uintptr_t)ws & 7) return fail(GNN_ERR_INVALID_ARG, "%s: misaligned workspace", who);
  return GNN_OK;
}

extern "C" gnn_status gnn_group_norm_fwd(const void* X, int64_t ldx, int32_t x_type, int64_t n,
                                         int32_t C, int32_t groups, const int64_t* seg_start,
                                         int32_t n_seg, const float* gamma, const float* beta,
                                         double eps, int32_t act, void* Y, int64_t ldy,
                                         int32_t y_type, float* mean, float* rstd, void* ws,
                                         size_t ws_bytes, gnn_stream_t stream) {
  const char* who = "gnn_group_norm_fwd";
  gnn_status s = check_norm(who, n, C, groups, n_seg);
  if (s != GNN_OK) return s;
  s = check_norm_args(who, x_type, y_type, act, seg_start, n_seg, {gamma, beta, mean, rstd}, ws);
  if (s != GNN_OK) return s;
  GNN_REQUIRE(eps >= 1.2e-38 && eps < 1e30, "gnn_group_norm_fwd: eps must be positive (a normal fp32 value)");
  GNN_REQUIRE(mean && rstd, "gnn_group_norm_fwd: NULL mean or rstd");
  GNN_REQUIRE(n == 0 || !bad_rows(X, ldx, x_type, C, false), "gnn_group_norm_fwd: X needs 16-byte aligned rows "
              "and ldx >= C");
  GNN_REQUIRE(n == 0 || !bad_rows(Y, ldy, y_type, C, true), "gnn_group_norm_fwd: Y needs 16-byte aligned rows and "
              "ldy >= C rounded up to 4 (fp32) or 16");
  GNN_REQUIRE(!clashes(Y, ldy, y_type, X, ldx, x_type, n, C), "gnn_group_norm_fwd: Y overlaps X and is not in its place");
  bool ok;
  const NormWs w = norm_ws(ws, ws_bytes, n, C, groups, n_seg, &ok);
  GNN_REQUIRE(ws && ok, "gnn_group_norm_fwd: workspace too small (%zu < %zu)", ws_bytes, w.bytes);
  NormArgs a{};
  a.X = X, a.ldx = ldx, a.out = Y, a.ldo = ldy, a.n = (int)n, a.C = C, a.groups = groups, a.cg = C / groups;
  a.n_seg = n_seg, a.act = act, a.seg = seg_start, a.gamma = gamma, a.beta = beta, a.eps = (float)eps;
  a.mean = mean, a.rstd = rstd, a.part = w.part, a.has_long = w.has_long;
  a.flags = device_flags();
  if (!a.flags) return fail(GNN_ERR_CUDA, "device flag word unavailable");
  cudaStream_t st = as_stream(stream);
  if (x_type == GNN_BF16) return norm_fwd<__nv_bfloat16, __nv_bfloat16, 8>(a, st);
  if (x_type == GNN_F16) return norm_fwd<__half, __half, 8>(a, st);
  if (y_type == GNN_BF16) return norm_fwd<float, __nv_bfloat16, 4>(a, st);
  if (y_type == GNN_F16) return norm_fwd<float, __half, 4>(a, st);
  return norm_fwd<float, float, 4>(a, st);
}

extern "C" gnn_status gnn_group_norm_bwd(const void* dY, int64_t ldy, int32_t y_type, const void* X,
                                         int64_t ldx, int32_t x_type, int64_t n, int32_t C,
                                         int32_t groups, const int64_t* seg_start, int32_t n_seg,
                                         const float* gamma, const float* beta, int32_t act,
                                         const float* mean, const float* rstd, void* dX, int64_t lddx,
                                         float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                         gnn_stream_t stream) {
  const char* who = "gnn_group_norm_bwd";
  gnn_status s = check_norm(who, n, C, groups, n_seg);
  if (s != GNN_OK) return s;
  s = check_norm_args(who, x_type, y_type, act, seg_start, n_seg, {gamma, beta, mean, rstd, dgamma, dbeta}, ws);
  if (s != GNN_OK) return s;
  GNN_REQUIRE(mean && rstd, "gnn_group_norm_bwd: NULL mean or rstd");
  GNN_REQUIRE(n == 0 || !bad_rows(X, ldx, x_type, C, false), "gnn_group_norm_bwd: X needs 16-byte aligned rows "
              "and ldx >= C");
  GNN_REQUIRE(n == 0 || !bad_rows(dY, ldy, y_type, C, false), "gnn_group_norm_bwd: dY needs 16-byte aligned rows "
              "and ldy >= C");
  GNN_REQUIRE(n == 0 || !bad_rows(dX, lddx, x_type, C, true), "gnn_group_norm_bwd: dX needs 16-byte aligned rows "
              "and lddx >= C rounded up to 4 (fp32) or 16");
  GNN_REQUIRE(!clashes(dX, lddx, x_type, X, ldx, x_type, n, C) && !clashes(dX, lddx, x_type, dY, ldy, y_type, n, C),
              "gnn_group_norm_bwd: dX overlaps X or dY and is not in its place");
  bool ok;
  const NormWs w = norm_ws(ws, ws_bytes, n, C, groups, n_seg, &ok);
  GNN_REQUIRE(ws && ok, "gnn_group_norm_bwd: workspace too small (%zu < %zu)", ws_bytes, w.bytes);
  NormArgs a{};
  a.X = X, a.ldx = ldx, a.dY = dY, a.ldy = ldy, a.out = dX, a.ldo = lddx, a.n = (int)n, a.C = C, a.groups = groups;
  a.cg = C / groups, a.n_seg = n_seg, a.act = act, a.seg = seg_start, a.gamma = gamma, a.beta = beta;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = w.part, a.has_long = w.has_long, a.joined = w.joined, a.dpart = dgamma || dbeta ? w.dpart : nullptr;
  a.dgamma = dgamma, a.dbeta = dbeta;
  a.flags = device_flags();
  if (!a.flags) return fail(GNN_ERR_CUDA, "device flag word unavailable");
  cudaStream_t st = as_stream(stream);
  if (x_type == GNN_BF16) return norm_bwd<__nv_bfloat16, __nv_bfloat16, 8>(a, st);
  if (x_type == GNN_F16) return norm_bwd<__half, __half, 8>(a, st);
  if (y_type == GNN_BF16) return norm_bwd<float, __nv_bfloat16, 4>(a, st);
  if (y_type == GNN_F16) return norm_bwd<float, __half, 4>(a, st);
  return norm_bwd<float, float, 4>(a, st);
}
