// Gated feed-forward projections H = act(X Wg) * (X Wu) and their backward
// pass on tcgen05 tensor cores.
//
// One persistent, warp-specialised kernel shape serves the four products:
//   FWD  G|U = X [Wg|Wu], epilogue H = act(G) * U
//   ACT  the same product again in the backward, epilogue dG|dU from dH, rounded to
//        the 2-byte type that the tensor cores read (an error of a gradient is
//        then sqrt(2) that of its own rounding, 0.0023 against 0.0017 of its norm
//        in bf16; a second 2-byte term each would double DX and DW)
//   DX   dX = [dG|dU] [Wg|Wu]^T (one accumulation over both halves)
//   DW   dWg|dWu = X^T [dG|dU], split over the rows
// A 256 x 256 tile belongs to a pair of CTAs (cta_group::2), each with 128 of
// its rows and half of B in shared memory.  On single CTAs (128 x 256 tiles) all
// four products ran at the rate their operands came from L2, 13.5-15 TB/s,
// 57-65% of the tensor rate; the pair halves B's share of that traffic.
// In FWD and ACT the first CTA's half of B is the gate's columns and the
// second's the same columns of up, so both factors of an output element meet in
// one thread and G, U never reach memory.  Weights are read as they lie
// ([F_in][F_mid], columns contiguous): MN-major operands in FWD/ACT, K-major in
// DX.
//
// Roles: warp 0 issues TMA loads into a ring of 128-byte-swizzled tiles, warp 1
// of the first CTA issues the MMAs from one thread, warps 2-9 drain one of two
// TMEM accumulators while the next tile is multiplied (eight of them:
// exponentials of 128 x 128 outputs would take longer than the product on
// four).  Every wait is bounded.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm.h"
#include "internal.h"
#include "nodewise.cuh"
#include "tc.cuh"

namespace gnn {

namespace {

enum Mode { FWD, ACT, DX, DW };

constexpr int BM = 256, BN = 256, BK = 64;  // of a pair of CTAs
constexpr int CM = BM / 2, CN = BN / 2;      // a CTA's rows of A and of B
constexpr int A_STAGE = CM * BK * 2;  // 16 KB
constexpr int B_STAGE = CN * BK * 2;  // 16 KB
constexpr int BOX = 64 * BK * 2;      // one 64-wide block of an MN-major operand: 8 KB
constexpr int SUB = 32 * 128;         // a warp's 32 rows x 128 bytes of staged output
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;

constexpr int stages(Mode m) { return m == ACT ? 5 : 6; }
constexpr int subs(Mode m) { return m == ACT ? 2 : m == DW ? 0 : 1; }  // staging tiles of an epilogue warp
constexpr int smem_bytes(Mode m) {
  return stages(m) * (A_STAGE + B_STAGE) + EPI_WARPS * subs(m) * SUB + 1024 /*barriers*/ + 1024 /*align*/;
}

struct Args {
  CUtensorMap a[2], b[2];  // the operands (of the gate and the up half where they differ)
  CUtensorMap out[2];      // H, or dG and dU, or dX
  CUtensorMap dh;
  int cols;                // FWD, DX: the output's columns without padding
  int bn;                  // DX: tile columns
  int num_m, num_n, num_kb;  // tiles; k blocks of one half
  int act, dh_f32;
  int splits, kb_per_split;  // DW
  float* part;
  unsigned* flags;
};

struct Smem {
  uint8_t *a, *b, *out;
  uint64_t *full, *empty, *tfull, *tempty, *dh;
  uint32_t* tmem;
  volatile int* abort_flag;
};

template <Mode M>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
  Smem s;
  uint8_t* p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.a = p;
  s.b = p + stages(M) * A_STAGE;
  s.out = s.b + stages(M) * B_STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s.out + EPI_WARPS * subs(M) * SUB);
  s.full = bars;
  s.empty = bars + 6;
  s.tfull = bars + 12;
  s.tempty = bars + 14;
  s.dh = bars + 16;
  s.tmem = reinterpret_cast<uint32_t*>(bars + 16 + EPI_WARPS);
  s.abort_flag = reinterpret_cast<volatile int*>(s.tmem + 1);
  return s;
}

// A tile's place: first row and column of the pair's, half (DW: gate or up), k blocks.
struct Tile {
  int m0, n0, half, split, kb0, kb1;
};
template <Mode M>
__device__ __forceinline__ Tile tile_at(const Args& g, int t) {
  Tile r;
  if (M == DW) {
    r.m0 = (t % g.num_m) * BM;
    t /= g.num_m;
    r.n0 = (t % g.num_n) * BN;
    t /= g.num_n;
    r.half = t & 1;
    r.split = t >> 1;
    r.kb0 = r.split * g.kb_per_split;
    r.kb1 = min(g.num_kb, r.kb0 + g.kb_per_split);
  } else {
    // the column blocks of one row block run side by side, so its rows are
    // read from memory once and from L2 after that
    r.n0 = (t % g.num_n) * (M == DX ? g.bn : BN / 2);
    r.m0 = (t / g.num_n) * BM;
    r.half = r.split = 0;
    r.kb0 = 0;
    r.kb1 = M == DX ? 2 * g.num_kb : g.num_kb;
  }
  return r;
}
template <Mode M>
__device__ __forceinline__ int num_tiles(const Args& g) {
  return g.num_m * g.num_n * (M == DW ? 2 * g.splits : 1);
}

// Bytes that both CTAs load in a stage.
template <Mode M>
__device__ __forceinline__ uint32_t stage_bytes(const Args& g) {
  return 2 * (A_STAGE + (M == DX ? g.bn / 2 * BK * 2 : B_STAGE));
}

// This CTA's share of a stage; `bar`: the first CTA's barrier.
template <Mode M>
__device__ __forceinline__ void load_stage(const Args& g, const Smem& s, const Tile& t, int kb, int st, int rank,
                                           uint32_t bar) {
  uint8_t* a = s.a + st * A_STAGE;
  uint8_t* b = s.b + st * B_STAGE;
  const int m = t.m0 + rank * CM;
  if (M == FWD || M == ACT) {
    tc::tma_load_2d_pair(a, &g.a[0], bar, kb * BK, m);
#pragma unroll
    for (int j = 0; j < 2; ++j) tc::tma_load_2d_pair(b + j * BOX, &g.b[rank], bar, t.n0 + 64 * j, kb * BK);
  } else if (M == DX) {
    const int half = kb >= g.num_kb;
    const int k = (half ? kb - g.num_kb : kb) * BK;
    tc::tma_load_2d_pair(a, &g.a[half], bar, k, m);
    tc::tma_load_2d_pair(b, &g.b[half], bar, k, t.n0 + rank * (g.bn / 2));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) tc::tma_load_2d_pair(a + j * BOX, &g.a[0], bar, m + 64 * j, kb * BK);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      tc::tma_load_2d_pair(b + j * BOX, &g.b[t.half], bar, t.n0 + rank * CN + 64 * j, kb * BK);
  }
}

// Eight 2-byte columns of a staged row: chunk k of row r of a swizzled tile.
__device__ __forceinline__ uint4* staged(uint8_t* tile, int r, int k) {
  return reinterpret_cast<uint4*>(tile + r * 128 + ((k ^ (r & 7)) << 4));
}

// Zero in the padding columns of a staged row, whose first one is column `cols`
// of its 64: a row that is not finite leaves NaN there (times the zeros past the
// weights' last column), and what reads the padding as an operand's counts on zero.
__device__ __forceinline__ void clear_staged(uint8_t* tile, int r, int cols) {
  for (int c = cols; c & 15; ++c) reinterpret_cast<uint16_t*>(staged(tile, r, c >> 3))[c & 7] = 0;
}

__device__ __forceinline__ float2 pair_at(const uint32_t* v, int i) {
  return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}

// The tiles pair, pair + pairs, ... of one product, by one pair of CTAs.  PAD: the
// output has padding columns.  FWD without any leaves their clearing out (716847 x
// 256 x 512: 296 us with the test for a last tile in its epilogue, 287 without).
template <Mode M, class T, bool PAD = true>
__device__ __forceinline__ void walk_tiles(const Args& g, uint8_t* smem_raw, int pair, int pairs) {
  const Smem s = carve<M>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int ST = stages(M);
  const int rank = (int)tc::cluster_rank();
  if (warp == 0 && lane < 2) {  // the maps arrive while the barriers are set up
    tc::prefetch_tmap(&g.a[M == DX ? lane : 0]);
    tc::prefetch_tmap(&g.b[lane]);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.tfull[i], 1);
      tc::mbar_init(&s.tempty[i], 2 * EPI_WARPS);  // a lane of each warp, of both CTAs
    }
    for (int i = 0; i < EPI_WARPS; ++i) tc::mbar_init(&s.dh[i], 1);
    *s.abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(s.tmem, 2 * BN);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the partner's barriers are there
  tc::fence_after_sync();
  cudaGridDependencySynchronize();
  const uint32_t tmem = *s.tmem;
  const int tiles = num_tiles<M>(g);

  if (warp == 0 && lane == 0) {
    int st = 0;
    uint32_t ph = 0;
    for (int t = pair; t < tiles; t += pairs) {
      const Tile w = tile_at<M>(g, t);
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (!tc::mbar_wait(&s.empty[st], ph ^ 1, g.flags, s.abort_flag)) goto done;
        if (rank == 0) tc::mbar_expect_tx(&s.full[st], stage_bytes<M>(g));
        load_stage<M>(g, s, w, kb, st, rank, tc::map_to_rank(&s.full[st], 0));
        if (++st == ST) { st = 0; ph ^= 1; }
      }
    }
    // every stage's release has arrived before this CTA may end
    for (int i = 0; i < ST; ++i) {
      if (!tc::mbar_wait(&s.empty[st], ph ^ 1, g.flags, s.abort_flag)) goto done;
      if (++st == ST) { st = 0; ph ^= 1; }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr bool a_mn = M == DW, b_mn = M != DX;
    const uint32_t idesc = tc::idesc_16(kBf16, BM, M == DX ? g.bn : BN, a_mn, b_mn);
    int st = 0, it = 0;
    uint32_t ph = 0;
    for (int t = pair; t < tiles; t += pairs, ++it) {
      const Tile w = tile_at<M>(g, t);
      const int acc = it & 1;
      if (!tc::mbar_wait<true>(&s.tempty[acc], ((it >> 1) & 1) ^ 1, g.flags, s.abort_flag)) goto done;
      tc::fence_after_sync();
      const uint32_t d = tmem + acc * BN;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (!tc::mbar_wait(&s.full[st], ph, g.flags, s.abort_flag)) goto done;
        tc::fence_after_sync();
        const uint32_t a0 = tc::smem_u32(s.a + st * A_STAGE), b0 = tc::smem_u32(s.b + st * B_STAGE);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)  // 16 elements of K: 32 bytes K-major, 16 rows of 128 bytes MN-major
          tc::mma_16_pair(d, tc::sw128_desc(a0 + k * (a_mn ? 2048 : 32), a_mn ? BOX : 16),
                          tc::sw128_desc(b0 + k * (b_mn ? 2048 : 32), b_mn ? BOX : 16), idesc,
                          kb > w.kb0 || k ? 1u : 0u);
        tc::mma_commit_pair(&s.empty[st]);
        if (++st == ST) { st = 0; ph ^= 1; }
      }
      tc::mma_commit_pair(&s.tfull[acc]);
    }
  } else if (warp >= 2) {
    const int e = warp - 2, q = warp & 3, h = e >> 2;  // TMEM lane quarter, column half
    uint8_t* stage = s.out + e * subs(M) * SUB;
    const uint32_t lane0 = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t freed0 = tc::map_to_rank(&s.tempty[0], 0), freed1 = tc::map_to_rank(&s.tempty[1], 0);
    // hands the accumulator back to the first CTA's MMA warp
    auto release = [&](int acc) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(acc ? freed1 : freed0);
    };
    int it = 0;
    for (int t = pair; t < tiles; t += pairs, ++it) {
      const Tile w = tile_at<M>(g, t);
      const int acc = it & 1;
      const uint32_t base = lane0 + acc * BN;
      const int row = w.m0 + rank * CM + q * 32;  // of the warp
      if (M == ACT) {
        // this warp's dH into its staging tiles, once the stores of the last
        // tile have read them
        if (lane == 0) {
          tc::bulk_wait_read<0>();
          tc::mbar_expect_tx(&s.dh[e], g.dh_f32 ? 2 * SUB : SUB);
          tc::tma_load_2d(stage, &g.dh, &s.dh[e], w.n0 + h * 64, row);
          if (g.dh_f32) tc::tma_load_2d(stage + SUB, &g.dh, &s.dh[e], w.n0 + h * 64 + 32, row);
        }
      }
      if (!tc::mbar_wait(&s.tfull[acc], (it >> 1) & 1, g.flags, s.abort_flag)) goto done;
      tc::fence_after_sync();
      if (M == FWD) {
        if (lane == 0) tc::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t gate[32], up[32];
          tc::tmem_ld32(base + h * 64 + c, gate);
          tc::tmem_ld32(base + BN / 2 + h * 64 + c, up);
          tc::tmem_wait_ld();
          if (c == 32) release(acc);
          with_act(g.act, [&](auto A) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int i = 8 * k + 2 * j;
                const float2 v = mul2_rn(act2(pair_at(gate, i), A), pair_at(up, i));
                o[j] = Pack2<T>::to(v.x, v.y);
              }
              *staged(stage, lane, (c >> 3) + k) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          });
        }
        const int cols = g.cols - (w.n0 + h * 64);
        if (PAD && cols > 0 && cols < 64) clear_staged(stage, lane, cols);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::tma_store_2d(&g.out[0], stage, w.n0 + h * 64, row);
          tc::bulk_commit();
        }
      } else if (M == ACT) {
        if (!tc::mbar_wait(&s.dh[e], it & 1, g.flags, s.abort_flag)) goto done;
        // columns 0-31 come first: with dH in fp32 they fill the first tile, and
        // the bf16 outputs of all 64 columns take half of each
        float dh[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (g.dh_f32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 v = *staged(stage + c * SUB, lane, k);
              dh[c][4 * k] = __uint_as_float(v.x), dh[c][4 * k + 1] = __uint_as_float(v.y);
              dh[c][4 * k + 2] = __uint_as_float(v.z), dh[c][4 * k + 3] = __uint_as_float(v.w);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 v = *staged(stage, lane, c * 4 + k);
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = Pack2<T>::from(x[j]);
                dh[c][8 * k + 2 * j] = f.x, dh[c][8 * k + 2 * j + 1] = f.y;
              }
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t gate[32], up[32];
          tc::tmem_ld32(base + h * 64 + c * 32, gate);
          tc::tmem_ld32(base + BN / 2 + h * 64 + c * 32, up);
          tc::tmem_wait_ld();
          if (c == 1) release(acc);
          with_act(g.act, [&](auto A) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t og[4], ou[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int i = 8 * k + 2 * j;
                const float2 d2 = make_float2(dh[c][i], dh[c][i + 1]);
                float2 a, d;
                act_grad2(pair_at(gate, i), A, a, d);
                const float2 x = mul2_rn(mul2_rn(d2, pair_at(up, i)), d), y = mul2_rn(d2, a);
                og[j] = Pack2<T>::to(x.x, x.y);
                ou[j] = Pack2<T>::to(y.x, y.y);
              }
              *staged(stage, lane, c * 4 + k) = make_uint4(og[0], og[1], og[2], og[3]);
              *staged(stage + SUB, lane, c * 4 + k) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            }
          });
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::tma_store_2d(&g.out[0], stage, w.n0 + h * 64, row);
          tc::tma_store_2d(&g.out[1], stage + SUB, w.n0 + h * 64, row);
          tc::bulk_commit();
        }
      } else if (M == DX) {
        // 64-column pieces of the tile, dealt to the two column halves in turn
        const int pieces = (g.bn + 63) / 64;
        for (int c = h; c < pieces; c += 2) {
          uint32_t v[64];
          tc::tmem_ld32(base + c * 64, *reinterpret_cast<uint32_t(*)[32]>(v));
          tc::tmem_ld32(base + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tc::tmem_wait_ld();
          if (lane == 0) tc::bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = Pack2<T>::to(__uint_as_float(v[8 * k + 2 * j]), __uint_as_float(v[8 * k + 2 * j + 1]));
            *staged(stage, lane, k) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          const int cols = g.cols - (w.n0 + c * 64);
          if (cols > 0 && cols < 64) clear_staged(stage, lane, cols);
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::tma_store_2d(&g.out[0], stage, w.n0 + c * 64, row);
            tc::bulk_commit();
          }
        }
        release(acc);
      } else {
        float* prow = g.part + (((int64_t)w.split * 2 + w.half) * g.num_m * BM + row + lane) * ((int64_t)g.num_n * BN) +
                      w.n0 + h * (BN / 2);
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
          uint32_t v[32];
          tc::tmem_ld32(base + h * (BN / 2) + c, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4*>(prow + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        release(acc);
      }
    }
  }
done:
  if (warp >= 2 && lane == 0) tc::bulk_wait_all();  // stores finish before the block exits
  __syncwarp();
  if (*s.abort_flag) {
    // a wait gave up: what is still in flight (loads, products) lands within
    // microseconds; nothing may end before that
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // nothing of the partner's arrives here any more
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 2 * BN);
  }
}

template <Mode M, class T, bool PAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) gated_kernel(const __grid_constant__ Args g) {
  extern __shared__ uint8_t smem_raw[];
  cudaTriggerProgrammaticLaunchCompletion();
  walk_tiles<M, T, PAD>(g, smem_raw, blockIdx.x >> 1, gridDim.x >> 1);
}

// DX on the first dx_pairs pairs of CTAs and DW on the others: neither needs the
// other, a small one alone leaves most SMs idle, and two uneven last rounds of
// tiles become one.
template <class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gated_grads_kernel(const __grid_constant__ Args dx, const __grid_constant__ Args dw, int dx_pairs) {
  extern __shared__ uint8_t smem_raw[];
  cudaTriggerProgrammaticLaunchCompletion();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (pair < dx_pairs)
    walk_tiles<DX, T>(dx, smem_raw, pair, dx_pairs);
  else
    walk_tiles<DW, T>(dw, smem_raw, pair - dx_pairs, pairs - dx_pairs);
}

// dWg and dWu from the split partials, added in split order; padding columns up
// to a multiple of 16 come out zero (their partials are zero or, beside an X that
// is not finite, NaN).
template <class T>
__global__ void __launch_bounds__(256) gated_dw_kernel(const float* part, int splits, int D, int F, int64_t ldp,
                                                       int64_t half_stride, T* dWg, int64_t ldg, T* dWu,
                                                       int64_t ldu) {
  cudaGridDependencySynchronize();
  const int per = (F + 15) / 16 * 2;  // chunks of 8 columns
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)2 * D * per) return;
  const int c = (int)(i % per) * 8;
  const int64_t r = i / per;
  const int half = r >= D;
  const int64_t d = half ? r - D : r;
  const float* p = part + half * half_stride + d * ldp + c;
  float acc[8] = {};
  for (int s = 0; s < splits; ++s) {
    float v[8];
    load_vec<8>(p + s * 2 * half_stride, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += v[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= F) acc[j] = 0.f;
  store_vec<8>((half ? dWu + d * ldu : dWg + d * ldg) + c, acc);
}

// H of up to NR rows without tensor cores.  A few rows read the weights once and
// do next to nothing with them, so what counts is that every SM reads, with
// much in flight: a block takes `cols` columns of both matrices, eight to a lane
// (16-byte loads), cols / 8 lanes side by side; its warps and their lane rows
// share the inner length, and a lane requests its next four rows of each matrix
// before it multiplies the last four.  On 128 columns to a pair of CTAs as above,
// F_mid = 1024 keeps 16 SMs busy.
constexpr int ROW_THREADS = 256, ROW_CHUNK = 2048;

template <class T, int NR>
__global__ void __launch_bounds__(ROW_THREADS)
    gated_rows_kernel(const T* __restrict__ X, int64_t ldx, int n, int D, const T* __restrict__ Wg, int64_t ldg,
                      const T* __restrict__ Wu, int64_t ldu, int F, int act, T* __restrict__ H, int64_t ldh,
                      int cols) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  constexpr int W = ROW_THREADS / 32, U = 4;
  __shared__ T xs[NR][ROW_CHUNK];
  __shared__ float red[W][NR][2][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int across = cols / 8, down = 32 / across;  // lanes of a row of weights, rows of a warp
  const int c = blockIdx.x * cols + 8 * (lane % across);
  const int k0 = warp * down + lane / across, step = W * down;
  const bool in = c < F;  // a row of weights has its stride, so its last eight columns are there
  float ag[NR][8] = {}, au[NR][8] = {};
  uint4 wg[U], wu[U];
  const T* pg = Wg + (int64_t)k0 * ldg + c;
  const T* pu = Wu + (int64_t)k0 * ldu + c;
  int left = in ? (D - k0 + step - 1) / step : 0;  // rows of weights not yet requested
  auto request = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wg[u] = wu[u] = make_uint4(0, 0, 0, 0);
      if (u < left) {
        wg[u] = *reinterpret_cast<const uint4*>(pg);
        wu[u] = *reinterpret_cast<const uint4*>(pu);
      }
      pg += step * ldg;
      pu += step * ldu;
    }
    left -= U;
  };
  request();
  for (int kb = 0; kb < D; kb += ROW_CHUNK) {
    const int len = min(ROW_CHUNK, D - kb);
    if (kb) __syncthreads();
    for (int i = threadIdx.x; i < NR * len; i += ROW_THREADS) {
      const int r = i / len, k = i - r * len;
      xs[r][k] = r < n ? X[r * ldx + kb + k] : from_f32<T>(0.f);
    }
    __syncthreads();
    // a chunk holds a whole number of batches of rows, so only the last ends early
    for (int k = k0; k < len; k += U * step) {
      uint4 g[U], p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) g[u] = wg[u], p[u] = wu[u];
      request();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u * step >= len) break;
        const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w}, pw[4] = {p[u].x, p[u].y, p[u].z, p[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 gv = Pack2<T>::from(gw[j]), uv = Pack2<T>::from(pw[j]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float x = to_f32(xs[r][k + u * step]);
            ag[r][2 * j] = fmaf(x, gv.x, ag[r][2 * j]);
            ag[r][2 * j + 1] = fmaf(x, gv.y, ag[r][2 * j + 1]);
            au[r][2 * j] = fmaf(x, uv.x, au[r][2 * j]);
            au[r][2 * j + 1] = fmaf(x, uv.y, au[r][2 * j + 1]);
          }
        }
      }
    }
  }
  // over a warp's lane rows, then over the warps, in order
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      for (int o = 16; o >= across; o >>= 1) {
        ag[r][j] += __shfl_xor_sync(0xffffffffu, ag[r][j], o);
        au[r][j] += __shfl_xor_sync(0xffffffffu, au[r][j], o);
      }
      if (lane < across) {
        red[warp][r][0][8 * lane + j] = ag[r][j];
        red[warp][r][1][8 * lane + j] = au[r][j];
      }
    }
  }
  __syncthreads();
  const int end = (F + 15) / 16 * 16;  // padding columns come out zero
  for (int i = threadIdx.x; i < NR * cols; i += ROW_THREADS) {
    const int r = i / cols, j = i % cols, col = blockIdx.x * cols + j;
    if (r >= n || col >= end) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      g += red[w][r][0][j];
      u += red[w][r][1][j];
    }
    H[r * ldh + col] = from_f32<T>(col < F ? act_f(g, act) * u : 0.f);
  }
}

// ---------------------------------------------------------------- host side
constexpr int PAIRS = 76;  // of CTAs, one an SM

// Pairs that the current device holds at once.
int pairs_there() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PAIRS;
  return std::max(n / 2, 1);
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// How the gradients' products share the card: which pairs of CTAs take DX and
// into how many parts DW's sum over the rows is split, by the rounds of tiles they
// take, counted in k blocks (a tile's start and drain as four).
struct GradPlan {
  int dw_m, dw_n, splits, kb_per_split;  // DW's tiles and split
  int dx_bn, dx_n;                       // DX's tile columns and column tiles
  int dx_pairs;                          // 0: DX and DW by themselves
  size_t part_floats;
};

int64_t dw_split(int64_t tiles, int64_t kb, int pairs, int* splits, int* per_split) {
  int64_t best = -1;
  for (int64_t s = 1; s <= PAIRS && (s == 1 || (s * 8 <= kb && s * tiles <= 4 * PAIRS)); ++s) {
    const int64_t per = std::max<int64_t>((kb + s - 1) / s, 1), used = std::max<int64_t>((kb + per - 1) / per, 1);
    const int64_t cost = (used * tiles + pairs - 1) / pairs * (per + 4);
    if (best < 0 || cost < best) {
      best = cost;
      *splits = (int)used;
      *per_split = (int)per;
    }
  }
  return best;
}

GradPlan grad_plan(int64_t n, int D, int F, bool both) {
  GradPlan p{};
  p.dw_m = (D + BM - 1) / BM, p.dw_n = (F + BN - 1) / BN;
  const int num_n = (D + BN - 1) / BN;
  p.dx_bn = (int)up((D + num_n - 1) / num_n, 64), p.dx_n = (D + p.dx_bn - 1) / p.dx_bn;
  const int64_t dw_tiles = 2ll * p.dw_m * p.dw_n, kb = (n + BK - 1) / BK;
  const int64_t dx_tiles = (n + BM - 1) / BM * p.dx_n, dx_len = 2 * ((F + BK - 1) / BK) + 4;
  int64_t best = dw_split(dw_tiles, kb, PAIRS, &p.splits, &p.kb_per_split);
  if (both) {
    best += (dx_tiles + PAIRS - 1) / PAIRS * dx_len + 10;  // one launch after the other
    for (int at = 4; at < PAIRS; at += 4) {
      const int pairs = (int)std::min<int64_t>(at, dx_tiles);
      int s, per;
      const int64_t cost = std::max((dx_tiles + pairs - 1) / pairs * dx_len,
                                    dw_split(dw_tiles, kb, PAIRS - pairs, &s, &per));
      if (cost < best) {
        best = cost;
        p.dx_pairs = pairs, p.splits = s, p.kb_per_split = per;
      }
      if (pairs < at) break;
    }
  }
  p.part_floats = (size_t)p.splits * 2 * p.dw_m * BM * p.dw_n * BN;
  return p;
}

struct GatedWs {
  void* dg;
  void* du;
  float* part;
  int64_t ldf;
  size_t bytes;
};
GatedWs gated_ws(void* base, size_t cap, int64_t n, int D, int F, bool* ok) {
  Arena ar(base, cap);
  GatedWs w{};
  w.ldf = up(F, 8);
  w.dg = ar.take<uint16_t>((size_t)n * w.ldf);
  w.du = ar.take<uint16_t>((size_t)n * w.ldf);
  w.part = ar.take<float>(std::max(grad_plan(n, D, F, true).part_floats, grad_plan(n, D, F, false).part_floats));
  w.bytes = ar.used;
  *ok = ar.ok();
  return w;
}

// A launch may start while the kernel before it ends; each waits for that before
// it touches memory.
template <class... P, class... A>
gnn_status launch(int grid, int block, size_t smem, cudaStream_t st, void (*k)(P...), const A&... args) {
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

#define GNN_TRY(expr)                 \
  do {                                \
    const gnn_status s_ = (expr);     \
    if (s_ != GNN_OK) return s_;      \
  } while (0)

template <Mode M, class T, bool PAD = true>
gnn_status launch_gated(const Args& g, cudaStream_t st) {
  static PerDevice done;
  GNN_TRY(allow_smem(gated_kernel<M, T, PAD>, smem_bytes(M), done));
  const int64_t tiles = (int64_t)g.num_m * g.num_n * (M == DW ? 2 * g.splits : 1);
  const int pairs = (int)std::min<int64_t>(tiles, pairs_there());
  return launch(2 * pairs, THREADS, smem_bytes(M), st, gated_kernel<M, T, PAD>, g);
}

// A map of a 2-byte matrix of `cols` used columns.
template <class T>
gnn_status map16(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_c, int box_r) {
  return encode_tmap_2d(m, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        p, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld * 2, (uint32_t)box_c, (uint32_t)box_r);
}

struct Mat {
  void* p;
  int64_t ld;
};

template <class T>
gnn_status product_args(Args& g, int64_t n, int D, int F, int act, Mat X, Mat Wg, Mat Wu) {
  g.flags = device_flags();
  if (!g.flags) return fail(GNN_ERR_CUDA, "device flag word unavailable");
  g.cols = F, g.act = act;
  g.num_m = (int)((n + BM - 1) / BM), g.num_n = (F + BN / 2 - 1) / (BN / 2), g.num_kb = (D + BK - 1) / BK;
  GNN_TRY(map16<T>(&g.a[0], X.p, n, D, X.ld, BK, CM));
  GNN_TRY(map16<T>(&g.b[0], Wg.p, D, F, Wg.ld, 64, BK));
  GNN_TRY(map16<T>(&g.b[1], Wu.p, D, F, Wu.ld, 64, BK));
  return GNN_OK;
}

template <class T, int NR>
gnn_status launch_rows(int n, int D, int F, int act, Mat X, Mat Wg, Mat Wu, Mat H, cudaStream_t st) {
  // as many columns to a block as leave every SM two: wide rows of weights are
  // read in longer pieces
  int cols = 64;
  while (cols > 16 && (F + cols - 1) / cols < 2 * 152) cols /= 2;
  const int grid = (int)((up(F, 16) + cols - 1) / cols);
  return launch(grid, ROW_THREADS, 0, st, gated_rows_kernel<T, NR>, static_cast<const T*>(X.p), X.ld, n, D,
                static_cast<const T*>(Wg.p), Wg.ld, static_cast<const T*>(Wu.p), Wu.ld, F, act, static_cast<T*>(H.p), H.ld,
                cols);
}

template <class T>
gnn_status gated_fwd(int64_t n, int D, int F, int act, Mat X, Mat Wg, Mat Wu, Mat H, cudaStream_t st) {
  // One or two rows (measured in us at 1024 x 4096, rows against tensor cores:
  // 1 row 6.8 / 10.4, 2 rows 8.0 / 10.5, 4 rows 18.4 / 10.7).
  if (n == 1) return launch_rows<T, 1>((int)n, D, F, act, X, Wg, Wu, H, st);
  if (n == 2) return launch_rows<T, 2>((int)n, D, F, act, X, Wg, Wu, H, st);
  Args g{};
  GNN_TRY(product_args<T>(g, n, D, F, act, X, Wg, Wu));
  GNN_TRY(map16<T>(&g.out[0], H.p, n, up(F, 16), H.ld, 64, 32));
  return F % 16 ? launch_gated<FWD, T>(g, st) : launch_gated<FWD, T, false>(g, st);
}

template <class T>
gnn_status gated_bwd(int64_t n, int D, int F, int act, int dh_f32, Mat dH, Mat X, Mat Wg, Mat Wu, Mat dX,
                     Mat dWg, Mat dWu, const GatedWs& w, cudaStream_t st) {
  if (n > 0) {
    Args g{};
    GNN_TRY(product_args<T>(g, n, D, F, act, X, Wg, Wu));
    g.dh_f32 = dh_f32;
    if (dh_f32)
      GNN_TRY(encode_tmap_2d(&g.dh, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dH.p, F, n, dH.ld * 4, 32, 32));
    else
      GNN_TRY(map16<T>(&g.dh, dH.p, n, F, dH.ld, 64, 32));
    GNN_TRY(map16<T>(&g.out[0], w.dg, n, F, w.ldf, 64, 32));
    GNN_TRY(map16<T>(&g.out[1], w.du, n, F, w.ldf, 64, 32));
    GNN_TRY((launch_gated<ACT, T>(g, st)));
  }
  const GradPlan p = grad_plan(n, D, F, dX.p && dWg.p);
  Args x{}, v{};
  if (n > 0 && dX.p) {
    x.flags = device_flags();
    x.cols = D, x.bn = p.dx_bn, x.num_m = (int)((n + BM - 1) / BM), x.num_n = p.dx_n, x.num_kb = (F + BK - 1) / BK;
    GNN_TRY(map16<T>(&x.a[0], w.dg, n, F, w.ldf, BK, CM));
    GNN_TRY(map16<T>(&x.a[1], w.du, n, F, w.ldf, BK, CM));
    GNN_TRY(map16<T>(&x.b[0], Wg.p, D, F, Wg.ld, BK, x.bn / 2));
    GNN_TRY(map16<T>(&x.b[1], Wu.p, D, F, Wu.ld, BK, x.bn / 2));
    GNN_TRY(map16<T>(&x.out[0], dX.p, n, up(D, 16), dX.ld, 64, 32));
  }
  if (n > 0 && dWg.p) {
    v.flags = device_flags();
    v.num_m = p.dw_m, v.num_n = p.dw_n, v.num_kb = (int)((n + BK - 1) / BK);
    v.splits = p.splits, v.kb_per_split = p.kb_per_split, v.part = w.part;
    GNN_TRY(map16<T>(&v.a[0], X.p, n, D, X.ld, 64, BK));
    GNN_TRY(map16<T>(&v.b[0], w.dg, n, F, w.ldf, 64, BK));
    GNN_TRY(map16<T>(&v.b[1], w.du, n, F, w.ldf, 64, BK));
  }
  // the plan shares PAIRS pairs; on a device with fewer the products run one by one
  if (n > 0 && p.dx_pairs && pairs_there() >= PAIRS) {
    static PerDevice done;
    constexpr int smem = smem_bytes(DX) > smem_bytes(DW) ? smem_bytes(DX) : smem_bytes(DW);
    GNN_TRY(allow_smem(gated_grads_kernel<T>, smem, done));
    const int64_t dw_tiles = 2ll * p.dw_m * p.dw_n * p.splits;
    const int pairs = p.dx_pairs + (int)std::min<int64_t>(dw_tiles, PAIRS - p.dx_pairs);
    GNN_TRY(launch(2 * pairs, THREADS, smem, st, gated_grads_kernel<T>, x, v, p.dx_pairs));
  } else if (n > 0) {
    if (dX.p) GNN_TRY((launch_gated<DX, T>(x, st)));
    if (dWg.p) GNN_TRY((launch_gated<DW, T>(v, st)));
  }
  if (dWg.p) {
    const int64_t work = 2ll * D * (up(F, 16) / 8), ldp = (int64_t)p.dw_n * BN;
    GNN_TRY(launch((int)((work + 255) / 256), 256, 0, st, gated_dw_kernel<T>, (const float*)w.part,
                   n > 0 ? p.splits : 0, D, F, ldp, (int64_t)p.dw_m * BM * ldp, static_cast<T*>(dWg.p), dWg.ld,
                   static_cast<T*>(dWu.p), dWu.ld));
  }
  return GNN_OK;
}

gnn_status check_gated(const char* who, int64_t n, int D, int F) {
  if (n < 0 || n > (int64_t)0x7fffffff - 256) return fail(GNN_ERR_INVALID_ARG, "%s: bad row count", who);
  if (D < 1 || F < 1) return fail(GNN_ERR_INVALID_ARG, "%s: F_in/F_mid must be >= 1", who);
  if (D > 65536 || F > 65536) return fail(GNN_ERR_UNSUPPORTED, "%s: F_in or F_mid > 65536", who);
  // tile counts are 32-bit
  if ((n / BM + 1) * (int64_t)(F / (BN / 2) + 1) > 0x3fffffff || (n / BM + 1) * (int64_t)(D / 64 + 1) > 0x3fffffff)
    return fail(GNN_ERR_UNSUPPORTED, "%s: too many tiles (n=%lld)", who, (long long)n);
  return GNN_OK;
}

bool bad_mat(const void* p, int64_t ld, int64_t cols, int elem) {
  return !p || ((uintptr_t)p & 15) || (ld * elem) % 16 || ld < cols || ld > ((int64_t)1 << 36);
}

// A 2-byte matrix's memory.
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld) { return {p, rows, 2 * ld, 2 * cols}; }

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_gated_workspace(int64_t n, int32_t F_in, int32_t F_mid, size_t* fwd_bytes,
                                          size_t* bwd_bytes) {
  gnn_status s = check_gated("gnn_gated_workspace", n, F_in, F_mid);
  if (s != GNN_OK) return s;
  GNN_REQUIRE(fwd_bytes || bwd_bytes, "gnn_gated_workspace: NULL result");
  bool ok;
  if (fwd_bytes) *fwd_bytes = 0;
  if (bwd_bytes) *bwd_bytes = gated_ws(nullptr, 0, n, F_in, F_mid, &ok).bytes;
  return GNN_OK;
}

extern "C" gnn_status gnn_gated_fwd(const void* X, int64_t ldx, int32_t type, int64_t n, int32_t F_in,
                                    const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu,
                                    int32_t F_mid, int32_t act, void* H, int64_t ldh, void* ws,
                                    size_t ws_bytes, gnn_stream_t stream) {
  (void)ws, (void)ws_bytes;
  gnn_status s = check_gated("gnn_gated_fwd", n, F_in, F_mid);
  if (s != GNN_OK) return s;
  GNN_REQUIRE((type == GNN_BF16 || type == GNN_F16) && is_act(act), "gnn_gated_fwd: type is bf16 or fp16, act GNN_ACT_*");
  if (n == 0) return GNN_OK;
  GNN_REQUIRE(!bad_mat(X, ldx, F_in, 2), "gnn_gated_fwd: X needs 16-byte aligned rows and ldx >= F_in");
  GNN_REQUIRE(!bad_mat(Wg, ldwg, F_mid, 2) && !bad_mat(Wu, ldwu, F_mid, 2),
              "gnn_gated_fwd: Wg and Wu need 16-byte aligned rows and strides >= F_mid");
  GNN_REQUIRE(!bad_mat(H, ldh, up(F_mid, 16), 2),
              "gnn_gated_fwd: H needs 16-byte aligned rows and ldh >= round_up(F_mid, 16)");
  const Span hs = span(H, n, up(F_mid, 16), ldh);
  GNN_REQUIRE(!overlap(hs, span(X, n, F_in, ldx)) && !overlap(hs, span(Wg, F_in, F_mid, ldwg)) &&
                  !overlap(hs, span(Wu, F_in, F_mid, ldwu)), "gnn_gated_fwd: H overlaps X, Wg or Wu");
  const Mat x{const_cast<void*>(X), ldx}, g{const_cast<void*>(Wg), ldwg}, u{const_cast<void*>(Wu), ldwu}, h{H, ldh};
  cudaStream_t st = as_stream(stream);
  return type == GNN_BF16 ? gated_fwd<__nv_bfloat16>(n, F_in, F_mid, act, x, g, u, h, st)
                          : gated_fwd<__half>(n, F_in, F_mid, act, x, g, u, h, st);
}

extern "C" gnn_status gnn_gated_bwd(const void* dH, int64_t lddh, int32_t dh_type, const void* X,
                                    int64_t ldx, int32_t type, int64_t n, int32_t F_in, const void* Wg,
                                    int64_t ldwg, const void* Wu, int64_t ldwu, int32_t F_mid,
                                    int32_t act, void* dX, int64_t lddx, void* dWg, int64_t lddwg,
                                    void* dWu, int64_t lddwu, void* ws, size_t ws_bytes,
                                    gnn_stream_t stream) {
  gnn_status s = check_gated("gnn_gated_bwd", n, F_in, F_mid);
  if (s != GNN_OK) return s;
  GNN_REQUIRE((type == GNN_BF16 || type == GNN_F16) && is_act(act), "gnn_gated_bwd: type is bf16 or fp16, act GNN_ACT_*");
  GNN_REQUIRE(dh_type == type || dh_type == GNN_F32, "gnn_gated_bwd: dh_type is type or GNN_F32");
  GNN_REQUIRE((dWg == nullptr) == (dWu == nullptr), "gnn_gated_bwd: dWg and dWu come together");
  GNN_REQUIRE(n == 0 || (!bad_mat(X, ldx, F_in, 2) && !bad_mat(dH, lddh, F_mid, dh_type == GNN_F32 ? 4 : 2)),
              "gnn_gated_bwd: X and dH need 16-byte aligned rows and strides >= their columns");
  GNN_REQUIRE(n == 0 || (!bad_mat(Wg, ldwg, F_mid, 2) && !bad_mat(Wu, ldwu, F_mid, 2)),
              "gnn_gated_bwd: Wg and Wu need 16-byte aligned rows and strides >= F_mid");
  GNN_REQUIRE(n == 0 || !dX || !bad_mat(dX, lddx, up(F_in, 16), 2),
              "gnn_gated_bwd: dX needs 16-byte aligned rows and lddx >= round_up(F_in, 16)");
  GNN_REQUIRE(!dWg || (!bad_mat(dWg, lddwg, up(F_mid, 16), 2) && !bad_mat(dWu, lddwu, up(F_mid, 16), 2)),
              "gnn_gated_bwd: dWg and dWu need 16-byte aligned rows and strides >= round_up(F_mid, 16)");
  // dH is read before anything is written, X, Wg and Wu before dWg and dWu are
  const Span dxs = span(dX, n, up(F_in, 16), lddx), dgs = span(dWg, F_in, up(F_mid, 16), lddwg),
             dus = span(dWu, F_in, up(F_mid, 16), lddwu);
  GNN_REQUIRE(!overlap(dxs, span(Wg, F_in, F_mid, ldwg)) && !overlap(dxs, span(Wu, F_in, F_mid, ldwu)),
              "gnn_gated_bwd: dX overlaps Wg or Wu");
  GNN_REQUIRE(!dWg || !overlap(dxs, span(X, n, F_in, ldx)), "gnn_gated_bwd: dX overlaps X, which dWg and dWu need");
  GNN_REQUIRE(!overlap(dxs, dgs) && !overlap(dxs, dus) && !overlap(dgs, dus), "gnn_gated_bwd: outputs overlap");
  bool ok;
  const GatedWs w = gated_ws(ws, ws_bytes, n, F_in, F_mid, &ok);
  GNN_REQUIRE(ws && ok && ((uintptr_t)ws & 15) == 0, "gnn_gated_bwd: workspace too small (%zu < %zu) or misaligned",
              ws_bytes, w.bytes);
  const Mat dh{const_cast<void*>(dH), lddh}, x{const_cast<void*>(X), ldx}, g{const_cast<void*>(Wg), ldwg},
      u{const_cast<void*>(Wu), ldwu}, dx{dX, lddx}, dg{dWg, lddwg}, du{dWu, lddwu};
  cudaStream_t st = as_stream(stream);
  const int f32 = dh_type == GNN_F32;
  return type == GNN_BF16 ? gated_bwd<__nv_bfloat16>(n, F_in, F_mid, act, f32, dh, x, g, u, dx, dg, du, w, st)
                          : gated_bwd<__half>(n, F_in, F_mid, act, f32, dh, x, g, u, dx, dg, du, w, st);
}
