// Newton-Schulz orthogonalisation of matrices, and the Muon step that uses it.
//
// X0 = u / (|u|_F + eps), taken on the side where it is wide (m <= n); each of the
// steps forms
//   A = X X',  P = a I + b A + c A A,  X <- P X.
// The map multiplies small singular values by a (3.44) a step, rounding errors among
// them: of X kept in bf16 a tenth of the result would be noise after five steps, in
// fp16 a hundredth.  So every operand is held as two fp16 limbs of 1024 times its
// value (22 bits; no entry exceeds the largest singular value, so 64 times the usual
// range is left), and a product is hi hi + hi lo + lo hi with fp32 sums.
//
// Operands lie in the workspace in blocks of 128 rows x 64 columns, the hi limb's
// 16 KB before the lo limb's: rows of 128 bytes, so that a few tensor maps over the
// whole workspace bring any of them, swizzled, to shared memory and back.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "gemm.h"
#include "internal.h"
#include "nodewise.cuh"
#include "tc.cuh"

namespace gnn {

namespace {

constexpr int MAX_MATS = 64;     // of one pass over the pipeline
constexpr int MAX_STEPS = 16;
constexpr int THREADS = 256;
constexpr int LIMB = 128 * 128;  // bytes of a block's limb
constexpr int BLOCK = 2 * LIMB;
constexpr int PARTS = 128;       // of a matrix's sum of squares
constexpr float UNIT = 1024.f;   // what the limbs hold is this many times the value

// One matrix: the caller's arrays, and its place in the workspace.
struct Mat {
  void* param;        // orthogonalise: the output
  const void* grad;   // orthogonalise: the input
  void* mom;
  uint16_t* copy;
  int64_t ldp, ldg, ldm, ldc;
  float scale;
  int rows, cols;
  int flip;           // X is the transpose
  int m, n;           // X's rows and columns
  int mb, nb;         // blocks of X: 128 rows, 64 columns
  int parts, slot;    // partial sums of squares; the matrix's number in the call
  int quads;          // bits: rows of param, grad, mom, copy lie on borders of four elements
  char *x[2], *a, *p;
};
// Warps that have finished their share of a tile, by matrix and product; and, of a pass's
// first matrix, whether a wait of the steps has run out: what X holds is then unfinished.
struct Done {
  int of[3];
  int gave_up;
};
constexpr int DONE_WORDS = MAX_MATS * sizeof(Done) / sizeof(int);
struct Table {
  Mat mat[MAX_MATS];
  int first[MAX_MATS + 1];  // blocks (or parts) before each matrix
  int count;
  int small;  // every matrix stays in one CTA's shared memory
  int bn;  // the steps' tiles: columns of a CTA's, or 0 for pairs of CTAs
  int half[3];  // pairs: tiles of 128 columns instead of 256, by product
  int64_t blocks;  // of the operands, from the workspace's start
  double* partial;
  Done* done;
};

struct Hyper {
  float momentum, grad_scale, decay, lr;
  double eps;
  int nesterov, orth;
  int pt, gt, mt;  // types of param (output), grad (input), momentum
};

// Four elements of a row from column c, zero past `cols`; in one access where the
// rows allow it.
__device__ __forceinline__ float4 load4(const void* p, int64_t row, int64_t c, int64_t cols, int type, bool quad) {
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (quad && c + 4 <= cols) {
    if (type == GNN_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + c);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + row + c);
    const float2 a = type == GNN_BF16 ? Pack2<__nv_bfloat16>::from(w.x) : Pack2<__half>::from(w.x);
    const float2 b = type == GNN_BF16 ? Pack2<__nv_bfloat16>::from(w.y) : Pack2<__half>::from(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (c + j < cols) {
      const int64_t i = row + c + j;
      v[j] = type == GNN_F32    ? static_cast<const float*>(p)[i]
             : type == GNN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                                : __half2float(static_cast<const __half*>(p)[i]);
    }
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(void* p, int64_t row, int64_t c, int64_t cols, int type, bool quad, float4 f) {
  if (quad && c + 4 <= cols) {
    if (type == GNN_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + row + c) = f;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + row + c) =
          type == GNN_BF16 ? make_uint2(Pack2<__nv_bfloat16>::to(f.x, f.y), Pack2<__nv_bfloat16>::to(f.z, f.w))
                           : make_uint2(Pack2<__half>::to(f.x, f.y), Pack2<__half>::to(f.z, f.w));
    }
    return;
  }
  const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (c + j < cols) {
      const int64_t i = row + c + j;
      if (type == GNN_F32)
        static_cast<float*>(p)[i] = v[j];
      else if (type == GNN_BF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[j]);
      else
        static_cast<__half*>(p)[i] = __float2half_rn(v[j]);
    }
  }
}
enum { PARAM = 1, GRAD = 2, MOM = 4, COPY = 8 };  // of Mat::quads

__device__ __forceinline__ float4 axpy4(float4 x, float a, float4 y) {
  return make_float4(fmaf(x.x, a, y.x), fmaf(x.y, a, y.y), fmaf(x.z, a, y.z), fmaf(x.w, a, y.w));
}

// A gradient and a momentum as they were, and the update that is orthogonalised.
struct Quad {
  float4 g, m;
  __device__ __forceinline__ void load(const Mat& t, const Hyper& h, int64_t row, int64_t c, int64_t cols) {
    g = load4(t.grad, row * t.ldg, c, cols, h.gt, t.quads & GRAD);
    if (!h.orth) m = load4(t.mom, row * t.ldm, c, cols, h.mt, t.quads & MOM);
  }
  // m becomes the new momentum
  __device__ __forceinline__ float4 update(const Hyper& h) {
    g = make_float4(g.x * h.grad_scale, g.y * h.grad_scale, g.z * h.grad_scale, g.w * h.grad_scale);
    if (h.orth) return g;
    m = axpy4(m, h.momentum, g);
    return h.nesterov ? axpy4(m, h.momentum, g) : m;
  }
};

__device__ __forceinline__ int mat_of(const Table& tab, int k) {
  int i = 0;
  while (i + 1 < tab.count && k >= tab.first[i + 1]) ++i;
  return i;
}

// Sums of u^2 over a share of a matrix's rows; the counts of the steps start at zero.
// It reads what begin_kernel reads again (a norm comes before the first limb): the three
// kernels around the steps take 105 us of six matrices of 1024 x 4096 cold, DRAM at half.
__global__ void __launch_bounds__(THREADS) square_kernel(const __grid_constant__ Table tab, const Hyper h) {
  __shared__ double sm[THREADS / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < DONE_WORDS; k += THREADS) reinterpret_cast<int*>(tab.done)[k] = 0;
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int part = blockIdx.x - tab.first[i];
  double sum = 0;
  // rows that lie end to end are one long row, and each part has a piece of it
  const bool flat = t.ldg == t.cols && (h.orth || t.ldm == t.cols);
  const int64_t cols = flat ? (int64_t)t.rows * t.cols : t.cols, rows = flat ? 1 : t.rows;
  const int64_t share = flat ? ((cols + t.parts - 1) / t.parts + 3) / 4 * 4 : (rows + t.parts - 1) / t.parts;
  const int64_t lo = part * share, hi = min(lo + share, flat ? cols : rows);
  const int64_t r0 = flat ? 0 : lo, r1 = flat ? 1 : hi, c0 = flat ? lo : 0, c1 = flat ? hi : cols;
  constexpr int AHEAD = 4;
  for (int64_t r = r0; r < r1; ++r) {
    for (int64_t c = c0 + 4 * threadIdx.x; c < c1; c += 4 * AHEAD * THREADS) {
      Quad q[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) q[k].load(t, h, r, c + 4 * k * THREADS, c1);
      float s = 0.f;
      float4 u[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        u[k] = q[k].update(h);
        s = fmaf(u[k].x, u[k].x, fmaf(u[k].y, u[k].y, fmaf(u[k].z, u[k].z, fmaf(u[k].w, u[k].w, s))));
      }
      if (s > 1e-28f && s < 1e38f) {
        sum += (double)s;
      } else {  // outside of what fp32 holds well
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          sum += (double)u[k].x * u[k].x + (double)u[k].y * u[k].y + (double)u[k].z * u[k].z + (double)u[k].w * u[k].w;
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
    for (int w = 0; w < THREADS / 32; ++w) s += sm[w];
    tab.partial[i * PARTS + part] = s;
  }
}

// sqrt(s) in fp32 without fp64's root, which an SM forms slowly: s by an even power of
// two, so that fp32 holds it.
__device__ __forceinline__ float root_of(double s) {
  if (!(s > 0) || !isfinite(s)) return (float)s;
  const int e = ilogb(s) & ~1;
  return ldexpf(sqrtf((float)scalbn(s, -e)), e / 2);
}
// UNIT / (norm + eps): what u is multiplied by.
__device__ __forceinline__ float scale_of(float norm, double eps) { return UNIT / (norm + (float)eps); }

// |u|_F, in every thread of the block; `sm` is one float.
__device__ __forceinline__ float norm_of(const double* partial, int i, int parts, float* sm) {
  if (threadIdx.x < 32) {
    double s = 0;
    for (int k = threadIdx.x; k < parts; k += 32) s += partial[i * PARTS + k];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) *sm = root_of(s);
  }
  __syncthreads();
  return *sm;
}

// Two values' limbs, packed.
__device__ __forceinline__ void limbs(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Byte of 8 columns (chunk k of 8) of row r in a block's limb.
__device__ __forceinline__ int chunk_at(int r, int k) { return r * 128 + k * 16; }

// u scaled into X's limbs, and the new momentum; a block of X a thread block.
__global__ void __launch_bounds__(THREADS) begin_kernel(const __grid_constant__ Table tab, const Hyper h, float* norms) {
  __shared__ float tile[128][65];
  __shared__ float sm;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int block = blockIdx.x - tab.first[i], r0 = block / t.nb * 128, c0 = block % t.nb * 64;
  // in the order of the caller's rows, 64 or (transposed) 128 columns of them
  const int across = t.flip ? 32 : 16, row0 = t.flip ? c0 : r0, col0 = t.flip ? r0 : c0;
  constexpr int QUADS = 128 * 64 / 4 / THREADS, AHEAD = 4;
  Quad q[AHEAD];
  auto place = [&](int k, int& row, int& col) {
    const int e = threadIdx.x + k * THREADS;
    row = e / across, col = e % across * 4;
  };
  auto load = [&](int k, Quad& to) {
    int row, col;
    place(k, row, col);
    to.load(t, h, min(row0 + row, t.rows - 1), col0 + col, row0 + row < t.rows ? t.cols : 0);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) load(k, q[k]);
  const float norm = norm_of(tab.partial, i, t.parts, &sm);
  const bool good = isfinite(norm);
  const float inv = scale_of(norm, h.eps);
  if (block == 0 && threadIdx.x == 0 && norms) norms[t.slot] = norm;
#pragma unroll
  for (int k0 = 0; k0 < QUADS; k0 += AHEAD) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      int row, col;
      place(k0 + k, row, col);
      float4 u = q[k].update(h);
      if (!h.orth && good && row0 + row < t.rows && col0 + col < t.cols)
        store4(t.mom, (int64_t)(row0 + row) * t.ldm, col0 + col, t.cols, h.mt, t.quads & MOM, q[k].m);
      u = good ? make_float4(u.x * inv, u.y * inv, u.z * inv, u.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (t.flip) {
        tile[col][row] = u.x, tile[col + 1][row] = u.y, tile[col + 2][row] = u.z, tile[col + 3][row] = u.w;
      } else {
        tile[row][col] = u.x, tile[row][col + 1] = u.y, tile[row][col + 2] = u.z, tile[row][col + 3] = u.w;
      }
      if (k0 + AHEAD < QUADS) load(k0 + AHEAD + k, q[k]);
    }
  }
  __syncthreads();
  char* x = t.x[0] + (int64_t)block * BLOCK;
  for (int e = threadIdx.x; e < 128 * 8; e += THREADS) {
    const int r = e >> 3, k = e & 7;
    uint4 hi, lo;
    limbs(tile[r][8 * k], tile[r][8 * k + 1], hi.x, lo.x);
    limbs(tile[r][8 * k + 2], tile[r][8 * k + 3], hi.y, lo.y);
    limbs(tile[r][8 * k + 4], tile[r][8 * k + 5], hi.z, lo.z);
    limbs(tile[r][8 * k + 6], tile[r][8 * k + 7], hi.w, lo.w);
    *reinterpret_cast<uint4*>(x + chunk_at(r, k)) = hi;
    *reinterpret_cast<uint4*>(x + LIMB + chunk_at(r, k)) = lo;
  }
}

// Parameters (or the output) from the orthogonalised X.
__global__ void __launch_bounds__(THREADS) apply_kernel(const __grid_constant__ Table tab, const Hyper h, int which) {
  __shared__ float tile[128][65];
  __shared__ float sm;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int block = blockIdx.x - tab.first[i], r0 = block / t.nb * 128, c0 = block % t.nb * 64;
  const bool good = isfinite(norm_of(tab.partial, i, t.parts, &sm)) && !tab.done->gave_up;
  if (!good && !h.orth) return;  // this matrix stays as it is
  const char* x = t.x[which] + (int64_t)block * BLOCK;
  for (int e = threadIdx.x; e < 128 * 8; e += THREADS) {
    const int r = e >> 3, k = e & 7;
    const uint4 hi = *reinterpret_cast<const uint4*>(x + chunk_at(r, k)),
                lo = *reinterpret_cast<const uint4*>(x + LIMB + chunk_at(r, k));
    const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = Pack2<__half>::from(hw[j]), b = Pack2<__half>::from(lw[j]);
      tile[r][8 * k + 2 * j] = (a.x + b.x) * (1.f / UNIT);
      tile[r][8 * k + 2 * j + 1] = (a.y + b.y) * (1.f / UNIT);
    }
  }
  __syncthreads();
  const int across = t.flip ? 32 : 16, row0 = t.flip ? c0 : r0, col0 = t.flip ? r0 : c0;
#pragma unroll 4
  for (int e = threadIdx.x; e < 128 * 64 / 4; e += THREADS) {
    const int row = e / across, col = e % across * 4;
    if (row0 + row >= t.rows || col0 + col >= t.cols) continue;
    float4 o = t.flip ? make_float4(tile[col][row], tile[col + 1][row], tile[col + 2][row], tile[col + 3][row])
                      : make_float4(tile[row][col], tile[row][col + 1], tile[row][col + 2], tile[row][col + 3]);
    const int64_t at = (int64_t)(row0 + row) * t.ldp;
    if (h.orth) {
      const float nan = __int_as_float(0x7fc00000);
      if (!good) o = make_float4(nan, nan, nan, nan);
      store4(t.param, at, col0 + col, t.cols, h.pt, t.quads & PARAM, o);
    } else {
      const float4 p = load4(t.param, at, col0 + col, t.cols, h.pt, t.quads & PARAM);
      const float4 n = axpy4(o, -h.lr * t.scale, make_float4(p.x * h.decay, p.y * h.decay, p.z * h.decay, p.w * h.decay));
      store4(t.param, at, col0 + col, t.cols, h.pt, t.quads & PARAM, n);
      if (t.copy) store4(t.copy, (int64_t)(row0 + row) * t.ldc, col0 + col, t.cols, GNN_BF16, t.quads & COPY, n);
    }
  }
}

// ------------------------------------------------------------------ products
enum Phase { GRAM, POLY, NEXT };  // A = X X', P = a I + b A + c A A, X <- P X

// Every product of every step in one launch of persistent, warp-specialised blocks:
// warp 0 loads a ring of tiles by TMA, warp 1 issues the MMAs from one thread, warps
// 2-9 drain one of two accumulators in TMEM while the next tile is multiplied.  A
// tile is 128 x 64 or 128 x 128 on one CTA, or 256 x 256 on a pair of CTAs
// (cta_group::2), which reads a third less from L2 for its flops.  Tiles are dealt in
// the order step, product, matrix; before a tile's first load its matrix's counts of
// the product before are waited for, so a matrix goes on when its own tiles are
// there, and no launch or barrier of the whole card comes between products.
//
// A and P are symmetric: only their blocks on and above the diagonal (of the tile's
// size) are formed, and a block below is read as the transpose of its mirror image,
// by loading that and setting the operand's major bit in the instruction.
//
// The tensor cores truncate at every 16 of k: a product's bits below 2^-25 of the
// largest term, and the sum's below its last place (measured on sums of powers of
// two).  Over a whole row of k that loss, of one sign with the sum, is what the result
// would be off by (4.7e-6 of its norm for 64 x 256, 1.7e-5 for 1000 x 1000, where fp32
// FMAs leave 1.3e-6 and 2.6e-6).  So an accumulator holds 64 of k only, the cross
// products first, while it is small; warps 2-9 add it, rounded, to the tile's sums in
// their registers, and put back what is lost on average, one unit in 2^23 where three
// or four sums of 16 are in it: 1.7e-6 and 1.0e-6 (without that 2.6e-6 and 1.5e-6;
// 128 of k: 2.4e-6 and 2.3e-6).
constexpr int BLOCK_ROWS = BLOCK / 128;
constexpr int EPI_WARPS = 8;
constexpr int PRODUCT_THREADS = 64 + 32 * EPI_WARPS;
constexpr int RING = 192 << 10;
constexpr int MAX_STAGES = 4;
constexpr int STAGED = 32 * 128;  // a warp's 32 rows of 128 bytes on their way out
constexpr int PRODUCT_SMEM = RING + EPI_WARPS * STAGED + 1024 /*barriers*/ + 1024 /*align*/;

// A matrix's operands by their first block of the workspace.
struct Rows {
  int x0, x1, a, p;
  int mb, nb;
  int kx, km;  // 16s of k with values: of X's columns, of its rows
};
struct Steps {
  // The workspace as rows of 64 columns: a block in one box, rows as they lie
  // (K-major operands of 128 rows); and 32 rows of a limb, to store.
  CUtensorMap block, out;
  // As [half of a block][block][limb][64 rows][64 columns]: both limbs of 64 rows of
  // one block, or of two neighbours (MN-major operands: columns of a mirror image or
  // of X; K-major ones of 64 rows).
  CUtensorMap one, two;
  char* base;
  Done* done;
  unsigned* flags;
  int count, steps;
  int half[3];  // pairs: tiles of 128 columns instead of 256
  float coeff[MAX_STEPS][3];
  int first[3][MAX_MATS + 1];  // a step's tiles before each matrix of each product
  Rows mat[MAX_MATS];
};

struct Ring {
  uint8_t *tiles, *staged;
  uint64_t *full, *empty, *tfull, *tempty;
  uint64_t *clear, *filled;  // tiles of 64 columns: the two warps of 32 rows meet
  uint32_t* tmem;
  volatile int* abort_flag;
};
__device__ __forceinline__ Ring carve(uint8_t* raw) {
  Ring s;
  s.tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.staged = s.tiles + RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s.staged + EPI_WARPS * STAGED);
  s.full = bars;
  s.empty = bars + MAX_STAGES;
  s.tfull = bars + 2 * MAX_STAGES;
  s.tempty = s.tfull + 2;
  s.clear = s.tempty + 2;
  s.filled = s.clear + 4;
  s.tmem = reinterpret_cast<uint32_t*>(s.filled + 4);
  s.abort_flag = reinterpret_cast<volatile int*>(s.tmem + 1);
  return s;
}

// A tile: its step, product and matrix, the first 128-row block and the first
// 64-column block of the pair's (or the CTA's), and the length of its sum in 16s and
// in blocks of 64.
struct Tile {
  Rows m;
  int step, phase, mat;
  int rb, cb, k16, kb;
  int cols;  // of the tile
};
template <int COLS>
__device__ __forceinline__ Tile tile_at(const Steps& g, int t) {
  constexpr bool PAIR = COLS == 256;
  const int n0 = g.first[0][g.count], n1 = g.first[1][g.count], each_step = n0 + n1 + g.first[2][g.count];
  Tile r;
  r.step = t / each_step;
  t -= r.step * each_step;
  r.phase = t < n0 ? GRAM : t < n0 + n1 ? POLY : NEXT;
  t -= r.phase == GRAM ? 0 : r.phase == POLY ? n0 : n0 + n1;
  const int* first = g.first[r.phase];
  int lo = 0, hi = g.count - 1;  // the last matrix that begins at t or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  t -= first[lo];
  r.mat = lo;
  r.m = g.mat[lo];
  r.cols = PAIR && g.half[r.phase] ? COLS / 2 : COLS;
  const int wide = r.cols >> 6;  // blocks of 64 across
  const int side = PAIR ? r.m.mb >> 1 : r.m.mb;
  if (r.phase == NEXT) {
    // the tiles that share columns of X side by side
    r.rb = t % side;
    r.cb = t / side * wide;
  } else if (COLS == 64) {
    // columns to the last with values
    const int cols = (r.m.km + 3) >> 2;
    int row = 0;
    while (t >= cols - 2 * row) t -= cols - 2 * row, ++row;
    r.rb = row;
    r.cb = 2 * row + t;
  } else {
    const int each = COLS / r.cols;  // tiles of a square
    int row = 0;
    while (t >= each * (side - row)) t -= each * (side - row), ++row;
    r.rb = row;
    r.cb = row * each * wide + t * wide;
  }
  if (PAIR) r.rb *= 2;
  r.k16 = r.phase == GRAM ? r.m.kx : r.m.km;
  r.kb = (r.k16 + 3) >> 2;
  return r;
}
template <int COLS>
__device__ __forceinline__ int tiles_of(const Steps& g) {
  return g.steps * (g.first[0][g.count] + g.first[1][g.count] + g.first[2][g.count]);
}

// Waits until what a tile reads has been written: the product before, of its matrix.
// False after the time limit or once another role has given up.
template <int COLS>
__device__ __forceinline__ bool wait_for(const Steps& g, const Tile& w, volatile int* abort_flag) {
  const int before = w.phase == GRAM ? NEXT : w.phase - 1;
  const int times = w.phase == GRAM ? w.step : w.step + 1;
  const int need = times * (g.first[before][w.mat + 1] - g.first[before][w.mat]) * (COLS == 256 ? 16 : 8);
  const int* at = &g.done[w.mat].of[before];
  int have;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(have) : "l"(at) : "memory");
  if (have >= need) return true;
  const long long t0 = clock64();
  while (true) {
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(have) : "l"(at) : "memory");
    if (have >= need) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > tc::kWaitCycles) {
      atomicOr(g.flags, 2u);
      *abort_flag = 1;
      return false;
    }
  }
}

// Whether rows of 128-row block b, columns of 64-block kb lie on or above the
// diagonal of a symmetric operand (in squares of the tile's size).
template <bool PAIR>
__device__ __forceinline__ bool above(int b, int kb) {
  return PAIR ? (b >> 1) <= (kb >> 2) : b <= (kb >> 1);
}

// 64 or 128 rows (from 64-row block r64) of an operand with `nb` column blocks from
// block `s`, at k block kb: as they lie (K-major), or, below the diagonal, the mirror
// image's columns (MN-major).  128 rows as they lie come as [limb][128][64], all else
// as [64 of them][limb][64][64].
template <bool PAIR>
__device__ __forceinline__ void load_rows(const Steps& g, uint8_t* to, uint32_t bar, int s, int nb, int r64, int kb,
                                          bool wide, bool direct) {
  if (direct && wide) {
    const int row = (s + (r64 >> 1) * nb + kb) * BLOCK_ROWS;
    if (PAIR)
      tc::tma_load_2d_pair(to, &g.block, bar, 0, row);
    else
      tc::tma_load_2d(to, &g.block, bar, 0, row);
  } else if (direct) {
    tc::tma_load_5d<PAIR>(to, &g.one, bar, s + (r64 >> 1) * nb + kb, r64 & 1);
  } else {
    tc::tma_load_5d<PAIR>(to, wide ? &g.two : &g.one, bar, s + (kb >> 1) * nb + r64, kb & 1);
  }
}

// Where an operand's limbs and 16s of k lie in a stage, in units of 16 bytes of its
// descriptor: K-major a row has its 128 bytes of k, MN-major 16 of k are 16 rows.
struct Operand {
  uint64_t desc;
  uint32_t limb, step;
};
__device__ __forceinline__ Operand operand(uint32_t at, bool mn, bool wide) {
  return {tc::sw128_desc(at, mn ? 2 * 8192 : 16), (uint32_t)(!mn && wide ? 16384 : 8192) >> 4, (uint32_t)(mn ? 2048 : 32) >> 4};
}

template <bool PAIR>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (PAIR)
    tc::mma_16_pair(d, a, b, idesc, acc);
  else
    tc::mma_bf16(d, a, b, idesc, acc);
}

// Of a warp: its lanes go on, or give up, together.
__device__ __forceinline__ bool all(bool x) { return __all_sync(0xffffffffu, x); }

// COLS: of a tile; 256: a pair's.
template <int COLS>
__device__ __forceinline__ void walk(const Steps& g, uint8_t* smem_raw) {
  constexpr bool PAIR = COLS == 256;
  const Ring s = carve(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)tc::cluster_rank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;
  constexpr int a_stage = BLOCK, stage = BLOCK + (PAIR ? COLS / 2 : COLS) * 256;
  constexpr int stages = RING / stage < MAX_STAGES ? RING / stage : MAX_STAGES;
  if (warp == 0 && lane < 4) tc::prefetch_tmap(lane == 0 ? &g.block : lane == 1 ? &g.one : lane == 2 ? &g.two : &g.out);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.tfull[i], 1);
      tc::mbar_init(&s.tempty[i], (PAIR ? 2 : 1) * EPI_WARPS);  // a lane of each warp
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&s.clear[i], 2);
      tc::mbar_init(&s.filled[i], 2);
    }
    *s.abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tc::tmem_alloc_pair(s.tmem, 512);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(s.tmem, 256);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (PAIR) tc::cluster_sync();  // the partner's barriers are there
  tc::fence_after_sync();
  const uint32_t tmem = *s.tmem;
  const int tiles = tiles_of<COLS>(g);

  if (warp == 0 && lane == 0) {
    int st = 0;
    uint32_t ph = 0;
    for (int t = unit; t < tiles; t += units) {
      const Tile w = tile_at<COLS>(g, t);
      const int bn = PAIR ? w.cols >> 1 : COLS;  // columns of a CTA's share of B
      const int x = w.step & 1 ? w.m.x1 : w.m.x0, sq = 2 * w.m.mb;
      const int left = w.phase == GRAM ? x : w.phase == POLY ? w.m.a : w.m.p, left_nb = w.phase == GRAM ? w.m.nb : sq;
      const int rb = w.rb + rank, cb = w.cb + rank * (bn >> 6);
      for (int kb = 0; kb < w.kb; ++kb) {
        if (!tc::mbar_wait(&s.empty[st], ph ^ 1, g.flags, s.abort_flag)) goto done;
        if (rank == 0) tc::mbar_expect_tx(&s.full[st], (PAIR ? 2 : 1) * (BLOCK + bn * 256));
        if (kb == 0) {
          if (!wait_for<COLS>(g, w, s.abort_flag)) goto done;
          tc::fence_async_global();  // what the count says is there, to TMA's reads too
        }
        uint8_t* a = s.tiles + st * stage;
        const uint32_t bar = PAIR ? tc::map_to_rank(&s.full[st], 0) : tc::smem_u32(&s.full[st]);
        load_rows<PAIR>(g, a, bar, left, left_nb, 2 * rb, kb, true, w.phase == GRAM || above<PAIR>(rb, kb));
        if (w.phase == NEXT)
          load_rows<PAIR>(g, a + a_stage, bar, x, w.m.nb, cb, kb, bn == 128, false);
        else
          load_rows<PAIR>(g, a + a_stage, bar, left, left_nb, cb, kb, bn == 128, w.phase == GRAM || above<PAIR>(cb >> 1, kb));
        if (++st == stages) { st = 0; ph ^= 1; }
      }
    }
    // every stage's release has arrived before this CTA may end
    for (int i = 0; i < stages; ++i) {
      if (!tc::mbar_wait(&s.empty[st], ph ^ 1, g.flags, s.abort_flag)) goto done;
      if (++st == stages) { st = 0; ph ^= 1; }
    }
  } else if (warp == 1 && rank == 0) {
    // the whole warp walks, one lane issues
    int st = 0, it = 0;
    uint32_t ph = 0;
    for (int t = unit; t < tiles; t += units) {
      const Tile w = tile_at<COLS>(g, t);
      const int bn = PAIR ? w.cols >> 1 : COLS;
      for (int kb = 0; kb < w.kb; ++kb, ++it) {
        const int acc = it & 1, some = min(w.k16 - 4 * kb, 4);
        const uint32_t d = tmem + acc * COLS;
        const bool a_mn = w.phase != GRAM && !above<PAIR>(w.rb, kb);
        const bool b_mn = w.phase == NEXT || (w.phase == POLY && !above<PAIR>(w.cb >> 1, kb));
        const uint32_t idesc = tc::idesc_16(false, PAIR ? 256 : 128, PAIR ? w.cols : COLS, a_mn, b_mn);
        if (!all(tc::mbar_wait<true>(&s.tempty[acc], ((it >> 1) & 1) ^ 1, g.flags, s.abort_flag))) goto done;
        if (!all(tc::mbar_wait(&s.full[st], ph, g.flags, s.abort_flag))) goto done;
        tc::fence_after_sync();
        const uint32_t at = tc::smem_u32(s.tiles + st * stage);
        const Operand l = operand(at, a_mn, true), r = operand(at + a_stage, b_mn, bn == 128);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= some) break;
            multiply<PAIR>(d, l.desc + k * l.step, r.desc + r.limb + k * r.step, idesc, k ? 1u : 0u);
            multiply<PAIR>(d, l.desc + l.limb + k * l.step, r.desc + k * r.step, idesc, 1u);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= some) break;
            multiply<PAIR>(d, l.desc + k * l.step, r.desc + k * r.step, idesc, 1u);
          }
          if (PAIR) {
            tc::mma_commit_pair(&s.empty[st]);
            tc::mma_commit_pair(&s.tfull[acc]);
          } else {
            tc::mma_commit(&s.empty[st]);
            tc::mma_commit(&s.tfull[acc]);
          }
        }
        __syncwarp();
        if (++st == stages) { st = 0; ph ^= 1; }
      }
    }
  } else if (warp >= 2) {
    const int e = warp - 2, q = warp & 3, half = e >> 2;  // TMEM lane quarter, column half
    const uint32_t lane0 = tmem + ((uint32_t)(q * 32) << 16);
    const int r = q * 32 + lane;  // of the 128-row block
    constexpr int MOST = COLS / 2;  // columns of this warp's half of a tile, at most
    // tiles of 64 columns: the two warps of 32 rows share a tile for each limb
    uint8_t* staged = s.staged + (MOST < 64 ? 2 * q : e) * STAGED;
    const uint32_t freed0 = tc::map_to_rank(&s.tempty[0], 0), freed1 = tc::map_to_rank(&s.tempty[1], 0);
    int it = 0;
    uint32_t met = 0;  // parity of the two warps' next meeting
    // The last tile's stores are waited for and counted when this warp would wait
    // anyway, or when it has drained an accumulator.
    int* pending = nullptr;
    auto count_it = [&] {
      if (!pending) return;
      if (lane == 0) {
        tc::bulk_wait_all();
        if (MOST < 64) tc::mbar_arrive(&s.clear[q]);
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(pending) : "memory");
      }
      pending = nullptr;
    };
    for (int t = unit; t < tiles; t += units) {
      const Tile w = tile_at<COLS>(g, t);
      const int rb = w.rb + rank, row = rb * 128 + r, mine = PAIR ? w.cols >> 1 : MOST;
      const int out = w.phase == GRAM ? w.m.a : w.phase == POLY ? w.m.p : w.step & 1 ? w.m.x0 : w.m.x1;
      const int out_nb = w.phase == NEXT ? w.m.nb : 2 * w.m.mb;
      const float ca = g.coeff[w.step][0], cb_ = g.coeff[w.step][1], cc = g.coeff[w.step][2];
      // this thread's place on P's diagonal, from the first column of its half
      const int on_diag = row - (w.cb * 64 + half * mine);
      if (w.phase == POLY) {  // A, by ordinary loads
        count_it();
        if (!all(lane || wait_for<COLS>(g, w, s.abort_flag))) goto done;
        __syncwarp();  // orders the other lanes' reads behind the first one's wait, as a vote does not
      }
      const int64_t a_at = (int64_t)w.m.a * BLOCK + ((int64_t)rb * out_nb + w.cb) * BLOCK + r * 128;
      uint4 a_hi[MOST < 64 ? 4 : 1], a_lo[MOST < 64 ? 4 : 1];
      if (MOST < 64 && w.phase == POLY) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a_hi[k] = __ldcg(reinterpret_cast<const uint4*>(g.base + a_at + half * 64 + k * 16));
          a_lo[k] = __ldcg(reinterpret_cast<const uint4*>(g.base + a_at + LIMB + half * 64 + k * 16));
        }
      }
      float2 sum[MOST / 2];
#pragma unroll
      for (int j = 0; j < MOST / 2; ++j) sum[j] = dup2(0.f);
      for (int kb = 0; kb < w.kb; ++kb, ++it) {
        const int acc = it & 1;
        const float2 back = dup2(w.k16 - 4 * kb > 2 ? 1.f + 0x1p-23f : 1.f);
        if (!all(tc::mbar_test(&s.tfull[acc], (it >> 1) & 1))) {
          count_it();
          if (!all(tc::mbar_wait(&s.tfull[acc], (it >> 1) & 1, g.flags, s.abort_flag))) goto done;
        }
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < MOST; c += 32) {
          if (c >= mine) break;
          uint32_t v[32];
          tc::tmem_ld32(lane0 + acc * COLS + half * mine + c, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            sum[c / 2 + j] = fma2_rn(back, make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sum[c / 2 + j]);
        }
        // hands the accumulator back to the MMA warp
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(acc ? freed1 : freed0);
        count_it();
      }
      // 64 columns at a time: a row of one limb is then 128 bytes
#pragma unroll
      for (int c = 0; c < MOST; c += 64) {
        if (c >= mine) break;
        const int col = half * mine + c, cb = w.cb + (col >> 6);
        constexpr int CHUNKS = MOST < 64 ? MOST / 8 : 8;  // of eight columns
        const int64_t block = out + (int64_t)rb * out_nb + cb;
        const char* from = g.base + a_at + (int64_t)(col >> 6) * BLOCK;
        uint4 hi[CHUNKS], lo[CHUNKS];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
          float2 f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = mul2_rn(sum[c / 2 + 4 * k + j], dup2(1.f / UNIT));
          if (w.phase == POLY) {
            const int diag = on_diag - (c + 8 * k);  // the diagonal's place among the eight
            uint4 h, l;
            if (MOST < 64) {
              h = a_hi[k], l = a_lo[k];
            } else {
              h = __ldcg(reinterpret_cast<const uint4*>(from + k * 16));
              l = __ldcg(reinterpret_cast<const uint4*>(from + LIMB + k * 16));
            }
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 a = add2_rn(Pack2<__half>::from(hw[j]), Pack2<__half>::from(lw[j]));
              f[j] = fma2_rn(dup2(cc), f[j], mul2_rn(dup2(cb_), a));
              if (diag == 2 * j) f[j].x += ca * UNIT;
              if (diag == 2 * j + 1) f[j].y += ca * UNIT;
            }
          }
          limbs(f[0].x, f[0].y, hi[k].x, lo[k].x), limbs(f[1].x, f[1].y, hi[k].y, lo[k].y);
          limbs(f[2].x, f[2].y, hi[k].z, lo[k].z), limbs(f[3].x, f[3].y, hi[k].w, lo[k].w);
        }
        // through shared memory: a warp's rows lie 128 bytes apart, and as ordinary
        // stores each of their 16-byte pieces would be a transaction of its own
        if (MOST < 64) {
          // both warps' last tile has left (each sends one limb of it)
          count_it();
          if (!all(tc::mbar_wait(&s.clear[q], met ^ 1, g.flags, s.abort_flag))) goto done;
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            uint4* to = reinterpret_cast<uint4*>(staged + lane * 128 + (((half * 4 + k) ^ (lane & 7)) << 4));
            to[0] = hi[k];
            to[STAGED / 16] = lo[k];
          }
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.filled[q]);
          if (!all(tc::mbar_wait(&s.filled[q], met, g.flags, s.abort_flag))) goto done;
          met ^= 1;
          if (lane == 0) {
            tc::tma_store_2d(&g.out, staged + half * STAGED, 0, (int)(block * BLOCK_ROWS) + half * 128 + q * 32);
            tc::bulk_commit();
          }
        } else {
#pragma unroll
          for (int l = 0; l < 2; ++l) {
            if (lane == 0) tc::bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
              *reinterpret_cast<uint4*>(staged + lane * 128 + ((k ^ (lane & 7)) << 4)) = l ? lo[k] : hi[k];
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tc::tma_store_2d(&g.out, staged, 0, (int)(block * BLOCK_ROWS) + l * 128 + q * 32);
              tc::bulk_commit();
            }
          }
        }
      }
      __syncwarp();
      pending = &g.done[w.mat].of[w.phase];
    }
    count_it();
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
  if (PAIR) tc::cluster_sync();  // nothing of the partner's arrives here any more
  if (threadIdx.x == 0 && *s.abort_flag) atomicExch(&g.done->gave_up, 1);
  if (warp == 1) {
    tc::fence_after_sync();
    if (PAIR)
      tc::tmem_dealloc_pair(tmem, 512);
    else
      tc::tmem_dealloc(tmem, 256);
  }
}

// 4096 x 4096: 554 us a step, 1.49 PFLOP/s of fp16 products; 36 of 1024 x 4096 1.35-1.5,
// at the card's power cap (a library's bf16 product sustains 1.70).
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PRODUCT_THREADS, 1)
    steps_pair_kernel(const __grid_constant__ Steps g) {
  extern __shared__ uint8_t smem_raw[];
  walk<256>(g, smem_raw);
}
// 256 x 512: 19 us a step, three products in dependence, of which 4 us each are a tile's
// store, its count, the poll for it and the next product's first load.
template <int COLS>
__global__ void __launch_bounds__(PRODUCT_THREADS, 1) steps_kernel(const __grid_constant__ Steps g) {
  extern __shared__ uint8_t smem_raw[];
  walk<COLS>(g, smem_raw);
}

// ------------------------------------------------------------- small matrices
// A matrix of up to 64 x 512 stays in one CTA's shared memory from its gradient to its
// update: no tile waits for another CTA's, which is what bounds small matrices above
// (16 of 64 x 256: 94 us, here 39, fifteen products of 1.2 us and the passes around).  The
// same limbs, products and sums; every 64 of k has an accumulator of its own in TMEM, so
// that a product is issued without a pause.  Operands have 64 rows; an MMA reads 128 of A,
// and what the other 64 give stays in lanes of TMEM that nobody reads.
constexpr int SMALL_M = 64, SMALL_N = 512;
constexpr int SMALL_THREADS = 512;
constexpr int HALF_LIMB = 64 * 128, HALF_BLOCK = 2 * HALF_LIMB;  // of 64 rows
struct SmallSteps {
  int steps;
  float coeff[MAX_STEPS][3];
  unsigned* flags;
};
constexpr int small_smem(int kb) { return (kb + 3) * HALF_BLOCK + 1024 /*barrier*/ + 1024 /*align*/; }

// Byte of 8 columns (chunk k of 8) of row r of a limb in shared memory.
__device__ __forceinline__ int small_at(int r, int k) { return r * 128 + ((k ^ (r & 7)) << 4); }

__global__ void __launch_bounds__(SMALL_THREADS, 1)
    small_kernel(const __grid_constant__ Table tab, const Hyper h, const __grid_constant__ SmallSteps g, float* norms) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ double part[SMALL_THREADS / 32];
  __shared__ float shared_norm;
  const Mat& t = tab.mat[blockIdx.x];
  uint8_t* const x = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int kbs = (t.n + 63) >> 6, kx = (t.n + 15) >> 4, km = (t.m + 15) >> 4;
  uint8_t* const a = x + kbs * HALF_BLOCK;
  uint8_t* const p = a + HALF_BLOCK;
  uint64_t* const bar = reinterpret_cast<uint64_t*>(p + 2 * HALF_BLOCK);
  uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(bar + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t tmem_cols = kbs <= 4 ? 256 : 512;
  if (threadIdx.x == 0) {
    tc::mbar_init(bar, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  for (int e = threadIdx.x; e < kbs * HALF_BLOCK / 16; e += SMALL_THREADS)
    reinterpret_cast<uint4*>(x)[e] = make_uint4(0, 0, 0, 0);
  cudaGridDependencySynchronize();
  // Columns of TMEM are asked for when the kernel before has given its own back, and the
  // kernel behind starts when they are there: on a shared SM neither can hold columns
  // that the other, which it waits for, has yet to get.  A block's first thread to trigger
  // counts for all of it, so only the warp that has them does.
  if (warp == 0) {
    tc::tmem_alloc(tmem_at, tmem_cols);
    tc::tmem_relinquish();
    __syncwarp();
    cudaTriggerProgrammaticLaunchCompletion();
  }
  tc::fence_before_sync();
  // |u|
  const int across = (t.cols + 3) >> 2, quads = t.rows * across;
  double sum = 0;
  for (int e = threadIdx.x; e < quads; e += 4 * SMALL_THREADS) {
    Quad q[4];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = e + k * SMALL_THREADS, row = min(i / across, t.rows - 1);
      q[k].load(t, h, row, i % across * 4, i < quads ? t.cols : 0);
    }
    float4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[k] = q[k].update(h);
      s = fmaf(u[k].x, u[k].x, fmaf(u[k].y, u[k].y, fmaf(u[k].z, u[k].z, fmaf(u[k].w, u[k].w, s))));
    }
    if (s > 1e-28f && s < 1e38f) {
      sum += (double)s;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sum += (double)u[k].x * u[k].x + (double)u[k].y * u[k].y + (double)u[k].z * u[k].z + (double)u[k].w * u[k].w;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  if (threadIdx.x == 0) {
    double s = 0;
    for (int w = 0; w < SMALL_THREADS / 32; ++w) s += part[w];
    shared_norm = root_of(s);
    if (norms) norms[t.slot] = shared_norm;
  }
  __syncthreads();
  const float norm = shared_norm;
  bool good = isfinite(norm);
  const float inv = scale_of(norm, h.eps);
  for (int e = threadIdx.x; e < quads; e += SMALL_THREADS) {
    const int row = e / across, col = e % across * 4;
    Quad q;
    q.load(t, h, row, col, t.cols);
    const float4 u = q.update(h);
    if (!good) continue;
    if (!h.orth) store4(t.mom, (int64_t)row * t.ldm, col, t.cols, h.mt, t.quads & MOM, q.m);
    uint32_t hi[2], lo[2];
    limbs(u.x * inv, u.y * inv, hi[0], lo[0]);
    limbs(u.z * inv, u.w * inv, hi[1], lo[1]);
    if (t.flip) {  // four rows of X; those past its last stay zero
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = col + j;
        if (r >= t.m) break;
        uint8_t* to = x + (row >> 6) * HALF_BLOCK + small_at(r, (row & 63) >> 3) + (row & 7) * 2;
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)(hi[j >> 1] >> (16 * (j & 1)));
        *reinterpret_cast<uint16_t*>(to + HALF_LIMB) = (uint16_t)(lo[j >> 1] >> (16 * (j & 1)));
      }
    } else {
      uint8_t* to = x + (col >> 6) * HALF_BLOCK + small_at(row, (col & 63) >> 3) + (col & 7) * 2;
      *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(to + HALF_LIMB) = make_uint2(lo[0], lo[1]);
    }
  }
  tc::fence_async_smem();
  __syncthreads();

  // 64 of k (or `some` 16s of it) of a product, from one lane
  auto multiply64 = [&](uint32_t d, uint32_t left, uint32_t right, bool right_mn, int cols, int some) {
    const uint32_t idesc = tc::idesc_16(false, 128, cols, false, right_mn);
    const uint64_t l = tc::sw128_desc(left, 16), r = tc::sw128_desc(right, right_mn ? HALF_BLOCK : 16);
    const uint32_t limb = HALF_LIMB >> 4, ls = 32 >> 4, rs = (right_mn ? 2048 : 32) >> 4;
    for (int k = 0; k < some; ++k) {
      tc::mma_bf16(d, l + k * ls, r + limb + k * rs, idesc, k ? 1u : 0u);
      tc::mma_bf16(d, l + limb + k * ls, r + k * rs, idesc, 1u);
    }
    for (int k = 0; k < some; ++k) tc::mma_bf16(d, l + k * ls, r + k * rs, idesc, 1u);
  };
  const uint32_t xs = tc::smem_u32(x), as = tc::smem_u32(a), ps = tc::smem_u32(p);
  uint32_t ph = 0;
  // every thread: the product is there, or all give up
  auto arrived = [&] {
    const bool ok = tc::mbar_wait(bar, ph, g.flags, abort_flag);
    ph ^= 1;
    const bool all_ok = !__syncthreads_or(!ok);
    tc::fence_after_sync();
    return all_ok;
  };
  // what was written is there for the next product
  auto written = [&] {
    tc::fence_before_sync();
    tc::fence_async_smem();
    __syncthreads();
    tc::fence_after_sync();
  };
  const int q = warp & 3, piece = warp >> 2, r = q * 32 + lane;  // TMEM lanes; 16 columns of 64
  const bool mine = q < 2;
  const uint32_t lane0 = tmem + ((uint32_t)(q * 32) << 16);
  auto put16 = [&](uint8_t* limb, int col, const float (&f)[16]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4 hi, lo;
      limbs(f[8 * k], f[8 * k + 1], hi.x, lo.x), limbs(f[8 * k + 2], f[8 * k + 3], hi.y, lo.y);
      limbs(f[8 * k + 4], f[8 * k + 5], hi.z, lo.z), limbs(f[8 * k + 6], f[8 * k + 7], hi.w, lo.w);
      uint8_t* to = limb + small_at(r, (col >> 3) + k);
      *reinterpret_cast<uint4*>(to) = hi;
      *reinterpret_cast<uint4*>(to + HALF_LIMB) = lo;
    }
  };
  // what truncated sums lose on average (see the steps' kernel)
  auto back_of = [](int k16) { return k16 > 2 ? 1.f + 0x1p-23f : 1.f; };
  bool done = true;  // false once a wait has run out: what X holds is unfinished
  for (int s = 0; s < g.steps; ++s) {
    const float ca = g.coeff[s][0], cb = g.coeff[s][1], cc = g.coeff[s][2];
    if (warp == 0 && tc::elect_one()) {
      for (int kb = 0; kb < kbs; ++kb)
        multiply64(tmem + 64 * kb, xs + kb * HALF_BLOCK, xs + kb * HALF_BLOCK, false, 64, min(kx - 4 * kb, 4));
      tc::mma_commit(bar);
    }
    __syncwarp();
    if (!(done = arrived())) break;
    float am[16];
    if (mine) {
#pragma unroll
      for (int j = 0; j < 16; ++j) am[j] = 0.f;
      for (int kb = 0; kb < kbs; ++kb) {
        float v[16];
        tc::tmem_ld16(lane0 + 64 * kb + 16 * piece, v);
        const float back = back_of(kx - 4 * kb);
#pragma unroll
        for (int j = 0; j < 16; ++j) am[j] = fmaf(back, v[j], am[j]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) am[j] *= 1.f / UNIT;
      put16(a, 16 * piece, am);
    }
    written();
    if (warp == 0 && tc::elect_one()) {
      multiply64(tmem, as, as, false, 64, km);
      tc::mma_commit(bar);
    }
    __syncwarp();
    if (!(done = arrived())) break;
    if (mine) {
      float v[16];
      tc::tmem_ld16(lane0 + 16 * piece, v);
      const float back = back_of(km) * (1.f / UNIT);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        // A as its limbs hold it
        const __half ah = __float2half_rn(am[j]);
        const float held = __half2float(ah) + __half2float(__float2half_rn(am[j] - __half2float(ah)));
        v[j] = fmaf(cc, v[j] * back, cb * held) + (r == 16 * piece + j ? ca * UNIT : 0.f);
      }
      put16(p, 16 * piece, v);
    }
    written();
    if (warp == 0 && tc::elect_one()) {
      for (int kb = 0; kb < kbs; kb += 4)
        multiply64(tmem + 64 * kb, ps, xs + kb * HALF_BLOCK, true, 64 * min(kbs - kb, 4), km);
      tc::mma_commit(bar);
    }
    __syncwarp();
    if (!(done = arrived())) break;
    if (mine) {
      const float back = back_of(km) * (1.f / UNIT);
      for (int kb = 0; kb < kbs; ++kb) {
        float v[16];
        tc::tmem_ld16(lane0 + 64 * kb + 16 * piece, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= back;
        put16(x + kb * HALF_BLOCK, 16 * piece, v);
      }
    }
    written();
  }
  good &= done;
  for (int e = threadIdx.x; e < quads; e += SMALL_THREADS) {
    const int row = e / across, col = e % across * 4;
    if (!good && !h.orth) break;  // this matrix stays as it is
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int xr = t.flip ? col + j : row, xc = t.flip ? row : col + j;
      const uint8_t* from = x + (xc >> 6) * HALF_BLOCK + small_at(xr, (xc & 63) >> 3) + (xc & 7) * 2;
      const bool there = xr < t.m && xc < t.n;
      o[j] = !good ? __int_as_float(0x7fc00000)
             : there ? (__half2float(*reinterpret_cast<const __half*>(from)) +
                        __half2float(*reinterpret_cast<const __half*>(from + HALF_LIMB))) * (1.f / UNIT)
                     : 0.f;
    }
    const float4 f = make_float4(o[0], o[1], o[2], o[3]);
    const int64_t at = (int64_t)row * t.ldp;
    if (h.orth) {
      store4(t.param, at, col, t.cols, h.pt, t.quads & PARAM, f);
    } else {
      const float4 w = load4(t.param, at, col, t.cols, h.pt, t.quads & PARAM);
      const float4 n = axpy4(f, -h.lr * t.scale, make_float4(w.x * h.decay, w.y * h.decay, w.z * h.decay, w.w * h.decay));
      store4(t.param, at, col, t.cols, h.pt, t.quads & PARAM, n);
      if (t.copy) store4(t.copy, (int64_t)row * t.ldc, col, t.cols, GNN_BF16, t.quads & COPY, n);
    }
  }
  if (*abort_flag) {
    // a wait gave up: products in flight land within microseconds
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, tmem_cols);
  }
}

// ---------------------------------------------------------------- host side
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// A launch may start while the kernel before it ends; each waits for that before
// it touches memory.  TOGETHER: its blocks wait on one another, so all are there or none
// starts.
template <bool TOGETHER = false, class... P, class... A>
gnn_status launch(int64_t grid, int block, size_t smem, cudaStream_t st, void (*k)(P...), const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (TOGETHER) {
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
  } else {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
  }
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

struct Shape {
  int rows, cols;
};
int64_t size_of(const Shape& s) {
  const int64_t m = std::min(s.rows, s.cols), n = std::max(s.rows, s.cols);
  return m * m * n;
}

// X's sides, padded to whole tiles.
void sides(Mat& t, int bn) {
  t.flip = t.rows > t.cols;
  t.m = std::min(t.rows, t.cols), t.n = std::max(t.rows, t.cols);
  t.mb = (int)up((t.m + 127) / 128, bn ? 1 : 2), t.nb = (int)up((t.n + 63) / 64, bn ? 2 : 4);
}
// Places of X's two copies, A and P in a pass's workspace.
void place(Mat& t, Arena& ar, int bn) {
  sides(t, bn);
  for (int k = 0; k < 2; ++k) t.x[k] = ar.take<char>((size_t)t.mb * t.nb * BLOCK);
  t.a = ar.take<char>((size_t)t.mb * 2 * t.mb * BLOCK);
  t.p = ar.take<char>((size_t)t.mb * 2 * t.mb * BLOCK);
  t.parts = (int)std::min<int64_t>(PARTS, ((int64_t)t.rows * t.cols + 16 * THREADS - 1) / (16 * THREADS));
}

// A matrix's tiles of one product; half: of 128 columns on pairs.
int64_t tiles_in(const Mat& t, Phase ph, int bn, int half) {
  const int64_t side = bn ? t.mb : t.mb / 2, km = (t.m + 63) / 64, kx = (t.n + 63) / 64;
  if (ph == NEXT) return side * (bn == 64 ? kx : bn || half ? t.nb / 2 : t.nb / 4);
  return bn == 64 ? side * km - side * (side - 1) : side * (side + 1) / 2 * (half ? 2 : 1);
}

constexpr int SMS = 152;
int sms_there() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SMS;
  return std::max(n, 2);
}

// One product's clocks on tiles of bn columns (0: pairs, 256 or with half 128
// columns): from a tile's last product to the first of what waits for it, and for
// every 64 of k what the MMAs, or shared memory for smaller tiles, take.  Fitted to steps
// of 1 to 12 matrices of 64 x 64 to 1024 x 4096 (within 15%; 36 of 1024 x 4096, at the power
// cap, take half as long again, on any tiles).  Several matrices fill each other's last rounds.
double clocks(const Table& tab, Phase ph, int bn, int half) {
  const double between = bn == 64 ? 7000 : bn ? 11000 : half ? 12000 : 18000;
  const double each = bn == 64 ? 1050 : bn ? 1130 : half ? 983 : 1490;
  const int units = bn ? SMS : SMS / 2;
  double total = 0, longest = 0;
  int64_t tiles = 0;
  for (int i = 0; i < tab.count; ++i) {
    Mat t = tab.mat[i];
    sides(t, bn);
    const double len = ((ph == GRAM ? t.n : t.m) + 63) / 64;
    const int64_t k = tiles_in(t, ph, bn, half);
    tiles += k, total += k * len, longest = std::max(longest, len);
  }
  const double rounds = tab.count == 1 ? (double)((tiles + units - 1) / units) * longest : total / units;
  return std::max(rounds, longest) * each + between;
}
double clocks(const Table& tab, int bn, const int (&half)[3]) {
  return clocks(tab, GRAM, bn, half[GRAM]) + clocks(tab, POLY, bn, half[POLY]) + clocks(tab, NEXT, bn, half[NEXT]);
}

// The tiles of a pass, and every matrix's place in its workspace.
void place_pass(Table& tab, Arena& ar) {
  // a pass of small matrices alone needs none; among larger ones theirs are hidden
  tab.small = 1;
  for (int i = 0; i < tab.count; ++i) {
    const int m = std::min(tab.mat[i].rows, tab.mat[i].cols), n = std::max(tab.mat[i].rows, tab.mat[i].cols);
    tab.small &= m <= SMALL_M && n <= SMALL_N;
  }
  tab.blocks = 0;
  if (tab.small) {
    for (int i = 0; i < tab.count; ++i) sides(tab.mat[i], 64);
    ar.take<int>(1);
    return;
  }
  const int whole[3] = {0, 0, 0};
  int half[3];
  for (Phase ph : {GRAM, POLY, NEXT}) half[ph] = clocks(tab, ph, 0, 1) < clocks(tab, ph, 0, 0);
  tab.bn = clocks(tab, 128, whole) < clocks(tab, 64, whole) ? 128 : 64;
  if (clocks(tab, 0, half) < clocks(tab, tab.bn, whole)) tab.bn = 0;
  for (int k = 0; k < 3; ++k) tab.half[k] = tab.bn ? 0 : half[k];
  for (int i = 0; i < tab.count; ++i) place(tab.mat[i], ar, tab.bn);
  tab.blocks = (int64_t)(ar.used / BLOCK);
  tab.partial = ar.take<double>((size_t)MAX_MATS * PARTS);
  tab.done = ar.take<Done>(MAX_MATS);
}

// Matrices in the order of their work, the largest first, MAX_MATS to a pass; every
// pass has the workspace from its start.
template <class Get>
std::vector<int> order_of(int count, Get shape) {
  std::vector<int> at;
  for (int i = 0; i < count; ++i) {
    const Shape s = shape(i);
    if (s.rows > 0 && s.cols > 0) at.push_back(i);
  }
  std::stable_sort(at.begin(), at.end(), [&](int a, int b) { return size_of(shape(a)) > size_of(shape(b)); });
  return at;
}

template <class Fill>
gnn_status each_pass(const std::vector<int>& order, void* ws, size_t cap, size_t* need, Fill fill) {
  *need = 0;
  for (size_t k = 0; k < order.size(); k += MAX_MATS) {
    Arena ar(ws, cap);
    Table tab;
    tab.count = (int)std::min<size_t>(MAX_MATS, order.size() - k);
    GNN_TRY(fill(tab, ar, (int)k));
    *need = std::max(*need, ar.used);
  }
  return GNN_OK;
}

gnn_status launch_steps(const Steps& g, int bn, cudaStream_t st) {
  const int64_t tiles = (int64_t)g.steps * (g.first[0][g.count] + g.first[1][g.count] + g.first[2][g.count]);
  const int widest = std::max(std::max(g.first[0][g.count], g.first[1][g.count]), g.first[2][g.count]);
  if (tiles > 0x3fffffff) return fail(GNN_ERR_UNSUPPORTED, "Newton-Schulz: too many tiles in one call");
  const int units = std::min(widest, bn ? sms_there() : sms_there() / 2);
  auto run = [&](auto* k, PerDevice& done, int grid) -> gnn_status {
    GNN_TRY(allow_smem(k, PRODUCT_SMEM, done));
    return launch<true>(grid, PRODUCT_THREADS, PRODUCT_SMEM, st, k, g);
  };
  static PerDevice done0, done64, done128;
  if (bn == 0) return run(steps_pair_kernel, done0, 2 * units);
  return bn == 64 ? run(steps_kernel<64>, done64, units) : run(steps_kernel<128>, done128, units);
}

gnn_status maps_of(Steps& g, const void* ws, uint64_t blocks) {
  const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  GNN_TRY(encode_tmap_2d(&g.block, t, ws, 64, blocks * BLOCK_ROWS, 128, 64, BLOCK_ROWS));
  GNN_TRY(encode_tmap_2d(&g.out, t, ws, 64, blocks * BLOCK_ROWS, 128, 64, 32));
  const uint64_t dims[5] = {64, 64, 2, blocks, 2}, strides[4] = {128, LIMB, BLOCK, LIMB / 2};
  const uint32_t one[5] = {64, 64, 2, 1, 1}, two[5] = {64, 64, 2, 2, 1};
  GNN_TRY(encode_tmap(&g.one, t, 5, ws, dims, strides, one));
  return encode_tmap(&g.two, t, 5, ws, dims, strides, two);
}

gnn_status run_pass(void* ws, Table& tab, const Hyper& h, const float* coeffs, int steps, float* norms, cudaStream_t st) {
  if (tab.blocks > 0x7fffff00 / BLOCK_ROWS) return fail(GNN_ERR_UNSUPPORTED, "Newton-Schulz: matrices too large together");
  auto blocks = [&](auto&& of) {
    tab.first[0] = 0;
    for (int i = 0; i < tab.count; ++i) tab.first[i + 1] = tab.first[i] + of(tab.mat[i]);
    return tab.first[tab.count];
  };
  if (tab.small) {
    static PerDevice done;
    GNN_TRY(allow_smem(small_kernel, small_smem(SMALL_N / 64), done));
    SmallSteps g;
    g.steps = steps;
    for (int s = 0; s < steps; ++s)
      for (int k = 0; k < 3; ++k) g.coeff[s][k] = coeffs[3 * s + k];
    g.flags = device_flags();
    if (!g.flags) return fail(GNN_ERR_CUDA, "device flag word unavailable");
    int kb = 0;
    for (int i = 0; i < tab.count; ++i) kb = std::max(kb, (tab.mat[i].n + 63) / 64);
    return launch(tab.count, SMALL_THREADS, small_smem(kb), st, small_kernel, tab, h, g, norms);
  }
  int grid = blocks([](const Mat& t) { return t.parts; });
  GNN_TRY(launch(grid, THREADS, 0, st, square_kernel, tab, h));
  grid = blocks([](const Mat& t) { return t.mb * t.nb; });
  GNN_TRY(launch(grid, THREADS, 0, st, begin_kernel, tab, h, norms));
  if (steps) {
    Steps g;
    g.base = static_cast<char*>(ws);
    g.done = tab.done;
    g.flags = device_flags();
    if (!g.flags) return fail(GNN_ERR_CUDA, "device flag word unavailable");
    GNN_TRY(maps_of(g, ws, (uint64_t)tab.blocks));
    for (int k = 0; k < 3; ++k) g.half[k] = tab.half[k];
    g.count = tab.count, g.steps = steps;
    for (int s = 0; s < steps; ++s)
      for (int k = 0; k < 3; ++k) g.coeff[s][k] = coeffs[3 * s + k];
    auto at = [&](const char* p) { return (int)((p - g.base) / BLOCK); };
    for (int i = 0; i < tab.count; ++i) {
      const Mat& t = tab.mat[i];
      g.mat[i] = {at(t.x[0]), at(t.x[1]), at(t.a), at(t.p), t.mb, t.nb, (t.n + 15) / 16, (t.m + 15) / 16};
    }
    for (Phase ph : {GRAM, POLY, NEXT}) {
      int64_t sum = 0;
      for (int i = 0; i <= tab.count; ++i) {
        if (sum > 0x3fffffff) return fail(GNN_ERR_UNSUPPORTED, "Newton-Schulz: too many tiles in one call");
        g.first[ph][i] = (int)sum;
        if (i < tab.count) sum += tiles_in(tab.mat[i], ph, tab.bn, tab.half[ph]);
      }
    }
    GNN_TRY(launch_steps(g, tab.bn, st));
  }
  grid = blocks([](const Mat& t) { return t.mb * t.nb; });
  return launch(grid, THREADS, 0, st, apply_kernel, tab, h, steps & 1);
}

constexpr int MOST = 65536;  // rows or columns of a matrix
constexpr int MOST_SIDE = 16384;  // the smaller of the two
gnn_status check_shape(const char* who, int i, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return fail(GNN_ERR_INVALID_ARG, "%s: matrix %d has a negative size", who, i);
  if (rows > MOST || cols > MOST || std::min(rows, cols) > MOST_SIDE)
    return fail(GNN_ERR_UNSUPPORTED, "%s: matrix %d is larger than %d x %d", who, i, MOST_SIDE, MOST);
  return GNN_OK;
}
gnn_status check_steps(const char* who, const float* coeffs, int steps, double eps) {
  if (steps < 0 || steps > MAX_STEPS) return fail(GNN_ERR_INVALID_ARG, "%s: steps is 0 to %d", who, MAX_STEPS);
  if (steps && !coeffs) return fail(GNN_ERR_INVALID_ARG, "%s: NULL coeffs", who);
  for (int i = 0; i < 3 * steps; ++i)
    if (!(std::fabs(coeffs[i]) <= 32.f)) return fail(GNN_ERR_INVALID_ARG, "%s: coeffs lie in [-32, 32]", who);
  if (!(eps >= 1e-30) || !(eps <= 1e30)) return fail(GNN_ERR_INVALID_ARG, "%s: eps lies in [1e-30, 1e30]", who);
  return GNN_OK;
}
bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
constexpr int64_t LD_MOST = (int64_t)1 << 36;
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) { return ld < cols || ld > LD_MOST; }

// The order of the matrices takes memory of the host's, which may run out.
template <class Fn>
gnn_status guarded(const char* who, Fn f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(GNN_ERR_CAPACITY, "%s: %s", who, e.what());
  }
}

// Whether four elements from a column that is a multiple of four are one access.
bool quad_rows(const void* p, int64_t ld, int elem) { return aligned_to(p, 4 * elem) && ld % 4 == 0; }

Span flat(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }
Span span(const void* p, const gnn_muon_tensor& t, int64_t ld, int elem) { return {p, t.rows, ld * elem, (int64_t)t.cols * elem}; }

// A batch of matrices, seen as whole matrices and as rows (of the distance that divides both
// strides): it lies apart from something else where either does.
struct Batch {
  Span whole, rows;
};
Batch batch(const void* p, int count, int rows, int cols, int64_t ld, int64_t stride, int elem) {
  if (count == 1) stride = 0;
  int64_t step = rows > 1 ? ld : 0;
  for (int64_t r = stride; r;) {
    const int64_t t = step % r;
    step = r, r = t;
  }
  const int64_t last = (count - 1) * stride + (rows > 1 ? (rows - 1) * ld : 0);  // the last row's place
  return {{p, count, stride * elem, (last - (count - 1) * stride + cols) * elem},
          {p, step ? last / step + 1 : 1, step * elem, (int64_t)cols * elem}};
}
bool overlap(const Batch& a, const Batch& b) {
  return gnn::overlap(a.whole, b.whole) && gnn::overlap(a.whole, b.rows) && gnn::overlap(a.rows, b.whole) &&
         gnn::overlap(a.rows, b.rows);
}
bool overlap(const Batch& a, const Span& b) { return gnn::overlap(a.whole, b) && gnn::overlap(a.rows, b); }

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_muon_workspace(const gnn_muon_tensor* tensors, int32_t n_tensors, size_t* ws_bytes) {
  GNN_REQUIRE(ws_bytes, "gnn_muon_workspace: NULL ws_bytes");
  GNN_REQUIRE(n_tensors >= 0 && (tensors || n_tensors == 0), "gnn_muon_workspace: bad tensor list");
  for (int i = 0; i < n_tensors; ++i) GNN_TRY(check_shape("gnn_muon_workspace", i, tensors[i].rows, tensors[i].cols));
  return guarded("gnn_muon_workspace", [&] {
    const auto order = order_of(n_tensors, [&](int i) { return Shape{tensors[i].rows, tensors[i].cols}; });
    return each_pass(order, nullptr, 0, ws_bytes, [&](Table& tab, Arena& ar, int k) {
      for (int i = 0; i < tab.count; ++i) {
        tab.mat[i] = Mat{};
        tab.mat[i].rows = tensors[order[k + i]].rows, tab.mat[i].cols = tensors[order[k + i]].cols;
      }
      place_pass(tab, ar);
      return GNN_OK;
    });
  });
}

extern "C" gnn_status gnn_muon_step(const gnn_muon_tensor* tensors, int32_t n_tensors, int32_t param_type,
                                    int32_t grad_type, int32_t m_type, double lr, double momentum, int32_t nesterov,
                                    double weight_decay, double grad_scale, const float* coeffs, int32_t steps,
                                    double eps, float* norms, void* ws, size_t ws_bytes, gnn_stream_t stream) {
  static const char* who = "gnn_muon_step";
  GNN_REQUIRE(n_tensors >= 0 && (tensors || n_tensors == 0), "%s: bad tensor list", who);
  GNN_REQUIRE(is_type(grad_type), "%s: unknown grad_type", who);
  if ((param_type != GNN_F32 && param_type != GNN_BF16) || (m_type != GNN_F32 && m_type != GNN_BF16))
    return fail(GNN_ERR_UNSUPPORTED, "%s: parameters and momentum are fp32 or bf16", who);
  GNN_REQUIRE(momentum >= 0 && momentum < 1, "%s: momentum lies in [0, 1)", who);
  GNN_REQUIRE(std::isfinite((float)lr) && std::isfinite((float)(1.0 - lr * weight_decay)) && std::isfinite((float)grad_scale),
              "%s: lr, 1 - lr weight_decay or grad_scale is not finite in fp32", who);
  GNN_TRY(check_steps(who, coeffs, steps, eps));
  GNN_REQUIRE(aligned_to(norms, 4), "%s: misaligned norms", who);
  const int ps = type_size(param_type), gs = type_size(grad_type), ms = type_size(m_type);
  for (int i = 0; i < n_tensors; ++i) {
    const gnn_muon_tensor& t = tensors[i];
    GNN_TRY(check_shape(who, i, t.rows, t.cols));
    if (t.rows == 0 || t.cols == 0) continue;
    GNN_REQUIRE(t.param && t.grad && t.m, "%s: matrix %d has a NULL array", who, i);
    GNN_REQUIRE(aligned_to(t.param, ps) && aligned_to(t.grad, gs) && aligned_to(t.m, ms) && aligned_to(t.copy, 2),
                "%s: matrix %d has a misaligned array", who, i);
    GNN_REQUIRE(!bad_ld(t.ldp, t.rows, t.cols) && !bad_ld(t.ldg, t.rows, t.cols) && !bad_ld(t.ldm, t.rows, t.cols) &&
                    (!t.copy || !bad_ld(t.ldc, t.rows, t.cols)), "%s: matrix %d has a stride below its columns", who, i);
    GNN_REQUIRE(std::isfinite(t.scale) && std::isfinite((float)lr * t.scale),
                "%s: matrix %d has a scale that is not finite, alone or times lr", who, i);
    const Span p = span(t.param, t, t.ldp, ps), g = span(t.grad, t, t.ldg, gs), m = span(t.m, t, t.ldm, ms),
               c = span(t.copy, t, t.ldc, 2);
    // bf16 parameters may be their own copy: a thread writes the same value twice
    const bool own = param_type == GNN_BF16 && t.copy == t.param && t.ldc == t.ldp;
    GNN_REQUIRE(!overlap(p, g) && !overlap(p, m) && !overlap(g, m) && (own || !overlap(c, p)) && !overlap(c, g) && !overlap(c, m),
                "%s: matrix %d has arrays that overlap", who, i);
  }
  size_t need = 0;
  GNN_TRY(gnn_muon_workspace(tensors, n_tensors, &need));
  if (need == 0) return GNN_OK;  // no elements
  GNN_REQUIRE(ws && ws_bytes >= need && aligned_to(ws, 256), "%s: workspace too small (%zu < %zu) or misaligned", who,
              ws_bytes, need);
  const Span taken[2] = {flat(ws, (int64_t)need), flat(norms, 4ll * n_tensors)};
  GNN_REQUIRE(!overlap(taken[0], taken[1]), "%s: norms overlaps the workspace", who);
  for (int i = 0; i < n_tensors; ++i) {
    const gnn_muon_tensor& t = tensors[i];
    for (const Span& s : taken)
      GNN_REQUIRE(!overlap(s, span(t.param, t, t.ldp, ps)) && !overlap(s, span(t.grad, t, t.ldg, gs)) &&
                      !overlap(s, span(t.m, t, t.ldm, ms)) && !overlap(s, span(t.copy, t, t.ldc, 2)),
                  "%s: matrix %d overlaps norms or the workspace", who, i);
  }
  const Hyper h{(float)momentum, (float)grad_scale, (float)(1.0 - lr * weight_decay), (float)lr, eps, nesterov != 0, 0,
                param_type, grad_type, m_type};
  return guarded(who, [&] {
    const auto order = order_of(n_tensors, [&](int i) { return Shape{tensors[i].rows, tensors[i].cols}; });
    return each_pass(order, ws, ws_bytes, &need, [&](Table& tab, Arena& ar, int k) {
      for (int i = 0; i < tab.count; ++i) {
        const gnn_muon_tensor& d = tensors[order[k + i]];
        Mat& t = tab.mat[i];
        t = Mat{d.param, d.grad, d.m, d.copy, d.ldp, d.ldg, d.ldm, d.ldc, d.scale, d.rows, d.cols};
        t.slot = order[k + i];
        t.quads = (quad_rows(d.param, d.ldp, ps) ? PARAM : 0) | (quad_rows(d.grad, d.ldg, gs) ? GRAD : 0) |
                  (quad_rows(d.m, d.ldm, ms) ? MOM : 0) | (d.copy && quad_rows(d.copy, d.ldc, 2) ? COPY : 0);
      }
      place_pass(tab, ar);
      return run_pass(ws, tab, h, coeffs, steps, norms, as_stream(stream));
    });
  });
}

extern "C" gnn_status gnn_orthogonalise_workspace(int32_t count, int32_t rows, int32_t cols, size_t* ws_bytes) {
  GNN_REQUIRE(ws_bytes, "gnn_orthogonalise_workspace: NULL ws_bytes");
  GNN_REQUIRE(count >= 0, "gnn_orthogonalise_workspace: negative count");
  GNN_TRY(check_shape("gnn_orthogonalise_workspace", 0, rows, cols));
  *ws_bytes = 0;
  if (!rows || !cols || !count) return GNN_OK;
  // the last pass may have fewer matrices than the others, and other tiles
  for (int left : {std::min(count, MAX_MATS), count % MAX_MATS}) {
    Arena ar(nullptr, 0);
    Table tab;
    tab.count = left;
    for (int i = 0; i < left; ++i) {
      tab.mat[i] = Mat{};
      tab.mat[i].rows = rows, tab.mat[i].cols = cols;
    }
    if (left) place_pass(tab, ar);
    *ws_bytes = std::max(*ws_bytes, ar.used);
  }
  return GNN_OK;
}

extern "C" gnn_status gnn_orthogonalise(const void* X, int64_t ldx, int64_t stride_x, int32_t x_type, int32_t count,
                                        int32_t rows, int32_t cols, const float* coeffs, int32_t steps, double eps,
                                        void* O, int64_t ldo, int64_t stride_o, int32_t o_type, float* norms, void* ws,
                                        size_t ws_bytes, gnn_stream_t stream) {
  static const char* who = "gnn_orthogonalise";
  GNN_REQUIRE(count >= 0, "%s: negative count", who);
  GNN_TRY(check_shape(who, 0, rows, cols));
  GNN_REQUIRE(is_type(x_type) && is_type(o_type), "%s: unknown type", who);
  GNN_TRY(check_steps(who, coeffs, steps, eps));
  GNN_REQUIRE(aligned_to(norms, 4), "%s: misaligned norms", who);
  if (!count || !rows || !cols) return GNN_OK;
  const int xs = type_size(x_type), os = type_size(o_type);
  GNN_REQUIRE(X && O && aligned_to(X, xs) && aligned_to(O, os), "%s: X or O is NULL or misaligned", who);
  GNN_REQUIRE(!bad_ld(ldx, rows, cols) && !bad_ld(ldo, rows, cols), "%s: a row stride below the columns", who);
  const int64_t x_size = (rows - 1) * ldx + cols, o_size = (rows - 1) * ldo + cols;
  GNN_REQUIRE(count == 1 || (stride_x >= x_size && stride_o >= o_size && stride_x <= LD_MOST && stride_o <= LD_MOST),
              "%s: matrices of a batch overlap", who);
  const Batch x_all = batch(X, count, rows, cols, ldx, stride_x, xs), o_all = batch(O, count, rows, cols, ldo, stride_o, os);
  // in place each element is read before anything is written
  GNN_REQUIRE((X == O && ldx == ldo && xs == os && (count == 1 || stride_x == stride_o)) ||
                  !overlap(x_all, o_all),
              "%s: O overlaps X (it may be X)", who);
  size_t need = 0;
  gnn_orthogonalise_workspace(count, rows, cols, &need);
  GNN_REQUIRE(ws && ws_bytes >= need && aligned_to(ws, 256), "%s: workspace too small (%zu < %zu) or misaligned", who,
              ws_bytes, need);
  const Span w_all = flat(ws, (int64_t)need), n_all = flat(norms, 4ll * count);
  GNN_REQUIRE(!overlap(x_all, w_all) && !overlap(o_all, w_all) && !overlap(w_all, n_all) && !overlap(x_all, n_all) &&
                  !overlap(o_all, n_all), "%s: norms or the workspace overlaps an array", who);
  const Hyper h{0.f, 1.f, 1.f, 0.f, eps, 0, 1, o_type, x_type, 0};
  return guarded(who, [&] {
    const auto order = order_of(count, [&](int) { return Shape{rows, cols}; });
    return each_pass(order, ws, ws_bytes, &need, [&](Table& tab, Arena& ar, int k) {
      for (int i = 0; i < tab.count; ++i) {
        Mat& t = tab.mat[i];
        t = Mat{static_cast<char*>(O) + (k + i) * stride_o * os, static_cast<const char*>(X) + (k + i) * stride_x * xs, nullptr,
                nullptr, ldo, ldx, 0, 0, 1.f, rows, cols};
        t.slot = k + i;
        t.quads = (quad_rows(t.param, ldo, os) ? PARAM : 0) | (quad_rows(t.grad, ldx, xs) ? GRAD : 0);
      }
      place_pass(tab, ar);
      return run_pass(ws, tab, h, coeffs, steps, norms, as_stream(stream));
    });
  });
}
