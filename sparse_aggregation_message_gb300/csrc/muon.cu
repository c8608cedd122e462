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
// Operands lie in the workspace as the tensor cores want them in shared memory:
// blocks of 128 rows x 64 columns, a row's 128 bytes swizzled, the hi limb's 16 KB
// before the lo limb's.
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
  char *x[2], *a, *p;
};
struct Table {
  Mat mat[MAX_MATS];
  int first[MAX_MATS + 1];  // blocks (or parts) before each matrix
  int count;
};

struct Hyper {
  float momentum, grad_scale, decay, lr;
  double eps;
  int nesterov, orth;
  int pt, gt, mt;  // types of param (output), grad (input), momentum
};

__device__ __forceinline__ float load_any(const void* p, int64_t i, int type) {
  if (type == GNN_F32) return static_cast<const float*>(p)[i];
  if (type == GNN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int type, float v) {
  if (type == GNN_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == GNN_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The momentum and the update that is orthogonalised, of one element.
__device__ __forceinline__ float update_of(const Mat& t, const Hyper& h, int64_t r, int64_t c, float* mom) {
  const float g = load_any(t.grad, r * t.ldg + c, h.gt) * h.grad_scale;
  if (h.orth) return g;
  const float m = fmaf(load_any(t.mom, r * t.ldm + c, h.mt), h.momentum, g);
  *mom = m;
  return h.nesterov ? fmaf(m, h.momentum, g) : m;
}

__device__ __forceinline__ int mat_of(const Table& tab, int k) {
  int i = 0;
  while (i + 1 < tab.count && k >= tab.first[i + 1]) ++i;
  return i;
}

// Sums of u^2 over a share of a matrix's rows.
__global__ void __launch_bounds__(THREADS) square_kernel(const __grid_constant__ Table tab, const Hyper h, double* partial) {
  __shared__ double sm[THREADS / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int part = blockIdx.x - tab.first[i];
  double sum = 0;
  float mom;
  // rows that lie end to end are one long row
  const bool flat = t.ldg == t.cols && (h.orth || t.ldm == t.cols);
  const int64_t cols = flat ? (int64_t)t.rows * t.cols : t.cols, rows = flat ? 1 : t.rows;
  const int64_t share = flat ? (cols + t.parts - 1) / t.parts : (rows + t.parts - 1) / t.parts;
  const int64_t lo = part * share, hi = min(lo + share, flat ? cols : rows);
  const int64_t r0 = flat ? 0 : lo, r1 = flat ? 1 : hi, c0 = flat ? lo : 0, c1 = flat ? hi : cols;
  for (int64_t r = r0; r < r1; ++r) {
    for (int64_t c = c0 + threadIdx.x; c < c1; c += 8 * THREADS) {
      float u[8], s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = c + k * THREADS < c1 ? update_of(t, h, r, c + k * THREADS, &mom) : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(u[k], u[k], s);
      if (s > 1e-28f && s < 1e38f) {
        sum += (double)s;
      } else {  // outside of what fp32 holds well
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += (double)u[k] * (double)u[k];
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
    partial[i * PARTS + part] = s;
  }
}

// |u|_F, in every thread of the block; `sm` is one double.
__device__ __forceinline__ double norm_of(const double* partial, int i, int parts, double* sm) {
  if (threadIdx.x < 32) {
    double s = 0;
    for (int k = threadIdx.x; k < parts; k += 32) s += partial[i * PARTS + k];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) *sm = sqrt(s);
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
__device__ __forceinline__ int chunk_at(int r, int k) { return r * 128 + ((k ^ (r & 7)) << 4); }

// u scaled into X's limbs, and the new momentum; a block of X a thread block.
__global__ void __launch_bounds__(THREADS) begin_kernel(const __grid_constant__ Table tab, const Hyper h,
                                                        const double* partial, float* norms) {
  __shared__ float tile[128][65];
  __shared__ double sm;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int block = blockIdx.x - tab.first[i], r0 = block / t.nb * 128, c0 = block % t.nb * 64;
  const double norm = norm_of(partial, i, t.parts, &sm);
  const bool good = isfinite((float)norm);
  const float inv = good ? (float)((double)UNIT / (norm + h.eps)) : 0.f;
  if (block == 0 && threadIdx.x == 0 && norms) norms[t.slot] = (float)norm;
  // in the order of the caller's rows
  const int across = t.flip ? 128 : 64;
  for (int e = threadIdx.x; e < 128 * 64; e += THREADS) {
    const int b = e % across, a = e / across;
    const int r = t.flip ? b : a, c = t.flip ? a : b;
    float u = 0.f;
    if (r0 + r < t.m && c0 + c < t.n && good) {
      const int64_t row = t.flip ? c0 + c : r0 + r, col = t.flip ? r0 + r : c0 + c;
      float mom;
      u = update_of(t, h, row, col, &mom) * inv;
      if (!h.orth) store_any(t.mom, row * t.ldm + col, h.mt, mom);
    }
    tile[r][c] = u;
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
__global__ void __launch_bounds__(THREADS) apply_kernel(const __grid_constant__ Table tab, const Hyper h,
                                                        const double* partial, int which) {
  __shared__ float tile[128][65];
  __shared__ double sm;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int block = blockIdx.x - tab.first[i], r0 = block / t.nb * 128, c0 = block % t.nb * 64;
  const double norm = norm_of(partial, i, t.parts, &sm);
  const bool good = isfinite((float)norm);
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
  const int across = t.flip ? 128 : 64;
  for (int e = threadIdx.x; e < 128 * 64; e += THREADS) {
    const int b = e % across, a = e / across;
    const int r = t.flip ? b : a, c = t.flip ? a : b;
    if (r0 + r >= t.m || c0 + c >= t.n) continue;
    const int64_t row = t.flip ? c0 + c : r0 + r, col = t.flip ? r0 + r : c0 + c;
    const float o = good ? tile[r][c] : __int_as_float(0x7fc00000);
    if (h.orth) {
      store_any(t.param, row * t.ldp + col, h.pt, o);
    } else {
      const float p = fmaf(-h.lr * t.scale, o, load_any(t.param, row * t.ldp + col, h.pt) * h.decay);
      store_any(t.param, row * t.ldp + col, h.pt, p);
      if (t.copy) reinterpret_cast<__nv_bfloat16*>(t.copy)[row * t.ldc + col] = __float2bfloat16_rn(p);
    }
  }
}

// ------------------------------------------------------------------ products
enum Phase { GRAM, POLY, NEXT };  // A = X X', P = a I + b A + c A A, X <- P X

__device__ __forceinline__ float value_at(const char* s, int nb, int r, int c) {
  const char* b = s + ((int64_t)(r >> 7) * nb + (c >> 6)) * BLOCK + chunk_at(r & 127, (c & 63) >> 3) + (c & 7) * 2;
  return __half2float(*reinterpret_cast<const __half*>(b)) + __half2float(*reinterpret_cast<const __half*>(b + LIMB));
}

// The plain form of a product: a thread block a block of the output, 64 of k at a time.
__global__ void __launch_bounds__(THREADS) product_kernel(const __grid_constant__ Table tab, Phase phase, int which, float ca,
                                                          float cb, float cc) {
  __shared__ float left[128][17], right[16][65];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int i = mat_of(tab, blockIdx.x);
  const Mat& t = tab.mat[i];
  const int out_nb = phase == NEXT ? t.nb : 2 * t.mb, block = blockIdx.x - tab.first[i];
  const int r0 = block / out_nb * 128, c0 = block % out_nb * 64, sq = 2 * t.mb;
  const char* x = t.x[which];
  const int K = phase == GRAM ? t.nb * 64 : t.mb * 128;
  float acc[32] = {};
  const int tc = threadIdx.x & 63, tr = threadIdx.x >> 6;
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int e = threadIdx.x; e < 128 * 16; e += THREADS) {
      const int r = e >> 4, k = e & 15;
      left[r][k] = phase == GRAM ? value_at(x, t.nb, r0 + r, k0 + k) : value_at(phase == POLY ? t.a : t.p, sq, r0 + r, k0 + k);
    }
    for (int e = threadIdx.x; e < 64 * 16; e += THREADS) {
      const int c = e >> 4, k = e & 15;
      right[k][c] = phase == GRAM ? value_at(x, t.nb, c0 + c, k0 + k) : phase == POLY ? value_at(t.a, sq, c0 + c, k0 + k)
                                                                                       : value_at(x, t.nb, k0 + k, c0 + c);
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = fmaf(left[tr + 4 * j][k], right[k][tc], acc[j]);
    __syncthreads();
  }
  char* out = phase == GRAM ? t.a : phase == POLY ? t.p : t.x[which ^ 1];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int r = r0 + tr + 4 * j, c = c0 + tc;
    float v = acc[j] * (1.f / UNIT);
    if (phase == POLY) v = cc * v + cb * value_at(t.a, sq, r, c) + (r == c ? ca * UNIT : 0.f);
    char* b = out + (int64_t)block * BLOCK + chunk_at(r & 127, (c & 63) >> 3) + (c & 7) * 2;
    const __half hi = __float2half_rn(v);
    *reinterpret_cast<__half*>(b) = hi;
    *reinterpret_cast<__half*>(b + LIMB) = __float2half_rn(v - __half2float(hi));
  }
}

// ---------------------------------------------------------------- host side
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

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

// Places of X's two copies, A and P in a pass's workspace.
void place(Mat& t, Arena& ar) {
  t.flip = t.rows > t.cols;
  t.m = std::min(t.rows, t.cols), t.n = std::max(t.rows, t.cols);
  t.mb = (t.m + 127) / 128, t.nb = (int)up((t.n + 63) / 64, 2);
  for (int k = 0; k < 2; ++k) t.x[k] = ar.take<char>((size_t)t.mb * t.nb * BLOCK);
  t.a = ar.take<char>((size_t)t.mb * 2 * t.mb * BLOCK);
  t.p = ar.take<char>((size_t)t.mb * 2 * t.mb * BLOCK);
  t.parts = (int)std::min<int64_t>(PARTS, ((int64_t)t.rows * t.cols + 16 * THREADS - 1) / (16 * THREADS));
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
    double* partial = ar.take<double>((size_t)MAX_MATS * PARTS);
    Table tab;
    tab.count = (int)std::min<size_t>(MAX_MATS, order.size() - k);
    GNN_TRY(fill(tab, ar, partial, (int)k));
    *need = std::max(*need, ar.used);
  }
  return GNN_OK;
}

gnn_status run_pass(Table& tab, const Hyper& h, const float* coeffs, int steps, double* partial, float* norms,
                    cudaStream_t st) {
  auto blocks = [&](auto&& of) {
    tab.first[0] = 0;
    for (int i = 0; i < tab.count; ++i) tab.first[i + 1] = tab.first[i] + of(tab.mat[i]);
    return tab.first[tab.count];
  };
  int grid = blocks([](const Mat& t) { return t.parts; });
  GNN_TRY(launch(grid, THREADS, 0, st, square_kernel, tab, h, partial));
  grid = blocks([](const Mat& t) { return t.mb * t.nb; });
  GNN_TRY(launch(grid, THREADS, 0, st, begin_kernel, tab, h, (const double*)partial, norms));
  for (int s = 0; s < steps; ++s) {
    const float* c = coeffs + 3 * s;
    grid = blocks([](const Mat& t) { return t.mb * 2 * t.mb; });
    GNN_TRY(launch(grid, THREADS, 0, st, product_kernel, tab, GRAM, s & 1, c[0], c[1], c[2]));
    GNN_TRY(launch(grid, THREADS, 0, st, product_kernel, tab, POLY, s & 1, c[0], c[1], c[2]));
    grid = blocks([](const Mat& t) { return t.mb * t.nb; });
    GNN_TRY(launch(grid, THREADS, 0, st, product_kernel, tab, NEXT, s & 1, c[0], c[1], c[2]));
  }
  grid = blocks([](const Mat& t) { return t.mb * t.nb; });
  return launch(grid, THREADS, 0, st, apply_kernel, tab, h, (const double*)partial, steps & 1);
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
  if (!(eps > 0) || !std::isfinite(eps)) return fail(GNN_ERR_INVALID_ARG, "%s: eps must be positive", who);
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

Span span(const void* p, const gnn_muon_tensor& t, int64_t ld, int elem) { return {p, t.rows, ld * elem, (int64_t)t.cols * elem}; }

}  // namespace

}  // namespace gnn

using namespace gnn;

extern "C" gnn_status gnn_muon_workspace(const gnn_muon_tensor* tensors, int32_t n_tensors, size_t* ws_bytes) {
  GNN_REQUIRE(ws_bytes, "gnn_muon_workspace: NULL ws_bytes");
  GNN_REQUIRE(n_tensors >= 0 && (tensors || n_tensors == 0), "gnn_muon_workspace: bad tensor list");
  for (int i = 0; i < n_tensors; ++i) GNN_TRY(check_shape("gnn_muon_workspace", i, tensors[i].rows, tensors[i].cols));
  return guarded("gnn_muon_workspace", [&] {
    const auto order = order_of(n_tensors, [&](int i) { return Shape{tensors[i].rows, tensors[i].cols}; });
    return each_pass(order, nullptr, 0, ws_bytes, [&](Table& tab, Arena& ar, double*, int k) {
      for (int i = 0; i < tab.count; ++i) {
        Mat t{};
        t.rows = tensors[order[k + i]].rows, t.cols = tensors[order[k + i]].cols;
        place(t, ar);
      }
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
  GNN_REQUIRE(std::isfinite(lr) && std::isfinite(weight_decay) && std::isfinite(grad_scale),
              "%s: lr, weight_decay or grad_scale is not finite", who);
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
    GNN_REQUIRE(std::isfinite(t.scale), "%s: matrix %d has a scale that is not finite", who, i);
    const Span p = span(t.param, t, t.ldp, ps), g = span(t.grad, t, t.ldg, gs), m = span(t.m, t, t.ldm, ms),
               c = span(t.copy, t, t.ldc, 2);
    GNN_REQUIRE(!overlap(p, g) && !overlap(p, m) && !overlap(g, m) && !overlap(c, p) && !overlap(c, g) && !overlap(c, m),
                "%s: matrix %d has arrays that overlap", who, i);
  }
  size_t need = 0;
  GNN_TRY(gnn_muon_workspace(tensors, n_tensors, &need));
  if (need == 0) return GNN_OK;  // no elements
  GNN_REQUIRE(ws && ws_bytes >= need && aligned_to(ws, 256), "%s: workspace too small (%zu < %zu) or misaligned", who,
              ws_bytes, need);
  const Hyper h{(float)momentum, (float)grad_scale, (float)(1.0 - lr * weight_decay), (float)lr, eps, nesterov != 0, 0,
                param_type, grad_type, m_type};
  return guarded(who, [&] {
    const auto order = order_of(n_tensors, [&](int i) { return Shape{tensors[i].rows, tensors[i].cols}; });
    return each_pass(order, ws, ws_bytes, &need, [&](Table& tab, Arena& ar, double* partial, int k) {
      for (int i = 0; i < tab.count; ++i) {
        const gnn_muon_tensor& d = tensors[order[k + i]];
        Mat& t = tab.mat[i];
        t = Mat{d.param, d.grad, d.m, d.copy, d.ldp, d.ldg, d.ldm, d.ldc, d.scale, d.rows, d.cols};
        t.slot = order[k + i];
        place(t, ar);
      }
      return run_pass(tab, h, coeffs, steps, partial, norms, as_stream(stream));
    });
  });
}

extern "C" gnn_status gnn_orthogonalise_workspace(int32_t count, int32_t rows, int32_t cols, size_t* ws_bytes) {
  GNN_REQUIRE(ws_bytes, "gnn_orthogonalise_workspace: NULL ws_bytes");
  GNN_REQUIRE(count >= 0, "gnn_orthogonalise_workspace: negative count");
  GNN_TRY(check_shape("gnn_orthogonalise_workspace", 0, rows, cols));
  *ws_bytes = 0;
  if (!rows || !cols || !count) return GNN_OK;
  Arena ar(nullptr, 0);
  ar.take<double>((size_t)MAX_MATS * PARTS);
  for (int i = 0; i < std::min(count, MAX_MATS); ++i) {
    Mat t{};
    t.rows = rows, t.cols = cols;
    place(t, ar);
  }
  *ws_bytes = ar.used;
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
  // in place each element is read before anything is written
  GNN_REQUIRE((X == O && ldx == ldo && xs == os && (count == 1 || stride_x == stride_o)) ||
                  !overlap(Span{X, count, stride_x * xs, x_size * xs}, Span{O, count, stride_o * os, o_size * os}),
              "%s: O overlaps X (it may be X)", who);
  size_t need = 0;
  gnn_orthogonalise_workspace(count, rows, cols, &need);
  GNN_REQUIRE(ws && ws_bytes >= need && aligned_to(ws, 256), "%s: workspace too small (%zu < %zu) or misaligned", who,
              ws_bytes, need);
  const Hyper h{0.f, 1.f, 1.f, 0.f, eps, 0, 1, o_type, x_type, 0};
  return guarded(who, [&] {
    const auto order = order_of(count, [&](int) { return Shape{rows, cols}; });
    return each_pass(order, ws, ws_bytes, &need, [&](Table& tab, Arena& ar, double* partial, int k) {
      for (int i = 0; i < tab.count; ++i) {
        Mat& t = tab.mat[i];
        t = Mat{static_cast<char*>(O) + (k + i) * stride_o * os, static_cast<const char*>(X) + (k + i) * stride_x * xs, nullptr,
                nullptr, ldo, ldx, 0, 0, 1.f, rows, cols};
        t.slot = k + i;
        place(t, ar);
      }
      return run_pass(tab, h, coeffs, steps, partial, norms, as_stream(stream));
    });
  });
}
