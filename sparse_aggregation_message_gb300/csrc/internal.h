// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "gnnagg.h"

namespace gnn {

// Records a message for gnn_last_error() and returns `code`.
gnn_status fail(gnn_status code, const char* fmt, ...);

// Device-side flag word raised by kernels (bit 0: bad data, bit 1: timeout).
unsigned* device_flags();

inline cudaStream_t as_stream(gnn_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

#define GNN_CUDA(expr)                                                              \
  do {                                                                              \
    cudaError_t e_ = (expr);                                                        \
    if (e_ != cudaSuccess)                                                          \
      return ::gnn::fail(GNN_ERR_CUDA, "%s failed: %s (%s:%d)", #expr,              \
                         cudaGetErrorString(e_), __FILE__, __LINE__);               \
  } while (0)

// Counts library kernel launches (reported by gnn_kernel_launches).
void count_launch();

#define GNN_CHECK_LAUNCH()        \
  do {                            \
    ::gnn::count_launch();        \
    GNN_CUDA(cudaGetLastError()); \
  } while (0)

#define GNN_REQUIRE(cond, ...)                                                      \
  do {                                                                              \
    if (!(cond)) return ::gnn::fail(GNN_ERR_INVALID_ARG, __VA_ARGS__);              \
  } while (0)

// Lets a kernel take `bytes` of shared memory on the current device: once for each
// device, which `done` remembers (one for each kernel; devices past its end are
// told at every call).
using PerDevice = std::atomic<bool>[16];
template <class K>
gnn_status allow_smem(K* kernel, int bytes, PerDevice& done) {
  int dev = 0;
  GNN_CUDA(cudaGetDevice(&dev));
  if (dev >= 16 || !done[dev].load(std::memory_order_acquire)) {
    GNN_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (dev < 16) done[dev].store(true, std::memory_order_release);
  }
  return GNN_OK;
}

// Carves 256-byte aligned pieces out of a caller workspace.  With base NULL
// it only measures.
struct Arena {
  char* base;
  size_t cap;
  size_t used = 0;
  Arena(void* b, size_t c) : base(static_cast<char*>(b)), cap(c) {}
  template <class T>
  T* take(size_t count) {
    size_t bytes = (count * sizeof(T) + 255) & ~size_t(255);
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += bytes;
    return p;
  }
  void* take_bytes(size_t bytes) { return take<char>(bytes); }
  bool ok() const { return base == nullptr || used <= cap; }
};

// `rows` rows of `width` bytes, `stride` bytes apart, in device memory.
struct Span {
  const void* p;
  int64_t rows, stride, width;
};
// Whether two of them may share a byte.  Rows that lie apart in a common period of
// the strides (columns of one buffer) do not.
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  const __int128 pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;  // strides may be anything
  if (pa + (__int128)(a.rows - 1) * a.stride + a.width <= pb || pb + (__int128)(b.rows - 1) * b.stride + b.width <= pa)
    return false;
  int64_t period = a.rows > 1 ? a.stride : 0;
  for (int64_t r = b.rows > 1 ? b.stride : 0; r;) {
    const int64_t t = period % r;
    period = r, r = t;
  }
  if (period == 0) return true;
  const int64_t d = ((int64_t)(pb - pa) % period + period) % period;  // b's place in a's period
  return d < a.width || d + b.width > period;
}

inline bool is_valid_bits(int b) { return b == 1 || b == 2 || b == 4 || b == 8 || b == 32; }

constexpr int kMaxF = 1024;

}  // namespace gnn
