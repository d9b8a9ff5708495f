// The library handle and the host-side helpers that every entry point's
// translation unit shares.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "gemm_ws.h"

// A tensor map the handle encoded before, and what it describes.
struct MapCacheEntry {
  const void* ptr;
  uint64_t d0, d1, d2;
  uint32_t b0, b1;
  int swizzle, promotion;
  bool valid;
  CUtensorMap map;
};
constexpr int kMapCache = 16;
// The operators' kernels that take more shared memory than a kernel has by default.
constexpr int kLargeKernels = 96;

struct gemm_ws {
  int device;
  int num_sms;
  int cta_group;                  // 0: chosen per problem (default); 1: single-CTA tiles; 2: CTA pairs
  int pdl;                        // launch with programmatic stream serialisation
  int group_m;                    // raster group: m-tiles walked per n step
  int max_pair_clusters;          // co-resident 2-CTA clusters of the pair kernel
  int stream_k;                   // 0 off, 1 where the cost model gains (default), 2 always
  int sk_inline;                  // two-piece tiles: fix-up inside the GEMM (default 1)
  int k_snake;                    // every other unit of a cluster walks K backwards
  uint32_t* work;                 // [0] stream-out counter, [1] status, [2] done count, [3] the
                                  // cross entropy's done count, then the in-kernel fix-up words
                                  // (work_words)
  float* partial;                 // stream-K partials: num_sms parts of 128 x 256 fp32
  int last_cuda_error;
  unsigned long long timeout_ns;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  MapCacheEntry map_cache[kMapCache];   // recently encoded tensor maps (host memory)
  int map_cache_next;
  const void* large[kLargeKernels];     // kernels allowed the shared memory they ask for, in
                                        // the order of their first use (see allow_smem)
#ifdef GEMM_WS_DEBUG
  int debug_fault;
  unsigned long long* trace;
  unsigned long long* phases;
#endif
};

namespace {

// The work area's counter [0], status [1], consumers done [2], blocks done [3]; the words for
// arrivals follow.
[[maybe_unused]] constexpr int kWorkWords = 4;
constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 40;
// Dynamic shared memory that a kernel has unasked: of 48 KB, which what it declares itself counts towards, so
// that 12280 fp32 columns and the 512 bytes of a sum's boxes would be too much.
[[maybe_unused]] constexpr size_t kDefaultSmem = 40 * 1024;

int cuda_fail(gemm_ws* h, cudaError_t e) {
  if (h) h->last_cuda_error = static_cast<int>(e);
  return GEMM_WS_ERR_CUDA;
}

// Allows `kernel` `bytes` of dynamic shared memory before its first launch by the handle
// (whose device is current). Not at the handle's creation: that would load every such
// kernel, some fifty of them, for callers that use none (21 ms instead of 0.6 with 22 of them).
[[maybe_unused]] cudaError_t allow_smem(gemm_ws* h, const void* kernel, size_t bytes) {
  for (const void*& k : h->large) {
    if (k == kernel) return cudaSuccess;
    if (k) continue;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes));
    if (e == cudaSuccess) k = kernel;
    return e;
  }
  return cudaErrorInvalidValue;   // more such kernels than kLargeKernels
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
    if (prev_ != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev_) cudaSetDevice(prev_);
  }

 private:
  int prev_ = -1;
};

}  // namespace
