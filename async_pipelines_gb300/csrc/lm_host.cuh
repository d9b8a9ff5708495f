// What the host sides of the operators of lm_norm.cu, lm_block.cu, lm_int8.cu and lm_logits.cu
// share: a matrix argument's checks, a row's team of threads and the launch.
#pragma once

#include "gemm_ws_lm.h"
#include "handle.cuh"
#include "lm_rows.cuh"

namespace {

[[maybe_unused]] int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

[[maybe_unused]] int element_size(int dtype) { return dtype == GEMM_WS_F32 ? 4 : 2; }

// A matrix argument as the checks see it.
struct Mat {
  const void* ptr;
  int64_t ld;
  int64_t size;   // bytes of an element
  bool given() const { return ptr != nullptr; }
  int64_t bytes(int64_t rows, int64_t cols) const { return ((rows - 1) * ld + cols) * size; }
  // Each row starts on a boundary of 8 elements (16 bytes at most).
  bool wide() const {
    const int64_t step = size * 8 < 16 ? size * 8 : 16;
    return reinterpret_cast<uintptr_t>(ptr) % step == 0 && (ld * size) % step == 0;
  }
};

// The output `out` may be exactly the input `in`, and else not overlap it.
[[maybe_unused]] bool clash(const Mat& out, const Mat& in, int64_t rows, int64_t cols, bool may_equal) {
  if (!out.given() || !in.given()) return false;
  if (may_equal && out.ptr == in.ptr && out.ld == in.ld && out.size == in.size) return false;
  return overlaps(out.ptr, out.bytes(rows, cols), in.ptr, in.bytes(rows, cols));
}

// The bytes that an argument takes up.
struct Span {
  const void* ptr;
  int64_t bytes;
};
[[maybe_unused]] Span span(const Mat& m, int64_t rows, int64_t cols) { return {m.ptr, m.given() ? m.bytes(rows, cols) : 0}; }

// Whether any output overlaps an input or another output.
template <int O, int I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I]) {
  for (int i = 0; i < O; ++i) {
    for (int j = 0; j < I; ++j)
      if (overlaps(out[i].ptr, out[i].bytes, in[j].ptr, in[j].bytes)) return true;
    for (int j = i + 1; j < O; ++j)
      if (overlaps(out[i].ptr, out[i].bytes, out[j].ptr, out[j].bytes)) return true;
  }
  return false;
}

[[maybe_unused]] bool bad_matrix(const Mat& m, int64_t cols) {
  return m.given() && (m.ld < cols || m.ld > kMaxElems ||
                       reinterpret_cast<uintptr_t>(m.ptr) % m.size != 0);
}

// A launch that may start while the stream's previous kernel ends; each of
// these kernels waits for that one before it touches global memory. `most`: the most
// shared memory that the kernel is ever launched with, where that is not always the same.
template <typename... P>
int launch_sized(gemm_ws* h, void (*kernel)(P...), int64_t blocks, int threads, size_t smem, size_t most,
                 cudaStream_t s, const P&... params) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (h->pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaSuccess;
  if (smem > kDefaultSmem)
    e = allow_smem(h, reinterpret_cast<const void*>(kernel), most > smem ? most : smem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, params...);
  return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
}
template <typename... P>
int launch(gemm_ws* h, void (*kernel)(P...), int64_t blocks, int threads, size_t smem, cudaStream_t s,
           const P&... params) {
  return launch_sized(h, kernel, blocks, threads, smem, smem, s, params...);
}

// The threads of a row and the groups that each holds.
struct Team {
  int threads, vpt, rows;   // rows: of a block
};

// Up to 256 columns, or 1024 of many rows, a warp holds a row and a block has
// several (no barrier). Longer rows take a block. With few rows (less than two for each SM) every
// thread takes one group, for the shortest row; with many, two, and from 2048
// columns four, so that an SM has more bytes in flight for the threads that it
// can hold (8192 x 8192 bf16: 78 us with four, 86 with two); beyond 8192 columns
// always four. On the general path, whose loads take many registers, a row longer
// than a warp's 32 groups takes a block with `any_vpt` groups a thread (8192 x 8191 bf16,
// forward: 163 us with two, 232 with one; 5000 x 4095 fp32 82 and 78; backward 8192 x 8191 bf16 314
// and 249).
[[maybe_unused]] Team pick_team(const gemm_ws* h, int64_t rows, int64_t cols, gws::Path path, int any_vpt) {
  const int64_t groups = ceil_div(cols, gws::GROUP);
  const bool any = path == gws::ANY;
  Team t;
  if (groups <= 32 || (!any && groups <= 128 && rows >= 2 * h->num_sms)) {
    t.vpt = groups <= 32 ? 1 : groups <= 64 ? 2 : 4;
    t.threads = 32;
    t.rows = rows >= 8 * h->num_sms ? 8 : rows >= 2 * h->num_sms ? 4 : 1;
    return t;
  }
  const bool many = rows >= (any ? 8 : 2) * h->num_sms;
  t.vpt = groups > 1024 ? 4 : !many ? 1 : any ? any_vpt : groups >= 256 ? 4 : 2;
  t.threads = static_cast<int>(ceil_div(ceil_div(groups, t.vpt), 32) * 32);
  t.rows = 1;
  return t;
}

}  // namespace
