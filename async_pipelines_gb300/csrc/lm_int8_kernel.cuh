// The product of 8-bit integers with a scale for each token and each channel:
//
//   d[m][n] = float(sum_k a[m][k] * w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
//
// with sums that are exact in 32-bit integers, so that neither the order of their
// terms nor a cut of K changes a bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "watchdog.cuh"

namespace gws {
namespace i8 {

enum OutType { OUT_BF16 = 0, OUT_F16 = 1, OUT_F32 = 2 };

struct Output {
  void* d;
  int64_t ldd;
  int type;
  const float *a_scales, *w_scales, *bias;   // bias may be NULL
};

__device__ __forceinline__ void put(const Output& o, int64_t m, int64_t n, int sum, float a_scale,
                                    float w_scale, float bias) {
  const float v = fmaf(static_cast<float>(sum) * a_scale, w_scale, bias);
  const int64_t at = m * o.ldd + n;
  if (o.type == OUT_F32)
    static_cast<float*>(o.d)[at] = v;
  else if (o.type == OUT_F16)
    static_cast<__half*>(o.d)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(o.d)[at] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------ few tokens

struct DotParams {
  const int8_t *a, *w;
  int64_t lda, ldw;
  int tokens, channels, k;
  int wide;            // a's rows lie on 16-byte boundaries
  int split;           // warps that share a group of channels
  Output out;
};

constexpr int DOT_THREADS = 256, DOT_WARPS = DOT_THREADS / 32;
constexpr int DOT_ROWS = 4;   // channels of a warp

// 16 bytes of a row, or as many as there are before its end.
__device__ __forceinline__ uint4 load16(const int8_t* row, int at, int k, bool whole) {
  if (whole && at + 16 <= k) return *reinterpret_cast<const uint4*>(row + at);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i < k) w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(row[at + i])) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// TOKENS rows of a (from blockIdx.y * TOKENS on) against all of w, by the integer dot products of
// the CUDA cores. `split` warps share DOT_ROWS channels, 16 bytes of K a lane and step.
template <int TOKENS>
__global__ void __launch_bounds__(DOT_THREADS) dot_kernel(const __grid_constant__ DotParams p) {
  __shared__ int box[DOT_WARPS][DOT_ROWS * TOKENS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = warp % p.split;
  const int n0 = (blockIdx.x * (DOT_WARPS / p.split) + warp / p.split) * DOT_ROWS;
  const int m0 = blockIdx.y * TOKENS;
  int acc[DOT_ROWS][TOKENS] = {};
  for (int k = (part * 32 + lane) * 16; k < p.k; k += p.split * 512) {
    uint4 w[DOT_ROWS];
#pragma unroll
    for (int r = 0; r < DOT_ROWS; ++r)
      w[r] = n0 + r < p.channels ? load16(p.w + static_cast<int64_t>(n0 + r) * p.ldw, k, p.k, true)
                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      if (m0 + t >= p.tokens) break;
      const uint4 a = load16(p.a + static_cast<int64_t>(m0 + t) * p.lda, k, p.k, p.wide);
#pragma unroll
      for (int r = 0; r < DOT_ROWS; ++r) {
        acc[r][t] = __dp4a(static_cast<int>(w[r].x), static_cast<int>(a.x), acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(w[r].y), static_cast<int>(a.y), acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(w[r].z), static_cast<int>(a.z), acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(w[r].w), static_cast<int>(a.w), acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < DOT_ROWS; ++r)
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
      if (lane == 0) box[warp][r * TOKENS + t] = s;
    }
  __syncthreads();
  if (part != 0 || lane >= DOT_ROWS * TOKENS) return;
  const int n = n0 + lane / TOKENS, m = m0 + lane % TOKENS;
  if (n >= p.channels || m >= p.tokens) return;
  int sum = 0;
  for (int i = 0; i < p.split; ++i) sum += box[warp + i][lane];
  put(p.out, m, n, sum, p.out.a_scales[m], p.out.w_scales[n], p.out.bias ? p.out.bias[n] : 0.0f);
}

}  // namespace i8
}  // namespace gws
