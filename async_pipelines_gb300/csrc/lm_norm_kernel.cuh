// Dropout, and the root-mean-square norm with the residual's addition,
// forward and backward: kernels that read each value once and are bound by
// memory.
//
//   dropout        d(x) = keep * x / (1 - p)
//   forward        h = residual + d(x);  r = 1 / sqrt(mean(h^2) + eps);
//                  y = h * r * weight  (in the type of x, or in e4m3 with a
//                  scale for each row or each 128 columns)
//   backward       a = dy * weight;  n = h * r;
//                  dres = dh + r * (a - n * mean(a * n));
//                  dx = keep * dres / (1 - p);  dweight = sum over rows dy * n
//
// A row belongs to a team of threads that hold it in registers, 8 columns (a
// "group", 16 bytes of a 16-bit type) at a time: group k * team + t is thread
// t's k-th, so that a warp's accesses are contiguous. The row's statistics
// are reduced over the team in 32 bits and the row is never read again.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gws {

constexpr int GROUP = 8;                 // columns of a group; Philox words of a counter
constexpr int QUANT_GROUP = 128;         // columns of one scale (Q == 2)
constexpr int MAX_VPT = 4;               // groups a thread holds
constexpr float E4M3_MAX = 448.0f;       // largest finite e4m3

// ------------------------------------------------------------ generator

// Philox4x32 with ten rounds (J. Salmon et al., "Parallel random numbers: as
// easy as 1, 2, 3", 2011): the key is the seed, the counter's low 64 bits are
// given and its high ones 0. The 128 bits serve the 8 columns of a group, 16
// bits each, lowest first: half the rounds' cost of 32 bits a column (which
// would take more issue slots than dropout's 4 bytes of traffic a column
// leave), for a p that is a multiple of 2^-16.
__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
  uint32_t c2 = 0, c3 = 0;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t m0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t m1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(m1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(m1);
    c2 = static_cast<uint32_t>(m0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(m0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// What a launch's dropout is: a column is dropped where its word is below
// `below` (0: no dropout; 65536: everything is dropped), else scaled.
struct Dropout {
  const uint64_t* rng;   // device: seed, first counter
  uint32_t below;
  float scale;           // 65536 / (65536 - below)
};

// v = d(v) for the group at `counter`. A dropped value is 0 whatever it was.
__device__ __forceinline__ void drop_group(const Dropout& d, uint64_t seed, uint64_t counter,
                                           float (&v)[GROUP]) {
  const uint4 w = philox(counter, seed);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (words[i] & 0xFFFFu) >= d.below ? v[2 * i] * d.scale : 0.0f;
    v[2 * i + 1] = (words[i] >> 16) >= d.below ? v[2 * i + 1] * d.scale : 0.0f;
  }
}

// ------------------------------------------------------------ groups

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

// A group as it lies in memory.
template <typename T>
struct alignas(16) Raw {
  uint4 w[sizeof(T) * GROUP / 16];
};

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& raw, float (&v)[GROUP]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < GROUP; ++i) v[i] = to_float(e[i]);
}

template <typename T>
__device__ __forceinline__ Raw<T> pack(const float (&v)[GROUP]) {
  Raw<T> raw;
  T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
  for (int i = 0; i < GROUP; ++i) e[i] = from_float<T>(v[i]);
  return raw;
}

// Columns [c, c + 8) of a row whose end is `cols`; past it zeros. `wide`: the
// row starts on a 16-byte boundary, so whole groups move in 16-byte pieces.
template <typename T>
__device__ __forceinline__ Raw<T> load_group(const T* row, int c, int cols, bool wide) {
  Raw<T> raw;
  if (wide && c + GROUP <= cols) {
    const uint4* src = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) * GROUP / 16); ++i) raw.w[i] = src[i];
  } else {
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) e[i] = c + i < cols ? row[c + i] : from_float<T>(0.0f);
  }
  return raw;
}

template <typename T>
__device__ __forceinline__ void store_group(T* row, int c, int cols, bool wide, const Raw<T>& raw) {
  if (wide && c + GROUP <= cols) {
    uint4* dst = reinterpret_cast<uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) * GROUP / 16); ++i) dst[i] = raw.w[i];
  } else {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
      if (c + i < cols) row[c + i] = e[i];
  }
}

// ------------------------------------------------------------ reductions

// The larger, or NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct SumMax {
  float sum, max;
};

// The sum (and the largest) over a team: a warp, or a whole block of `warps`
// warps through `box` (one slot a warp; a block's next use of the same box
// needs a barrier in between). Each thread adds the warps' sums in the same
// order, so the result does not depend on timing.
template <bool MAX>
__device__ __forceinline__ SumMax reduce_team(SumMax v, int warps, SumMax* box) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    if (MAX) v.max = max_nan(v.max, __shfl_xor_sync(0xffffffffu, v.max, o));
  }
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
  __syncthreads();
  SumMax all = box[0];
  for (int w = 1; w < warps; ++w) {
    all.sum += box[w].sum;
    if (MAX) all.max = max_nan(all.max, box[w].max);
  }
  return all;
}

// ------------------------------------------------------------ forward

struct NormParams {
  const void *x, *residual, *weight;   // residual may be NULL
  void *h, *y;                         // h may be NULL
  float *rstd, *scales;                // may be NULL (scales iff Q == 0)
  int64_t ldx, ldr, ldh, ldy;          // elements between rows
  int64_t rows;
  int cols;
  int team;                            // threads a row: 32 (blockDim / 32 rows a block), or all
  float eps;
  int wide;                            // rows of x, residual, h, y and weight allow wide accesses
  Dropout drop;
};

// One row a team. Q: 0 y has the type of x; 1 e4m3 with one scale a row; 2
// e4m3 with a scale for each 128 columns.
template <typename T, int VPT, int Q>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ SumMax box[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const bool wide = p.wide;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  const T* weight = static_cast<const T*>(p.weight);
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;

  Raw<T> xr[VPT], rr[VPT], wr[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      xr[k] = load_group(x, g * GROUP, cols, wide);
      if (res) rr[k] = load_group(res, g * GROUP, cols, wide);
      wr[k] = load_group(weight, g * GROUP, cols, wide);
    }
  }
  uint64_t seed = 0, first = 0;
  if (p.drop.below) {
    seed = p.drop.rng[0];
    first = p.drop.rng[1] + static_cast<uint64_t>(row) * groups;
  }
  float v[VPT][GROUP];
  SumMax s = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      unpack(xr[k], v[k]);
      if (p.drop.below) drop_group(p.drop, seed, first + g, v[k]);
      float w[GROUP];
      unpack(wr[k], w);
      if (res) {
        float r[GROUP];
        unpack(rr[k], r);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) v[k][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        s.sum = fmaf(v[k][i], v[k][i], s.sum);
        if (Q == 1) s.max = max_nan(s.max, fabsf(v[k][i] * w[i]));
      }
      if (p.h) store_group(static_cast<T*>(p.h) + row * p.ldh, g * GROUP, cols, wide, pack<T>(v[k]));
    }
  }
  s = reduce_team<Q == 1>(s, team / 32, box);
  // r of the unrounded h, in 32 bits
  const float r = rsqrtf(s.sum / static_cast<float>(cols) + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = r;
  // Q == 1: max |y| = r * max |h * weight|, so one reduction serves both
  float scale = 0.0f;
  if (Q == 1) {
    scale = max_nan(s.max * r / E4M3_MAX, 1.17549435e-38f);
    if (t == 0) p.scales[row] = scale;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    float w[GROUP];
    if (g < groups) {
      unpack(wr[k], w);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[k][i] = v[k][i] * r * w[i];
    }
    if (Q == 0) {
      if (g < groups)
        store_group(static_cast<T*>(p.y) + row * p.ldy, g * GROUP, cols, wide, pack<T>(v[k]));
    } else {
      if (Q == 2) {
        // the 16 groups of 128 columns sit on 16 neighbouring lanes
        float m = 0.0f;
        if (g < groups) {
#pragma unroll
          for (int i = 0; i < GROUP; ++i) m = max_nan(m, fabsf(v[k][i]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        scale = max_nan(m / E4M3_MAX, 1.17549435e-38f);
        if ((t & 15) == 0 && g < groups)
          p.scales[row * ((cols + QUANT_GROUP - 1) / QUANT_GROUP) + g / 16] = scale;
      }
      if (g < groups) {
        const float inv = 1.0f / scale;
        uint32_t out[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(v[k][4 * i] * inv, v[k][4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(
              make_float2(v[k][4 * i + 2] * inv, v[k][4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          out[i] = lo | (hi << 16);
        }
        uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.ldy + g * GROUP;
        if (wide && (g + 1) * GROUP <= cols) {
          *reinterpret_cast<uint2*>(y) = make_uint2(out[0], out[1]);
        } else {
#pragma unroll
          for (int i = 0; i < GROUP; ++i)
            if (g * GROUP + i < cols) y[i] = static_cast<uint8_t>(out[i / 4] >> (8 * (i % 4)));
        }
      }
    }
  }
}

// ------------------------------------------------------------ backward

struct NormGradParams {
  const void *dy, *dh, *h, *weight;    // dh may be NULL
  const float* rstd;
  void *dx, *dres;                     // dres may be NULL
  float* partial;                      // dweight partials, one row of `cols` a block; NULL: no dweight
  int64_t lddy, lddh, ldh, lddx, lddres;
  int64_t rows;
  int cols;
  int team;
  int wide;
  Dropout drop;
};

// Persistent: a team takes rows blockIdx * teams + team, + all teams of the
// grid, and keeps its columns' share of dweight in registers; a block leaves
// one partial row, and dweight_kernel adds those in block order. So dweight
// has the same bits on every run, whatever the timing.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) add_rms_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ SumMax box[2][32];
  extern __shared__ float share[];   // where a team is a warp: the block's sum of dweight
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, teams = blockDim.x / team;
  const bool wide = p.wide;
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  const T* weight = static_cast<const T*>(p.weight);
  uint64_t seed = 0, first = 0;
  if (p.drop.below) {
    seed = p.drop.rng[0];
    first = p.drop.rng[1];
  }
  float acc[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP; ++i) acc[k][i] = 0.0f;

  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * teams + threadIdx.x / team; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * teams, turn ^= 1) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* h = static_cast<const T*>(p.h) + row * p.ldh;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + row * p.lddh : nullptr;
    Raw<T> yr[VPT], hr[VPT], dr[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        yr[k] = load_group(dy, g * GROUP, cols, wide);
        hr[k] = load_group(h, g * GROUP, cols, wide);
        if (dh) dr[k] = load_group(dh, g * GROUP, cols, wide);
      }
    }
    const float r = p.rstd[row];
    SumMax s = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], n[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], n);
        unpack(load_group(weight, g * GROUP, cols, wide), w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          const float ni = n[i] * r;
          acc[k][i] = fmaf(a[i], ni, acc[k][i]);
          s.sum = fmaf(a[i] * w[i], ni, s.sum);
        }
      }
    }
    const float c = reduce_team<false>(s, team / 32, box[turn]).sum / static_cast<float>(cols);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], n[GROUP], w[GROUP], d[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], n);
        unpack(load_group(weight, g * GROUP, cols, wide), w);
        if (dh) {
          unpack(dr[k], d);
        } else {
#pragma unroll
          for (int i = 0; i < GROUP; ++i) d[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) d[i] = fmaf(r, a[i] * w[i] - n[i] * r * c, d[i]);
        if (p.dres)
          store_group(static_cast<T*>(p.dres) + row * p.lddres, g * GROUP, cols, wide, pack<T>(d));
        if (p.drop.below)
          drop_group(p.drop, seed, first + static_cast<uint64_t>(row) * groups + g, d);
        store_group(static_cast<T*>(p.dx) + row * p.lddx, g * GROUP, cols, wide, pack<T>(d));
      }
    }
  }
  if (!p.partial) return;
  float* out = p.partial + static_cast<size_t>(blockIdx.x) * cols;
  if (teams == 1) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * team + t) * GROUP;
#pragma unroll
      for (int i = 0; i < GROUP; ++i)
        if (c + i < cols) out[c + i] = acc[k][i];
    }
    return;
  }
  for (int c = threadIdx.x; c < cols; c += blockDim.x) share[c] = 0.0f;
  for (int w = 0; w < teams; ++w) {   // the teams in turn: a fixed order
    __syncthreads();
    if (static_cast<int>(threadIdx.x) / team == w) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int c = (k * team + t) * GROUP;
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
          if (c + i < cols) share[c + i] += acc[k][i];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += blockDim.x) out[c] = share[c];
}

constexpr int DW_COLS = 32, DW_LANES = 8;   // a block's columns, and partial rows in flight

struct DweightParams {
  const float* partial;
  int blocks, cols;
  void* dweight;
};

// dweight[c] = the sum of the blocks' partial rows, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(DW_COLS* DW_LANES)
    dweight_kernel(const __grid_constant__ DweightParams p) {
  __shared__ float box[DW_LANES][DW_COLS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int x = threadIdx.x % DW_COLS, lane = threadIdx.x / DW_COLS;
  const int c = blockIdx.x * DW_COLS + x;
  float s = 0.0f;
  if (c < p.cols) {
#pragma unroll 8
    for (int b = lane; b < p.blocks; b += DW_LANES)
      s += p.partial[static_cast<size_t>(b) * p.cols + c];
  }
  box[lane][x] = s;
  __syncthreads();
  if (lane == 0 && c < p.cols) {
    for (int l = 1; l < DW_LANES; ++l) s += box[l][x];
    static_cast<T*>(p.dweight)[c] = from_float<T>(s);
  }
}

// ------------------------------------------------------------ dropout alone

struct DropoutParams {
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int64_t groups;      // of all rows
  int row_groups;      // of one row
  int cols;
  int wide;
  Dropout drop;
};

constexpr int DROP_THREADS = 256, DROP_VPT = 4;

template <typename T>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t seed = p.drop.below ? p.drop.rng[0] : 0, first = p.drop.below ? p.drop.rng[1] : 0;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (DROP_THREADS * DROP_VPT) + threadIdx.x;
  Raw<T> raw[DROP_VPT];
  int64_t row[DROP_VPT];
  int col[DROP_VPT];
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) {
      row[k] = g / p.row_groups;
      col[k] = static_cast<int>(g - row[k] * p.row_groups) * GROUP;
      raw[k] = load_group(static_cast<const T*>(p.x) + row[k] * p.ldx, col[k], p.cols, p.wide);
    }
  }
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) {
      float v[GROUP];
      unpack(raw[k], v);
      if (p.drop.below) drop_group(p.drop, seed, first + g, v);
      store_group(static_cast<T*>(p.y) + row[k] * p.ldy, col[k], p.cols, p.wide, pack<T>(v));
    }
  }
}

}  // namespace gws
