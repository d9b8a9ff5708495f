// The norms around a block, with its gate and the scaled residual, forward and
// backward, and the quantisation of rows to 8-bit integers: kernels that read each
// value once and are bound by memory.
//
//   forward        n = x * r1,  r1 = 1 / sqrt(mean(x^2) + eps);  b = post * n
//                  h = alpha * residual + gate * b
//                  y = weight * h * r2,  r2 = 1 / sqrt(mean(h^2) + eps)
//   backward       a = dy * weight;  m = h * r2
//                  g = dh + r2 * (a - m * mean(a * m))
//                  dresidual = alpha * g;  dweight = sum over rows dy * m
//                  dgate = g * b;  e = gate * g;  dpost = sum over rows e * n
//                  dx = r1 * (e * post - n * mean(e * post * n))
//
// Without the norm after the block n is x and r1 is 1. A gate for each channel needs
// no sum of its own: with S = sum over rows g * n, dgate = post * S and dpost = gate * S.
#pragma once

#include <stdint.h>

#include "lm_rows.cuh"

namespace gws {

enum Quant { Q_SAME = 0, Q_E4M3_ROW = 1, Q_E4M3_GROUP = 2, Q_INT8_ROW = 3 };
constexpr float INT8_MAX_F = 127.0f;

// The scale of a row whose largest magnitude is `top`, to integers up to 127. What has no
// largest magnitude (an infinity or a NaN) has the scale NaN, which then marks all
// that is computed from the row.
__device__ __forceinline__ float int8_scale(float top) {
  const float s = max_nan(__fdiv_rn(top, INT8_MAX_F), 1.17549435e-38f);
  return s < INFINITY ? s : __int_as_float(0x7FC00000);
}

// ------------------------------------------------------------ forward

struct BlockParams {
  const void *x, *residual, *gate, *post, *weight;   // gate and post may be NULL
  void *h, *y;                                       // h may be NULL
  float *post_rstd, *rstd, *scales;                  // may be NULL (scales iff quant == Q_SAME)
  int64_t ldx, ldr, ldg, ldh, ldy;                   // elements between rows; ldg 0: a gate for each channel
  int64_t rows;
  int cols;
  int team;                                          // threads a row: 32, or all
  int quant;                                         // Quant
  float alpha, eps;
};

// The scale of a row in 8 bits whose largest |h * weight| is `top`.
__device__ __forceinline__ float row_scale(int quant, float top, float r2) {
  return quant == Q_INT8_ROW ? int8_scale(top * r2) : max_nan(top * r2 / E4M3_MAX, 1.17549435e-38f);
}

// The scale of the 128 columns that a thread's group belongs to; their 16 groups sit on 16
// neighbouring lanes. The first of them writes it down.
__device__ __forceinline__ float group_scale(const float (&v)[GROUP], float* scales, int g, int groups) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < GROUP; ++i) m = max_nan(m, fabsf(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float scale = max_nan(m / E4M3_MAX, 1.17549435e-38f);
  if (g % 16 == 0 && g < groups) scales[g / 16] = scale;
  return scale;
}

// h of a group, from x, the gate and the residual in 32 bits.
struct Join {
  bool post, gate;
  float alpha, r1;
  __device__ __forceinline__ void operator()(float (&v)[GROUP], const float (&post_w)[GROUP],
                                             const float (&gates)[GROUP], const float (&res)[GROUP]) const {
    if (post) {
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[i] = v[i] * r1 * post_w[i];
    }
    if (gate) {
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[i] *= gates[i];
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i) v[i] = fmaf(alpha, res[i], v[i]);
  }
};

// Rows that lie FAST: a team holds one in registers, so that each value moves once (8192 x 8192 bf16:
// 537 MB in 84 us, 6.4 TB/s). BYTES: y in 8 bits. LATE: many rows, and no gate for each
// value; the vectors are then loaded, from L2 or L1, when they are needed, as their registers would cost
// the SM a row (8192 x 8192 bf16 84 us, 96 with all loads first; 600 x 4096 5.3 and 4.0).
template <typename T, int VPT, int MOST, bool BYTES, bool LATE>
__global__ void __launch_bounds__(MOST, LATE && MOST == 256 ? 3 : 1)
    block_norm_kernel(const __grid_constant__ BlockParams p) {
  __shared__ SumMax box[2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const int cols = p.cols, groups = cols / GROUP;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  auto group = [&](const void* m, int64_t ld, int g) {
    return reinterpret_cast<const Raw<T>*>(static_cast<const T*>(m) + row * ld)[g];
  };
  Raw<T> xr[VPT] = {}, rr[VPT] = {}, gr[VPT] = {}, pr[VPT] = {};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      xr[k] = group(p.x, p.ldx, g);
      rr[k] = group(p.residual, p.ldr, g);
      if (!LATE && p.gate) gr[k] = group(p.gate, p.ldg, g);
      if (!LATE && p.post) pr[k] = group(p.post, 0, g);
    }
  }
  float r1 = 1.0f;
  if (p.post) {
    SumMax s = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float v[GROUP];
      unpack(xr[k], v);   // zeros past the row's end
#pragma unroll
      for (int i = 0; i < GROUP; ++i) s.sum = fmaf(v[i], v[i], s.sum);
    }
    s = reduce_team<false>(s, team / 32, box[0]);
    r1 = rsqrtf(s.sum * inv_cols + p.eps);
    if (p.post_rstd && t == 0) p.post_rstd[row] = r1;
  }
  const Join join{p.post != nullptr, p.gate != nullptr, p.alpha, r1};
  Raw<T> wr[VPT] = {};
  float v[VPT][GROUP];
  SumMax s = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    float f[GROUP], post[GROUP], gates[GROUP];
    unpack(xr[k], v[k]);
    unpack(rr[k], f);
    if (LATE && g < groups) {
      if (p.post) pr[k] = group(p.post, 0, g);
      if (p.gate) gr[k] = group(p.gate, 0, g);
    }
    unpack(pr[k], post);
    unpack(gr[k], gates);
    join(v[k], post, gates, f);
    if (g < groups) wr[k] = group(p.weight, 0, g);
    if (BYTES) unpack(wr[k], f);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      s.sum = fmaf(v[k][i], v[k][i], s.sum);
      if (BYTES) s.max = max_nan(s.max, fabsf(v[k][i] * f[i]));
    }
    if (p.h && g < groups)
      reinterpret_cast<Raw<T>*>(static_cast<T*>(p.h) + row * p.ldh)[g] = pack<T>(v[k]);
  }
  s = reduce_team<BYTES>(s, team / 32, box[1]);
  // of the unrounded h, in 32 bits
  const float r2 = rsqrtf(s.sum * inv_cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = r2;
  // max |y| = r2 * max |h * weight|, so one reduction serves both
  float scale = 0.0f;
  if (BYTES && p.quant != Q_E4M3_GROUP) {
    scale = row_scale(p.quant, s.max, r2);
    if (t == 0) p.scales[row] = scale;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    float w[GROUP];
    unpack(wr[k], w);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) v[k][i] = v[k][i] * r2 * w[i];
    if (!BYTES) {
      if (g < groups) reinterpret_cast<Raw<T>*>(static_cast<T*>(p.y) + row * p.ldy)[g] = pack<T>(v[k]);
    } else {
      if (p.quant == Q_E4M3_GROUP)
        scale = group_scale(v[k], p.scales + row * ((cols + QUANT_GROUP - 1) / QUANT_GROUP), g, groups);
      const uint2 out = p.quant == Q_INT8_ROW ? int8_quotients(v[k], scale) : quotients(v[k], scale);
      if (g < groups) reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.ldy)[g] = out;
    }
  }
}

// A row of groups in 32 bits in shared memory: the groups' lower halves before the upper
// ones, so that a warp's 16-byte accesses meet no bank twice.
struct Cells {
  float4* at;
  int groups;
  __device__ __forceinline__ void get(int g, float (&v)[GROUP]) const {
    const float4 a = at[g], b = at[groups + g];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void put(int g, const float (&v)[GROUP]) const {
    at[g] = make_float4(v[0], v[1], v[2], v[3]);
    at[groups + g] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

constexpr int ANY_MOST = 512;   // threads of a block on the general path

// Rows that lie anywhere: a team walks its row's groups, and keeps what later passes over the
// row need in shared memory, so that one kernel serves all lengths.
template <typename T>
__global__ void __launch_bounds__(ANY_MOST) block_norm_any_kernel(const __grid_constant__ BlockParams p) {
  __shared__ SumMax box[2][32];
  extern __shared__ __align__(16) float row_smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, which = threadIdx.x / team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + which;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const Row<T> x = row_of<T>(p.x, row, p.rows, p.ldx), res = row_of<T>(p.residual, row, p.rows, p.ldr),
               gate = p.ldg ? row_of<T>(p.gate, row, p.rows, p.ldg) : row_of<T>(p.gate, 0, 1, 0),
               post = row_of<T>(p.post, 0, 1, 0), weight = row_of<T>(p.weight, 0, 1, 0);
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  const Cells cells{reinterpret_cast<float4*>(row_smem) + which * 2 * groups, groups};
  for (int g = t; g < groups; g += team) {
    prefetch_group(x, g * GROUP);
    prefetch_group(res, g * GROUP);
    if (p.gate) prefetch_group(gate, g * GROUP);
  }
  SumMax s = {0.0f, 0.0f};
  for (int g = t; g < groups; g += team) {
    float v[GROUP];
    unpack(load_group<false>(x, g * GROUP, cols), v);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) s.sum = fmaf(v[i], v[i], s.sum);
    cells.put(g, v);   // read by this thread alone
  }
  float r1 = 1.0f;
  if (p.post) {
    r1 = rsqrtf(reduce_team<false>(s, team / 32, box[0]).sum * inv_cols + p.eps);
    if (p.post_rstd && t == 0) p.post_rstd[row] = r1;
  }
  const Join join{p.post != nullptr, p.gate != nullptr, p.alpha, r1};
  const bool by_row = p.quant == Q_E4M3_ROW || p.quant == Q_INT8_ROW;
  s = {0.0f, 0.0f};
  for (int g0 = 0; g0 < groups; g0 += team) {   // whole warps stay together for the stores
    const int g = g0 + t;
    float v[GROUP] = {};
    if (g < groups) {
      float r[GROUP], f[GROUP] = {}, gates[GROUP] = {};
      cells.get(g, v);
      unpack(load_group<false>(res, g * GROUP, cols), r);
      if (p.post) unpack(load_group<false>(post, g * GROUP, cols), f);
      if (p.gate) unpack(load_group<false>(gate, g * GROUP, cols), gates);
      join(v, f, gates, r);
      cells.put(g, v);
      if (by_row) unpack(load_group<false>(weight, g * GROUP, cols), f);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        s.sum = fmaf(v[i], v[i], s.sum);
        if (by_row) s.max = max_nan(s.max, fabsf(v[i] * f[i]));
      }
    }
    if (p.h)
      store_group<false>(static_cast<T*>(p.h) + row * p.ldh, column_of(g, groups, cols), cols, t, team,
                         pack<T>(v));
  }
  s = reduce_team<true>(s, team / 32, box[1]);
  const float r2 = rsqrtf(s.sum * inv_cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = r2;
  float scale = 0.0f;
  if (by_row) {
    scale = row_scale(p.quant, s.max, r2);
    if (t == 0) p.scales[row] = scale;
  }
  for (int g0 = 0; g0 < groups; g0 += team) {
    const int g = g0 + t, c = column_of(g, groups, cols);
    float v[GROUP] = {};
    if (g < groups) {
      float w[GROUP];
      cells.get(g, v);
      unpack(load_group<false>(weight, c, cols), w);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[i] = v[i] * r2 * w[i];
    }
    if (p.quant == Q_SAME) {
      store_group<false>(static_cast<T*>(p.y) + row * p.ldy, c, cols, t, team, pack<T>(v));
      continue;
    }
    if (p.quant == Q_E4M3_GROUP)
      scale = group_scale(v, p.scales + row * ((cols + QUANT_GROUP - 1) / QUANT_GROUP), g, groups);
    const uint2 out = p.quant == Q_INT8_ROW ? int8_quotients(v, scale) : quotients(v, scale);
    store_bytes<false>(static_cast<uint8_t*>(p.y) + row * p.ldy, c, cols, t, team, out);
  }
}

// How a launch's rows pass through the ring in shared memory.
struct RingPlan {
  int stages, teams;    // stages of a team
  uint32_t row_bytes;   // of one matrix
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;      // 3: only the first stages are ever filled; 5: the next row is given up
#endif
};

// A team's place in the ring.
struct TeamRing {
  int which, t;
  RingRows rows;
  uint32_t stage0, stage_bytes, bars;
  int stages;
  int s = 0;            // this row's stage and its phase
  uint32_t ph = 0;
  __device__ __forceinline__ uint32_t full(int stage) const { return bars + 8 * (which * stages + stage); }
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
  // Given up at row k, those before row `fetched` on their way: they land before the CTA ends.
  __device__ __forceinline__ void drain(int64_t k, int64_t fetched) const {
    if (t == 0)
      for (int64_t j = k; j < rows.count && j < fetched; ++j)
        wait_drain(full(static_cast<int>(j % stages)), static_cast<uint32_t>(j / stages) & 1);
  }
#ifdef GEMM_WS_DEBUG
  // Injected fault: false, as if the wait for a row that has come had run out.
  __device__ __forceinline__ bool give_up(const Watchdog& wd) const {
    if (t == 0) {
      *wd.abort = 1;
      atomicExch(wd.status, STATUS_TIMEOUT);
    }
    return false;
  }
#endif
};

// Sets the barriers up and finds the team's place (all threads of the CTA call it).
__device__ __forceinline__ TeamRing enter_ring(const RingPlan& q, int64_t rows, int team, int inputs,
                                               uint8_t* ring, uint64_t* bars, uint32_t* aborted) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.teams * q.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    *aborted = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  TeamRing r;
  r.t = threadIdx.x % team;
  r.which = threadIdx.x / team;
  r.rows = ring_rows(rows, q.teams, r.which);
  r.stage_bytes = inputs * q.row_bytes;
  r.stage0 = smem_addr(ring) + r.which * q.stages * r.stage_bytes;
  r.bars = smem_addr(bars);
  r.stages = q.stages;
  return r;
}

// Up to three vectors over the columns, for all of a launch's rows: a thread's groups of them in its
// registers, or in 16 bits, where the threads have more groups, in shared memory behind the ring (in registers
// they would spill, and what shared memory leaves of the L1 cache does not hold that: gradient of
// 8192 x 8192 213 us, 165 like this).
template <typename T, int VPT>
struct Vectors {
  static constexpr bool SHARED = sizeof(T) == 2;
  Raw<T> held[SHARED ? 1 : 3][SHARED ? 1 : VPT];
  const Raw<T>* at;
  int groups, team;
  // All threads of the CTA call it; `vectors` NULL: zeros.
  __device__ __forceinline__ Vectors(uint8_t* behind, const void* const (&vectors)[3], int groups_, int team_, int t)
      : at(reinterpret_cast<const Raw<T>*>(behind) + t), groups(groups_), team(team_) {
#pragma unroll
    for (int v = 0; v < 3; ++v) {
      const Raw<T>* from = static_cast<const Raw<T>*>(vectors[v]);
      if constexpr (SHARED) {
        for (int g = threadIdx.x; g < groups; g += blockDim.x)
          reinterpret_cast<Raw<T>*>(behind)[v * groups + g] = from ? from[g] : Raw<T>{};
      } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          held[v][j] = {};
          if (from && j * team + t < groups) held[v][j] = from[j * team + t];
        }
      }
    }
    if (SHARED) __syncthreads();
  }
  // Vector v, the thread's group j (which has to be there).
  __device__ __forceinline__ Raw<T> get(int v, int j) const {
    if constexpr (SHARED)
      return at[v * groups + j * team];
    else
      return held[v][j];
  }
};

// Many rows that lie FAST come through a ring of bulk copies, so that the next rows are on their
// way while a team waits for its row's two sums. One thread of a team fetches; the barrier of the
// second sum says that all of it has the row in registers, and the stage is filled anew.
template <typename T, int VPT, bool BYTES>
__global__ void __launch_bounds__(RING_THREADS, 1)
    block_norm_ring_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ RingPlan q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ SumMax box[2][RING_WARPS];
  __shared__ float box1[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const bool each = p.ldg != 0;
  TeamRing at = enter_ring(q, p.rows, team, each ? 3 : 2, ring, bars, &aborted);
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  const int t = at.t, which = at.which;
  const void* const vectors[3] = {p.weight, p.post, each ? nullptr : p.gate};
  const Vectors<T, VPT> vec(ring + q.teams * q.stages * at.stage_bytes, vectors, groups, team, t);
  if (at.rows.count == 0) return;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
    if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
    const int64_t row = at.rows.first + k * at.rows.step;
    const uint32_t dst = at.stage0 + s * at.stage_bytes, bar = at.full(s);
    mbar_arrive_expect_tx(bar, at.stage_bytes);
    bulk_load_1d(dst, static_cast<const T*>(p.x) + row * p.ldx, q.row_bytes, bar);
    bulk_load_1d(dst + q.row_bytes, static_cast<const T*>(p.residual) + row * p.ldr, q.row_bytes, bar);
    if (each)
      bulk_load_1d(dst + 2 * q.row_bytes, static_cast<const T*>(p.gate) + row * p.ldg, q.row_bytes, bar);
  };
  if (t == 0)
    for (int k = 0; k < q.stages && k < at.rows.count; ++k) fetch(k, k);
  int turn = 0;
  int64_t k = 0;
  for (; k < at.rows.count; ++k, turn ^= 1) {
    const int64_t row = at.rows.first + k * at.rows.step;
    bool ok = warp_wait_cta(at.full(at.s), at.ph, wd);
#ifdef GEMM_WS_DEBUG
    if (q.debug_fault == 5 && k == q.stages) ok = at.give_up(wd);
#endif
    const uint8_t* stage = ring + (which * q.stages + at.s) * at.stage_bytes;
    const Raw<T>* x = reinterpret_cast<const Raw<T>*>(stage) + t;
    const Raw<T>* res = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
    const Raw<T>* gate = reinterpret_cast<const Raw<T>*>(stage + 2 * q.row_bytes) + t;
    float r1 = 1.0f;
    if (p.post) {
      Pair sums = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (j * team + t < groups) {
          Pair v[GROUP / 2];
          unpack(x[j * team], v);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) sums = fma2(v[i], v[i], sums);
        }
      const float sum =
          ring_sum(values_of(sums).x + values_of(sums).y, which, team, box1[turn], &ok);
      if (!ok) break;
      r1 = rsqrtf(sum * inv_cols + p.eps);
      if (p.post_rstd && t == 0) p.post_rstd[row] = r1;
    }
    const Pair r11 = pair_of(r1, r1), alpha = pair_of(p.alpha, p.alpha);
    Raw<T>* h = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.h) + row * p.ldh) + t;
    float v[VPT][GROUP];
    Pair sums = 0;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool mine = j * team + t < groups;
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[j][i] = 0.0f;
      if (mine) {
        Pair a[GROUP / 2], f[GROUP / 2];
        unpack(x[j * team], a);
        if (p.post) {
          unpack(vec.get(1, j), f);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) a[i] = mul2(mul2(a[i], r11), f[i]);
        }
        if (p.gate) {
          unpack(each ? gate[j * team] : vec.get(2, j), f);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) a[i] = mul2(a[i], f[i]);
        }
        unpack(res[j * team], f);
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) {
          a[i] = fma2(alpha, f[i], a[i]);
          sums = fma2(a[i], a[i], sums);
          v[j][2 * i] = values_of(a[i]).x;
          v[j][2 * i + 1] = values_of(a[i]).y;
        }
        if (BYTES) {
          unpack(vec.get(0, j), f);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            const float2 b = values_of(mul2(a[i], f[i]));
            top = max_nan(top, max_nan(fabsf(b.x), fabsf(b.y)));
          }
        }
        if (p.h) h[j * team] = pack<T>(v[j]);
      }
    }
    const SumMax all = ring_sum_max({values_of(sums).x + values_of(sums).y, top}, which, team, box[turn], &ok);
    if (!ok) break;
    if (t == 0 && k + q.stages < at.rows.count) fetch(k + q.stages, at.s);   // the row is in registers
    const float r2 = rsqrtf(all.sum * inv_cols + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r2;
    float scale = 0.0f;
    if (BYTES && p.quant != Q_E4M3_GROUP) {
      scale = row_scale(p.quant, all.max, r2);
      if (t == 0) p.scales[row] = scale;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int g = j * team + t;
      if (g < groups) {
        float w[GROUP];
        unpack(vec.get(0, j), w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) v[j][i] = v[j][i] * r2 * w[i];
      }
      if (!BYTES) {
        if (g < groups) (reinterpret_cast<Raw<T>*>(static_cast<T*>(p.y) + row * p.ldy))[g] = pack<T>(v[j]);
      } else {
        if (p.quant == Q_E4M3_GROUP)
          scale = group_scale(v[j], p.scales + row * ((cols + QUANT_GROUP - 1) / QUANT_GROUP), g, groups);
        const uint2 out = p.quant == Q_INT8_ROW ? int8_quotients(v[j], scale) : quotients(v[j], scale);
        if (g < groups) reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.ldy)[g] = out;
      }
    }
    at.next();
  }
  at.drain(k, k + q.stages);
}

// ------------------------------------------------------------ backward

struct BlockGradParams {
  const void *dy, *dh, *x, *h, *gate, *post, *weight;   // dh, gate and post may be NULL
  const float *post_rstd, *rstd;
  void *dx, *dres, *dgate;            // dres and dgate (of a gate for each value) may be NULL
  float *partial, *partial_s;         // partial sums of dweight and S, one row of whole groups a block; may be NULL
  int64_t lddy, lddh, ldx, ldh, ldg, lddx, lddres, lddg;
  int64_t rows;
  int cols;
  int team;
  float alpha;
};

// What the passes over a group make of it, forward's names: from dy, h, dh and weight g (in d),
// what goes to the residual, and the share of dweight.
struct GradRow {
  bool post, each, gate;   // a norm after the block; a gate for each value; a gate
  float alpha, r1, r2;
  // The first pass: this group's terms of mean(a * m), and of dweight.
  __device__ __forceinline__ float first(const float (&a)[GROUP], const float (&h)[GROUP],
                                         const float (&w)[GROUP], float (&acc)[GROUP]) const {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const float m = h[i] * r2;
      acc[i] = fmaf(a[i], m, acc[i]);
      sum = fmaf(a[i] * w[i], m, sum);
    }
    return sum;
  }
  // g, in d, which holds dh; c2 = r2 * mean(a * m).
  __device__ __forceinline__ void second(const float (&a)[GROUP], const float (&h)[GROUP],
                                         const float (&w)[GROUP], float c2, float (&d)[GROUP]) const {
#pragma unroll
    for (int i = 0; i < GROUP; ++i) d[i] = fmaf(r2, a[i] * w[i] - h[i] * c2, d[i]);
  }
  // From g in d: e * post in d, the gate's gradient, and this group's terms of mean(e post n) and of S.
  __device__ __forceinline__ float third(const float (&x)[GROUP], const float (&gates)[GROUP],
                                         const float (&w)[GROUP], float (&d)[GROUP], float (&acc)[GROUP],
                                         float (&dgate)[GROUP]) const {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const float n = x[i] * r1;
      if (each) {
        dgate[i] = d[i] * (post ? n * w[i] : n);
        d[i] *= gates[i];
      }
      acc[i] = fmaf(d[i], n, acc[i]);
      if (gate && !each) d[i] *= gates[i];
      if (post) {
        d[i] *= w[i];
        sum = fmaf(d[i], n, sum);
      }
    }
    return sum;
  }
  // dx, in d; c1 = r1 * mean(e post n).
  __device__ __forceinline__ void fourth(const float (&x)[GROUP], float c1, float (&d)[GROUP]) const {
    if (!post) return;
#pragma unroll
    for (int i = 0; i < GROUP; ++i) d[i] = r1 * (d[i] - x[i] * c1);
  }
};

// Persistent, rows that lie FAST: a team takes rows blockIdx * teams + team, + all teams of the
// grid, and keeps its columns' shares of the two sums over the rows in registers; a block
// leaves one partial row of each, which block_sums_kernel adds in block order, so that the
// sums have the same bits on every run.
template <typename T, int VPT, int MOST>
__global__ void __launch_bounds__(MOST, 1)
    block_norm_grad_kernel(const __grid_constant__ BlockGradParams p) {
  __shared__ SumMax box[2][2][32];
  extern __shared__ __align__(16) float share[];   // where a team is a warp: their shares of a sum
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, teams = blockDim.x / team;
  const int cols = p.cols, groups = cols / GROUP;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  float acc[VPT][GROUP], acc_s[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP; ++i) acc[k][i] = acc_s[k][i] = 0.0f;

  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * teams + threadIdx.x / team; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * teams, turn ^= 1) {
    auto group = [&](const void* m, int64_t ld, int g) {
      return reinterpret_cast<const Raw<T>*>(static_cast<const T*>(m) + row * ld)[g];
    };
    auto place = [&](void* m, int64_t ld, int g) -> Raw<T>& {
      return reinterpret_cast<Raw<T>*>(static_cast<T*>(m) + row * ld)[g];
    };
    Raw<T> yr[VPT] = {}, hr[VPT] = {}, dr[VPT] = {}, xr[VPT] = {}, gr[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        yr[k] = group(p.dy, p.lddy, g);
        hr[k] = group(p.h, p.ldh, g);
        if (p.dh) dr[k] = group(p.dh, p.lddh, g);
        xr[k] = group(p.x, p.ldx, g);
        if (p.gate) gr[k] = group(p.gate, p.ldg, g);
      }
    }
    const GradRow of{p.post != nullptr, p.ldg != 0, p.gate != nullptr, p.alpha,
                     p.post ? p.post_rstd[row] : 1.0f, p.rstd[row]};
    SumMax s = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], h[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], h);
        unpack(group(p.weight, 0, g), w);
        s.sum += of.first(a, h, w, acc[k]);
      }
    }
    const float c2 = reduce_team<false>(s, team / 32, box[turn][0]).sum * inv_cols * of.r2;
    float d[VPT][GROUP];
    s = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], h[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], h);
        unpack(group(p.weight, 0, g), w);
        unpack(dr[k], d[k]);
        of.second(a, h, w, c2, d[k]);
        if (p.dres) {
#pragma unroll
          for (int i = 0; i < GROUP; ++i) a[i] = p.alpha * d[k][i];
          place(p.dres, p.lddres, g) = pack<T>(a);
        }
        unpack(xr[k], h);
        unpack(gr[k], a);
        if (p.post) unpack(group(p.post, 0, g), w);
        float dgate[GROUP];
        s.sum += of.third(h, a, w, d[k], acc_s[k], dgate);
        if (p.dgate) place(p.dgate, p.lddg, g) = pack<T>(dgate);
      }
    }
    float c1 = 0.0f;
    if (p.post) c1 = reduce_team<false>(s, team / 32, box[turn][1]).sum * inv_cols * of.r1;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float x[GROUP];
        unpack(xr[k], x);
        of.fourth(x, c1, d[k]);
        place(p.dx, p.lddx, g) = pack<T>(d[k]);
      }
    }
  }
  if (p.partial) leave_partial(acc, share, p.partial, groups, team, teams, threadIdx.x / team, t);
  if (p.partial_s) {
    if (p.partial && teams > 1) __syncthreads();   // `share` has been read
    leave_partial(acc_s, share, p.partial_s, groups, team, teams, threadIdx.x / team, t);
  }
}

// The gradient of many rows that lie FAST, through the ring (loaded straight into registers the
// rows of an SM stop at each of a row's two sums). The barrier of a row's second sum says that all of the
// team has what it still needs of it in registers; without the norm after the block that of the next row's first sum. Two groups a thread, so
// that its shares of the two sums over the rows fit its registers. 8192 x 8192 bf16 with dh and dresidual: 805 MB
// in 165 us, 4.9 TB/s; bound by latency: an SM has 16 warps, two rows in its ring, and two barriers a row
// (warps issue in 45 of 100 cycles, a quarter of their time they wait for the row).
template <typename T, int VPT>
__global__ void __launch_bounds__(RING_THREADS, 1)
    block_norm_grad_ring_kernel(const __grid_constant__ BlockGradParams p, const __grid_constant__ RingPlan q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ float box[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const bool each = p.ldg != 0, post = p.post != nullptr;
  const int gate_at = p.dh ? 4 : 3;
  TeamRing at = enter_ring(q, p.rows, team, gate_at + (each ? 1 : 0), ring, bars, &aborted);
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  const int t = at.t, which = at.which;
  const void* const vectors[3] = {p.weight, p.post, each ? nullptr : p.gate};
  const Vectors<T, VPT> vec(ring + q.teams * q.stages * at.stage_bytes, vectors, groups, team, t);
  const float inv_cols = 1.0f / static_cast<float>(cols);

  Pair acc[VPT][GROUP / 2], acc_s[VPT][GROUP / 2];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < GROUP / 2; ++i) acc[j][i] = acc_s[j][i] = 0;

  if (at.rows.count > 0) {
    auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
      if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
      const int64_t row = at.rows.first + k * at.rows.step;
      const uint32_t dst = at.stage0 + s * at.stage_bytes, bar = at.full(s), each_row = q.row_bytes;
      mbar_arrive_expect_tx(bar, at.stage_bytes);
      bulk_load_1d(dst, static_cast<const T*>(p.dy) + row * p.lddy, each_row, bar);
      bulk_load_1d(dst + each_row, static_cast<const T*>(p.h) + row * p.ldh, each_row, bar);
      bulk_load_1d(dst + 2 * each_row, static_cast<const T*>(p.x) + row * p.ldx, each_row, bar);
      if (p.dh) bulk_load_1d(dst + 3 * each_row, static_cast<const T*>(p.dh) + row * p.lddh, each_row, bar);
      if (each)
        bulk_load_1d(dst + gate_at * each_row, static_cast<const T*>(p.gate) + row * p.ldg, each_row, bar);
    };
    if (t == 0)
      for (int k = 0; k < q.stages && k < at.rows.count; ++k) fetch(k, k);
    int turn = 0, before = q.stages - 1;   // the row before's stage
    float next2 = p.rstd[at.rows.first], next1 = post ? p.post_rstd[at.rows.first] : 1.0f;
    const Pair alpha = pair_of(p.alpha, p.alpha);
    int64_t k = 0;
    for (; k < at.rows.count; ++k) {
      const int64_t row = at.rows.first + k * at.rows.step;
      const float r2 = next2, r1 = next1;
      if (k + 1 < at.rows.count) {
        next2 = p.rstd[row + at.rows.step];
        if (post) next1 = p.post_rstd[row + at.rows.step];
      }
      bool ok = warp_wait_cta(at.full(at.s), at.ph, wd);
#ifdef GEMM_WS_DEBUG
      if (q.debug_fault == 5 && k == q.stages) ok = at.give_up(wd);
#endif
      const uint8_t* stage = ring + (which * q.stages + at.s) * at.stage_bytes;
      const Raw<T>* dy = reinterpret_cast<const Raw<T>*>(stage) + t;
      const Raw<T>* h = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
      const Raw<T>* x = reinterpret_cast<const Raw<T>*>(stage + 2 * q.row_bytes) + t;
      const Raw<T>* dh = reinterpret_cast<const Raw<T>*>(stage + 3 * q.row_bytes) + t;
      const Raw<T>* gate = reinterpret_cast<const Raw<T>*>(stage + gate_at * q.row_bytes) + t;
      const Pair r22 = pair_of(r2, r2), r11 = pair_of(r1, r1);
      Pair d[VPT][GROUP / 2];
      Pair sums = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (j * team + t < groups) {
          Pair a[GROUP / 2], m[GROUP / 2], w[GROUP / 2];
          unpack(dy[j * team], a);
          unpack(h[j * team], m);
          unpack(vec.get(0, j), w);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            acc[j][i] = fma2(mul2(a[i], m[i]), r22, acc[j][i]);
            d[j][i] = mul2(a[i], w[i]);
            sums = fma2(d[j][i], m[i], sums);
          }
        }
      float sum = ring_sum(values_of(sums).x + values_of(sums).y, which, team, box[turn], &ok);
      turn ^= 1;
      if (!ok) break;
      // The whole team has been in the sum, so it has done with the row before.
      if (!post && t == 0 && k > 0 && k - 1 + q.stages < at.rows.count) fetch(k - 1 + q.stages, before);
      // g = dh + r2 dy weight - h r2^2 mean(dy weight h r2), then e * post
      const float c2 = -r2 * r2 * (r2 * sum * inv_cols);
      const Pair c22 = pair_of(c2, c2);
      Raw<T>* dres = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dres) + row * p.lddres) + t;
      Raw<T>* dgate = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dgate) + row * p.lddg) + t;
      Raw<T>* dx = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dx) + row * p.lddx) + t;
      auto put = [](Raw<T>& to, const Pair (&v)[GROUP / 2]) {
        float f[GROUP];
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) {
          f[2 * i] = values_of(v[i]).x;
          f[2 * i + 1] = values_of(v[i]).y;
        }
        to = pack<T>(f);
      };
      Raw<T> xr[VPT];
      sums = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j * team + t >= groups) continue;
        Pair a[GROUP / 2], f[GROUP / 2];
        {
          Raw<T> dr = {};
          if (p.dh) dr = dh[j * team];
          unpack(dr, f);
        }
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) d[j][i] = fma2(d[j][i], r22, f[i]);
        unpack(h[j * team], a);
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) d[j][i] = fma2(a[i], c22, d[j][i]);
        if (p.dres) {
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) a[i] = mul2(d[j][i], alpha);
          put(dres[j * team], a);
        }
        Pair n[GROUP / 2];
        xr[j] = x[j * team];
        unpack(xr[j], n);
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) n[i] = mul2(n[i], r11);
        if (post) unpack(vec.get(1, j), f);
        if (each) {
          if (p.dgate) {
#pragma unroll
            for (int i = 0; i < GROUP / 2; ++i) {
              a[i] = mul2(d[j][i], n[i]);
              if (post) a[i] = mul2(a[i], f[i]);
            }
            put(dgate[j * team], a);
          }
          unpack(gate[j * team], a);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) d[j][i] = mul2(d[j][i], a[i]);
        }
#pragma unroll
        for (int i = 0; i < GROUP / 2; ++i) acc_s[j][i] = fma2(d[j][i], n[i], acc_s[j][i]);
        if (p.gate && !each) {
          unpack(vec.get(2, j), a);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) d[j][i] = mul2(d[j][i], a[i]);
        }
        if (post) {
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            d[j][i] = mul2(d[j][i], f[i]);
            sums = fma2(d[j][i], n[i], sums);
          }
        } else {
          put(dx[j * team], d[j]);
        }
      }
      if (post) {
        sum = ring_sum(values_of(sums).x + values_of(sums).y, which, team, box[turn], &ok);
        turn ^= 1;
        if (!ok) break;
        if (t == 0 && k + q.stages < at.rows.count) fetch(k + q.stages, at.s);   // what is left is in registers
        const float c1 = -r1 * (r1 * sum * inv_cols);
        const Pair c11 = pair_of(c1, c1);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          if (j * team + t >= groups) continue;
          Pair n[GROUP / 2];
          unpack(xr[j], n);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) d[j][i] = fma2(n[i], c11, mul2(d[j][i], r11));
          put(dx[j * team], d[j]);
        }
      }
      before = at.s;
      at.next();
    }
    at.drain(k, k + q.stages - (!post && k > 0));   // without `post` a stage is filled anew one row later
  }
  float mine[VPT][GROUP];
  auto leave = [&](const Pair (&of)[VPT][GROUP / 2], float* partial) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < GROUP / 2; ++i) {
        mine[j][2 * i] = values_of(of[j][i]).x;
        mine[j][2 * i + 1] = values_of(of[j][i]).y;
      }
    __syncthreads();   // all teams have done with the ring, or with the sum before
    leave_partial(mine, reinterpret_cast<float*>(ring), partial, groups, team, q.teams, which, t);
  };
  static_assert(RING_THREADS * VPT * GROUP * sizeof(float) <= RING_BYTES, "the teams' rows fit the ring");
  if (p.partial) leave(acc, p.partial);
  if (p.partial_s) leave(acc_s, p.partial_s);
}

// The same for rows that lie anywhere, and (WHOLE) for long aligned ones, whose shares of the sums no
// registers hold: e * post and the columns' shares are in shared memory, and the rows' values are read once more
// (from L2) for the second pass. The team's next row is called into L2 meanwhile. (8192 x 8191 bf16 600 us, 1.3 TB/s: the
// pieces that unaligned groups are cut from, and put together to, cost most; 4096 x 16384 298, 2.7.)
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(WHOLE ? 1024 : ANY_MOST)
    block_norm_grad_any_kernel(const __grid_constant__ BlockGradParams p) {
  __shared__ SumMax box[2][2][32];
  extern __shared__ __align__(16) float row_smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, teams = blockDim.x / team, which = threadIdx.x / team;
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  float4* base = reinterpret_cast<float4*>(row_smem);
  const Cells sums{base + which * 2 * groups, groups}, sums_s{base + (teams + which) * 2 * groups, groups},
      cells{base + (2 * teams + which) * 2 * groups, groups};
  const Row<T> weight = row_of<T>(p.weight, 0, 1, 0), post = row_of<T>(p.post, 0, 1, 0);
  for (int g = t; g < groups; g += team) {
    const float zero[GROUP] = {};
    sums.put(g, zero);
    sums_s.put(g, zero);
  }
  auto fetch = [&](int64_t row) {
    if (row >= p.rows) return;
    for (int g = t; g < groups; g += team) {
      auto ahead = [&](const void* m, int64_t ld) { prefetch_group(row_of<T>(m, row, p.rows, ld), g * GROUP); };
      ahead(p.dy, p.lddy);
      ahead(p.h, p.ldh);
      ahead(p.x, p.ldx);
      if (p.dh) ahead(p.dh, p.lddh);
      if (p.ldg) ahead(p.gate, p.ldg);
    }
  };
  int turn = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * teams + which;
  fetch(row);
  for (; row < p.rows; row += step, turn ^= 1) {
    fetch(row + step);
    const Row<T> dy = row_of<T>(p.dy, row, p.rows, p.lddy), h = row_of<T>(p.h, row, p.rows, p.ldh),
                 dh = row_of<T>(p.dh, row, p.rows, p.lddh), x = row_of<T>(p.x, row, p.rows, p.ldx),
                 gate = p.ldg ? row_of<T>(p.gate, row, p.rows, p.ldg) : row_of<T>(p.gate, 0, 1, 0);
    const GradRow of{p.post != nullptr, p.ldg != 0, p.gate != nullptr, p.alpha,
                     p.post ? p.post_rstd[row] : 1.0f, p.rstd[row]};
    SumMax s = {0.0f, 0.0f};
    for (int g = t; g < groups; g += team) {
      float a[GROUP], v[GROUP], w[GROUP], acc[GROUP];
      unpack(load_group<WHOLE>(dy, g * GROUP, cols), a);
      unpack(load_group<WHOLE>(h, g * GROUP, cols), v);
      unpack(load_group<WHOLE>(weight, g * GROUP, cols), w);
      sums.get(g, acc);
      s.sum += of.first(a, v, w, acc);
      sums.put(g, acc);
    }
    const float c2 = reduce_team<false>(s, team / 32, box[turn][0]).sum * inv_cols * of.r2;
    s = {0.0f, 0.0f};
    // dy and dh are read for the last time before anything is written over them: by a group's
    // own thread, and its neighbours take nothing of it that counts
    for (int g0 = 0; g0 < groups; g0 += team) {   // whole warps stay together for the stores
      const int g = g0 + t, c = column_of(g, groups, cols);
      float d[GROUP] = {}, a[GROUP] = {}, dgate[GROUP] = {};
      if (g < groups) {
        float v[GROUP], w[GROUP], acc[GROUP];
        unpack(load_group<WHOLE>(dy, c, cols), a);
        unpack(load_group<WHOLE>(h, c, cols), v);
        unpack(load_group<WHOLE>(weight, c, cols), w);
        if (p.dh) unpack(load_group<WHOLE>(dh, c, cols), d);
        of.second(a, v, w, c2, d);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) a[i] = p.alpha * d[i];
        unpack(load_group<WHOLE>(x, c, cols), v);
        float gates[GROUP] = {};
        if (p.gate) unpack(load_group<WHOLE>(gate, c, cols), gates);
        if (p.post) unpack(load_group<WHOLE>(post, c, cols), w);
        sums_s.get(g, acc);
        s.sum += of.third(v, gates, w, d, acc, dgate);
        sums_s.put(g, acc);
        cells.put(g, d);
      }
      __syncwarp();
      if (WHOLE && g >= groups) continue;
      if (p.dres)
        store_group<WHOLE>(static_cast<T*>(p.dres) + row * p.lddres, c, cols, t, team, pack<T>(a));
      if (p.dgate)
        store_group<WHOLE>(static_cast<T*>(p.dgate) + row * p.lddg, c, cols, t, team, pack<T>(dgate));
    }
    float c1 = 0.0f;
    if (p.post) c1 = reduce_team<false>(s, team / 32, box[turn][1]).sum * inv_cols * of.r1;
    for (int g0 = 0; g0 < groups; g0 += team) {
      const int g = g0 + t, c = column_of(g, groups, cols);
      float d[GROUP] = {};
      if (g < groups) {
        float v[GROUP];
        cells.get(g, d);
        unpack(load_group<WHOLE>(x, c, cols), v);
        of.fourth(v, c1, d);
      }
      if (!WHOLE || g < groups)
        store_group<WHOLE>(static_cast<T*>(p.dx) + row * p.lddx, c, cols, t, team, pack<T>(d));
    }
  }
  __syncthreads();
  // the teams' shares added in the teams' order
  auto leave = [&](const float4* of_teams, float* partial) {
    float4* out = reinterpret_cast<float4*>(partial) + static_cast<size_t>(blockIdx.x) * 2 * groups;
    for (int j = threadIdx.x; j < 2 * groups; j += blockDim.x) {
      float4 sum = of_teams[j];
      for (int v = 1; v < teams; ++v) {
        const float4 a = of_teams[v * 2 * groups + j];
        sum.x += a.x, sum.y += a.y, sum.z += a.z, sum.w += a.w;
      }
      out[j < groups ? 2 * j : 2 * (j - groups) + 1] = sum;
    }
  };
  if (p.partial) leave(base, p.partial);
  if (p.partial_s) leave(base + teams * 2 * groups, p.partial_s);
}

struct BlockSumsParams {
  const float *partial, *partial_s;   // NULL: without that sum
  int blocks, cols, pitch;
  int columns;                        // blocks of columns; those of the second sum follow
  const void *gate, *post;            // of a gate for each channel; NULL: 1
  void *dweight, *dpost, *dgate;      // NULL: not written
};

// dweight, and from S dpost and dgate.
template <typename T>
__global__ void __launch_bounds__(DW_THREADS)
    block_sums_kernel(const __grid_constant__ BlockSumsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const bool second = !p.partial || blockIdx.x >= static_cast<unsigned>(p.columns);
  const int block = second && p.partial ? blockIdx.x - p.columns : blockIdx.x;
  auto at = [](const void* v, int c) { return v ? to_float(static_cast<const T*>(v)[c]) : 1.0f; };
  column_sums(second ? p.partial_s : p.partial, block, p.blocks, p.cols, p.pitch, [&](int c, float sum) {
    if (!second) {
      static_cast<T*>(p.dweight)[c] = round_to(sum, T());
      return;
    }
    if (p.dpost) static_cast<T*>(p.dpost)[c] = round_to(sum * at(p.gate, c), T());
    if (p.dgate) static_cast<T*>(p.dgate)[c] = round_to(sum * at(p.post, c), T());
  });
}

// ------------------------------------------------------------ rows to 8-bit integers

struct QuantizeParams {
  const void* x;
  int8_t* y;
  float* scales;
  int64_t ldx, ldy;
  int64_t rows;
  int cols;
  int team;
};

// The largest magnitude of a thread's groups, NaN if there is one. Without their signs 16-bit floats are in the
// order of their bits as integers, with NaN on top: two at a time.
template <typename T, int VPT>
__device__ __forceinline__ float largest(const Raw<T> (&x)[VPT]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      uint32_t w[WORDS<T>];
      words_of(x[k], w);
#pragma unroll
      for (int i = 0; i < WORDS<T>; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    }
    const uint16_t lo = static_cast<uint16_t>(top), hi = static_cast<uint16_t>(top >> 16), most = lo > hi ? lo : hi;
    return to_float(*reinterpret_cast<const T*>(&most));
  } else {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float v[GROUP];
      unpack(x[k], v);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) top = max_nan(top, fabsf(v[i]));
    }
    return top;
  }
}

// A row in registers: read once for its largest magnitude and for its integers. 8192 x 8192 bf16: 201 MB in
// 37.7 us, 5.3 TB/s; bound by the arithmetic of the exact quotients with what blocks the registers leave (42.2 with the
// magnitudes taken in fp32; through a ring of bulk copies 1.14 times as long). fp32 4096 x 8192: 25.6 us, 6.5 TB/s.
template <typename T, int VPT, int MOST>
__global__ void __launch_bounds__(MOST, VPT == 4 && MOST == 512 ? (sizeof(T) == 2 ? 3 : 2) : 1)
    quantize_rows_kernel(const __grid_constant__ QuantizeParams p) {
  __shared__ SumMax box[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const int groups = p.cols / GROUP;
  const Raw<T>* x = reinterpret_cast<const Raw<T>*>(static_cast<const T*>(p.x) + row * p.ldx);
  uint2* y = reinterpret_cast<uint2*>(p.y + row * p.ldy);
  Raw<T> xr[VPT] = {};
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    if (k * team + t < groups) xr[k] = x[k * team + t];
  SumMax s = {0.0f, largest(xr)};
  const float scale = int8_scale(reduce_team<true>(s, team / 32, box).max);
  if (t == 0) p.scales[row] = scale;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float v[GROUP];
    unpack(xr[k], v);
    if (k * team + t < groups) y[k * team + t] = int8_quotients(v, scale);
  }
}

// Rows that lie anywhere, read twice (the second time from L2).
template <typename T>
__global__ void __launch_bounds__(ANY_MOST)
    quantize_rows_any_kernel(const __grid_constant__ QuantizeParams p) {
  __shared__ SumMax box[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const Row<T> x = row_of<T>(p.x, row, p.rows, p.ldx);
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  for (int g = t; g < groups; g += team) prefetch_group(x, g * GROUP);
  SumMax s = {0.0f, 0.0f};
  for (int g = t; g < groups; g += team) {
    float v[GROUP];
    unpack(load_group<false>(x, g * GROUP, cols), v);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) s.max = max_nan(s.max, fabsf(v[i]));
  }
  const float scale = int8_scale(reduce_team<true>(s, team / 32, box).max);
  if (t == 0) p.scales[row] = scale;
  for (int g0 = 0; g0 < groups; g0 += team) {   // whole warps stay together for the stores
    const int g = g0 + t, c = column_of(g, groups, cols);
    float v[GROUP] = {};
    if (g < groups) unpack(load_group<false>(x, c, cols), v);
    store_bytes<false>(reinterpret_cast<uint8_t*>(p.y) + row * p.ldy, c, cols, t, team,
                       int8_quotients(v, scale));
  }
}

}  // namespace gws
