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

#include <stdint.h>

#include "lm_rows.cuh"

namespace gws {

// ------------------------------------------------------------ generator

// Philox4x32 with ten rounds (J. Salmon et al., "Parallel random numbers: as
// easy as 1, 2, 3", 2011): the key is the seed, the counter's low 64 bits are
// given and its high ones 0. The 128 bits serve the 8 columns of a group, 16
// bits each, lowest first: half the rounds' cost of 32 bits a column (which
// would take more issue slots than dropout's 4 bytes of traffic a column
// leave), for a p that is a multiple of 2^-16.
//
// N counters at a time: they share the rounds' keys, and the rounds of one fill
// the latency of the others'.
template <int N>
__device__ __forceinline__ void philox(const uint64_t (&counter)[N], uint64_t seed,
                                       uint32_t (&words)[N][4]) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    words[n][0] = static_cast<uint32_t>(counter[n]);
    words[n][1] = static_cast<uint32_t>(counter[n] >> 32);
    words[n][2] = words[n][3] = 0;
  }
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t(&c)[4] = words[n];
      const uint64_t m0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
      const uint64_t m1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
      c[0] = static_cast<uint32_t>(m1 >> 32) ^ c[1] ^ k0;
      c[1] = static_cast<uint32_t>(m1);
      c[2] = static_cast<uint32_t>(m0 >> 32) ^ c[3] ^ k1;
      c[3] = static_cast<uint32_t>(m0);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// What a launch's dropout is: a column is kept, and scaled, where its word,
// shifted to the top of 32 bits, is above `limit`.
struct Dropout {
  const uint64_t* rng;   // device: seed, first counter (readable, if unused, without dropout)
  int on;
  uint32_t limit;        // (round(65536 p) << 16) - 1
  float scale;           // 65536 / (65536 - round(65536 p)); 0 where all is dropped
};

// v = d(v) for N groups by their words. A dropped value is 0 whatever it was.
// Words are compared in the upper half of a register: the high one as it
// stands (what is below it cannot change the verdict), the low one shifted up.
template <int N>
__device__ __forceinline__ void drop_by(const Dropout& d, const uint32_t (&words)[N][4],
                                        float (&v)[N][GROUP]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[n][2 * i] = (words[n][i] << 16) > d.limit ? v[n][2 * i] * d.scale : 0.0f;
      v[n][2 * i + 1] = words[n][i] > d.limit ? v[n][2 * i + 1] * d.scale : 0.0f;
    }
}

// v = d(v) for N groups at their counters.
template <int N>
__device__ __forceinline__ void drop_groups(const Dropout& d, uint64_t seed,
                                            const uint64_t (&counter)[N], float (&v)[N][GROUP]) {
  uint32_t words[N][4];
  philox(counter, seed, words);
  drop_by(d, words, v);
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
  Dropout drop;
};

// Blocks of `most` threads that an SM has to hold, which bounds their registers: so that
// another row's loads are under way while one waits for its sum. On the general path in
// 16 bits two rows of 512 threads (8192 x 8191 bf16: 164 us, with one of them 270).
constexpr int rows_at_once(bool any, int bytes, int vpt, int most) {
  return most == 256 ? (bytes == 2 ? 3 : 2) : any && bytes == 2 && vpt == 2 ? 2 : 1;
}

// One row a team. Q: 0 y has the type of x; 1 e4m3 with one scale a row; 2
// e4m3 with a scale for each 128 columns.
template <typename T, Path PATH, int VPT, int MOST, int Q>
__global__ void __launch_bounds__(MOST, rows_at_once(PATH == ANY, sizeof(T), VPT, MOST))
    add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ SumMax box[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const Row<T> x = row_of<T>(p.x, row, p.rows, p.ldx), res = row_of<T>(p.residual, row, p.rows, p.ldr),
               weight = row_of<T>(p.weight, 0, 1, 0);
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  constexpr bool WHOLE = PATH != ANY;

  if constexpr (!WHOLE) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * team + t) * GROUP;
      if (c < cols) {
        prefetch_group(x, c);
        if (p.residual) prefetch_group(res, c);
      }
    }
  }
  Raw<T> xr[VPT] = {}, rr[VPT], wr[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      xr[k] = load_group<WHOLE>(x, g * GROUP, cols);
      if (p.residual) rr[k] = load_group<WHOLE>(res, g * GROUP, cols);
      wr[k] = load_group<WHOLE>(weight, g * GROUP, cols);
    }
  }
  const uint64_t seed = p.drop.rng[0];
  const uint64_t first = p.drop.rng[1] + static_cast<uint64_t>(row) * groups;
  float v[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k) unpack(xr[k], v[k]);
  if (PATH == DROP || (PATH == ANY && p.drop.on)) {
    constexpr int PAIR = VPT < 2 ? VPT : 2;   // generators side by side; more would cost registers
#pragma unroll
    for (int k = 0; k < VPT; k += PAIR) {
      uint64_t counter[PAIR];
#pragma unroll
      for (int j = 0; j < PAIR; ++j) counter[j] = first + (k + j) * team + t;
      drop_groups(p.drop, seed, counter, reinterpret_cast<float(&)[PAIR][GROUP]>(v[k]));
    }
  }
  SumMax s = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      float w[GROUP];
      if (Q == 1) unpack(wr[k], w);
      if (p.residual) {
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
    }
    if (p.h && (PATH == ANY || g < groups))
      store_group<WHOLE>(static_cast<T*>(p.h) + row * p.ldh, g * GROUP, cols, t, team, pack<T>(v[k]));
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
      if (PATH == ANY || g < groups)
        store_group<WHOLE>(static_cast<T*>(p.y) + row * p.ldy, g * GROUP, cols, t, team, pack<T>(v[k]));
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
      const uint2 out = quotients(v[k], scale);
      if (PATH == ANY || g < groups)
        store_bytes<WHOLE>(static_cast<uint8_t*>(p.y) + row * p.ldy, g * GROUP, cols, t, team,
                           out);
    }
  }
}

struct NormRing {
  NormParams p;
  int stages, teams;    // stages of a team
  uint32_t row_bytes;   // of one matrix
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;      // 3: only the first stages are ever filled
#endif
};

// The forward pass with dropout for many rows of a 16-bit type that lie FAST: as
// the gradient's ring (see there), since the generator's rounds leave the plain
// kernel too few threads on an SM to cover a row's wait (8192 x 8192 bf16: 100 us,
// here 95, 0.84 of the copy rate; 4096 x 8192 fp32, with half the rounds a byte,
// is faster without: 82 against 97). A team has its row in registers at its
// barrier, so the row's own stage is free then.
template <typename T, int VPT>
__global__ void __launch_bounds__(RING_THREADS, 1)
    add_rms_norm_ring_kernel(const __grid_constant__ NormRing q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ float box[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const NormParams& p = q.p;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const int inputs = p.residual ? 2 : 1;
  const uint32_t stage_bytes = inputs * q.row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.teams * q.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    aborted = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x % team, which = threadIdx.x / team;
  const RingRows rows = ring_rows(p.rows, q.teams, which);
  if (rows.count == 0) return;
  const uint32_t stage0 = smem_addr(ring) + which * q.stages * stage_bytes;
  auto full = [&](int s) { return smem_addr(&bars[which * q.stages + s]); };
  auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
    if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
    const int64_t row = rows.first + k * rows.step;
    const uint32_t dst = stage0 + s * stage_bytes;
    mbar_arrive_expect_tx(full(s), stage_bytes);
    bulk_load_1d(dst, static_cast<const T*>(p.x) + row * p.ldx, q.row_bytes, full(s));
    if (p.residual)
      bulk_load_1d(dst + q.row_bytes, static_cast<const T*>(p.residual) + row * p.ldr, q.row_bytes,
                   full(s));
  };
  if (t == 0)
    for (int k = 0; k < q.stages && k < rows.count; ++k) fetch(k, k);
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  Raw<T> wr[VPT] = {};
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (j * team + t < groups) wr[j] = static_cast<const Raw<T>*>(p.weight)[j * team + t];
  int s = 0, turn = 0;
  uint32_t ph = 0;
  int64_t k = 0;
  for (; k < rows.count; ++k, turn ^= 1) {
    const int64_t row = rows.first + k * rows.step;
    uint64_t counter[VPT];
    uint32_t words[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      counter[j] = first + static_cast<uint64_t>(row) * groups + j * team + t;
    philox(counter, seed, words);
    bool ok = __all_sync(0xffffffffu, ring_wait(full(s), ph, wd));
    const uint8_t* stage = ring + (which * q.stages + s) * stage_bytes;
    const Raw<T>* x = reinterpret_cast<const Raw<T>*>(stage) + t;
    const Raw<T>* res = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
    Raw<T>* h = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.h) + row * p.ldh) + t;
    float v[VPT][GROUP];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * team + t < groups) {
        unpack(x[j * team], v[j]);
        drop_by(p.drop, reinterpret_cast<const uint32_t(&)[1][4]>(words[j]),
                reinterpret_cast<float(&)[1][GROUP]>(v[j]));
        if (p.residual) {
          float r[GROUP];
          unpack(res[j * team], r);
#pragma unroll
          for (int i = 0; i < GROUP; ++i) v[j][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) sum = fmaf(v[j][i], v[j][i], sum);
        if (p.h) h[j * team] = pack<T>(v[j]);
      }
    }
    sum = ring_sum(sum, which, team, box[turn], &ok);
    if (!ok) break;
    if (t == 0 && k + q.stages < rows.count) fetch(k + q.stages, s);   // the row is in registers
    const float r = rsqrtf(sum / static_cast<float>(cols) + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r;
    Raw<T>* y = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.y) + row * p.ldy) + t;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * team + t < groups) {
        float w[GROUP];
        unpack(wr[j], w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) v[j][i] = v[j][i] * r * w[i];
        y[j * team] = pack<T>(v[j]);
      }
    }
    if (++s == q.stages) {
      s = 0;
      ph ^= 1;
    }
  }
  // Given up: the copies under way land before the CTA ends.
  if (k < rows.count && t == 0)
    for (int64_t j = k; j < rows.count && j < k + q.stages; ++j)
      wait_drain(full(static_cast<int>(j % q.stages)), static_cast<uint32_t>(j / q.stages) & 1);
}

// ------------------------------------------------------------ backward

struct NormGradParams {
  const void *dy, *dh, *h, *weight;    // dh may be NULL
  const float* rstd;
  void *dx, *dres;                     // dres may be NULL
  float* partial;                      // dweight partials, one row of whole groups a block; NULL: no dweight
  int64_t lddy, lddh, ldh, lddx, lddres;
  int64_t rows;
  int cols;
  int team;
  Dropout drop;
};

// Persistent: a team takes rows blockIdx * teams + team, + all teams of the
// grid, and keeps its columns' share of dweight in registers; a block leaves
// one partial row, and dweight_kernel adds those in block order. So dweight
// has the same bits on every run, whatever the timing.
template <typename T, Path PATH, int VPT, int MOST>
__global__ void __launch_bounds__(MOST, 1)
    add_rms_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ SumMax box[2][32];
  extern __shared__ __align__(16) float share[];   // where a team is a warp: their shares of dweight
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, teams = blockDim.x / team;
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  constexpr bool WHOLE = PATH != ANY;
  const Row<T> weight = row_of<T>(p.weight, 0, 1, 0);
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  float acc[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP; ++i) acc[k][i] = 0.0f;

  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * teams + threadIdx.x / team; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * teams, turn ^= 1) {
    const Row<T> dy = row_of<T>(p.dy, row, p.rows, p.lddy), h = row_of<T>(p.h, row, p.rows, p.ldh),
                 dh = row_of<T>(p.dh, row, p.rows, p.lddh);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int c = (k * team + t) * GROUP;
        if (c < cols) {
          prefetch_group(dy, c);
          prefetch_group(h, c);
          if (p.dh) prefetch_group(dh, c);
        }
      }
    }
    Raw<T> yr[VPT], hr[VPT], dr[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        yr[k] = load_group<WHOLE>(dy, g * GROUP, cols);
        hr[k] = load_group<WHOLE>(h, g * GROUP, cols);
        if (p.dh) dr[k] = load_group<WHOLE>(dh, g * GROUP, cols);
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
        unpack(load_group<WHOLE>(weight, g * GROUP, cols), w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          const float ni = n[i] * r;
          acc[k][i] = fmaf(a[i], ni, acc[k][i]);
          s.sum = fmaf(a[i] * w[i], ni, s.sum);
        }
      }
    }
    const float c = reduce_team<false>(s, team / 32, box[turn]).sum / static_cast<float>(cols);
    const float rc = r * c;
    float d[VPT][GROUP];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], n[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], n);
        unpack(load_group<WHOLE>(weight, g * GROUP, cols), w);
        unpack(dr[k], d[k]);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) d[k][i] = fmaf(r, a[i] * w[i] - n[i] * rc, d[k][i]);
      }
      if (p.dres && (PATH == ANY || g < groups))
        store_group<WHOLE>(static_cast<T*>(p.dres) + row * p.lddres, g * GROUP, cols, t, team,
                           pack<T>(d[k]));
    }
    if (PATH == DROP || (PATH == ANY && p.drop.on)) {
      uint64_t counter[VPT];
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        counter[k] = first + static_cast<uint64_t>(row) * groups + k * team + t;
      drop_groups(p.drop, seed, counter, d);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (PATH == ANY || g < groups)
        store_group<WHOLE>(static_cast<T*>(p.dx) + row * p.lddx, g * GROUP, cols, t, team, pack<T>(d[k]));
    }
  }
  if (p.partial) leave_partial(acc, share, p.partial, groups, team, teams, threadIdx.x / team, t);
}

// The same for many rows that lie FAST: the rows come through a ring in shared
// memory by bulk copies, so that the next rows are on their way while a team
// waits for its row's sum (loaded straight into registers the rows of an SM stop
// at each such wait: 8192 x 8192 bf16 took 124 us, with dropout 171, against 87
// and 107: 0.91 and 0.93 of the copy rate). RING_WARPS warps form teams of `team`
// threads; row k of a CTA goes to its team k % teams, each of which has its own
// stages. There is no producer warp: a team's barrier of a row says that all of it
// is done with the row before, whose stage one thread then fills again. (With such
// a warp the CTA's 17 warps count as 20, which leaves 96 registers a thread instead
// of 128, and four groups a thread spill.) Both passes over a row read it from the
// ring: holding it in registers in between cost more (130 us) than the second
// reading.
struct NormGradRing {
  NormGradParams p;
  int stages, teams;    // stages of a team
  uint32_t row_bytes;   // of one matrix
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;      // 3: only the first stages are ever filled
#endif
};

template <typename T, bool ON, int VPT>
__global__ void __launch_bounds__(RING_THREADS, 1)
    add_rms_norm_grad_ring_kernel(const __grid_constant__ NormGradRing q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ float box[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const NormGradParams& p = q.p;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const int inputs = p.dh ? 3 : 2;
  const uint32_t stage_bytes = inputs * q.row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.teams * q.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    aborted = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x % team, which = threadIdx.x / team;
  const RingRows rows = ring_rows(p.rows, q.teams, which);

  Pair acc[VPT][GROUP / 2];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP / 2; ++i) acc[k][i] = 0;

  if (rows.count > 0) {
    const uint32_t stage0 = smem_addr(ring) + which * q.stages * stage_bytes;
    auto full = [&](int s) { return smem_addr(&bars[which * q.stages + s]); };
    // One thread of the team fetches row k into stage s.
    auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
      if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
      const int64_t row = rows.first + k * rows.step;
      const uint32_t dst = stage0 + s * stage_bytes;
      mbar_arrive_expect_tx(full(s), stage_bytes);
      bulk_load_1d(dst, static_cast<const T*>(p.dy) + row * p.lddy, q.row_bytes, full(s));
      bulk_load_1d(dst + q.row_bytes, static_cast<const T*>(p.h) + row * p.ldh, q.row_bytes, full(s));
      if (p.dh)
        bulk_load_1d(dst + 2 * q.row_bytes, static_cast<const T*>(p.dh) + row * p.lddh, q.row_bytes,
                     full(s));
    };
    if (t == 0)
      for (int k = 0; k < q.stages && k < rows.count; ++k) fetch(k, k);
    const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
    Raw<T> wr[VPT] = {};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (j * team + t < groups) wr[j] = static_cast<const Raw<T>*>(p.weight)[j * team + t];
    int s = 0, turn = 0, before = q.stages - 1;   // this row's stage, and the one before's
    uint32_t ph = 0;
    float next_r = p.rstd[rows.first];
    int64_t k = 0;
    for (; k < rows.count; ++k, turn ^= 1) {
      const int64_t row = rows.first + k * rows.step;
      const float r = next_r;
      if (k + 1 < rows.count) next_r = p.rstd[row + rows.step];
      // The mask needs nothing of the row: its rounds fill the wait for it.
      uint32_t words[VPT][4];
      if (ON) {
        uint64_t counter[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          counter[j] = first + static_cast<uint64_t>(row) * groups + j * team + t;
        philox(counter, seed, words);
      }
      bool ok = __all_sync(0xffffffffu, ring_wait(full(s), ph, wd));
      const uint8_t* stage = ring + (which * q.stages + s) * stage_bytes;
      const Raw<T>* dy = reinterpret_cast<const Raw<T>*>(stage) + t;
      const Raw<T>* h = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
      const Raw<T>* dh = reinterpret_cast<const Raw<T>*>(stage + 2 * q.row_bytes) + t;
      // acc += dy h r, and the sum of dy weight h
      const Pair r2 = pair_of(r, r);
      Pair sums = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j * team + t < groups) {
          Pair a[GROUP / 2], n[GROUP / 2], w[GROUP / 2];
          unpack(dy[j * team], a);
          unpack(h[j * team], n);
          unpack(wr[j], w);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            const Pair an = mul2(a[i], n[i]);
            acc[j][i] = fma2(an, r2, acc[j][i]);
            sums = fma2(an, w[i], sums);
          }
        }
      }
      const float sum =
          ring_sum(values_of(sums).x + values_of(sums).y, which, team, box[turn], &ok);
      if (!ok) break;
      // The whole team has been in the sum, so it has done with the row before.
      if (t == 0 && k > 0 && k - 1 + q.stages < rows.count) fetch(k - 1 + q.stages, before);
      // dres = dh + r dy weight - h r^2 mean(dy weight h r)
      const float m = -r * r * (r * sum / static_cast<float>(cols));
      const Pair m2 = pair_of(m, m);
      Raw<T>* dres = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dres) + row * p.lddres) + t;
      Raw<T>* dx = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dx) + row * p.lddx) + t;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j * team + t < groups) {
          Pair a[GROUP / 2], n[GROUP / 2], w[GROUP / 2], e[GROUP / 2];
          unpack(dy[j * team], a);
          unpack(h[j * team], n);
          unpack(wr[j], w);
          Raw<T> dr = {};
          if (p.dh) dr = dh[j * team];
          unpack(dr, e);
          float d[1][GROUP];
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            e[i] = fma2(n[i], m2, fma2(mul2(a[i], w[i]), r2, e[i]));
            d[0][2 * i] = values_of(e[i]).x;
            d[0][2 * i + 1] = values_of(e[i]).y;
          }
          if (p.dres) dres[j * team] = pack<T>(d[0]);
          if (ON) drop_by(p.drop, reinterpret_cast<const uint32_t(&)[1][4]>(words[j]), d);
          dx[j * team] = pack<T>(d[0]);
        }
      }
      before = s;
      if (++s == q.stages) {
        s = 0;
        ph ^= 1;
      }
    }
    // Given up: the copies under way land before the CTA ends.
    if (k < rows.count && t == 0)
      for (int64_t j = k; j < rows.count && j < k + q.stages - (k > 0); ++j)
        wait_drain(full(static_cast<int>(j % q.stages)), static_cast<uint32_t>(j / q.stages) & 1);
  }
  if (!p.partial) return;
  float mine[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP / 2; ++i) {
      mine[k][2 * i] = values_of(acc[k][i]).x;
      mine[k][2 * i + 1] = values_of(acc[k][i]).y;
    }
  __syncthreads();   // all teams have done with the ring
  static_assert(RING_THREADS * VPT * GROUP * sizeof(float) <= RING_BYTES, "the teams' rows fit the ring");
  leave_partial(mine, reinterpret_cast<float*>(ring), p.partial, groups, team, q.teams, which, t);
}

struct DweightParams {
  const float* partial;
  int blocks, cols, pitch;
  void* dweight;
};

// dweight[c] = the sum of the blocks' partial rows.
template <typename T>
__global__ void __launch_bounds__(DW_THREADS)
    dweight_kernel(const __grid_constant__ DweightParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  column_sums(p.partial, blockIdx.x, p.blocks, p.cols, p.pitch,
              [&](int c, float sum) { static_cast<T*>(p.dweight)[c] = round_to(sum, T()); });
}

// ------------------------------------------------------------ dropout alone

struct DropoutParams {
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int64_t rows;
  int cols;
  int64_t groups;      // FLAT: of the whole matrix; else of a row
  int row_threads;     // not FLAT: threads of a row, a power of two
  Dropout drop;
};

constexpr int DROP_THREADS = 256, DROP_VPT = 2;

// FLAT: rows follow one another without gaps in whole groups, so the matrix is
// one run of groups and no row has to be found. ON: p > 0.
template <typename T, bool ON>
__global__ void __launch_bounds__(DROP_THREADS) dropout_flat_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (DROP_THREADS * DROP_VPT) + threadIdx.x;
  Raw<T> raw[DROP_VPT] = {};
  float v[DROP_VPT][GROUP];
  uint64_t counter[DROP_VPT];
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) raw[k] = static_cast<const Raw<T>*>(p.x)[g];
    counter[k] = first + g;
  }
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) unpack(raw[k], v[k]);
  if (ON) drop_groups(p.drop, seed, counter, v);
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) static_cast<Raw<T>*>(p.y)[g] = pack<T>(v[k]);
  }
}

// Any rows: row_threads threads walk one, DROP_THREADS / row_threads rows a block.
template <typename T>
__global__ void __launch_bounds__(DROP_THREADS) dropout_rows_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  const int team = p.row_threads, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (DROP_THREADS / team) + threadIdx.x / team;
  const bool there = row < p.rows;
  const Row<T> x = row_of<T>(p.x, there ? row : 0, p.rows, p.ldx);
  T* y = static_cast<T*>(p.y) + (there ? row : 0) * p.ldy;
  const int groups = static_cast<int>(p.groups);
  for (int g0 = 0; g0 < groups; g0 += team) {   // whole warps stay together for the stores
    const int g = g0 + t;
    const bool mine = there && g < groups;
    Raw<T> raw = {};
    if (mine) raw = load_group<false>(x, column_of(g, groups, p.cols), p.cols);
    float v[1][GROUP];
    unpack(raw, v[0]);
    const uint64_t counter[1] = {first + static_cast<uint64_t>(row) * groups + g};
    if (p.drop.on) drop_groups(p.drop, seed, counter, v);
    store_group<false>(y, column_of(mine ? g : groups, groups, p.cols), p.cols, t, team, pack<T>(v[0]));
  }
}

}  // namespace gws
