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
  int type, channels;
  bool pairs;      // d's rows allow accesses of two elements
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
// the CUDA cores. `split` warps share DOT_ROWS channels, 16 bytes of K a lane and step: four rows of w at a
// time are enough bytes in flight, and a lane's 16 bytes of each token serve all four. Bound by w's bytes
// (one token x 4096 over 131072: 82 us, 6.5 TB/s; four 102).
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

// ------------------------------------------------------------ tensor cores

// This chip's tensor cores multiply 16-bit floats several times as fast as 8-bit integers, and an
// 8-bit integer is exact in fp16. So is a product of two in the fp32 accumulator, and the sum of 1024
// of them (2^10 * 2^14 = 2^24): the accumulator is handed over every 1024 of K, and the epilogue
// adds what it held in 32-bit integers.
//
// w's rows are A of the product, from tensor memory: converted on their way there from
// shared memory by warps of their own, they cost the shared memory 2 bytes of traffic each (in and
// out) instead of the 5 that a copy in fp16 there would (1 in, 1 out, 2 back and 2 out to the
// tensor cores, for the half that a CTA of a pair holds). a's rows, the tokens, are B: a small kernel
// writes them in fp16 first, once for all channels.
//
// A pair of CTAs has a tile of 256 channels x bn tokens, each its 128 channels as
// TMEM lanes. Tensor memory: two accumulators of bn columns, up to 160, and in what is left of its 512
// columns buffers of w, 128 x 128 in 64 columns each: three to seven. A buffer's way from its hand-over
// until it is seen free again (both CTAs' warps, the MMAs, and between the CTAs) takes the time of
// two stages' MMAs, which is why there have to be several.
//
// One warp issues all MMAs, and what it does beside that has to fit into their time: for 128 of K it
// polls the two operands' barriers and commits once, to w's buffer. That the tokens' stage of the same step
// is free again a warp of its own tells on, when it sees w's buffer free.
//
// Times in a graph: 8192 x 8192 over 8192 653 us (1.68 P operations a second, 0.87 of a bf16 product's
// rate; from 645 to 680 between chips), bound by how fast w's stages get into tensor memory, some 800 cycles
// a stage against some 720 of its MMAs. 64 x 4096 over 131072 103 us (w at 5.2 TB/s). Small products are bound by
// what comes one after the other: 64 x 4096 over 4096 takes 16 us, of which the tokens' kernel 3, set-up
// and first loads 3.5, a joined cut's end 2.5.

constexpr int BM = 128;              // channels of a CTA's tile
constexpr int BN_MAX = 160;          // tokens of a tile, at most
constexpr int BK = 128;              // K of a stage: one 128-byte swizzle row of 8-bit integers
constexpr int HALF_K = 64;           // of a stage: one 128-byte swizzle row of fp16
constexpr int UMMA_K = 16;
constexpr int ACC_BUFS = 2, MAX_W_BUFS = 7;
constexpr int W_COLS = BK / 2;       // TMEM columns of a buffer of w
constexpr int TMEM_COLS = 512;
__host__ __device__ constexpr int w_bufs(int bn) { return (TMEM_COLS - ACC_BUFS * bn) / W_COLS; }
static_assert(w_bufs(BN_MAX) >= 3 && w_bufs(32) <= MAX_W_BUFS, "tensor memory");
constexpr int CUT_STAGES = 1024 / BK;   // stages of one accumulator
// Warpgroups: producers, the MMA warp and the teller; two that convert; two of the epilogue.
constexpr int WARP_W = 0, WARP_MMA = 1, WARP_A = 2, WARP_TELL = 3, WARP_CONV0 = 4, CONV_WARPS = 8, WARP_EPI0 = WARP_CONV0 + CONV_WARPS,
              EPI_WARPS = 8;
constexpr int THREADS = (WARP_EPI0 + EPI_WARPS) * 32;
// Registers a thread at launch, and after the warpgroups have shared them out: the epilogue holds 80 sums.
constexpr int REGS_LAUNCH = 96, REGS_FEW = 72, REGS_EPI = 128;
static_assert(WARP_EPI0 * REGS_FEW + EPI_WARPS * REGS_EPI <= THREADS / 32 * REGS_LAUNCH, "registers of a block");
constexpr int MAX_STAGES = 12;
constexpr uint32_t W_STAGE = BM * BK;                  // 16 KB
constexpr uint32_t RING_ROOM = 222 * 1024;
constexpr int BAR_W_FULL = 0, BAR_W_EMPTY = BAR_W_FULL + MAX_STAGES, BAR_A_FULL = BAR_W_EMPTY + MAX_STAGES,
              BAR_A_EMPTY = BAR_A_FULL + MAX_STAGES, BAR_T_FULL = BAR_A_EMPTY + MAX_STAGES,
              BAR_T_EMPTY = BAR_T_FULL + MAX_W_BUFS, BAR_ACC_FULL = BAR_T_EMPTY + MAX_W_BUFS,
              BAR_ACC_EMPTY = BAR_ACC_FULL + ACC_BUFS, BAR_DRAIN = BAR_ACC_EMPTY + ACC_BUFS,
              NUM_BARS = BAR_DRAIN + 1;
constexpr uint32_t OFF_SCALES = RING_ROOM;              // the tokens' scales, for each epilogue warp
constexpr uint32_t OFF_BAR = OFF_SCALES + EPI_WARPS * (BN_MAX / 2) * 4;
constexpr uint32_t OFF_TMEM = OFF_BAR + NUM_BARS * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t SMEM_BYTES = OFF_ABORT + 4 + 1024;   // + slack to align the base
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KiB per-CTA shared memory");

__host__ __device__ constexpr uint32_t a_stage(int bn) { return static_cast<uint32_t>(bn / 2) * BK * 2; }

// Arrivals that fill a buffer of w: a warpgroup's warps that convert, of both CTAs, and both CTAs' tellers, which
// so have seen the step before in the buffer go before the next can. Without theirs a teller that is late by
// the time of all buffers would find the barrier's other parity, and wait for a phase that cannot come: the tokens'
// ring has more stages than there are buffers, and does not hold the next step back.
constexpr int TELLERS = 2, T_FULL_ARRIVALS = CONV_WARPS + TELLERS;

// Stages of the two rings. The tokens' are freed later than w's, which take what those leave.
struct Rings {
  int bufs, w_stages, a_stages;
};
__host__ __device__ constexpr Rings rings_of(int bn) {
  const int bufs = w_bufs(bn), a_stages = bufs + 2 < 6 ? 6 : bufs + 2;
  const int room = static_cast<int>((RING_ROOM - a_stages * a_stage(bn)) / W_STAGE);
  return {bufs, room < MAX_STAGES ? room : MAX_STAGES, a_stages};
}
// The two warpgroups that convert take w's stages in turn. One of them, at step i, has seen the buffer of step i - 2 - bufs free, so
// all steps up to that have been converted, by the other as well; with these many stages the one before in its own
// stage is among them.
constexpr bool rings_fit() {
  for (int bn = 32; bn <= BN_MAX; bn += 32) {
    const Rings r = rings_of(bn);
    if (r.w_stages < r.bufs + 2 || r.a_stages > MAX_STAGES || r.bufs > MAX_W_BUFS) return false;
  }
  return true;
}
static_assert(rings_fit(), "a wait by parity is at most one phase behind");

struct Params {
  CUtensorMap tmW, tmA;
  int tokens, channels, stages;   // stages of K
  int bn;                         // tokens of a tile, a multiple of 32
  int w_stages, a_stages;         // of the two rings in shared memory
  int bufs;                       // w_bufs(bn)
  int tiles_m, tiles_n;           // tiles of tokens, of channels
  int whole;                      // tiles of their own; of those after them K is cut
  int splits;                     // into so many units, all of which run at once
  int* total;                     // [cut tile][CTA of the pair][token][channel], zero at launch: the cuts' sums
  uint32_t* arrived;              // [cut tile][CTA of the pair][epilogue warp], zero at launch
  Output out;
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;                // 3: w's producer brings nothing; 4: the tellers are late; 5: the MMA warp gives up
#endif
};

// A unit of work: a tile, or a cut of its K.
struct Unit {
  int n0, m0;      // first channel of the pair, first token
  int cut_tile;    // the tile's number among those whose K is cut, or -1
  int s0, s1;      // stages of K
};

constexpr int GROUP_N = 8;   // tiles walk 8 tiles of channels down, then step on in the tokens (L2 reuse)

__device__ __forceinline__ bool unit_of(const Params& p, int u, Unit& w) {
  int t = u;
  w.cut_tile = -1;
  w.s0 = 0;
  w.s1 = p.stages;
  if (u >= p.whole) {
    w.cut_tile = (u - p.whole) / p.splits;
    t = p.whole + w.cut_tile;
    if (t >= p.tiles_m * p.tiles_n) return false;
    const int cut = u - p.whole - w.cut_tile * p.splits;
    w.s0 = static_cast<int>(static_cast<int64_t>(cut) * p.stages / p.splits);
    w.s1 = static_cast<int>(static_cast<int64_t>(cut + 1) * p.stages / p.splits);
  }
  const int group = t / (GROUP_N * p.tiles_m), first = group * GROUP_N;
  const int r = t - group * GROUP_N * p.tiles_m;
  const int high = min(GROUP_N, p.tiles_n - first);
  w.m0 = r / high * p.bn;
  w.n0 = (first + r % high) * 2 * BM;
  return true;
}

// Four 8-bit integers in fp16, in the order 0 2 1 3: a byte's offset value b + 128 under the
// exponent of 1024 is 1152 + b, and subtracting 1152 is exact. Both operands are laid out in this
// order of K, which a sum does not see.
__device__ __forceinline__ uint2 to_fp16(uint32_t w) {
  const uint32_t even = (w & 0x00FF00FFu) ^ 0x64806480u, odd = (w >> 8 & 0x00FF00FFu) ^ 0x64806480u;
  const uint32_t shift = 0x64806480u;   // 1152, 1152
  const __half2 s = *reinterpret_cast<const __half2*>(&shift);
  const __half2 e = __hsub2(*reinterpret_cast<const __half2*>(&even), s);
  const __half2 o = __hsub2(*reinterpret_cast<const __half2*>(&odd), s);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&e), *reinterpret_cast<const uint32_t*>(&o));
}

// Returns how many stages it has armed.
__device__ __forceinline__ uint32_t produce_w(const Params& p, uint32_t sbase, uint32_t rank, const Watchdog& wd) {
  auto full = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_W_FULL + s); };
  auto empty = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_W_EMPTY + s); };
  const uint32_t stages = p.w_stages;
  uint32_t s = 0, ph = 0, g = 0;
  Unit w;
#ifdef GEMM_WS_DEBUG
  if (p.debug_fault == 3) return 0;   // injected fault: no stage ever fills
#endif
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2)
    for (int st = w.s0; st < w.s1; ++st) {
      if (!wait_suspended(empty(s), ph ^ 1, wd)) return g;
      mbar_arrive_expect_tx(full(s), W_STAGE);
      tma_load_3d(sbase + s * W_STAGE, &p.tmW, full(s), st * BK, w.n0 + static_cast<int>(rank) * BM, 0);
      ++g;
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
  return g;
}

// After an abort, whichever warp gave up, and when nothing more is issued: the copies of the stages armed last land
// before the CTA ends. `full`: the first stage's barrier.
__device__ __forceinline__ void drain(uint32_t full, uint32_t stages, uint32_t g) {
  for (uint32_t j = g > stages ? g - stages : 0; j < g; ++j) wait_drain(full + 8 * (j % stages), (j / stages) & 1);
}

__device__ __forceinline__ uint32_t produce_a(const Params& p, uint32_t sbase, uint32_t rank, const Watchdog& wd) {
  auto full = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_A_FULL + s); };
  auto empty = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_A_EMPTY + s); };
  const uint32_t stages = p.a_stages, bytes = a_stage(p.bn), ring = sbase + p.w_stages * W_STAGE;
  const bool leader = rank == 0;   // arms full[s] for the pair
  uint32_t s = 0, ph = 0, g = 0;
  Unit w;
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2)
    for (int st = w.s0; st < w.s1; ++st) {
      if (!wait_suspended(empty(s), ph ^ 1, wd)) return g;
      if (leader) mbar_arrive_expect_tx(full(s), 2 * bytes);
      const uint32_t bar = mapa_shared(full(s), 0u), dst = ring + s * bytes;
      const int row = w.m0 + static_cast<int>(rank) * (p.bn / 2);
      tma_load_3d_pair(dst, &p.tmA, bar, st * BK, row, 0);
      tma_load_3d_pair(dst + bytes / 2, &p.tmA, bar, st * BK + HALF_K, row, 0);
      ++g;
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
  return g;
}

// A ring's place and phase, some steps on.
__device__ __forceinline__ void advance(uint32_t& at, uint32_t& phase, uint32_t by, uint32_t size) {
  at += by;
  if (at >= size) {
    at -= size;
    phase ^= 1;
  }
}

// A warp's 32 channels of every other stage, from shared memory to tensor memory. The two
// warpgroups take the stages in turn: what a stage costs a warp besides its conversions (the waits and
// arrivals) so has the time of two.
__device__ __forceinline__ void convert(const Params& p, uint32_t sbase, const uint8_t* smem, uint32_t tmem,
                                        int warp, const Watchdog& wd) {
  auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
  const int lane = threadIdx.x & 31, row = 32 * (warp & 3) + lane;
  const uint32_t mine = tmem + ACC_BUFS * p.bn + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  const uint32_t t_full = mapa_shared(bar(BAR_T_FULL), 0u);   // the leader's
  const uint32_t stages = p.w_stages, bufs = p.bufs;
  uint32_t next = (warp - WARP_CONV0) / 4;                    // this warpgroup's next step of all units'
  uint32_t s = next, ph = 0, t = next, tph = 0, end = 0;
  Unit w;
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2)
    for (end += w.s1 - w.s0; static_cast<int>(end - next) > 0; next += 2) {
      if (!warp_wait_cta(bar(BAR_W_FULL + s), ph, wd)) return;
      const uint8_t* from = smem + s * W_STAGE + row * BK;
      uint4 raw[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)   // the TMA's 128-byte swizzle
        raw[c] = *reinterpret_cast<const uint4*>(from + ((c ^ (row & 7)) << 4));
      bool free = mbar_test_wait(bar(BAR_T_EMPTY + t), tph ^ 1);   // mostly it is by now
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 r = raw[4 * half + c];
          const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 two = to_fp16(x[i]);
            v[8 * c + 2 * i] = two.x;
            v[8 * c + 2 * i + 1] = two.y;
          }
        }
        if (half == 0) {
          __syncwarp();   // the stage has been read
          if (lane == 0) mbar_arrive(bar(BAR_W_EMPTY + s));
          if (!__all_sync(0xffffffffu, free) && !warp_wait_cta(bar(BAR_T_EMPTY + t), tph ^ 1, wd)) return;
          tc_fence_after_sync();
        }
        tmem_st_32x32b_x32(mine + t * W_COLS + half * (W_COLS / 2), v);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(t_full + 8 * t);
      advance(s, ph, 2, stages);
      advance(t, tph, 2, bufs);
    }
}

// Frees the tokens' stages: the MMAs that have read w's buffer of a step have read the step's tokens. The
// arrival on the buffer's own barrier holds its next step back until this one has been seen (see
// T_FULL_ARRIVALS); in time it is early, as the buffer is still to be filled then.
__device__ __forceinline__ void tell(const Params& p, uint32_t sbase, const Watchdog& wd) {
  const uint32_t bufs = p.bufs, t_full = mapa_shared(sbase + OFF_BAR + 8 * BAR_T_FULL, 0u);   // the leader's
  const bool first = (threadIdx.x & 31) == 0;
  uint32_t s = 0, t = 0, tph = 0;
  Unit w;
  if (first)
    for (uint32_t i = 0; i < bufs; ++i) mbar_arrive_cluster_relaxed(t_full + 8 * i);   // none before the first
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2)
    for (int st = w.s0; st < w.s1; ++st) {
#ifdef GEMM_WS_DEBUG
      if (p.debug_fault == 4)   // injected delay: many steps' time
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 20000ull;) __nanosleep(1000);
#endif
      if (!warp_wait_cta(sbase + OFF_BAR + 8 * (BAR_T_EMPTY + t), tph, wd)) return;
      if (first) {
        mbar_arrive(sbase + OFF_BAR + 8 * (BAR_A_EMPTY + s));
        mbar_arrive_cluster_relaxed(t_full + 8 * t);
      }
      if (++t == bufs) {
        t = 0;
        tph ^= 1;
      }
      if (++s == static_cast<uint32_t>(p.a_stages)) s = 0;
    }
}

// The whole warp walks, so that addresses and descriptors stay in uniform registers; one lane waits and
// issues. Once a wait has given up, the rest of the walk does nothing.
__device__ __forceinline__ void issue(const Params& p, uint32_t sbase, uint32_t tmem, const Watchdog& wd) {
  auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
  constexpr uint16_t BOTH = 0x3;
  const uint32_t bytes = a_stage(p.bn), ring = sbase + p.w_stages * W_STAGE;
  const uint32_t idesc = idesc_f16_f32(2 * BM, p.bn);
  const bool mine = elect_one();
  const uint32_t bufs = p.bufs;
  uint32_t s = 0, ph = 0, t = 0, tph = 0, handed = 0;
  bool ok = true, issued = false;
  Unit w;
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2)
    for (int first = w.s0; first < w.s1; first += CUT_STAGES, ++handed) {
      const uint32_t b = handed & 1;
      if (mine && ok) {
        ok = wait_inline(bar(BAR_ACC_EMPTY + b), ((handed >> 1) & 1) ^ 1, wd);
        tc_fence_after_sync();
      }
      const uint32_t d = tmem + b * p.bn;
      const int end = min(first + CUT_STAGES, w.s1);
      for (int st = first; st < end; ++st) {
        const uint32_t b_addr = ring + s * bytes, from = tmem + ACC_BUFS * p.bn + t * W_COLS;
#ifdef GEMM_WS_DEBUG
        if (mine && ok && p.debug_fault == 5 && st == w.s0 + 1) {   // injected fault: it gives up while all others work
          ok = false;
          *wd.abort = 1;
          atomicExch(wd.status, STATUS_TIMEOUT);
        }
#endif
        if (mine && ok) {
          ok = wait_inline(bar(BAR_A_FULL + s), ph, wd) &&
               wait_inline(bar(BAR_T_FULL + t), tph, wd);
          if (ok) {
            tc_fence_after_sync();
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              umma_16bit_pair_ts(d, from + k * (UMMA_K / 2),
                                 sdesc_kmajor_sw128(b_addr + (k >= 4 ? bytes / 2 : 0) + (k & 3) * UMMA_K * 2),
                                 idesc, st != first || k != 0 ? 1u : 0u);
            umma_commit_pair(bar(BAR_T_EMPTY + t), BOTH);
            issued = true;
          }
        }
        if (++t == bufs) {
          t = 0;
          tph ^= 1;
        }
        if (++s == static_cast<uint32_t>(p.a_stages)) {
          s = 0;
          ph ^= 1;
        }
      }
      if (mine && ok) umma_commit_pair(bar(BAR_ACC_FULL + b), BOTH);
    }
  if (issued) {
    // Every MMA issued has finished once this arrives (also after an abort).
    umma_commit_pair(bar(BAR_DRAIN), static_cast<uint16_t>(0x1));
    wait_drain(bar(BAR_DRAIN), 0);
  }
  __syncwarp();
}

// 16 tokens of a thread's channel. In 16 bits neighbouring lanes exchange two tokens' values at a
// time, so that each stores two channels of one of them.
__device__ __forceinline__ void store_tokens(const Output& o, int m, int tokens, int n, bool both,
                                             const int (&sum)[16], const float4* scales, float w_scale,
                                             float bias) {
  asm volatile("" ::: "memory");   // nothing of this ahead: the other sums fill the registers
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = scales[i];
    v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fmaf(static_cast<float>(sum[i]) * v[i], w_scale, bias);
  const int64_t at = static_cast<int64_t>(m) * o.ldd + n;
  if (o.type == OUT_F32) {
    float* d = static_cast<float*>(o.d) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i, d += o.ldd)
      if (n < o.channels && m + i < tokens) *d = v[i];
    return;
  }
  const bool odd = threadIdx.x & 1;
  const uint32_t pick = odd ? 0x3276 : 0x5410;   // even lanes: both channels' token i, odd ones: token i + 1
  uint16_t* d = static_cast<uint16_t*>(o.d) + at + (odd ? o.ldd - 1 : 0);
#pragma unroll
  for (int i = 0; i < 16; i += 2, d += 2 * o.ldd) {
    uint32_t own;
    if (o.type == OUT_F16) {
      const __half2 h = __floats2half2_rn(v[i], v[i + 1]);
      own = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      own = pack_bf16x2(v[i], v[i + 1]);
    }
    const uint32_t two = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), pick);
    if (m + i + odd >= tokens) continue;
    if (both) {
      *reinterpret_cast<uint32_t*>(d) = two;
    } else {   // an unaligned row, or the last channel
      const int c = n - odd;
      if (c < o.channels) d[0] = static_cast<uint16_t>(two);
      if (c + 1 < o.channels) d[1] = static_cast<uint16_t>(two >> 16);
    }
  }
}

// A thread has one channel, and half of the tile's tokens in registers.
__device__ __forceinline__ void epilogue(const Params& p, uint32_t sbase, uint8_t* smem, uint32_t tmem,
                                         uint32_t rank, int warp, const Watchdog& wd) {
  auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
  constexpr int BLOCKS = BN_MAX / 2 / 16;   // of 16 tokens
  const int lane = threadIdx.x & 31, q = warp & 3, hf = (warp - WARP_EPI0) / 4;
  const int col0 = hf * (p.bn / 2), blocks = p.bn / 32;
  float* scales = reinterpret_cast<float*>(smem + OFF_SCALES) + (warp - WARP_EPI0) * (BN_MAX / 2);
  uint32_t handed = 0;
  Unit w;
  for (int u = blockIdx.x / 2; unit_of(p, u, w); u += gridDim.x / 2) {
    int sum[BLOCKS][16];
    // what the tile's end needs, loaded ahead
    const int in_cta = 32 * q + lane, n = w.n0 + static_cast<int>(rank) * BM + in_cta, m = w.m0 + col0;
    const bool there = n < p.channels;
    const float w_scale = there ? p.out.w_scales[n] : 0.0f, bias = there && p.out.bias ? p.out.bias[n] : 0.0f;
    __syncwarp();   // the tile before has been stored
    for (int i = lane; i < p.bn / 2; i += 32) scales[i] = m + i < p.tokens ? p.out.a_scales[m + i] : 0.0f;
    __syncwarp();
    for (int first = w.s0; first < w.s1; first += CUT_STAGES, ++handed) {
      const uint32_t b = handed & 1;
      if (!warp_wait_cta(bar(BAR_ACC_FULL + b), (handed >> 1) & 1, wd)) return;
      tc_fence_after_sync();
      const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + b * p.bn + col0;
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        if (k >= blocks) continue;
        uint32_t v[16];
        tmem_ld_32x32b_x16(from + 16 * k, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = __float2int_rn(__uint_as_float(v[i]));
          sum[k][i] = first == w.s0 ? x : sum[k][i] + x;
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        const uint32_t e = bar(BAR_ACC_EMPTY + b);
        if (rank == 0)
          mbar_arrive(e);
        else
          mbar_arrive_cluster_relaxed(mapa_shared(e, 0));
      }
    }
    if (w.cut_tile >= 0) {
      // The cuts' sums meet in the workspace, which is zero at launch: integers, so in any order.
      // The warp that arrives last takes what is there.
      const int64_t which = static_cast<int64_t>(w.cut_tile) * 2 + rank;
      int* total = p.total + (which * p.bn + col0) * BM + in_cta;
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        if (k >= blocks) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) atomicAdd(total + (16 * k + i) * BM, sum[k][i]);
      }
      __threadfence();
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0) before = atomicAdd(p.arrived + which * EPI_WARPS + (warp - WARP_EPI0), 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before + 1 != static_cast<uint32_t>(p.splits)) continue;
      __threadfence();
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        if (k >= blocks) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[k][i] = __ldcg(total + (16 * k + i) * BM);
      }
    }
    const bool both = p.out.pairs && (n | 1) < p.channels;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
      if (k >= blocks) continue;
      store_tokens(p.out, m + 16 * k, p.tokens, n, both, sum[k], reinterpret_cast<const float4*>(scales) + 4 * k, w_scale, bias);
    }
  }
}

__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
  if (warp == WARP_W && lane == 0) {
    auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(bar(BAR_W_FULL + s), 1);
      mbar_init(bar(BAR_W_EMPTY + s), CONV_WARPS / 2);
      mbar_init(bar(BAR_A_FULL + s), 1);
      mbar_init(bar(BAR_A_EMPTY + s), 1);
    }
    for (int t = 0; t < MAX_W_BUFS; ++t) {
      mbar_init(bar(BAR_T_FULL + t), T_FULL_ARRIVALS);   // of each CTA 4 that convert, and the teller
      mbar_init(bar(BAR_T_EMPTY + t), 1);
    }
    for (int b = 0; b < ACC_BUFS; ++b) {
      mbar_init(bar(BAR_ACC_FULL + b), 1);
      mbar_init(bar(BAR_ACC_EMPTY + b), 2 * EPI_WARPS);
    }
    mbar_init(bar(BAR_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tmW);
    prefetch_tensormap(&p.tmA);
  }
  if (warp == WARP_MMA) {
    tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  // The set-up above, and w's way into tensor memory, overlap the end of the kernel that writes the tokens in
  // fp16: that one has waited for everything before it, and does not touch w. Who needs its results waits.
  if (threadIdx.x == 0) grid_launch_dependents();

  uint32_t loaded = 0;   // stages, of the two producers
  if (warp >= WARP_EPI0) {
    more_registers<REGS_EPI>();
    grid_dependency_wait();
    epilogue(p, sbase, smem, tmem, rank, warp, wd);
  } else {
    fewer_registers<REGS_FEW>();
    if (warp >= WARP_CONV0) {
      convert(p, sbase, smem, tmem, warp, wd);
    } else if (warp == WARP_W) {
      if (lane == 0) loaded = produce_w(p, sbase, rank, wd);
    } else if (warp == WARP_A) {
      grid_dependency_wait();
      if (lane == 0) loaded = produce_a(p, sbase, rank, wd);
    } else if (warp == WARP_TELL) {
      tell(p, sbase, wd);
    } else if (warp == WARP_MMA) {
      if (rank == 0) issue(p, sbase, tmem, wd);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  // No warp of the CTA gives up after this, and without that every copy has been waited for.
  if (*abort_flag && lane == 0) {
    if (warp == WARP_W) {
      drain(sbase + OFF_BAR + 8 * BAR_W_FULL, p.w_stages, loaded);
    } else if (warp == WARP_A && rank == 0) {
      drain(sbase + OFF_BAR + 8 * BAR_A_FULL, p.a_stages, loaded);
    } else if (warp == WARP_A) {
      // Its copies have the leader's barriers: give them 100 us (they take a few).
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------ the tokens in fp16

struct ExpandParams {
  const int8_t* a;
  int64_t lda;
  int tokens, k;
  int wide;          // a's rows lie on 16-byte boundaries
  int chunks;        // of 16 in a row
  uint16_t* out;     // rows of 16 * chunks fp16, zeros after k, in the order of to_fp16
  uint4* zero;       // what is to be zero before the product, and how many
  int64_t zeros;
};

constexpr int EXPAND_THREADS = 256;

// 16 of K a thread, which are one load and two stores; bound by memory where tokens are many (8192 x 8192 within
// the product's 653 us: 201 MB), by its launch where they are few (3 us).
__global__ void __launch_bounds__(EXPAND_THREADS) expand_kernel(const __grid_constant__ ExpandParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * EXPAND_THREADS + threadIdx.x;
  const int64_t chunks = static_cast<int64_t>(p.tokens) * p.chunks;
  if (v >= chunks) {
    if (v - chunks < p.zeros) p.zero[v - chunks] = make_uint4(0, 0, 0, 0);
    return;
  }
  // 32-bit divisions where they do
  const int64_t row = chunks < (int64_t{1} << 31) ? static_cast<uint32_t>(v) / static_cast<uint32_t>(p.chunks)
                                                  : v / p.chunks;
  const int c = static_cast<int>(v - row * p.chunks) * 16;
  const uint4 raw = load16(p.a + row * p.lda, c, p.k, p.wide);
  const uint2 w[4] = {to_fp16(raw.x), to_fp16(raw.y), to_fp16(raw.z), to_fp16(raw.w)};
  uint4* to = reinterpret_cast<uint4*>(p.out + (row * p.chunks) * 16 + c);
  to[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
  to[1] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
}

}  // namespace i8
}  // namespace gws
