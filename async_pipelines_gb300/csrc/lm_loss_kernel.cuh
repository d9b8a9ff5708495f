// Softmax cross entropy of x * weight^T over a vocabulary, and its gradients,
// without the logits in memory.
//
//   z = x * weight^T (T x V);  lse_i = log sum_j exp(z_ij);
//   loss_i = lse_i - z_i,target(i)
//   G_ij = g_i / s * (exp(z_ij - lse_i) - [j == target(i)])
//   dx = s * G * weight;  dweight = s * G^T * x
// where s is the largest |g|, or g itself if all tokens have one.
//
// Tokens that are not counted (target == ignore) are left out before the
// first product: a gather packs the counted rows of x, so such a row costs
// no product, and cannot put a NaN into dweight. How many rows are counted is
// known on the device only; every kernel reads it there. (A loss of few rows or
// of few tiles takes x as it lies: there an uncounted row is multiplied like any
// other, and its sums, which are its own, are left out at the end.)
//
// One persistent warp-specialised product kernel serves all of it, with the
// roles of the GEMM (two TMA producer warps, one MMA thread, eight epilogue
// warps, two TMEM accumulators) and one of three epilogues:
//   LSE    the logits' tile stays in TMEM; each row's running maximum and sum
//          of exponentials leave, and the target's logit.
//   GRAD   the tile is computed again for a piece of the vocabulary and G
//          leaves in bf16, since the tensor cores multiply 16-bit operands. That
//          rounds G once, by up to 2^-8 of each value. It is rounded without s: the
//          targets' -1 of tokens that the model does not expect, which are most
//          of dx and dweight, are then exact, where -g, the same for all of them,
//          would be off by one and the same share (3.9e-3 for the mean of 255
//          tokens). In the norm dx and dweight are off by 1.6e-3 to 2.1e-3 (1 to 8192
//          tokens), where their own rounding to bf16 alone makes 1.7e-3. A second product
//          with what G's rounding leaves would take them to that, for twice the operations.
//   SUMS   the two products of that piece in one launch, dx's units (fp32,
//          added to by later pieces) before dweight's (bf16, final). G^T, x
//          and weight are read as they lie, as MN-major operands, so nothing
//          is transposed in memory.
// The work is 8 T V H operations for both gradients (6 without computing the
// logits twice), for a workspace of one piece of G instead of T x V.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "watchdog.cuh"

namespace gws {
namespace ce {

constexpr int BM = 128;                   // rows of a CTA's tile = TMEM lanes
constexpr int BN_MAX = 256;               // columns of a tile, at most
constexpr int BK = 64;                    // k-block: one 128-byte swizzle row of bf16
constexpr int UMMA_K = 16;
constexpr int ACC_BUFS = 2;
constexpr int EPI_N = 32;                 // columns of one TMEM load
constexpr int EPI_WARPS = 8;              // two for each 32-lane quarter
constexpr int WARP_A = 0, WARP_MMA = 1, WARP_EPI0 = 2, WARP_B = WARP_EPI0 + EPI_WARPS;
constexpr int THREADS = (WARP_B + 1) * 32;
constexpr int MAX_STAGES = 8;
constexpr uint32_t A_BLOCK = BM * BK * 2;              // 16 KiB: 128 x 64 of A
constexpr uint32_t MN_BOX = 64 * BK * 2;               // 8 KiB: a 64 x 64 box of an MN-major operand
constexpr uint32_t RING_BYTES = 192 * 1024;
constexpr uint32_t OUT_BYTES = 32 * 128;               // an epilogue warp's 32 rows x 128 bytes
constexpr uint32_t OFF_OUT = RING_BYTES;
constexpr uint32_t OFF_BAR = OFF_OUT + EPI_WARPS * OUT_BYTES;
constexpr int BAR_FULL = 0, BAR_EMPTY = BAR_FULL + MAX_STAGES, BAR_ACC_FULL = BAR_EMPTY + MAX_STAGES,
              BAR_ACC_EMPTY = BAR_ACC_FULL + ACC_BUFS, BAR_DRAIN = BAR_ACC_EMPTY + ACC_BUFS,
              NUM_BARS = BAR_DRAIN + 1;
constexpr uint32_t OFF_TMEM = OFF_BAR + NUM_BARS * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t SMEM_BYTES = OFF_ABORT + 4 + 1024;   // + slack to align the base
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KiB per-CTA shared memory");
// The tensor cores cut off what an addition to the accumulator shifts out, so a
// logit that grows over a long K ends too near to zero: by 5e-6 of lse with 8192
// hidden, and the loss of a token that the model is nearly sure of by more than
// that. So the logits' sums are cut, and the epilogue adds the cuts in registers
// with rounding. Each cut costs the tensor cores the time in which the accumulator is
// read (0.28 us for 256 x 256: 4096 x 4096 over 131072 takes 2.36 ms in one cut,
// 2.44 in cuts of 1024, 2.58 in cuts of 512), so it is 1024 of K; and 256 where few
// tokens leave them waiting for memory anyway. Loss, off by in the root of the mean
// square, of 9 to 10 in 8192 hidden: 2.5e-6 in cuts of 1024, 1.2e-6 in 512, 7e-7 in
// 256, 5e-7 in 128 (which takes 1.5 % longer), and 1.6e-6 by a matrix product in
// fp32. (The gradients' products, which end in bf16, need none of it.)
constexpr int CUT_K = 1024, CUT_K_FEW = 256;
constexpr int JOIN_FEW = 8;
constexpr float LOG2E = 1.4426950408889634f;

enum Mode { LSE = 0, GRAD = 1, SUMS = 2 };
enum Output { OUT_LSE = 0, OUT_GRAD = 1, OUT_ADD = 2, OUT_BF16 = 3 };

// 64-deep k-blocks of a ring stage: two for a CTA pair (half the barrier
// round trips for each MMA), one for a single CTA (finer stages).
template <int CG>
__host__ __device__ constexpr int ksub() { return CG; }
template <int CG>
__host__ __device__ constexpr uint32_t stage_bytes(int bn) {
  return ksub<CG>() * (A_BLOCK + static_cast<uint32_t>(bn / CG) * BK * 2);
}

// One product: D (M x N) from A and B over K. The M and K that are the
// counted rows are read from the device.
struct Job {
  CUtensorMap tmA, tmB, tmD;
  int m, n, k;          // extents; -1: the counted rows
  int a_mn, b_mn;       // the operand lies MN-major
  int b_row0;           // added to B's row coordinate (a piece's first vocabulary row)
  int d_row0;           // added to D's row coordinate
  int splits;           // cuts of K, each with a D of its own (third coordinate)
  int add;              // OUT_ADD: add to D (later pieces) instead of storing
  int out;              // Output
};

// The targets as the caller gives them.
struct Targets {
  const void* at;
  int wide;         // int64, else int32
  int64_t ignore;
  int vocab;
  __device__ __forceinline__ int64_t raw(int row) const {
    return wide ? static_cast<const int64_t*>(at)[row]
                : static_cast<int64_t>(static_cast<const int*>(at)[row]);
  }
  __device__ __forceinline__ bool inside(int64_t t) const { return t >= 0 && t < vocab; }
};

// Where the forward pass's results go.
struct Results {
  float *loss, *lse;
  float* mean;      // two, or NULL
};

struct Params {
  Job job[2];
  int jobs;
  int bn, stages;            // tile columns; ring stages
  int a_rows;                // rows of A that a box brings: 128, or all there are if fewer (what
                             // lies below them in a stage is never looked at)
  const int* count;          // counted rows
  // LSE and GRAD: the logits' rows and columns
  int cols;                  // valid columns of the launch (its piece of the vocabulary)
  int col0;                  // the first of them in the vocabulary
  const int* target;         // [row] of the packed rows, -1: outside the vocabulary
  float* target_logit;       // [row]
  float2* part;              // [slot][row]: maximum and sum of exponentials
  int64_t part_stride;
  int cut_k;                 // K of one accumulator, a multiple of 128 (the same in both)
  int carry;                 // one row of tiles: a CTA keeps its sums over its tiles
  const float *lse, *grad;   // [row]: lse, and g / s (0: no gradient)
  const float* scale;        // SUMS: s
  // LSE of few rows or tiles: x itself is A, so nothing is packed; and with at most
  // JOIN_FEW rows the CTA that ends last joins the sums, so that the pass is one
  // launch. (It is one SM's work: 61 rows so take 10 us longer than with a launch.)
  int direct;
  int join;
  int rows;
  int slots;
  Targets given;
  Results result;
  uint32_t* done;            // CTAs that ended; zero at launch, left zero
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;           // 3: A's producer brings nothing
#endif
};

// A unit of work: a tile of a job, or of one cut of its K.
struct Unit {
  const Job* job;
  int m0, n0;      // first row of the cluster's tile, first column
  int nb;          // tile column
  int cut;
  int s0, s1;      // ring stages of K
};

constexpr int GROUP_M = 8;   // tiles walk 8 rows of tiles down, then step a column (L2 reuse)

// ceil(a / b); a may be any int (a + b - 1 may not be one).
__host__ __device__ constexpr int parts_of(int a, int b) { return a / b + (a % b != 0); }

// The tiles of a job, and the ring stages of its K.
struct Grid {
  int tm, tn, tiles, units, stages;
};
template <int CG>
__host__ __device__ __forceinline__ Grid grid_of(const Params& p, const Job& job, int count) {
  Grid g;
  const int m = job.m < 0 ? count : job.m, k = job.k < 0 ? count : job.k;
  g.tm = parts_of(m, BM * CG);
  g.tn = parts_of(job.n, p.bn);
  g.tiles = g.tm * g.tn;
  g.units = g.tiles * job.splits;
  g.stages = parts_of(k, BK * ksub<CG>());
  return g;
}

// What every role of a cluster walks: units first, first + clusters, ... of
// the jobs' units one after the other. With two jobs, the first one's units
// (dx's, usually the longer) leave the clusters from `heavy` on with one unit
// less; those then take `extra` units of the second job before all go on in
// turn, so that no cluster ends more than about one of the shorter units
// after the others. (Without it dx's quarter-full last wave of long units
// held the launch up: 4096 x 4096 over 131072, both gradients of a piece,
// 1378 us instead of 1290.) All that does not change from unit to unit is kept
// here: a division costs a role that walks short units more than its unit.
struct Walk {
  int cluster, clusters;
  Grid a, b;        // of the two jobs
  int heavy, extra;
  int turns, rank;  // units of the first job that this cluster has; its place after them
  bool light;
};

template <int CG>
__host__ __device__ __forceinline__ Walk make_walk(const Params& p, int count, int cluster,
                                                   int clusters) {
  Walk k;
  k.cluster = cluster;
  k.clusters = clusters;
  k.a = grid_of<CG>(p, p.job[0], count);
  k.b = k.a;
  k.heavy = k.extra = k.turns = k.rank = 0;
  k.light = true;
  if (p.jobs == 2) {
    k.b = grid_of<CG>(p, p.job[1], count);
    k.heavy = k.a.units % k.clusters;
    // Short units take about a stage's time on top, for their stores.
    const int each = k.b.stages < 8 ? k.b.stages + 1 : k.b.stages;
    if (k.heavy) k.extra = k.a.stages / p.job[0].splits / each;
    k.light = k.cluster >= k.heavy;
    k.turns = k.a.units / k.clusters + (k.light ? 0 : 1);
    k.rank = k.light ? k.cluster - k.heavy : k.cluster + k.clusters - k.heavy;
  }
  return k;
}

// The i-th unit of the walk.
template <int CG>
__host__ __device__ __forceinline__ bool next_unit(const Params& p, const Walk& k, int i, Unit& w) {
  int u = k.cluster + i * k.clusters;
  const bool second = p.jobs == 2 && u >= k.a.units;
  if (second) {
    if (k.extra == 0) {
      u -= k.a.units;
    } else {
      const int t = i - k.turns, lights = k.clusters - k.heavy;
      if (k.light && t < k.extra)
        u = t * lights + k.rank;
      else
        u = k.extra * lights + (k.light ? t - k.extra : t) * k.clusters + k.rank;
    }
  }
  Grid g;   // chosen value by value, so that the walk stays in registers
  g.tm = second ? k.b.tm : k.a.tm;
  g.tn = second ? k.b.tn : k.a.tn;
  g.tiles = second ? k.b.tiles : k.a.tiles;
  g.units = second ? k.b.units : k.a.units;
  g.stages = second ? k.b.stages : k.a.stages;
  if (u >= g.units) return false;
  const Job& job = p.job[second];
  w.job = &job;
  int t = u;
  w.cut = 0;
  w.s0 = 0;
  w.s1 = g.stages;
  if (job.splits > 1) {
    w.cut = u / g.tiles;
    t = u - w.cut * g.tiles;
    w.s0 = static_cast<int>(static_cast<int64_t>(w.cut) * g.stages / job.splits);
    w.s1 = static_cast<int>(static_cast<int64_t>(w.cut + 1) * g.stages / job.splits);
  }
  const int group = t / (GROUP_M * g.tn), first = group * GROUP_M;
  const int r = t - group * GROUP_M * g.tn;
  int dm;
  if (g.tm - first >= GROUP_M) {
    dm = r % GROUP_M;
    w.nb = r / GROUP_M;
  } else {
    w.nb = r / (g.tm - first);
    dm = r - w.nb * (g.tm - first);
  }
  w.m0 = (first + dm) * BM * CG;
  w.n0 = w.nb * p.bn;
  return true;
}

// Ring stages that one accumulator takes before it is handed over, and how often
// a unit's is.
template <int CG, int MODE>
__device__ __forceinline__ int cut_stages(const Params& p, const Unit& w) {
  return MODE == SUMS ? max(w.s1 - w.s0, 1) : p.cut_k / (BK * ksub<CG>());
}
template <int CG, int MODE>
__device__ __forceinline__ int cuts(const Params& p, const Unit& w) {
  if (MODE == SUMS) return 1;
  const int n = cut_stages<CG, MODE>(p, w);
  return (w.s1 - w.s0 + n - 1) / n;
}

// ------------------------------------------------------------ producers

template <int CG>
__device__ __forceinline__ void producer(const Params& p, uint32_t sbase, uint32_t rank, bool a_part,
                                         int count, const Watchdog& wd) {
  auto full = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_FULL + s); };
  auto empty = [&](uint32_t s) { return sbase + OFF_BAR + 8 * (BAR_EMPTY + s); };
  const Walk walk = make_walk<CG>(p, count, blockIdx.x / CG, gridDim.x / CG);
  const bool leader = a_part && rank == 0;   // arms full[s] for the pair
  const uint32_t stages = p.stages, sbytes = stage_bytes<CG>(p.bn);
  const uint32_t b_block = static_cast<uint32_t>(p.bn / CG) * BK * 2;
  const uint32_t tx = CG * ksub<CG>() * (p.a_rows * BK * 2 + b_block);
  uint32_t s = 0, ph = 0, g = 0;
  bool ok = true;
  Unit w;
#ifdef GEMM_WS_DEBUG
  if (p.debug_fault == 3 && a_part) return;   // injected fault: no stage ever fills
#endif
  for (int i = 0; ok && next_unit<CG>(p, walk, i, w); ++i) {
    const Job& job = *w.job;
    const CUtensorMap* map = a_part ? &job.tmA : &job.tmB;
    const bool mn = a_part ? job.a_mn : job.b_mn;
    // this CTA's first row (or column) of the operand, and how much it holds
    const int at = a_part ? w.m0 + static_cast<int>(rank) * BM
                          : w.n0 + static_cast<int>(rank) * (p.bn / CG);
    const int boxes = (a_part ? BM : p.bn / CG) / 64;
    const int row0 = a_part ? 0 : job.b_row0;
    for (int st = w.s0; st < w.s1; ++st) {
      if (!wait_spin<false>(empty(s), ph ^ 1, wd)) {
        ok = false;
        break;
      }
      if (leader) mbar_arrive_expect_tx(full(s), tx);
      const uint32_t bar = CG == 1 ? full(s) : mapa_shared(full(s), 0u);
      uint32_t dst = sbase + s * sbytes + (a_part ? 0u : ksub<CG>() * A_BLOCK);
#pragma unroll
      for (int ks = 0; ks < ksub<CG>(); ++ks) {
        const int k0 = (st * ksub<CG>() + ks) * BK;
        auto load = [&](uint32_t to, int x, int y) {
          if constexpr (CG == 1)
            tma_load_3d(to, map, bar, x, y, 0);
          else
            tma_load_3d_pair(to, map, bar, x, y, 0);
        };
        if (mn) {
          for (int b = 0; b < boxes; ++b) load(dst + b * MN_BOX, at + 64 * b, k0 + row0);
        } else {
          load(dst, k0, at + row0);
        }
        dst += a_part ? A_BLOCK : b_block;
      }
      ++g;
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  if (!ok && leader) {
    // Abort: the copies of the stages armed last land before the CTA goes on.
    for (uint32_t j = g > stages ? g - stages : 0; j < g; ++j)
      wait_drain(full(j % stages), (j / stages) & 1);
  } else if (!ok) {
    // Copies into a stage that the leader never armed have no barrier: give
    // them 100 us (they take a few).
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
  }
}

// ------------------------------------------------------------ MMA issuer

template <int CG, int MODE>
__device__ __forceinline__ void mma_issuer(const Params& p, uint32_t sbase, uint32_t tmem,
                                           uint32_t rank, int count, const Watchdog& wd) {
  auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
  auto commit = [&](uint32_t b) {
    if constexpr (CG == 1)
      umma_commit(b);
    else
      umma_commit_pair(b, static_cast<uint16_t>(0x3u));
  };
  const Walk walk = make_walk<CG>(p, count, blockIdx.x / CG, gridDim.x / CG);
  const uint32_t stages = p.stages, sbytes = stage_bytes<CG>(p.bn);
  const uint32_t b_block = static_cast<uint32_t>(p.bn / CG) * BK * 2;
  uint32_t s = 0, ph = 0;
  uint32_t handed = 0;   // accumulators handed over so far
  bool issued = false;
  Unit w;
  for (int i = 0; next_unit<CG>(p, walk, i, w); ++i) {
    const Job& job = *w.job;
    const bool a_mn = job.a_mn, b_mn = job.b_mn;
    const uint32_t idesc = idesc_bf16_f32(BM * CG, p.bn, a_mn, b_mn);
    // 16 of K: 32 bytes along a K-major row, or 16 rows of 128 bytes
    const uint32_t a_step = a_mn ? UMMA_K * 128 : UMMA_K * 2;
    const uint32_t b_step = b_mn ? UMMA_K * 128 : UMMA_K * 2;
    bool ok = true;
    const int n = cuts<CG, MODE>(p, w), len = cut_stages<CG, MODE>(p, w);
    for (int c = 0; ok && c < n; ++c, ++handed) {
      const uint32_t b = handed & 1, aph = (handed >> 1) & 1;
      if (!wait_spin<true>(bar(BAR_ACC_EMPTY + b), aph ^ 1, wd)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d = tmem + b * BN_MAX;
      const int first = w.s0 + c * len, end = min(first + len, w.s1);
      for (int st = first; st < end; ++st) {
        if (!wait_spin<true>(bar(BAR_FULL + s), ph, wd)) {
          ok = false;
          break;
        }
        const uint32_t a_addr = sbase + s * sbytes, b_addr = a_addr + ksub<CG>() * A_BLOCK;
#pragma unroll
        for (int kk = 0; kk < ksub<CG>() * (BK / UMMA_K); ++kk) {
          const int blk = kk / (BK / UMMA_K), kin = kk % (BK / UMMA_K);
          const uint32_t aa = a_addr + blk * A_BLOCK + kin * a_step;
          const uint32_t bb = b_addr + blk * b_block + kin * b_step;
          const uint64_t ad = a_mn ? sdesc_mnmajor_sw128(aa) : sdesc_kmajor_sw128(aa);
          const uint64_t bd = b_mn ? sdesc_mnmajor_sw128(bb) : sdesc_kmajor_sw128(bb);
          const uint32_t acc = (st != first || kk != 0) ? 1u : 0u;
          if constexpr (CG == 1)
            umma_bf16(d, ad, bd, idesc, acc);
          else
            umma_bf16_pair(d, ad, bd, idesc, acc);
        }
        issued = true;
        commit(bar(BAR_EMPTY + s));
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (end > first) {
        commit(bar(BAR_ACC_FULL + b));
      } else {   // nothing to sum: signal the accumulator barriers directly
        for (int r = 0; r < CG; ++r) {
          if constexpr (CG == 1)
            mbar_arrive(bar(BAR_ACC_FULL + b));
          else
            mbar_arrive_cluster(mapa_shared(bar(BAR_ACC_FULL + b), r));
        }
      }
    }
    if (!ok) break;
  }
  if (issued) {
    // Every MMA issued has finished once this arrives (also after an abort).
    if constexpr (CG == 1)
      umma_commit(bar(BAR_DRAIN));
    else
      umma_commit_pair(bar(BAR_DRAIN), static_cast<uint16_t>(1u << rank));
    wait_drain(bar(BAR_DRAIN), 0);
  }
}

// ------------------------------------------------------------ epilogue

// exp(x - y). The difference is taken before the change of base: a logit that
// is the maximum, or all of the sum, gives exactly 1, so the gradient of a token
// that the model is sure of does not drown in the rounding of a large logit.
__device__ __forceinline__ float exp_diff(float x, float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((x - y) * LOG2E));
  return r;
}

// What an epilogue warp knows of its place, and its side of the hand-overs.
template <int CG>
struct Epilogue {
  uint32_t sbase, tmem, rank;
  int lane;
  int e;        // 0 .. 7
  int q;        // the TMEM lane quarter that the warp may read
  int hf;       // it takes the unit's column blocks of 64 (or 32) b with b % 2 == hf
  uint8_t* out;
  uint32_t handed;

  __device__ __forceinline__ Epilogue(uint32_t sbase_, uint8_t* smem, uint32_t tmem_, uint32_t rank_,
                                      int warp)
      : sbase(sbase_), tmem(tmem_), rank(rank_), lane(threadIdx.x & 31), e(warp - WARP_EPI0),
        q(warp & 3), hf((warp - WARP_EPI0) / 4), out(smem + OFF_OUT + (warp - WARP_EPI0) * OUT_BYTES),
        handed(0) {}
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + OFF_BAR + 8 * i; }
  // Waits for the next accumulator; its address for this warp's lanes.
  __device__ __forceinline__ bool take(const Watchdog& wd, uint32_t* tacc) const {
    if (!warp_wait_spin(bar(BAR_ACC_FULL + (handed & 1)), (handed >> 1) & 1, wd)) return false;
    tc_fence_after_sync();
    *tacc = tmem + (static_cast<uint32_t>(32 * q) << 16) + (handed & 1) * BN_MAX;
    return true;
  }
  // Gives it back to the MMA thread (of the pair's even CTA).
  __device__ __forceinline__ void release() {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      const uint32_t b = bar(BAR_ACC_EMPTY + (handed & 1));
      if (CG == 1 || rank == 0)
        mbar_arrive(b);
      else
        mbar_arrive_cluster(mapa_shared(b, 0));
    }
    ++handed;
  }
  // Rows of 128 bytes with the TMA's 128-byte swizzle: 16-byte piece c of this lane's row.
  __device__ __forceinline__ uint4* piece(int c) const {
    return reinterpret_cast<uint4*>(out + lane * 128 + ((c ^ (lane & 7)) << 4));
  }
  // The warp's block may be written again: its last store has read it.
  __device__ __forceinline__ void reuse() const {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  __device__ __forceinline__ void store(const CUtensorMap* map, int x, int y, int z, bool add) const {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add)
        tma_add_3d(map, smem_addr(out), x, y, z);
      else
        tma_store_3d(map, smem_addr(out), x, y, z);
      bulk_commit();
    }
  }
};

// Two fp32 values times s, in bf16 (one instruction for both products).
__device__ __forceinline__ uint32_t scaled_bf16x2(float lo, float hi, float s) {
  unsigned long long v, f;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  asm("mov.b64 %0, {%1, %1};" : "=l"(f) : "f"(s));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(f));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return pack_bf16x2(lo, hi);
}

// 64 fp32 values of a row in bf16 to the warp's block.
template <int CG>
__device__ __forceinline__ void put_bf16(const Epilogue<CG>& w, const float (&lo)[32],
                                         const float (&hi)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float* a = c < 4 ? lo : hi;
    const int o = 8 * (c & 3);
    *w.piece(c) = make_uint4(pack_bf16x2(a[o], a[o + 1]), pack_bf16x2(a[o + 2], a[o + 3]),
                             pack_bf16x2(a[o + 4], a[o + 5]), pack_bf16x2(a[o + 6], a[o + 7]));
  }
}

// LSE and GRAD: a thread has one row and, in registers, the logits of its warp's
// column blocks, two of 64.
template <int CG, int MODE>
__device__ __forceinline__ void epilogue_logits(const Params& p, uint32_t sbase, uint8_t* smem,
                                                uint32_t tmem, uint32_t rank, int warp, int count,
                                                const Watchdog& wd) {
  Epilogue<CG> me(sbase, smem, tmem, rank, warp);
  const Walk walk = make_walk<CG>(p, count, blockIdx.x / CG, gridDim.x / CG);
  float top = -INFINITY, sum = 0.0f;
  int row = 0;
  bool any = false;
  auto flush = [&](int slot) {
    if (row < count) p.part[static_cast<int64_t>(slot) * p.part_stride + row] = make_float2(top, sum);
    top = -INFINITY;
    sum = 0.0f;
  };
  Unit w;
  for (int i = 0; next_unit<CG>(p, walk, i, w); ++i) {
    any = true;
    const int part0 = w.m0 + static_cast<int>(rank) * BM;   // this CTA's first row
    row = part0 + 32 * me.q + me.lane;
    const int width = part0 < count ? min(p.bn, p.cols - w.n0) : 0;   // valid columns
    int target = -1;   // the target's column in this tile, if in it
    float lse = 0.0f, grad = 0.0f;
    if (row < count) {
      int t;
      if (MODE == LSE && p.direct) {
        const int64_t raw = p.given.raw(row);
        t = raw != p.given.ignore && p.given.inside(raw) ? static_cast<int>(raw) : -1;
      } else {
        t = p.target[row];
      }
      target = t - p.col0 - w.n0;
      if (MODE == GRAD) {
        lse = p.lse[row];
        grad = p.grad[row];
      }
    }
    // block k of 32 columns: the halves of the warp's 64-column blocks
    auto column = [&](int k) { return 128 * (k / 2) + 64 * me.hf + 32 * (k % 2); };
    float z[4][32];
    bool ok = true;
    const int n = cuts<CG, MODE>(p, w);
    for (int c = 0; c < n; ++c) {
      uint32_t tacc;
      if (!me.take(wd, &tacc)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (column(k) >= width) continue;
#pragma unroll
        for (int x0 = 0; x0 < 32; x0 += 16) {
          uint32_t part[16];
          tmem_ld_32x32b_x16(tacc + column(k) + x0, part);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; ++x)
            z[k][x0 + x] = c == 0 ? __uint_as_float(part[x]) : z[k][x0 + x] + __uint_as_float(part[x]);
        }
      }
      me.release();
    }
    if (!ok) break;
    if constexpr (MODE == LSE) {
      float next = top;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (column(k) >= width) continue;
        const int valid = width - column(k);
        const int hit = target - column(k);
        if (hit >= 0 && hit < 32) {
          float at = 0.0f;
#pragma unroll
          for (int x = 0; x < 32; ++x) at = x == hit ? z[k][x] : at;
          p.target_logit[row] = at;
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (x >= valid) z[k][x] = -INFINITY;
          next = fmaxf(next, z[k][x]);
        }
      }
      const float base = next == -INFINITY ? 0.0f : next;   // nothing finite yet: all terms 0
      sum *= exp_diff(top, base);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (column(k) >= width) continue;
        float add = 0.0f;
#pragma unroll
        for (int x = 0; x < 32; ++x) add += exp_diff(z[k][x], base);
        sum += add;
      }
      top = next;
      if (!p.carry) flush(2 * w.nb + me.hf);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        if (column(k) >= width) continue;
        // Rows that are not there (or have no gradient) and columns past the
        // vocabulary are 0: the products after this one run over them.
        const int valid = grad != 0.0f ? width - column(k) : 0;
        const int hit = target - column(k);
        auto gradient = [&](float logit, int x) {
          float pr = exp_diff(logit, lse);
          if (x == hit) pr -= 1.0f;
          return x < valid ? pr * grad : 0.0f;
        };
        const bool second = column(k + 1) < width;   // else its z holds nothing
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          z[k][x] = gradient(z[k][x], x);
          z[k + 1][x] = second ? gradient(z[k + 1][x], 32 + x) : 0.0f;
        }
        me.reuse();
        put_bf16(me, z[k], z[k + 1]);
        me.store(&w.job->tmD, w.n0 + column(k), part0 + 32 * me.q, 0, false);
      }
    }
  }
  if (MODE == LSE && p.carry && any) flush(2 * walk.cluster + me.hf);
  if (MODE == GRAD) me.reuse();
}

// SUMS: dx's tiles leave in fp32 (stored, or added to the pieces before), dweight's
// times s in bf16. (The product with s costs 4 % where the tiles' stores bound the
// launch, gradients of one token over 131072 x 4096 566 us, and below 1 % from 128 tokens on.)
template <int CG>
__device__ __forceinline__ void epilogue_sums(const Params& p, uint32_t sbase, uint8_t* smem,
                                              uint32_t tmem, uint32_t rank, int warp, int count,
                                              const Watchdog& wd) {
  Epilogue<CG> me(sbase, smem, tmem, rank, warp);
  const Walk walk = make_walk<CG>(p, count, blockIdx.x / CG, gridDim.x / CG);
  const float scale = *p.scale;
  Unit w;
  for (int i = 0; next_unit<CG>(p, walk, i, w); ++i) {
    const Job& job = *w.job;
    const int part0 = w.m0 + static_cast<int>(rank) * BM;   // this CTA's first row
    const bool f32 = job.out == OUT_ADD;
    const int step = f32 ? EPI_N : 2 * EPI_N;   // columns of a block
    const int blocks = part0 < (job.m < 0 ? count : job.m)
                           ? (min(p.bn, job.n - w.n0) + step - 1) / step : 0;
    const bool has_acc = w.s1 > w.s0;
    uint32_t tacc;
    if (!me.take(wd, &tacc)) break;
    if (me.hf >= blocks) me.release();
    for (int j = me.hf; j < blocks; j += 2) {
      uint32_t a0[32] = {}, a1[32] = {};
      if (has_acc) {
        tmem_ld_32x32b_x32(tacc + j * step, a0);
        if (!f32) tmem_ld_32x32b_x32(tacc + j * step + EPI_N, a1);
        tmem_wait_ld();
      }
      if (j + 2 >= blocks) me.release();
      if (f32) {
        me.reuse();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *me.piece(c) = make_uint4(a0[4 * c], a0[4 * c + 1], a0[4 * c + 2], a0[4 * c + 3]);
      } else {
        // scaled and rounded while the block's last store may still be read
        uint32_t v[32];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          v[x] = scaled_bf16x2(__uint_as_float(a0[2 * x]), __uint_as_float(a0[2 * x + 1]), scale);
          v[16 + x] = scaled_bf16x2(__uint_as_float(a1[2 * x]), __uint_as_float(a1[2 * x + 1]), scale);
        }
        me.reuse();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *me.piece(c) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
      me.store(&job.tmD, w.n0 + j * step, job.d_row0 + part0 + 32 * me.q, w.cut, job.add);
    }
  }
  me.reuse();
}

// ------------------------------------------------------------ joining the sums

// (top, sum) and (v.x, v.y) as one maximum and sum.
__device__ __forceinline__ void join_pair(float& top, float& sum, float2 v) {
  const float next = fmaxf(top, v.x), base = next == -INFINITY ? 0.0f : next;
  sum = sum * exp_diff(top, base) + v.y * exp_diff(v.x, base);
  top = next;
}

// The pairs of the lanes that are equal modulo `group`, in each of them. The lower
// lane's pair comes first on both sides, so that both get the same bits.
__device__ __forceinline__ void join_lanes(float& top, float& sum, int group) {
  for (int o = 16; o >= group; o >>= 1) {
    const float2 a = make_float2(top, sum);
    const float2 b =
        make_float2(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, sum, o));
    const bool low = (threadIdx.x & o) == 0;
    top = low ? a.x : b.x;
    sum = low ? a.y : b.y;
    join_pair(top, sum, low ? b : a);
  }
}

__device__ __forceinline__ void write_mean(const Results& r, float total, int counted) {
  if (!r.mean) return;
  const float share = counted > 0 ? 1.0f / static_cast<float>(counted) : 0.0f;
  r.mean[0] = counted > 0 ? total * share : 0.0f;
  r.mean[1] = share;
}

// lse and loss of all rows, at most JOIN_FEW, and the mean, by the CTA that ends
// last, from the CTAs' partial maxima and sums. A warp's lanes are the rows,
// rounded up to a power of two, and as many slots side by side as fit; the order in
// which they are joined is fixed.
__device__ __forceinline__ void join_last(const Params& p, uint8_t* smem) {
  constexpr int WARPS = THREADS / 32;
  float2* box = reinterpret_cast<float2*>(smem);
  uint32_t* ended = reinterpret_cast<uint32_t*>(smem + WARPS * 32 * sizeof(float2));
  __threadfence();   // this thread's partial sums, before the count of CTAs
  __syncthreads();
  if (threadIdx.x == 0) *ended = atomicAdd(p.done, 1u);
  __syncthreads();
  if (*ended != gridDim.x - 1) return;
  __threadfence();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int group = 1;
  while (group < p.rows) group *= 2;
  const int row = lane % group;
  float top = -INFINITY, sum = 0.0f;
  if (row < p.rows) {
#pragma unroll 8
    for (int s = warp * (32 / group) + lane / group; s < p.slots; s += WARPS * (32 / group))
      join_pair(top, sum, __ldcg(p.part + s * p.part_stride + row));
  }
  join_lanes(top, sum, group);
  box[warp * 32 + lane] = make_float2(top, sum);
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < WARPS; ++w) join_pair(top, sum, box[w * 32 + lane]);
  float loss = 0.0f;
  int counted = 0;
  if (lane < p.rows) {
    const int64_t t = p.given.raw(row);
    counted = t != p.given.ignore;
    const float rest = counted ? logf(sum) : 0.0f;
    const float logit = p.given.inside(t) ? __ldcg(p.target_logit + row) : NAN;
    loss = counted ? (top - logit) + rest : 0.0f;
    p.result.lse[row] = counted ? top + rest : 0.0f;
    p.result.loss[row] = loss;
  }
  for (int o = 16; o > 0; o >>= 1) {
    loss += __shfl_xor_sync(0xffffffffu, loss, o);
    counted += __shfl_xor_sync(0xffffffffu, counted, o);
  }
  if (lane == 0) {
    write_mean(p.result, loss, counted);
    *p.done = 0u;
  }
}

// ------------------------------------------------------------ product kernel

template <int CG, int MODE>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_ctarank();
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
  if (warp == WARP_A && lane == 0) {
    auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(bar(BAR_FULL + s), 1);
      mbar_init(bar(BAR_EMPTY + s), 1);
    }
    for (int b = 0; b < ACC_BUFS; ++b) {
      mbar_init(bar(BAR_ACC_FULL + b), 1);
      mbar_init(bar(BAR_ACC_EMPTY + b), EPI_WARPS * CG);
    }
    mbar_init(bar(BAR_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int j = 0; j < p.jobs; ++j) {
      prefetch_tensormap(&p.job[j].tmA);
      prefetch_tensormap(&p.job[j].tmB);
      if (MODE != LSE) prefetch_tensormap(&p.job[j].tmD);
    }
  }
  if (warp == WARP_MMA) {
    if constexpr (CG == 1) {
      tmem_alloc(smem_addr(tmem_slot), ACC_BUFS * BN_MAX);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(smem_addr(tmem_slot), ACC_BUFS * BN_MAX);
      tmem_relinquish_pair();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG > 1) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  // The set-up above overlaps the previous kernel's end; nothing below does.
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int count = MODE == LSE && p.direct ? p.rows : *p.count;

  if (warp == WARP_A || warp == WARP_B) {
    if (lane == 0) producer<CG>(p, sbase, rank, warp == WARP_A, count, wd);
  } else if (warp == WARP_MMA) {
    if (lane == 0 && rank == 0) mma_issuer<CG, MODE>(p, sbase, tmem, rank, count, wd);
  } else {
    if constexpr (MODE == SUMS)
      epilogue_sums<CG>(p, sbase, smem, tmem, rank, warp, count, wd);
    else
      epilogue_logits<CG, MODE>(p, sbase, smem, tmem, rank, warp, count, wd);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG > 1) cluster_sync();
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    if constexpr (CG == 1)
      tmem_dealloc(tmem, ACC_BUFS * BN_MAX);
    else
      tmem_dealloc_pair(tmem, ACC_BUFS * BN_MAX);
  }
  if constexpr (MODE == LSE && CG == 1)
    if (p.join) join_last(p, smem);
}

// ------------------------------------------------------------ packing the counted rows

struct PackParams {
  const uint16_t* x;          // T x H bf16
  int64_t ldx;
  Targets given;
  int rows, cols;
  int padded;                 // rows, rounded up to a multiple of 128
  int wide;                   // x's rows allow 16-byte accesses
  int chunk;                  // rows of a block, at most PACK_THREADS
  uint16_t* packed;           // T x H, `pitch` elements between rows
  int64_t pitch;
  int* place;                 // [row]: its packed row, -1 if not counted
  int* target_out;            // [packed row]
  int* count;
  float* target_logit;        // LSE: [packed row], NaN where the target is outside the vocabulary
  const float *lse, *grad;    // GRAD: [row] (grad: grad_step 0 has one for all)
  int grad_step;
  float *lse_out, *grad_out;  // GRAD: [packed row]
  float* scale;               // GRAD: s
};

constexpr int PACK_THREADS = 256;
constexpr int NO_ROW = -0x7FFFFFFF - 1;

// The sum over the block of a value a thread, in every thread.
__device__ __forceinline__ int block_sum(int v, int* box) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < PACK_THREADS / 32; ++w) s += box[w];
  __syncthreads();
  return s;
}

// The largest over the block, in every thread.
__device__ __forceinline__ int block_max(int v, int* box) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
  __syncthreads();
  int m = box[0];
  for (int w = 1; w < PACK_THREADS / 32; ++w) m = max(m, box[w]);
  __syncthreads();
  return m;
}

// Block b packs the counted rows of [b * chunk, (b + 1) * chunk). Each block
// counts all targets itself (8 bytes a row, from L2 after the first block), which
// saves a scan of its own before it, and all g for s. The rows that follow the last counted
// one up to a multiple of 128 are zeroed, since dweight's product sums over
// them; the uncounted rows' blocks do that, and rows that are there only to make up
// the 128 count as uncounted.
__global__ void __launch_bounds__(PACK_THREADS) pack_kernel(const __grid_constant__ PackParams p) {
  __shared__ int box[PACK_THREADS / 32];
  __shared__ int dst_row[PACK_THREADS];   // [row of the chunk]: packed row; -1 - packed row: zeros; NO_ROW
  grid_dependency_wait();
  grid_launch_dependents();
  const int r0 = blockIdx.x * p.chunk, r1 = min(p.padded, r0 + p.chunk);
  int before = 0, all = 0;
  float top = 0.0f;   // |g| of what has a gradient, at most
#pragma unroll 4
  for (int r = threadIdx.x; r < p.rows; r += PACK_THREADS) {
    const int64_t t = p.given.raw(r);
    const int c = t != p.given.ignore;
    all += c;
    before += r < r0 ? c : 0;
    if (p.grad_step && c && p.given.inside(t)) top = fmaxf(top, fabsf(p.grad[r]));
  }
  before = block_sum(before, box);
  all = block_sum(all, box);
  if (p.scale) {
    // as integers, which order the same where nothing is negative
    top = p.grad_step ? __int_as_float(block_max(__float_as_int(top), box)) : *p.grad;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = top;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = all;
  const int row = r0 + threadIdx.x;
  const bool mine = threadIdx.x < p.chunk && row < r1;
  const int64_t t = mine && row < p.rows ? p.given.raw(row) : p.given.ignore;
  const bool counted = mine && t != p.given.ignore;
  const unsigned vote = __ballot_sync(0xffffffffu, counted);
  if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = __popc(vote);
  __syncthreads();
  bool empty = false;   // counted, but without a gradient: its packed row is zeros
  int rank = before + __popc(vote & ((1u << (threadIdx.x & 31)) - 1u));
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) rank += box[w];
  if (mine) {
    if (row < p.rows) p.place[row] = counted ? rank : -1;
    if (counted) {
      const bool inside = p.given.inside(t);
      p.target_out[rank] = inside ? static_cast<int>(t) : -1;
      if (p.target_logit) p.target_logit[rank] = inside ? 0.0f : __int_as_float(0x7FC00000);
      if (p.lse_out) {
        const float g = inside ? p.grad[static_cast<int64_t>(row) * p.grad_step] : 0.0f;
        p.lse_out[rank] = p.lse[row];
        p.grad_out[rank] = g == 0.0f ? 0.0f : g / top;
        empty = g == 0.0f;
      }
    }
    // the k-th uncounted row zeroes the k-th packed row after the counted ones
    const int behind = all + (row - rank);
    dst_row[threadIdx.x] = empty     ? -1 - rank
                           : counted ? rank
                           : behind < (all + 127) / 128 * 128 ? -1 - behind : NO_ROW;
  }
  __syncthreads();
  const int groups = p.cols / 8;   // cols is a multiple of 8
  for (int v = threadIdx.x; v < (r1 - r0) * groups; v += PACK_THREADS) {
    const int r = v / groups, c = (v - r * groups) * 8;
    const int to = dst_row[r];
    if (to == NO_ROW) continue;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (to >= 0) {
      const uint16_t* src = p.x + static_cast<int64_t>(r0 + r) * p.ldx + c;
      if (p.wide) {
        w = *reinterpret_cast<const uint4*>(src);
      } else {
        w.x = src[0] | static_cast<uint32_t>(src[1]) << 16;
        w.y = src[2] | static_cast<uint32_t>(src[3]) << 16;
        w.z = src[4] | static_cast<uint32_t>(src[5]) << 16;
        w.w = src[6] | static_cast<uint32_t>(src[7]) << 16;
      }
    }
    *reinterpret_cast<uint4*>(p.packed + static_cast<int64_t>(to >= 0 ? to : -1 - to) * p.pitch + c) = w;
  }
}

// ------------------------------------------------------------ joining the sums

struct JoinParams {
  const float2* part;
  int64_t part_stride;
  int slots;
  int direct;           // the rows are the tokens: `given`; else `place` and `count` say which
  Targets given;
  const int* place;
  const int* count;
  const float* target_logit;
  int rows;
  Results result;
  float* block_sum;     // [block]
  uint32_t* done;       // blocks finished; zero at launch, left zero
};

constexpr int JOIN_ROWS = 32, JOIN_LANES = 32;

// lse and loss of 32 rows a block, from the partial maxima and sums: a warp
// reads a slot's 32 rows at once, JOIN_LANES slots apart; then a warp joins the
// lanes of one row. The order is fixed. The block that finishes last adds the
// blocks' loss sums in block order, so the mean's bits do not depend on which
// one that is.
__global__ void __launch_bounds__(JOIN_ROWS* JOIN_LANES)
    join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float2 box[JOIN_LANES][JOIN_ROWS + 1];
  __shared__ float sums[JOIN_LANES], logit[JOIN_ROWS];
  __shared__ bool last, counted[JOIN_ROWS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int x = threadIdx.x % JOIN_ROWS, lane = threadIdx.x / JOIN_ROWS;
  {
    const int row = blockIdx.x * JOIN_ROWS + x;
    int at = -1;
    bool known = true;   // the target is in the vocabulary
    if (row < p.rows) {
      if (p.direct) {
        const int64_t t = p.given.raw(row);
        at = t != p.given.ignore ? row : -1;
        known = p.given.inside(t);
      } else {
        at = p.place[row];
      }
    }
    float top = -INFINITY, sum = 0.0f;
    if (lane == 0) {
      counted[x] = at >= 0;
      logit[x] = at < 0 ? 0.0f : known ? p.target_logit[at] : NAN;
    }
    if (at >= 0) {
      constexpr int AHEAD = 8;   // loads in flight
      for (int s0 = lane; s0 < p.slots; s0 += AHEAD * JOIN_LANES) {
        float2 v[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const int s = s0 + k * JOIN_LANES;
          v[k] = s < p.slots ? p.part[s * p.part_stride + at] : make_float2(-INFINITY, 0.0f);
        }
        float next = top;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) next = fmaxf(next, v[k].x);
        const float base = next == -INFINITY ? 0.0f : next;
        sum *= exp_diff(top, base);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) sum = fmaf(v[k].y, exp_diff(v[k].x, base), sum);
        top = next;
      }
    }
    box[lane][x] = make_float2(top, sum);
  }
  __syncthreads();
  const int row = blockIdx.x * JOIN_ROWS + lane;   // this warp's row
  const float2 mine = box[x][lane];
  float top = mine.x, sum = mine.y, loss = 0.0f;
  join_lanes(top, sum, 1);
  if (x == 0) {
    if (row < p.rows) {
      const float rest = counted[lane] ? logf(sum) : 0.0f;
      loss = counted[lane] ? (top - logit[lane]) + rest : 0.0f;
      p.result.lse[row] = counted[lane] ? top + rest : 0.0f;
      p.result.loss[row] = loss;
    }
    sums[lane] = loss;
  }
  __syncthreads();
  if (lane == 0) {
    loss = sums[x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
  }
  if (!p.result.mean) return;
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      p.block_sum[blockIdx.x] = loss;
      __threadfence();
      last = atomicAdd(p.done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    loss = 0.0f;
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += blockDim.x)
      loss += __ldcg(p.block_sum + b);
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    if (x == 0) sums[lane] = loss;
    __syncthreads();
    loss = 0.0f;
    for (int l = 0; l < JOIN_LANES; ++l) loss += sums[l];
  }
  int n = 0;
  if (!p.direct) n = *p.count;
  else
    for (int t0 = 0; t0 < p.rows; t0 += JOIN_ROWS * JOIN_LANES) {
      const int t = t0 + threadIdx.x;
      n += __syncthreads_count(t < p.rows && p.given.raw(t) != p.given.ignore);
    }
  if (threadIdx.x == 0) {
    write_mean(p.result, loss, n);
    *p.done = 0u;
  }
}

// ------------------------------------------------------------ dx

struct SpreadParams {
  const float* sums;    // [cut][packed row][col] fp32
  int cuts;
  int64_t cut_stride;
  const int* place;
  const float *grad, *scale;   // [packed row]: g / s; s
  int rows, cols;
  uint16_t* dx;
  int64_t lddx;
};

constexpr int SPREAD_THREADS = 256;

// dx of every row: the cuts' sums of its packed row added in order, times s, and
// rounded once, or zeros. Four columns a thread.
__global__ void __launch_bounds__(SPREAD_THREADS) spread_kernel(const __grid_constant__ SpreadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int quads = p.cols / 4;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * SPREAD_THREADS + threadIdx.x;
  const int64_t row = v / quads;
  if (row >= p.rows) return;
  const int c = static_cast<int>(v - row * quads) * 4;
  const int at = p.place[row];
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (at >= 0 && p.grad[at] != 0.0f) {
    const float scale = *p.scale;
    const float* src = p.sums + static_cast<int64_t>(at) * p.cols + c;
#pragma unroll 4
    for (int k = 0; k < p.cuts; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(src + k * p.cut_stride);
      s.x += f.x;
      s.y += f.y;
      s.z += f.z;
      s.w += f.w;
    }
    s.x *= scale;
    s.y *= scale;
    s.z *= scale;
    s.w *= scale;
  }
  uint2 out;
  out.x = pack_bf16x2(s.x, s.y);
  out.y = pack_bf16x2(s.z, s.w);
  *reinterpret_cast<uint2*>(p.dx + row * p.lddx + c) = out;
}

}  // namespace ce
}  // namespace gws
