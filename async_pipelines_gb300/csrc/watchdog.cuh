// Bounded waits (every wait of every kernel ends by its watchdog) and the
// bf16 packing that the epilogues share.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gws {

constexpr uint32_t STATUS_TIMEOUT = 5;   // == GEMM_WS_ERR_TIMEOUT
constexpr uint32_t WAIT_HINT_NS = 1000000;   // suspend bound of one try_wait

struct Watchdog {
  volatile uint32_t* abort;   // shared-memory abort flag of this CTA
  uint32_t* status;           // global status word
  unsigned long long limit_ns;
};

// Bounded wait on an mbarrier phase. The probe may suspend the thread until
// the phase completes (or WAIT_HINT_NS passes), so waiting costs few issue
// slots. Returns false if the CTA is aborting or this wait exceeded the limit
// (which then starts the abort). kCluster selects cluster-scope acquire, for
// barriers that the peer CTA arrives on.
template <bool kCluster>
__device__ __noinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  auto probe = [&]() {
    uint32_t ok;
    if (kCluster)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity), "r"(WAIT_HINT_NS)
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity), "r"(WAIT_HINT_NS)
          : "memory");
    return ok != 0;
  };
  if (probe()) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (probe()) return true;
    if (*wd.abort) return false;
    if (global_timer_ns() - t0 > wd.limit_ns) {
      *wd.abort = 1;
      atomicExch(wd.status, STATUS_TIMEOUT);
      return false;
    }
  }
}

// Non-blocking cluster-scope probe.
__device__ __forceinline__ bool mbar_test_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <bool kCluster>
__device__ __noinline__ bool spin_slow(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
    if ((it & 255) == 0) {
      if (*wd.abort) return false;
      if (global_timer_ns() - t0 > wd.limit_ns) {
        *wd.abort = 1;
        atomicExch(wd.status, STATUS_TIMEOUT);
        return false;
      }
    }
  }
}

// Bounded wait for the latency-critical producer and MMA threads: polls
// without ever suspending, because the wake-up delay of a suspended try_wait
// lands directly on the load -> MMA critical path.
template <bool kCluster>
__device__ __forceinline__ bool wait_spin(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  if (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
  return spin_slow<kCluster>(bar, parity, wd);
}

// Short bounded wait used only while draining after an abort.
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (global_timer_ns() - t0 > 100000000ull) return;   // 100 ms
  }
}

// Warp-uniform wait: lane 0 waits, the verdict is broadcast to the warp.
// On success every lane then probes the (already completed) phase once, so
// each thread itself observes the completion (acquire) before touching the
// data it guards. The phase cannot move on meanwhile: its next completion
// needs an arrival that this warp makes only later.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  uint32_t ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_bounded<true>(bar, parity, wd) ? 1u : 0u;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  if (ok) (void)mbar_try_wait_cluster(bar, parity);
  __syncwarp();
  return ok != 0;
}

// Warp-uniform wait for the epilogue's short, latency-critical handoffs (C
// arrival, a free D slot): lane 0 polls without suspending.
__device__ __forceinline__ bool warp_wait_spin(uint32_t bar, uint32_t parity,
                                               const Watchdog& wd) {
  uint32_t ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_spin<true>(bar, parity, wd) ? 1u : 0u;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  if (ok) (void)mbar_try_wait_cluster(bar, parity);
  __syncwarp();
  return ok != 0;
}

// A probe that may suspend the thread until the phase completes or WAIT_HINT_NS pass.
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(WAIT_HINT_NS)
      : "memory");
  return ok != 0;
}

// What a wait does now and then: whether it is to give up.
__device__ __forceinline__ bool wait_over(uint64_t& t0, const Watchdog& wd) {
  if (*wd.abort) return true;
  const uint64_t now = global_timer_ns();
  if (t0 == 0) t0 = now;
  if (now - t0 <= wd.limit_ns) return false;
  *wd.abort = 1;
  atomicExch(wd.status, STATUS_TIMEOUT);
  return true;
}

// Waits on a barrier that only this CTA, its copies and its tensor cores arrive on, without a call (a
// call's conventions would spill what lives across it). The warp is suspended meanwhile: warps that
// poll take issue slots from those that work.
__device__ __forceinline__ bool warp_wait_cta(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  uint64_t t0 = 0;
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xffffffffu, wait_over(t0, wd))) return false;
  return true;
}
// The same by one thread.
__device__ __forceinline__ bool wait_suspended(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity))
    if (wait_over(t0, wd)) return false;
  return true;
}
// By one thread whose wake-up counts: it polls.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_test_wait(bar, parity); ++it)
    if ((it & 255) == 0 && wait_over(t0, wd)) return false;
  return true;
}

// Warp-uniform bounded wait for a flag in global memory that another CTA
// sets with release semantics (the in-kernel fix-up's partial-written flag):
// lane 0 polls with acquire loads; on success every lane loads the flag once
// more with acquire, so each thread itself is ordered after the writer's
// partial stores.
inline __device__ __noinline__ bool flag_wait_slow(const uint32_t* f, const Watchdog& wd) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire_gpu(f) != 0u) return true;
    if ((it & 63) == 0) {
      if (*wd.abort) return false;
      if (global_timer_ns() - t0 > wd.limit_ns) {
        *wd.abort = 1;
        atomicExch(wd.status, STATUS_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool warp_wait_flag(const uint32_t* f, const Watchdog& wd) {
  uint32_t ok = 0;
  if ((threadIdx.x & 31) == 0) ok = (ld_acquire_gpu(f) != 0u || flag_wait_slow(f, wd)) ? 1u : 0u;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  if (ok) (void)ld_acquire_gpu(f);
  __syncwarp();
  return ok != 0;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

}  // namespace gws
