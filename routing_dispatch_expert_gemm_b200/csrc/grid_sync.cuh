// What the CTAs of a grid wait for each other with.  Either all CTAs are resident (a cooperative
// launch) and arrive once each, or the work waited for is handed out by tickets: a CTA waits only
// once all tickets are taken, so by CTAs that run and, before they wait themselves, finish it.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// Words in the workspace header, zero between launches: the last CTA to leave clears them.
struct GridSync {
  unsigned int* count;   // arrivals, or finished tickets, so far in this launch
  unsigned int* left;    // CTAs that have left
  unsigned int* ticket;  // next ticket
};

// One thread, after a barrier.
__device__ __forceinline__ void grid_arrive(const GridSync& g, unsigned int n = 1u) {
  __threadfence();
  atomicAdd(g.count, n);
}
// One thread.  Bounded: returns false (and records MOE_ERR_TIMEOUT) when the arrivals do not come.
static __device__ __noinline__ bool grid_wait(const GridSync& g, unsigned int target,
                                              volatile int* abort_flag, int32_t* status) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(g.count) : "memory");
    if (v >= target) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag != 0) return false;
      if (static_cast<int64_t>(global_timer_ns() - t0) > kWaitLimitNs) {
        *abort_flag = 1;
        record_status(status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void grid_leave(const GridSync& g) {  // one thread, waits all passed
  __threadfence();
  if (atomicAdd(g.left, 1u) == gridDim.x - 1) {
    *g.count = 0;
    *g.left = 0;
    *g.ticket = 0;
  }
}

}  // namespace moe
