// Test-only probe of what a warp and a role do as they give up (pa_wait.cuh), with
// short limits, on barriers of its own.  Nothing here can hang: every wait has a limit
// of at most `other_ns`.
#include <cuda_runtime.h>

#include "pa_wait.cuh"

// One CTA of two warps, two mbarriers of one arrival each.
//   mode 0: warp 0's lanes wait as a warp, the lower half on a barrier whose phase is
//           complete, the upper half on one that nothing completes.
//   mode 1: the whole of warp 0 on the completed one.
//   mode 2: warp 0 drains a barrier that nothing completes, the abort flag set.
//   mode 3: the same, and warp 1 arrives after 0.1 ms.
// result[0 .. 31] = what each lane of warp 0 was told (waits), result[32] = the abort
// flag at the end, result[33] = warp 0's time in microseconds.
__global__ void give_up_probe_kernel(int* status, int* result, unsigned long long limit_ns,
                                     unsigned long long other_ns, int mode) {
  __shared__ __align__(8) unsigned long long bars[2];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t done = (uint32_t)__cvta_generic_to_shared(&bars[0]);
  const uint32_t open = (uint32_t)__cvta_generic_to_shared(&bars[1]);
  if (threadIdx.x == 0) {
    pa::mbar_init(done, 1);
    pa::mbar_init(open, 1);
    abort_flag = mode >= 2;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pa::mbar_arrive(done);
  }
  __syncthreads();
  volatile int* vabort = &abort_flag;
  if (warp == 0) {
    const uint64_t t0 = pa::globaltimer();
    if (mode < 2) {
      const bool upper = mode == 0 && lane >= 16;
      result[lane] = pa::wait_bar_warp(upper ? open : done, 0, vabort, status, limit_ns);
    } else {
      pa::drain_bar(open, 0, t0, mode == 2 ? limit_ns : other_ns);
    }
    const uint64_t t1 = pa::globaltimer();
    if (lane == 0) result[33] = (int)((t1 - t0) / 1000);
  } else if (mode == 3 && lane == 0) {
    // (by the clock: a sleep may end at any time up to twice what it is given)
    const uint64_t t0 = pa::globaltimer();
    while (pa::globaltimer() - t0 < 100000) {
    }
    pa::mbar_arrive(open);
  }
  __syncthreads();
  if (threadIdx.x == 0) result[32] = abort_flag;
}

// status: one device int; result: 34 device ints.  Returns a cudaError_t value.
extern "C" int give_up_probe(int* status, int* result, unsigned long long limit_ns,
                             unsigned long long other_ns, int mode) {
  give_up_probe_kernel<<<1, 64>>>(status, result, limit_ns, other_ns, mode);
  return (int)cudaGetLastError();
}
