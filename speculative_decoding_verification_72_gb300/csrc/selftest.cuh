// Self-test of the failure paths that the kernels share: bounded mbarrier waits
// that nothing completes give up after their limit, and the kernel reports
// SV_STATUS_TIMEOUT and returns instead of hanging.
#pragma once

#include "tc_common.cuh"

namespace sv {

// One thread-block of one warp: lane 0 initialises an mbarrier that expects
// one arrival, never arrives on it, and waits on its first phase with
// mbar_wait_bounded, then with the tensor-core kernels' wait_or_fail: once until
// that gives up and sets its flag, and once more, when the flag ends it at once.
// No bulk copy is issued, so nothing is in flight when the block exits.
__global__ void __launch_bounds__(32) selftest_wait_kernel(int32_t* out_status) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t fail;
  if (threadIdx.x != 0) return;
  fail = 0;
  mbar_init(smem_u32(&bar), 1);
  fence_barrier_init();
  bool gave_up = !mbar_wait_bounded(smem_u32(&bar), 0);
  volatile uint32_t* flag = &fail;
  gave_up = gave_up && !wait_or_fail(smem_u32(&bar), 0, flag) && *flag != 0;
  const uint64_t t = global_timer_ns();
  gave_up = gave_up && !wait_or_fail(smem_u32(&bar), 0, flag) && global_timer_ns() - t < kWaitNs / 2;
  out_status[0] = gave_up ? SV_STATUS_TIMEOUT : 0;
}

}  // namespace sv
