// selftest.cu -- exercises the bounded mbarrier waits every pipeline uses,
// on the GPU, without a fault: one CTA waits on barriers that nothing ever
// completes, so the waits must give up, set the error flag and let the CTA
// leave.
#include "internal.h"
#include "ptx.cuh"

namespace decattn {
namespace {

// Thread 0 waits on barrier A with a limit of limit_ns and, when it gives up,
// raises the CTA's abort word (as a pipeline role does).  Thread 32 waits on
// barrier B with a limit 1000x longer but watching the abort word, so it must
// leave because of thread 0, long before its own limit.
__global__ void __launch_bounds__(64) wait_timeout_kernel(int* err_flag, int* result,
                                                           uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int abort_word;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    abort_word = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort = &abort_word;
  if (threadIdx.x == 0) {
    const uint64_t t0 = global_timer_ns();
    const bool ok = mbar_wait_or_abort(smem_u32(&bars[0]), 0, err_flag, abort, false, limit_ns);
    result[0] = ok ? 0 : 1;
    result[2] = static_cast<int>((global_timer_ns() - t0) / 1000);  // us waited
  } else if (threadIdx.x == 32) {
    const uint64_t t0 = global_timer_ns();
    const bool ok =
        mbar_wait_or_abort(smem_u32(&bars[1]), 0, err_flag, abort, false, limit_ns * 1000);
    const uint64_t waited = global_timer_ns() - t0;
    result[1] = (!ok && waited < limit_ns * 100) ? 1 : 0;
    result[3] = static_cast<int>(waited / 1000);
  }
  // The plain bounded wait (no abort word) gives up the same way.
  if (threadIdx.x == 1) result[4] = mbar_wait(smem_u32(&bars[0]), 0, err_flag, limit_ns) ? 0 : 1;
}

// One warp, whose lanes 16..31 wait on a barrier that nothing completes and the
// others on one that is complete: all must get the same answer, no; and yes where
// all wait on the complete one.
__global__ void __launch_bounds__(32) warp_wait_kernel(int* err_flag, int* result,
                                                       uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int abort_word;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    abort_word = 0;
    fence_barrier_init();
    mbar_arrive(smem_u32(&bars[0]));
  }
  __syncthreads();
  const uint32_t done = smem_u32(&bars[0]), mixed = smem_u32(&bars[threadIdx.x >> 4]);
  const bool a = mbar_wait_warp(mixed, 0, err_flag, limit_ns);
  const bool b = mbar_wait_or_abort_warp(mixed, 0, err_flag, &abort_word, limit_ns);
  const bool c = mbar_wait_warp(done, 0, err_flag, limit_ns);
  const bool d = mbar_wait_or_abort_warp(done, 0, err_flag, &abort_word, limit_ns);
  const bool yes[4] = {a, b, c, d};
  for (int k = 0; k < 4; ++k) {
    const int lanes = __popc(__ballot_sync(0xffffffffu, yes[k]));
    if (threadIdx.x == 0) result[k] = lanes;
  }
}

}  // namespace

cudaError_t launch_warp_wait_selftest(int* err_flag, int* result, uint64_t limit_ns,
                                      cudaStream_t stream) {
  warp_wait_kernel<<<1, 32, 0, stream>>>(err_flag, result, limit_ns);
  return cudaGetLastError();
}

cudaError_t launch_wait_selftest(int* err_flag, int* result, uint64_t limit_ns,
                                 cudaStream_t stream) {
  wait_timeout_kernel<<<1, 64, 0, stream>>>(err_flag, result, limit_ns);
  return cudaGetLastError();
}

}  // namespace decattn
