// selftest.cu -- one bounded mbarrier wait of each kind that the pipelined
// kernels here use (a thread's, a warp's), so that the give-up path can be exercised without a real hang.
//
// With expire set, nothing ever arrives on the barrier: the wait gives up
// after limit_ns, the kernel records DSA_STATUS_TIMEOUT in the status word and
// returns, and the context stays usable.  Without it the barrier is completed
// before the wait, which must then succeed and record nothing.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {

using namespace sm100;

__global__ void k_bounded_wait(int* status, int expire, unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x != 0) return;
  abort_flag = 0;
  mbar_init(&bar, 1);
  fence_mbar_init();
  if (!expire) mbar_arrive(&bar);
  if (!mbar_wait(&bar, 0, &abort_flag, limit_ns)) flag_status(status, DSA_STATUS_TIMEOUT);
}

// The whole-warp wait of the CTA-pair kernel, on one warp.  Mode 0: the barrier
// is completed first; 1: nothing arrives; 2: nothing arrives and another warp
// raises the abort flag after 5 ms.
__global__ void k_warp_wait(int* status, int mode, unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar, 1);
    fence_mbar_init();
    if (mode == 0) mbar_arrive(&bar);
  }
  __syncthreads();
  if (warp == 1) {
    const uint64_t t0 = globaltimer_ns();
    if (mode == 2 && lane == 0) {
      while (globaltimer_ns() - t0 < 5000000ull) {
      }
      *reinterpret_cast<volatile int*>(&abort_flag) = 1;
    }
    return;
  }
  if (!pair_wait(smem_u32(&bar), 0, &abort_flag, limit_ns) && lane == 0)
    flag_status(status, DSA_STATUS_TIMEOUT);
}

}  // namespace

int warp_wait_selftest(int mode, unsigned long long limit_ns, int* status, cudaStream_t s) {
  k_warp_wait<<<1, 64, 0, s>>>(status, mode, limit_ns);
  count_launch();
  return check_launch("warp wait self-test");
}

int bounded_wait_selftest(int expire, unsigned long long limit_ns, int* status, cudaStream_t s) {
  k_bounded_wait<<<1, 32, 0, s>>>(status, expire, limit_ns);
  count_launch();
  return check_launch("bounded wait self-test");
}

}  // namespace dsa
