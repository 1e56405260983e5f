// Self-test of the kernels' bounded waits (no paper counterpart).  Every wait of the
// tensor-core kernels on an mbarrier gives up after a time limit or a number of tries, records
// an error bit and lets the kernel leave instead of hanging the device.  This launch makes one
// wait of each kind run out on purpose -- on a barrier that nothing arrives on -- so that the
// give-up path, the error bit and the device's continued use can be checked.  Nothing faults or
// traps: the waits end by themselves after the (clamped) limit.
#include "kda_internal.cuh"
#include "tc_prims.cuh"

namespace kda {
namespace {

__device__ unsigned int g_selftest_error;  // bit 3: the self-test's waits gave up (expected)

__global__ void bounded_wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);  // one arrival expected; none is ever made
    tc::fence_mbar_init();
  }
  __syncthreads();
  bool gave_up = true;  // of the two waiting threads, one in each warp
  if (threadIdx.x == 0) gave_up = !tc::mbar_wait(&bar, 0, limit_ns);
  if (threadIdx.x == 32) {
    gave_up = false;
    for (int i = 0; !tc::mbar_try_wait_short(&bar, 0); ++i)
      if (i == (int)(limit_ns / 1000)) {
        gave_up = true;
        break;
      }
  }
  if (__syncthreads_and(gave_up) && threadIdx.x == 0) atomicOr(&g_selftest_error, 8u);
}

}  // namespace

cudaError_t launch_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  bounded_wait_selftest_kernel<<<1, 64, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

unsigned int selftest_read_error(bool reset) {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_selftest_error, sizeof(v));
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_selftest_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace kda
