// fp8_selftest.cu -- test-only kernels around the waits of the product kernels.
// Built by the GPU tests; never part of libnvfp4.
#include "fp8_tiles.cuh"

using namespace nvfp4;

namespace {

// Thread 0 waits for a phase that nothing completes, or (signal) for one that
// thread 1 completes; result: 1 when the phase came, 0 when the wait gave up.
__global__ void wait_kernel(unsigned* status, int signal, int* result) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (signal && threadIdx.x == 1) fp8::mbar_arrive(&bar);
  if (threadIdx.x == 0) {
    const bool came = fp8::mbar_wait(&bar, 0);
    if (!came) fp8::report_timeout(status);
    *result = came;
  }
}

}  // namespace

extern "C" int selftest_product_wait(unsigned* status, int signal, int* result) {
  wait_kernel<<<1, 32>>>(status, signal, result);
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : 1;
}
