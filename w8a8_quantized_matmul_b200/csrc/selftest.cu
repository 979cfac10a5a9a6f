// Self-test of the bounded device-side wait that every kernel of the library
// uses: one CTA waits on an mbarrier phase that nothing completes. The wait
// gives up after its time limit and the CTA records I8MM_ERR_TIMEOUT in a status
// word, exactly as the kernels do when a wait runs out; a second wait then gives up
// at once, copies in flight get their time, and the CTA leaves normally.
// No fault, trap or endless loop is involved; the GPU context stays usable.
#include <cuda_runtime.h>

#include <cstdint>

#include "int8mm.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace i8mm {
namespace {

__global__ void wait_timeout_kernel(int32_t* status) {
  __shared__ uint64_t bar;
  __shared__ int32_t stop;
  if (threadIdx.x == 0) {
    stop = 0;
    mbar_init(&bar, 1);   // one arrival expected; none ever comes
    fence_mbarrier_init();
  }
  __syncthreads();
  for (int i = 0; i < 2; ++i) wait_or_give_up(&bar, 0, &stop, status);
  __syncthreads();
  if (stop) let_copies_land();
}

}  // namespace
}  // namespace i8mm

extern "C" int int8_selftest_wait_timeout(int32_t* status, i8mm_stream_t stream) {
  if (!status) return I8MM_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(status, 0, 4, s) != cudaSuccess) return I8MM_ERR_CUDA;
  i8mm::wait_timeout_kernel<<<1, 32, 0, s>>>(status);
  return cudaGetLastError() == cudaSuccess ? I8MM_OK : I8MM_ERR_CUDA;
}

extern "C" int int8_selftest_product_status(int gemm, i8mm_stream_t stream) {
  const int st = i8mm::abi_check_device();
  if (st != I8MM_OK) return st;
  int32_t* word = nullptr;
  const cudaError_t e = gemm ? i8mm::gemm_status_word(&word) : i8mm::weight_stream_status_word(&word);
  if (e != cudaSuccess) return i8mm::abi_cuda_fail("address of the status word", e);
  return int8_selftest_wait_timeout(word, stream);
}
