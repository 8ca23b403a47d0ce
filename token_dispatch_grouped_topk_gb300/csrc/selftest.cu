// Self-test of the device-side failure path: the two bounded waits the
// pipelined kernels use -- an mbarrier wait, and the acquire wait on a global
// completion counter that gates the down tiles of the one-launch GEMM form --
// each run on something that nothing will complete.  Both give up after their
// time limit; the kernel reports MOE_DEV_TIMEOUT in dev_status[0], which of
// the two waits gave up as bits of dev_status[1] (1: mbarrier, 2: counter),
// and returns normally, so the context stays usable.
// moe_selftest_fp4_wait: the 4-bit products' own way out.  One block computes
// gate/up tiles, then waits for a count that never fills: the producer gives up,
// the other warps leave their waits, copies and MMAs are drained, TMEM is freed.
#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// A counter nothing increments.
__device__ int g_selftest_counter = 0;

__global__ void bounded_wait_selftest_kernel(int32_t* dev_status) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);   // one arrival expected; none will come
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0 && !mbar_wait(&bar, 0, &abort_flag)) {
    atomicOr(dev_status, kDevTimeout);
    atomicOr(dev_status + 1, 1);
  }
  if (threadIdx.x == 32 && !wait_count(&g_selftest_counter, 1, &abort_flag)) {
    atomicOr(dev_status, kDevTimeout);
    atomicOr(dev_status + 1, 2);
  }
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_selftest_bounded_wait(int32_t* dev_status, moe_stream_t stream) {
  if (dev_status == nullptr) return MOE_ERR_INVALID_ARG;
  moe::bounded_wait_selftest_kernel<<<1, 64, 0, reinterpret_cast<cudaStream_t>(stream)>>>(dev_status);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

namespace {
// One expert of 128 rows, H = 512, I = 256, NVFP4: two stages a gate/up tile.
constexpr int kStH = 512, kStI = 256, kStRows = 128;
constexpr size_t kStXq = 0, kStXs = kStXq + kStRows * kStH / 2, kStW13 = kStXs + kStRows * kStH / 16,
                 kStS13 = kStW13 + 2 * kStI * kStH / 2, kStW2 = kStS13 + 2 * kStI * kStH / 16,
                 kStS2 = kStW2 + kStH * kStI / 2, kStZq = kStS2 + kStH * kStI / 16,
                 kStZs = kStZq + kStRows * kStI / 2, kStOut = kStZs + kStRows * kStI / 16,
                 kStCounts = kStOut + kStRows * kStH * 2, kStSync = kStCounts + 16, kStBytes = kStSync + 16;
}  // namespace

extern "C" size_t moe_selftest_fp4_scratch_size(void) { return kStBytes; }

extern "C" moe_status moe_selftest_fp4_wait(void* scratch, size_t scratch_bytes, int32_t* dev_status,
                                            moe_stream_t stream) {
  if (scratch == nullptr || dev_status == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 15u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (scratch_bytes < kStBytes) return MOE_ERR_WORKSPACE;
  const moe::RowLayout rl{kStRows, 0, kStRows};
  if (moe::gemm_fp4_sync_ints(1, rl, kStRows) * sizeof(int) > kStBytes - kStSync) return MOE_ERR_WORKSPACE;
  uint8_t* p = static_cast<uint8_t*>(scratch);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // zero codes and scales; more rows than the expert has room for; counts of the
  // row blocks so far below zero that the tiles cannot fill them; ticket 0
  cudaError_t err = cudaMemsetAsync(p, 0, kStBytes, s);
  if (err == cudaSuccess) err = cudaMemsetAsync(p + kStCounts, 1, 4, s);
  if (err == cudaSuccess) err = cudaMemsetAsync(p + kStSync + 4, 0x80, 4, s);
  if (err == cudaSuccess)
    err = moe::launch_gemm_both_fp4(p + kStXq, p + kStXs, nullptr, reinterpret_cast<int32_t*>(p + kStCounts),
                                    1, rl, kStH, kStI, p + kStW13, p + kStS13, nullptr, p + kStW2, p + kStS2,
                                    nullptr, nullptr, 0, p + kStZq, p + kStZs, p + kStOut,
                                    reinterpret_cast<int*>(p + kStSync), dev_status, 1, true, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
