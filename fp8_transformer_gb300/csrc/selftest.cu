// Self-test of the bounded-wait path (no counterpart on the pages; it checks this library's own
// failure reporting).  One thread waits on an mbarrier that nothing completes, with a short
// limit: the wait gives up, records TE_ERR_TIMEOUT in the device status word and returns, the
// kernel exits normally and the context stays usable.  This is the same wait, with the same
// bookkeeping, that every pipeline of the GEMM and the norm backward goes through.
#include "kernels.h"
#include "sync.cuh"
#include "umma.cuh"

namespace te {
namespace {

__global__ void wait_timeout_kernel(int* status, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    mbar_init_fence();
  }
  __syncthreads();
  // phase 0 of a fresh barrier with one expected arrival and no arriving thread: never completes
  if (threadIdx.x == 0) wait_bounded(smem_u32(&bar), 0, nullptr, status, limit_ns, false);
}

// The end of a kernel whose CTAs read one another's sums (dense_few.cu): one CTA of a cluster gives up a wait, and
// none of them may write.  out[rank] = 1 where a CTA would.
constexpr int kClusterTest = 8;
__global__ void __cluster_dims__(kClusterTest, 1, 1) cluster_abort_kernel(int* status, uint64_t limit_ns, int waits, int* out) {
  __shared__ uint64_t bar;
  __shared__ volatile int abort_flag;
  const int rank = int(cluster_rank());
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  if (threadIdx.x == 0 && rank == waits) wait_bounded(smem_u32(&bar), 0, &abort_flag, status, limit_ns, true);
  __syncthreads();
  cluster_sync();
  const bool stop = ClusterFlags<kClusterTest>(&abort_flag, kClusterTest, rank).raised();
  const bool all = __syncthreads_and(!stop) != 0, any = __syncthreads_or(!stop) != 0;
  if (threadIdx.x == 0) out[rank] = all ? 1 : any ? 2 : 0;
  cluster_sync();
}

}  // namespace
}  // namespace te

extern "C" te_status te_selftest_wait_timeout(int64_t limit_us, void* stream) {
  if (limit_us <= 0 || limit_us > 1000000) return TE_ERR_INVALID_ARG;
  te::wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      te::device_status_ptr(), uint64_t(limit_us) * 1000u);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

extern "C" te_status te_selftest_cluster_abort(int64_t limit_us, int rank, int32_t* out, void* stream) {
  if (limit_us <= 0 || limit_us > 1000000 || rank < -1 || rank >= te::kClusterTest || !out ||
      reinterpret_cast<uintptr_t>(out) % 4)
    return TE_ERR_INVALID_ARG;
  te::cluster_abort_kernel<<<te::kClusterTest, 64, 0, static_cast<cudaStream_t>(stream)>>>(
      te::device_status_ptr(), uint64_t(limit_us) * 1000u, rank, out);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}
