// Self-check of the bounded waits every kernel relies on: a grid barrier that
// one participant never reaches, an mbarrier phase that nothing completes, and
// such a phase in one CTA of a cluster, of which the others learn.
// All give up after the wait limit, record DT_DEV_TIMEOUT in the status word
// and return, so the context stays usable; nothing faults, traps or hangs.
#include "chainlib.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"

namespace dt {

namespace {

// which = 0: a grid barrier of two CTAs where CTA 1 leaves without arriving;
// which = 1: one CTA waits on an mbarrier that no thread arrives on;
// which = 2: the last CTA of a cluster does, and the first records it.
__global__ void __launch_bounds__(cl::kThreads, 1) k_wait_check(unsigned* bar, int* status, int which) {
  __shared__ int s_abort;
  __shared__ uint32_t s_gave_up;
  __shared__ __align__(8) uint64_t s_mbar;
  if (which == 0) {
    if (blockIdx.x != 0) return;  // the missing participant
    unsigned epoch = 0;
    cl::grid_barrier(bar, epoch, status, &s_abort);
    return;
  }
  if (threadIdx.x == 0) {
    s_gave_up = 0;
    mbar_init(&s_mbar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (which == 2) {
    if (threadIdx.x == 0 && blockIdx.x + 1 == gridDim.x && !mbar_wait(&s_mbar, 0u, nullptr)) s_gave_up = 1;
    __syncthreads();
    cluster_barrier();
    if (blockIdx.x == 0 && threadIdx.x < 32 && __any_sync(0xFFFFFFFFu, gave_up_beside(&s_gave_up, static_cast<int>(gridDim.x)) != 0) && threadIdx.x == 0)
      dt_report(status, DT_DEV_TIMEOUT);
    cluster_barrier();  // (no CTA leaves while its word is read)
    return;
  }
  if (threadIdx.x == 0) mbar_wait(&s_mbar, 0u, status);
  __syncthreads();
}

}  // namespace

cudaError_t launch_wait_check(unsigned* bar, int* status, int which, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const unsigned cluster = 4;
  cfg.gridDim = dim3(which == 0 ? 2 : which == 1 ? 1 : cluster);
  cfg.blockDim = dim3(cl::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (which == 0) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = which == 1 ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, k_wait_check, bar, status, which);
}

}  // namespace dt
