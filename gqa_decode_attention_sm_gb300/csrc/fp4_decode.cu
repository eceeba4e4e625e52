// The split kernel's instances for an e2m1 (4-bit) cache, in a translation unit
// of their own so that they compile beside the other formats'.
#include <cuda_runtime.h>

#include "gqa_decode.h"
#include "kernels/split_launch.cuh"

namespace gqa {

cudaError_t e2m1_setup(ClusterFit (&fit)[2]) {
  cudaError_t e = set_split_attributes<kKvE2M1, kQF16>();
  if (e == cudaSuccess) e = set_split_attributes<kKvE2M1, kQBF16>();
  if (e == cudaSuccess) e = query_cluster_fits<kKvE2M1, kQF16>(fit[kQF16]);
  if (e == cudaSuccess) e = query_cluster_fits<kKvE2M1, kQBF16>(fit[kQBF16]);
  return e;
}

cudaError_t e2m1_launch_split(const SplitParams& sp, int qf, int q_len, int bal_ctas, int cluster,
                              cudaStream_t stream) {
  return qf == kQBF16 ? launch_split_t<kKvE2M1, kQBF16>(sp, q_len, bal_ctas, cluster, stream)
                      : launch_split_t<kKvE2M1, kQF16>(sp, q_len, bal_ctas, cluster, stream);
}

}  // namespace gqa
