// Launching the split kernel of one KV format: the one-time set-up of its
// instances and the launch itself.  Shared by the translation units that hold
// the kernel's instances (the formats are compiled side by side).
#pragma once

#include <cuda_runtime.h>

#include "split_kv_mma.cuh"

namespace gqa {

constexpr int kClusterMaxSplits = 8;  // the on-chip merge: clusters of 2..8 splits (portable sizes)

// The most clusters of s CTAs of one format's cluster-merge kernel that can be
// resident at once, by [q_len - 1][s] (cudaOccupancyMaxActiveClusters).
using ClusterFit = int[kMaxQLen][kClusterMaxSplits + 1];

template <int KVF, int QF>
cudaError_t set_split_attributes() {
  cudaError_t e = cudaSuccess;
  const auto set = [&](auto kernel, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set(split_kv_mma_kernel<KVF, QF, 1, false, false>, mma_smem_bytes(KVF, 1));
  set(split_kv_mma_kernel<KVF, QF, 2, false, false>, mma_smem_bytes(KVF, 2));
  set(split_kv_mma_kernel<KVF, QF, 3, false, false>, mma_smem_bytes(KVF, 3));
  set(split_kv_mma_kernel<KVF, QF, 4, false, false>, mma_smem_bytes(KVF, 4));
  set(split_kv_mma_kernel<KVF, QF, 1, true, false>, mma_smem_bytes(KVF, 1, true));
  set(split_kv_mma_kernel<KVF, QF, 2, true, false>, mma_smem_bytes(KVF, 2, true));
  set(split_kv_mma_kernel<KVF, QF, 3, true, false>, mma_smem_bytes(KVF, 3, true));
  set(split_kv_mma_kernel<KVF, QF, 4, true, false>, mma_smem_bytes(KVF, 4, true));
  set(split_kv_mma_kernel<KVF, QF, 1, false, true>, mma_smem_bytes(KVF, 1));
  set(split_kv_mma_kernel<KVF, QF, 2, false, true>, mma_smem_bytes(KVF, 2));
  set(split_kv_mma_kernel<KVF, QF, 3, false, true>, mma_smem_bytes(KVF, 3));
  set(split_kv_mma_kernel<KVF, QF, 4, false, true>, mma_smem_bytes(KVF, 4));
  return e;
}

template <int KVF, int QF, int NQ>
cudaError_t query_cluster_fit(ClusterFit& fit) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMmaThreads, 1, 1);
  cfg.dynamicSmemBytes = mma_smem_bytes(KVF, NQ);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (int s = 2; s <= kClusterMaxSplits; ++s) {
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)s;
    cfg.gridDim = dim3(kHkv, 1, (unsigned)s);
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, split_kv_mma_kernel<KVF, QF, NQ, false, true>, &cfg);
    if (e != cudaSuccess) return e;
    fit[NQ - 1][s] = n;
  }
  return cudaSuccess;
}

template <int KVF, int QF>
cudaError_t query_cluster_fits(ClusterFit& fit) {
  cudaError_t e = query_cluster_fit<KVF, QF, 1>(fit);
  if (e == cudaSuccess) e = query_cluster_fit<KVF, QF, 2>(fit);
  if (e == cudaSuccess) e = query_cluster_fit<KVF, QF, 3>(fit);
  if (e == cudaSuccess) e = query_cluster_fit<KVF, QF, 4>(fit);
  return e;
}

// `bal_ctas` > 0: the balanced schedule on that many CTAs (single token).
// `cluster`: the one-piece grid as clusters of its `cluster` splits, merged
// on chip (no combine kernel).
template <int KVF, int QF, bool BAL, bool CL>
cudaError_t launch_nq(cudaLaunchConfig_t& cfg, const SplitParams& sp, int q_len) {
  switch (q_len) {
    case 1: return cudaLaunchKernelEx(&cfg, split_kv_mma_kernel<KVF, QF, 1, BAL, CL>, sp);
    case 2: return cudaLaunchKernelEx(&cfg, split_kv_mma_kernel<KVF, QF, 2, BAL, CL>, sp);
    case 3: return cudaLaunchKernelEx(&cfg, split_kv_mma_kernel<KVF, QF, 3, BAL, CL>, sp);
    default: return cudaLaunchKernelEx(&cfg, split_kv_mma_kernel<KVF, QF, 4, BAL, CL>, sp);
  }
}

template <int KVF, int QF>
cudaError_t launch_split_t(const SplitParams& sp, int q_len, int bal_ctas, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMmaThreads, 1, 1);
  cfg.stream = stream;
  // programmatic dependent launch: CTAs may become resident while the
  // previous grid in the stream drains; they wait (griddepcontrol.wait)
  // before reading any input
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (bal_ctas > 0) {
    cfg.gridDim = dim3(bal_ctas, 1, 1);
    cfg.dynamicSmemBytes = mma_smem_bytes(KVF, q_len, true);
    return launch_nq<KVF, QF, true, false>(cfg, sp, q_len);
  }
  cfg.gridDim = dim3(kHkv, sp.batch, sp.splits_eff);
  cfg.dynamicSmemBytes = mma_smem_bytes(KVF, q_len);
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)cluster;
    cfg.numAttrs = 2;
    return launch_nq<KVF, QF, false, true>(cfg, sp, q_len);
  }
  return launch_nq<KVF, QF, false, false>(cfg, sp, q_len);
}

// The e2m1 cache's instances (fp4_decode.cu); qf is a QFormat.
cudaError_t e2m1_setup(ClusterFit (&fit)[2]);
cudaError_t e2m1_launch_split(const SplitParams& sp, int qf, int q_len, int bal_ctas, int cluster,
                              cudaStream_t stream);

}  // namespace gqa
