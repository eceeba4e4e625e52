// The kernels that verify drafts, sum softmax weights and make a cache smaller, in a
// translation unit of their own.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gqa_decode.h"
#include "kernels/serving.h"

namespace gqa {

namespace {

constexpr int kSelectThreads = kSelectBins / 2;

// Programmatic dependent launch, as the split kernel (each kernel waits for the
// previous grid before its first read), in clusters of `cluster` CTAs.
template <class... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                   const P&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p...);
}

}  // namespace

cudaError_t launch_verify_drafts(const DraftParams& p, int pf, cudaStream_t stream) {
  constexpr int S = kDraftCluster;
  const dim3 grid((unsigned)(p.batch * S));
  switch (pf) {
    case kPF16: return launch(verify_drafts_kernel<kPF16>, grid, kDraftThreads, 0, S, stream, p);
    case kPBF16: return launch(verify_drafts_kernel<kPBF16>, grid, kDraftThreads, 0, S, stream, p);
    default: return launch(verify_drafts_kernel<kPF32>, grid, kDraftThreads, 0, S, stream, p);
  }
}

// f(KVF, QF) as integral constants
template <class F>
cudaError_t with_formats(int kvf, int qf, const F& f) {
  const auto of = [&](auto k) {
    return qf == kQBF16 ? f(k, std::integral_constant<int, kQBF16>()) : f(k, std::integral_constant<int, kQF16>());
  };
  switch (kvf) {
    case kKvF16: return f(std::integral_constant<int, kKvF16>(), std::integral_constant<int, kQF16>());
    case kKvBF16: return f(std::integral_constant<int, kKvBF16>(), std::integral_constant<int, kQBF16>());
    case kKvE4M3: return of(std::integral_constant<int, kKvE4M3>());
    case kKvI8: return of(std::integral_constant<int, kKvI8>());
    default: return of(std::integral_constant<int, kKvE2M1>());
  }
}

cudaError_t serving_setup() {
  cudaError_t e = cudaFuncSetAttribute(select_kv_kernel<kSelectThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectKeys * 4);
  for (int kvf = kKvF16; kvf <= kKvE2M1 && e == cudaSuccess; ++kvf)
    for (int qf = kQF16; qf <= kQBF16 && e == cudaSuccess; ++qf)
      e = with_formats(kvf, qf, [](auto k, auto q) {
        const cudaError_t x = cudaFuncSetAttribute(fused_weights_kernel<k(), q(), 1>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreBytes);
        return x != cudaSuccess ? x : cudaFuncSetAttribute(fused_weights_kernel<k(), q(), 2>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreBytes);
      });
  return e;
}

cudaError_t launch_sum_weights(const WeightParams& params, int kvf, int qf, int q_len, int sms, cudaStream_t stream) {
  WeightParams p = params;
  // One launch where a cluster of 8 CTAs holds a row's scores and such clusters fill
  // the GPU, or the rows are short (every CTA of a row then has a few slabs of slots).
  const long long part = ((p.c.capacity + kRowCluster - 1LL) / kRowCluster + kSlab - 1) / kSlab * kSlab, bytes = part * 16 * q_len;
  if (bytes <= kScoreBytes && ((long long)kRowCluster * kHkv * p.c.batch >= sms || p.c.capacity <= 8192)) {
    p.held = (int)part;
    return with_formats(kvf, qf, [&](auto k, auto q) {
      return q_len <= 2 ? launch(fused_weights_kernel<k(), q(), 1>, dim3((unsigned)(kRowCluster * kHkv * p.c.batch)), kScoreThreads,
                                 (size_t)bytes, kRowCluster, stream, p, q_len)
                        : launch(fused_weights_kernel<k(), q(), 2>, dim3((unsigned)(kRowCluster * kHkv * p.c.batch)), kScoreThreads,
                                 (size_t)bytes, kRowCluster, stream, p, q_len);
    });
  }
  const dim3 scores((unsigned)p.chunks, kHkv, (unsigned)p.c.batch);
  const cudaError_t e = with_formats(kvf, qf, [&](auto k, auto q) {
    return q_len <= 2 ? launch(score_kv_kernel<k(), q(), 1>, scores, kScoreThreads, 0, 1, stream, p, q_len)
                      : launch(score_kv_kernel<k(), q(), 2>, scores, kScoreThreads, 0, 1, stream, p, q_len);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.c.capacity + kSumSlots - 1) / kSumSlots), kHkv, (unsigned)p.c.batch);
  switch (q_len) {
    case 1: return launch(sum_weights_kernel<4>, grid, kSumThreads, 0, 1, stream, p);
    case 2: return launch(sum_weights_kernel<8>, grid, kSumThreads, 0, 1, stream, p);
    case 3: return launch(sum_weights_kernel<12>, grid, kSumThreads, 0, 1, stream, p);
    default: return launch(sum_weights_kernel<16>, grid, kSumThreads, 0, 1, stream, p);
  }
}

cudaError_t launch_evict(const EvictParams& p, int kvf, int sms, cudaStream_t stream) {
  EvictParams e = p;
  e.cluster = 1;
  const int C = p.src.capacity;
  cudaError_t err;
  if (C <= kFewSlots) {
    const auto few = [&](auto kernel) { return launch(kernel, dim3((unsigned)(p.batch * kHkv)), kFewThreads, 0, 1, stream, e); };
    err = C <= 2 * kFewThreads   ? few(select_few_kernel<2>)
          : C <= 8 * kFewThreads ? few(select_few_kernel<8>)
                                 : few(select_few_kernel<16>);
  } else {
    // CTAs a head: one wave of them, 8 at most (each adds to the cluster's barriers and
    // to the histograms that every one reads), as many as hold the weights if need be
    while (e.cluster < 8 && (2LL * e.cluster * p.batch * kHkv <= sms || C > (long long)kSelectKeys * e.cluster)) e.cluster *= 2;
    const long long seg = ((C + e.cluster - 1LL) / e.cluster + 31) / 32 * 32;
    e.held = seg <= kSelectKeys ? (int)seg : 0;
    err = launch(select_kv_kernel<kSelectThreads>, dim3((unsigned)(p.batch * kHkv * e.cluster)), kSelectThreads,
                 (size_t)e.held * 4, e.cluster, stream, e);
  }
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)((long long)p.batch * kHkv * 2 * p.chunks));
  switch (kvf) {
    case kKvF16: return launch(move_kv_kernel<kKvF16>, grid, kMoveThreads, 0, 1, stream, e);
    case kKvBF16: return launch(move_kv_kernel<kKvF16>, grid, kMoveThreads, 0, 1, stream, e);
    case kKvE4M3: return launch(move_kv_kernel<kKvE4M3>, grid, kMoveThreads, 0, 1, stream, e);
    case kKvI8: return launch(move_kv_kernel<kKvI8>, grid, kMoveThreads, 0, 1, stream, e);
    default: return launch(move_kv_kernel<kKvE2M1>, grid, kMoveThreads, 0, 1, stream, e);
  }
}

}  // namespace gqa
