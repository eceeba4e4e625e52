// The kernels that verify drafts, sum softmax weights and make a cache smaller, in a
// translation unit of their own.
#include <cuda_runtime.h>

#include <algorithm>

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

cudaError_t serving_setup() {
  return cudaFuncSetAttribute(select_kv_kernel<kSelectThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectKeys * 4);
}

cudaError_t launch_verify_drafts(const DraftParams& p, int pf, int sms, cudaStream_t stream) {
  const int S = 8;
  const dim3 grid((unsigned)(p.batch * S));
  switch (pf) {
    case kPF16: return launch(verify_drafts_kernel<kPF16>, grid, kDraftThreads, 0, S, stream, p);
    case kPBF16: return launch(verify_drafts_kernel<kPBF16>, grid, kDraftThreads, 0, S, stream, p);
    default: return launch(verify_drafts_kernel<kPF32>, grid, kDraftThreads, 0, S, stream, p);
  }
}

template <int KVF, int QF>
cudaError_t launch_score(const WeightParams& p, int q_len, cudaStream_t stream) {
  const dim3 grid((unsigned)p.chunks, kHkv, (unsigned)p.c.batch);
  return q_len <= 2 ? launch(score_kv_kernel<KVF, QF, 1>, grid, kScoreThreads, 0, 1, stream, p, q_len)
                    : launch(score_kv_kernel<KVF, QF, 2>, grid, kScoreThreads, 0, 1, stream, p, q_len);
}

cudaError_t launch_sum_weights(const WeightParams& p, int kvf, int qf, int q_len, cudaStream_t stream) {
  const bool bf = qf == kQBF16;
  cudaError_t e;
  switch (kvf) {
    case kKvF16: e = launch_score<kKvF16, kQF16>(p, q_len, stream); break;
    case kKvBF16: e = launch_score<kKvBF16, kQBF16>(p, q_len, stream); break;
    case kKvE4M3: e = bf ? launch_score<kKvE4M3, kQBF16>(p, q_len, stream) : launch_score<kKvE4M3, kQF16>(p, q_len, stream); break;
    case kKvI8: e = bf ? launch_score<kKvI8, kQBF16>(p, q_len, stream) : launch_score<kKvI8, kQF16>(p, q_len, stream); break;
    default: e = bf ? launch_score<kKvE2M1, kQBF16>(p, q_len, stream) : launch_score<kKvE2M1, kQF16>(p, q_len, stream);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.c.capacity + kSumSlots - 1) / kSumSlots), kHkv, (unsigned)p.c.batch);
  switch (q_len) {
    case 1: return launch(sum_weights_kernel<4>, grid, kSumThreads, 0, 1, stream, p);
    case 2: return launch(sum_weights_kernel<8>, grid, kSumThreads, 0, 1, stream, p);
    case 3: return launch(sum_weights_kernel<12>, grid, kSumThreads, 0, 1, stream, p);
    default: return launch(sum_weights_kernel<16>, grid, kSumThreads, 0, 1, stream, p);
  }
}

cudaError_t launch_evict(const EvictParams& p, int kvf, cudaStream_t stream) {
  // as many CTAs a head as hold its weights, 4096 each at least (each adds to the
  // cluster barriers' time), 8 at most
  int S = 1;
  while (S < 8 && (p.src.capacity + S - 1) / S > 4096) S *= 2;
  EvictParams e = p;
  const long long seg = ((p.src.capacity + S - 1) / S + 31) / 32 * 32;
  e.cluster = S;
  e.held = seg <= kSelectKeys ? (int)seg : 0;
  cudaError_t err = launch(select_kv_kernel<kSelectThreads>, dim3((unsigned)(p.batch * kHkv * S)), kSelectThreads, (size_t)e.held * 4, S,
                           stream, e);
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
