// Launchers of the prompt attention (prefill.cu) and of the draft verification, the
// weight sums and the eviction (serving.cu).
#pragma once

#include <cuda_runtime.h>

#include "evict_kv.cuh"
#include "prefill.cuh"
#include "sum_weights.cuh"
#include "verify_drafts.cuh"

namespace gqa {

// kvf: KvFormat, qf: QFormat, pf: ProbFormat; sms: the current device's SM count.
cudaError_t serving_setup();  // once a device
cudaError_t prefill_setup();  // once a device
cudaError_t launch_prefill(const PrefillParams& p, int kvf, int qf, cudaStream_t stream);
cudaError_t launch_verify_drafts(const DraftParams& p, int pf, cudaStream_t stream);
cudaError_t launch_sum_weights(const WeightParams& p, int kvf, int qf, int q_len, int sms, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, int kvf, int sms, cudaStream_t stream);

}  // namespace gqa
