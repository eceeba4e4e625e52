// The attention of chunks of new tokens, in a translation unit of its own.
#include <cuda_runtime.h>

#include "gqa_decode.h"
#include "kernels/serving.h"

namespace gqa {

cudaError_t launch_prefill(const PrefillParams& p, int kvf, int qf, int sms, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.tokens + 3) / 4), kHkv);
  const auto go = [&](auto kernel) {
    kernel<<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
  };
  const bool bf = qf == kQBF16;
  switch (kvf) {
    case kKvF16: return go(prefill_kernel<kKvF16, kQF16>);
    case kKvBF16: return go(prefill_kernel<kKvBF16, kQBF16>);
    case kKvE4M3: return bf ? go(prefill_kernel<kKvE4M3, kQBF16>) : go(prefill_kernel<kKvE4M3, kQF16>);
    case kKvI8: return bf ? go(prefill_kernel<kKvI8, kQBF16>) : go(prefill_kernel<kKvI8, kQF16>);
    default: return bf ? go(prefill_kernel<kKvE2M1, kQBF16>) : go(prefill_kernel<kKvE2M1, kQF16>);
  }
}

}  // namespace gqa
