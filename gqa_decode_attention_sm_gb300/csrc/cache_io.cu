// The kernels that write many tokens into a cache and read a cache back, in a
// translation unit of their own.
#include <cuda_runtime.h>

#include <algorithm>

#include "gqa_decode.h"
#include "kernels/cache_io.h"

namespace gqa {

namespace {

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  // programmatic dependent launch, as the split kernel: the kernel waits for
  // the previous grid before its first read
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_write_kv(WriteParams& p, int kvf, int qf, int sms, cudaStream_t stream) {
  // Few tokens: a warp for each unit of four heads, so that the call's latency
  // is one unit's; many: a warp for each token, so that its angles are formed
  // once.
  p.parts = p.tokens <= 8 * sms ? kWriteUnits : 1;
  const long long items = (long long)p.tokens * p.parts;
  const dim3 grid((unsigned)std::min<long long>((items + kWriteWarps - 1) / kWriteWarps, 2LL * sms));
  const bool bf = qf == kQBF16;
  switch (kvf) {
    case kKvF16: return launch(write_kv_kernel<kKvF16, kQF16>, p, grid, kWriteThreads, stream);
    case kKvBF16: return launch(write_kv_kernel<kKvBF16, kQBF16>, p, grid, kWriteThreads, stream);
    case kKvE4M3:
      return launch(bf ? write_kv_kernel<kKvE4M3, kQBF16> : write_kv_kernel<kKvE4M3, kQF16>, p, grid, kWriteThreads,
                    stream);
    case kKvI8:
      return launch(bf ? write_kv_kernel<kKvI8, kQBF16> : write_kv_kernel<kKvI8, kQF16>, p, grid, kWriteThreads,
                    stream);
    default:
      return launch(bf ? write_kv_kernel<kKvE2M1, kQBF16> : write_kv_kernel<kKvE2M1, kQF16>, p, grid, kWriteThreads,
                    stream);
  }
}

cudaError_t launch_read_kv(const ReadParams& p, int kvf, int of, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.out_capacity + kReadChunk - 1) / kReadChunk), 2 * kHkv, (unsigned)p.batch);
  const bool bf = of == kQBF16;
  switch (kvf) {
    case kKvF16: return launch(bf ? read_kv_kernel<kKvF16, kQBF16> : read_kv_kernel<kKvF16, kQF16>, p, grid, kReadThreads, stream);
    case kKvBF16: return launch(bf ? read_kv_kernel<kKvBF16, kQBF16> : read_kv_kernel<kKvBF16, kQF16>, p, grid, kReadThreads, stream);
    case kKvE4M3: return launch(bf ? read_kv_kernel<kKvE4M3, kQBF16> : read_kv_kernel<kKvE4M3, kQF16>, p, grid, kReadThreads, stream);
    case kKvI8: return launch(bf ? read_kv_kernel<kKvI8, kQBF16> : read_kv_kernel<kKvI8, kQF16>, p, grid, kReadThreads, stream);
    default: return launch(bf ? read_kv_kernel<kKvE2M1, kQBF16> : read_kv_kernel<kKvE2M1, kQF16>, p, grid, kReadThreads, stream);
  }
}

}  // namespace gqa
