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

template <int U>
cudaError_t launch_write_u(const WriteParams& p, int kvf, int qf, int sms, cudaStream_t stream) {
  const long long items = (long long)p.tokens * (kWriteUnits / U);
  const dim3 grid((unsigned)std::min<long long>((items + kWriteWarps - 1) / kWriteWarps, 2LL * sms));
  const bool bf = qf == kQBF16;
  const auto go = [&](auto kernel) { return launch(kernel, p, grid, kWriteThreads, stream); };
  switch (kvf) {
    case kKvF16: return go(write_kv_kernel<kKvF16, kQF16, U>);
    case kKvBF16: return go(write_kv_kernel<kKvBF16, kQBF16, U>);
    case kKvE4M3: return bf ? go(write_kv_kernel<kKvE4M3, kQBF16, U>) : go(write_kv_kernel<kKvE4M3, kQF16, U>);
    case kKvI8: return bf ? go(write_kv_kernel<kKvI8, kQBF16, U>) : go(write_kv_kernel<kKvI8, kQF16, U>);
    default: return bf ? go(write_kv_kernel<kKvE2M1, kQBF16, U>) : go(write_kv_kernel<kKvE2M1, kQF16, U>);
  }
}

cudaError_t launch_write_kv(const WriteParams& p, int kvf, int qf, int sms, cudaStream_t stream) {
  // Few tokens: a warp for each unit, so that the call's latency is one unit's, as
  // long as all are resident at once (202 tokens on 152 SMs), or three times that
  // where the cache's rounding makes a part of four units long.  In a CUDA graph,
  // us, units / parts: bf16 64 tokens 2.4 / 2.6, 200 2.5 / 3.1, 256 3.4 / 3.1, 768
  // 5.6 / 3.5; int8 64 3.0 / 5.0, 512 5.1 / 6.1, 768 6.9 / 5.9; e2m1 64 4.2 / 7.2,
  // 512 7.1 / 8.5, 768 8.9 / 8.2; e4m3, which rounds by one instruction, as the
  // 16-bit caches: 256 3.4 / 3.1, 512 4.6 / 3.6.
  const long long waves = kvf == kKvI8 || kvf == kKvE2M1 ? 3 : 1;
  return (long long)p.tokens * kWriteUnits <= waves * 2 * kWriteWarps * sms
             ? launch_write_u<1>(p, kvf, qf, sms, stream)
             : launch_write_u<4>(p, kvf, qf, sms, stream);
}

// About 64 CTAs an SM (8 waves) over the rows: lengths are on the device, so the
// grid covers the capacity and short rows leave early; with fewer CTAs the long
// rows finish late (8 x U[16k, 32k] e2m1 tokens: 148 us; 155 with 32).
template <int KVF>
cudaError_t launch_read_t(const ReadParams& p, int of, int sms, cudaStream_t stream) {
  const long long rows = 2LL * kHkv * p.batch;
  const long long chunks = ((long long)p.out_capacity + kReadChunk - 1) / kReadChunk;
  const long long want = (64LL * sms + rows - 1) / rows;
  const dim3 grid((unsigned)std::min(chunks, want), 2 * kHkv, (unsigned)p.batch);
  return launch(of == kQBF16 ? read_kv_kernel<KVF, kQBF16> : read_kv_kernel<KVF, kQF16>, p, grid, kReadThreads, stream);
}

cudaError_t launch_read_kv(const ReadParams& p, int kvf, int of, int sms, cudaStream_t stream) {
  switch (kvf) {
    case kKvF16: return launch_read_t<kKvF16>(p, of, sms, stream);
    case kKvBF16: return launch_read_t<kKvBF16>(p, of, sms, stream);
    case kKvE4M3: return launch_read_t<kKvE4M3>(p, of, sms, stream);
    case kKvI8: return launch_read_t<kKvI8>(p, of, sms, stream);
    default: return launch_read_t<kKvE2M1>(p, of, sms, stream);
  }
}

}  // namespace gqa
