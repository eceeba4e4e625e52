// Launchers of the cache write and read-back kernels (cache_io.cu).
#pragma once

#include <cuda_runtime.h>

#include "read_kv.cuh"
#include "write_kv.cuh"

namespace gqa {

// kvf: KvFormat, qf and of: QFormat; sms: the current device's SM count.
cudaError_t launch_write_kv(const WriteParams& p, int kvf, int qf, int sms, cudaStream_t stream);
cudaError_t launch_read_kv(const ReadParams& p, int kvf, int of, int sms, cudaStream_t stream);

}  // namespace gqa
