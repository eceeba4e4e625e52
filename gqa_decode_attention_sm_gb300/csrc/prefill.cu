// The attention of chunks of new tokens, in a translation unit of its own.
#include <cuda_runtime.h>

#include <atomic>

#include "gqa_decode.h"
#include "kernels/serving.h"

namespace gqa {

namespace {

// The driver's encoder of tensor maps, looked up at a device's first call (no link to the
// driver library; two devices' first calls may meet, and find the same).
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<Encode> g_encode{nullptr};

// A cache's rows in boxes of `box`: of a 16-bit cache 64 elements wide and swizzled, of
// a narrow one whole rows as they are.
CUresult encode(CUtensorMap* map, const CacheView& c, int kvf, int box) {
  const cuuint32_t steps[2] = {1, 1};
  if (is_narrow(kvf)) {
    const cuuint64_t width = (cuuint64_t)kv_row_bytes(kvf), dims[2] = {width, c.rows}, strides[1] = {width};
    const cuuint32_t tile[2] = {(cuuint32_t)width, (cuuint32_t)box};
    return g_encode.load()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(c.kv), dims, strides, tile, steps,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  const cuuint64_t dims[2] = {kD, c.rows}, strides[1] = {2 * kD};
  const cuuint32_t tile[2] = {kD / 2, (cuuint32_t)box};
  return g_encode.load()(map, kvf == kKvBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                         const_cast<void*>(c.kv), dims, strides, tile, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

cudaError_t encode_rows(CUtensorMap* map, const CacheView& c, int kvf, int box) {
  if (encode(map, c, kvf, box) == CUDA_SUCCESS) return cudaSuccess;
  // A thread that has not called the runtime yet has no current context, which the
  // driver's encoder asks for; setting the device that it has gives it one.
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);
  if (e != cudaSuccess) return e;
  return encode(map, c, kvf, box) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int KVF, int QF>
cudaError_t set_attributes() {
  return cudaFuncSetAttribute(prefill_kernel<KVF, QF>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PfShared));
}

template <int KVF, int QF>
cudaError_t launch_t(const PrefillParams& p, const CUtensorMap& map, cudaStream_t stream) {
  // programmatic dependent launch, as the split kernel: the kernels wait for the
  // previous grid before their first read
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = sizeof(PfShared);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_kernel<KVF, QF>, p, map);
  if (e != cudaSuccess || p.ctas == 1) return e;
  cfg.gridDim = dim3((unsigned)p.ctas - 1, 2 * kPfRows / 32);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<QF>, p);
}

}  // namespace

static_assert(sizeof(PfShared) <= 227 * 1024, "shared memory of a CTA");

cudaError_t prefill_setup() {
  if (!g_encode.load()) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<Encode>(fn);
  }
  // (the merge kernel keeps the split of shared memory and L1 that the other needs:
  // changing it between the two would wait until an SM is empty)
  cudaError_t e = cudaFuncSetAttribute(prefill_merge_kernel<kQF16>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prefill_merge_kernel<kQBF16>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess) e = set_attributes<kKvF16, kQF16>();
  if (e == cudaSuccess) e = set_attributes<kKvBF16, kQBF16>();
  if (e == cudaSuccess) e = set_attributes<kKvE4M3, kQF16>();
  if (e == cudaSuccess) e = set_attributes<kKvE4M3, kQBF16>();
  if (e == cudaSuccess) e = set_attributes<kKvI8, kQF16>();
  if (e == cudaSuccess) e = set_attributes<kKvI8, kQBF16>();
  if (e == cudaSuccess) e = set_attributes<kKvE2M1, kQF16>();
  if (e == cudaSuccess) e = set_attributes<kKvE2M1, kQBF16>();
  return e;
}

cudaError_t launch_prefill(const PrefillParams& params, int kvf, int qf, cudaStream_t stream) {
  PrefillParams p = params;
  CUtensorMap map = {};
  p.box = p.c.block_table && p.c.page_log2 < 7 ? 1 << p.c.page_log2 : kPfTile;
  const cudaError_t e = encode_rows(&map, p.c, kvf, p.box);
  if (e != cudaSuccess) return e;
  const bool bf = qf == kQBF16;
  switch (kvf) {
    case kKvF16: return launch_t<kKvF16, kQF16>(p, map, stream);
    case kKvBF16: return launch_t<kKvBF16, kQBF16>(p, map, stream);
    case kKvE4M3: return bf ? launch_t<kKvE4M3, kQBF16>(p, map, stream) : launch_t<kKvE4M3, kQF16>(p, map, stream);
    case kKvI8: return bf ? launch_t<kKvI8, kQBF16>(p, map, stream) : launch_t<kKvI8, kQF16>(p, map, stream);
    default: return bf ? launch_t<kKvE2M1, kQBF16>(p, map, stream) : launch_t<kKvE2M1, kQF16>(p, map, stream);
  }
}

}  // namespace gqa
