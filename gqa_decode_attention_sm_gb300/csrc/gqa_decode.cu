// Host side of libgqa_decode.so: argument validation, the one-time device
// check, the split planner, workspace layout and kernel launches behind the C
// ABI declared in include/gqa_decode.h.
//
// The API shape follows the "FlashInfer sm110_gqa_decode" article: a
// convenience call, a prepared call that allocates nothing and reads nothing
// back (capturable in a CUDA graph), fail-fast validation before any launch
// (its "prepare" step: contiguous/aligned tensors, output not aliasing an
// input, finite positive q_scale, a compatible device), and a split-KV
// workspace owned by the caller.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "gqa_decode.h"
#include "kernels/append_kv.cuh"
#include "kernels/cache_io.h"
#include "kernels/combine.cuh"
#include "kernels/common.cuh"
#include "kernels/serving.h"
#include "kernels/split_launch.cuh"

static_assert(GQA_MAX_SPLITS <= 32 * gqa::kCombineChunks, "the combine's chunks cover every split slot");

namespace {

using namespace gqa;

thread_local std::string g_last_error;

gqa_status_t fail(gqa_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

gqa_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(GQA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// ---------------------------------------------------------------- devices

constexpr int kMaxDevices = 64;

// Per-device result of the one-time check.  Kept once known for good: the
// device is ready (sm_count set) or is not a compute capability 10.3 part.  A
// CUDA error during the check is not kept, so a later call retries it.
struct DeviceState {
  std::mutex mu;
  std::atomic<int> state{0};  // 0 unknown, 1 ready, 2 unsupported
  gqa_status_t status = GQA_ERR_UNSUPPORTED_DEVICE;
  int sm_count = 0;
  std::string message;
  // The most clusters of s CTAs of the cluster-merge split kernel that can be
  // resident at once, by [KV format][q format][q_len - 1][s]
  // (cudaOccupancyMaxActiveClusters).  A cluster's CTAs share one GPC, so a
  // grid that nearly fills the SMs can hold fewer clusters than slots / s.
  ClusterFit cluster_fit[5][2] = {};
};
DeviceState g_devices[kMaxDevices];

// One-time per-device check (compute capability 10.3), opt-in to the split
// kernel's dynamic shared memory, and the cluster occupancy table.  Runs
// with `dev` current.
void init_device(int dev, DeviceState& st) {
  int major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    st.status = GQA_ERR_CUDA;
    st.message = std::string("device query failed: ") + cudaGetErrorString(e);
    return;
  }
  if (major != 10 || minor != 3) {
    st.status = GQA_ERR_UNSUPPORTED_DEVICE;
    char buf[160];
    snprintf(buf, sizeof buf, "GQA decode requires compute capability 10.3 (sm_103); device %d is %d.%d",
             dev, major, minor);
    st.message = buf;
    return;
  }
  int prev = -1;
  cudaGetDevice(&prev);
  if (prev != dev) cudaSetDevice(dev);
  cudaError_t a = set_split_attributes<kKvF16, kQF16>();
  if (a == cudaSuccess) a = set_split_attributes<kKvBF16, kQBF16>();
  if (a == cudaSuccess) a = set_split_attributes<kKvE4M3, kQBF16>();
  if (a == cudaSuccess) a = set_split_attributes<kKvE4M3, kQF16>();
  if (a == cudaSuccess) a = set_split_attributes<kKvI8, kQBF16>();
  if (a == cudaSuccess) a = set_split_attributes<kKvI8, kQF16>();
  const char* what = "cudaFuncSetAttribute";
  if (a == cudaSuccess) {
    what = "cudaOccupancyMaxActiveClusters";
    a = query_cluster_fits<kKvF16, kQF16>(st.cluster_fit[kKvF16][kQF16]);
    if (a == cudaSuccess) a = query_cluster_fits<kKvBF16, kQBF16>(st.cluster_fit[kKvBF16][kQBF16]);
    if (a == cudaSuccess) a = query_cluster_fits<kKvE4M3, kQBF16>(st.cluster_fit[kKvE4M3][kQBF16]);
    if (a == cudaSuccess) a = query_cluster_fits<kKvE4M3, kQF16>(st.cluster_fit[kKvE4M3][kQF16]);
    if (a == cudaSuccess) a = query_cluster_fits<kKvI8, kQBF16>(st.cluster_fit[kKvI8][kQBF16]);
    if (a == cudaSuccess) a = query_cluster_fits<kKvI8, kQF16>(st.cluster_fit[kKvI8][kQF16]);
  }
  if (a == cudaSuccess) {
    what = "setting up the e2m1 kernels";
    a = e2m1_setup(st.cluster_fit[kKvE2M1]);
  }
  if (a == cudaSuccess) {
    what = "setting up the serving kernels";
    a = serving_setup();
    if (a == cudaSuccess) a = prefill_setup();
  }
  if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  if (a != cudaSuccess) {
    st.status = GQA_ERR_CUDA;
    st.message = std::string(what) + " failed: " + cudaGetErrorString(a);
    return;
  }
  st.sm_count = sms;
  st.status = GQA_OK;
}

gqa_status_t device_ready(int dev, int* sm_count) {
  if (dev < 0 || dev >= kMaxDevices) return fail(GQA_ERR_UNSUPPORTED_DEVICE, "device %d out of range", dev);
  DeviceState& st = g_devices[dev];
  int known = st.state.load(std::memory_order_acquire);
  if (known == 0) {
    std::lock_guard<std::mutex> lock(st.mu);
    known = st.state.load(std::memory_order_relaxed);
    if (known == 0) {
      init_device(dev, st);
      if (st.status == GQA_OK) known = 1;
      else if (st.status == GQA_ERR_UNSUPPORTED_DEVICE) known = 2;
      else return fail(st.status, "%s", st.message.c_str());  // not kept: retried next call
      st.state.store(known, std::memory_order_release);
    }
  }
  if (known == 2) return fail(GQA_ERR_UNSUPPORTED_DEVICE, "%s", st.message.c_str());
  if (sm_count) *sm_count = st.sm_count;
  return GQA_OK;
}

gqa_status_t current_device_ready(int* sm_count) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  return device_ready(dev, sm_count);
}

// ------------------------------------------------------------- validation

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool known_format(int fmt) { return fmt >= kKvF16 && fmt <= kKvE2M1; }

size_t partial_o_bytes(int batch, int splits) {
  return align_up((size_t)batch * kHq * splits * kD * sizeof(float), 256);
}
size_t partial_ml_bytes(int batch, int splits) {
  return align_up((size_t)batch * kHq * splits * sizeof(float), 256);
}

size_t workspace_bytes_for(int batch, int splits) {
  if (splits <= 1) return GQA_WORKSPACE_HEADER_BYTES;
  return GQA_WORKSPACE_HEADER_BYTES + partial_o_bytes(batch, splits) + 2 * partial_ml_bytes(batch, splits);
}

struct Call {
  const void* q;
  int q_dtype;
  const void* kv;
  int kv_format;
  const int32_t* lens;
  void* out;
  int batch, capacity;
  float q_scale, k_scale, v_scale;
  int num_splits;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
  uint64_t wait_budget_ns = kWaitBudgetNs;
  int skip_tile = -1;
  const void* kv_scales = nullptr;  // int8 (bf16) and e2m1 (e4m3) caches only
  const int32_t* block_table = nullptr;  // paged cache only
  int page_log2 = 0, max_pages = 0, num_pages = 0;
  int q_len = 1;  // query tokens per request (verify window)
  int sms = 0;    // SM count of the current device (set once validated)
};

gqa_status_t validate_shape(int batch, int capacity) {
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_INVALID_ARGUMENT, "batch %d outside [1, 65535]", batch);
  if (capacity < 1 || capacity > (1 << 30))
    return fail(GQA_ERR_INVALID_ARGUMENT, "capacity %d outside [1, 2^30]", capacity);
  return GQA_OK;
}

// Checks that need no CUDA call.  `q_scale_min_exclusive`: the prepared entry
// requires q_scale > 0, the others q_scale >= 0.
gqa_status_t validate(const Call& c, bool q_scale_positive, bool need_q) {
  if ((need_q && !c.q) || !c.kv || !c.lens || !c.out || !c.workspace)
    return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  gqa_status_t st = validate_shape(c.batch, c.capacity);
  if (st != GQA_OK) return st;
  if (c.q_dtype != GQA_F16 && c.q_dtype != GQA_BF16)
    return fail(GQA_ERR_INVALID_ARGUMENT, "unknown q/out dtype %d", c.q_dtype);
  if (!known_format(c.kv_format))
    return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", c.kv_format);
  if (!is_narrow(c.kv_format) && c.kv_format != c.q_dtype)
    return fail(GQA_ERR_INVALID_ARGUMENT, "fp16/bf16 KV must have the dtype of q");
  if (c.kv_format == kKvI8 && (!c.kv_scales || !aligned(c.kv_scales, 16) || c.capacity % 8 != 0))
    return fail(GQA_ERR_INVALID_ARGUMENT,
                "an int8 cache needs a 16-byte aligned bf16 scale array and a capacity that is a multiple of 8");
  if (c.kv_format == kKvE2M1 && (!c.kv_scales || !aligned(c.kv_scales, 16) || c.capacity % 2 != 0))
    return fail(GQA_ERR_INVALID_ARGUMENT,
                "an e2m1 cache needs a 16-byte aligned e4m3 scale array and a capacity that is a multiple of 2");
  if (!std::isfinite(c.q_scale) || c.q_scale < 0.f || (q_scale_positive && c.q_scale == 0.f))
    return fail(GQA_ERR_INVALID_ARGUMENT, "q_scale must be finite and %s 0", q_scale_positive ? ">" : ">=");
  if (!std::isfinite(c.k_scale) || c.k_scale <= 0.f || !std::isfinite(c.v_scale) || c.v_scale <= 0.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be finite and > 0");
  if (c.num_splits < 1 || c.num_splits > GQA_MAX_SPLITS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits %d outside [1, %d]", c.num_splits, GQA_MAX_SPLITS);
  if ((need_q && !aligned(c.q, 16)) || !aligned(c.kv, 16) || !aligned(c.out, 16) ||
      !aligned(c.workspace, 16) || !aligned(c.lens, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "q, kv, out, workspace must be 16-byte aligned, lens 4-byte");
  const size_t need = workspace_bytes_for(c.batch * c.q_len, c.num_splits);
  if (c.workspace_bytes < need)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", c.workspace_bytes, need);
  const size_t qo_bytes = (size_t)c.batch * c.q_len * kHq * kD * 2;
  const size_t kv_rows = c.block_table ? (size_t)c.num_pages * 2 * kHkv * ((size_t)1 << c.page_log2)
                                       : (size_t)c.batch * 2 * kHkv * (size_t)c.capacity;
  const size_t kv_bytes = kv_rows * kv_row_bytes(c.kv_format);
  const size_t lens_bytes = (size_t)c.batch * 4;
  if ((need_q && overlap(c.out, qo_bytes, c.q, qo_bytes)) || overlap(c.out, qo_bytes, c.kv, kv_bytes) ||
      overlap(c.out, qo_bytes, c.lens, lens_bytes) || overlap(c.out, qo_bytes, c.workspace, need))
    return fail(GQA_ERR_ALIASING, "out overlaps q, kv, lens or the workspace");
  if ((need_q && overlap(c.workspace, need, c.q, qo_bytes)) || overlap(c.workspace, need, c.kv, kv_bytes) ||
      overlap(c.workspace, need, c.lens, lens_bytes))
    return fail(GQA_ERR_ALIASING, "workspace overlaps q, kv or lens");
  if (c.block_table) {
    const size_t bt_bytes = (size_t)c.batch * c.max_pages * 4;
    if (overlap(c.out, qo_bytes, c.block_table, bt_bytes) || overlap(c.workspace, need, c.block_table, bt_bytes))
      return fail(GQA_ERR_ALIASING, "out or the workspace overlaps the block table");
  }
  if (scale_row_bytes(c.kv_format) > 0) {
    const size_t sc_bytes = kv_rows * scale_row_bytes(c.kv_format);
    if (overlap(c.out, qo_bytes, c.kv_scales, sc_bytes) || overlap(c.workspace, need, c.kv_scales, sc_bytes))
      return fail(GQA_ERR_ALIASING, "out or the workspace overlaps the cache's scales");
  }
  return GQA_OK;
}

// ------------------------------------------------ static (no-alloc) scratch

// Scratch for gqa_decode_noalloc.  In host code this name is only a stand-in
// for the device symbol: its device address comes from cudaGetSymbolAddress,
// once per device, with that device current.
constexpr size_t kStaticWorkspaceBytes = GQA_STATIC_WORKSPACE_BYTES;
static __device__ __align__(256) unsigned char g_static_workspace[kStaticWorkspaceBytes];

struct StaticWorkspace {
  std::mutex mu;
  std::atomic<void*> ptr{nullptr};  // set once set-up has succeeded on the device
};
StaticWorkspace g_static_ws[kMaxDevices];

// Device address of the static scratch on the current device `dev`.  Set-up
// (the first successful call per device): look the address up and zero the
// header (the status word) on `stream`.  Only a successful set-up is kept: a
// failed lookup (no context yet, a transient error) is retried by the next
// call.  The address stays valid for the life of the device's primary
// context; it goes stale after cudaDeviceReset.
gqa_status_t static_workspace(int dev, cudaStream_t stream, void** ptr) {
  if (dev < 0 || dev >= kMaxDevices) return fail(GQA_ERR_UNSUPPORTED_DEVICE, "device %d out of range", dev);
  StaticWorkspace& s = g_static_ws[dev];
  void* p = s.ptr.load(std::memory_order_acquire);
  if (!p) {
    std::lock_guard<std::mutex> lock(s.mu);
    p = s.ptr.load(std::memory_order_relaxed);
    if (!p) {
      cudaError_t e = cudaGetSymbolAddress(&p, g_static_workspace);
      if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(static workspace)");
      e = cudaMemsetAsync(p, 0, GQA_WORKSPACE_HEADER_BYTES, stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(static workspace header)");
      s.ptr.store(p, std::memory_order_release);
    }
  }
  *ptr = p;
  return GQA_OK;
}

// --------------------------------------------------------------- planning

int plan_splits(int batch, int capacity, int kv_format, int sm_count) {
  const long long tile = tile_tokens(kv_format);
  const long long units = (long long)batch * kHkv;
  const long long ctas_per_sm = mma_ctas_per_sm(kv_format, 1);
  const long long slots = ctas_per_sm * (sm_count > 0 ? sm_count : 148);
  const long long nmax = (capacity + tile - 1) / tile;
  long long per;
  if (units * nmax <= 16 * slots) {
    // Latency-bound sizes (at most 16 tiles per resident slot over the worst
    // case): one wave of work items at most, about sqrt(6 nmax) splits per
    // row — fewer leave each CTA more tiles to stream, more leave the merge
    // more partials.  Measured in CUDA graphs on GB300 (us per call, the
    // 8-wave rule -> this): bf16 1 x 4096 10.7 -> 9.0, 1 x 16384 20.6 -> 17.1,
    // 4 x 4096 16.4 -> 14.6, e4m3 1 x 8192 11.5 -> 10.3, fp16 1 x 1024 6.3.
    //
    // Batches of 8 or more rows of 4096 slots or more are not capped at one
    // wave, so they run the balanced schedule: a decode batch's lengths are
    // ragged, and only the balanced schedule spreads the actual tokens over
    // all the resident CTAs (a one-wave grid waits for the CTAs of its
    // longest rows).  Warm, in a CUDA graph, us per call, one wave ->
    // balanced, lengths U[C/4, C] and all = C: bf16 8 x 4096 22.7 -> 18.9 and
    // 24.2 -> 25.7, e4m3 16 x 4096 24.8 -> 21.2 and 26.4 -> 27.1, e4m3 8 x
    // 4096 15.6 -> 14.7 and 17.2 -> 17.6, int8 8 x 8192 26.8 -> 22.6 and 28.3
    // -> 28.3.  Shorter rows or smaller batches keep the one-wave grid: there
    // the balanced grid's extra pieces and combine cost more than it
    // balances (bf16 32 x 512 12.8 -> 14.9 and 13.7 -> 18.3, e4m3 16 x 1024
    // 10.4 -> 12.6 and 11.1 -> 14.3; bf16 4 x 8192 22.2 -> 20.2 but 24.1 ->
    // 26.1).
    long long s = (long long)std::llround(std::sqrt(6.0 * (double)nmax));
    // An e2m1 tile brings half the bytes and takes as long to compute, so more
    // splits pay: about sqrt(16 nmax), 32 at most (one request in a CUDA graph,
    // us per call, the rule above -> this: 512 tokens 4.4 -> 3.8, 2048 5.0 -> 4.4,
    // 4096 5.7 -> 5.0, 16384 9.4 -> 8.6, 32768 14.3 -> 12.5, there with 64
    // splits 14.4).
    if (kv_format == kKvE2M1) s = std::min(32LL, (long long)std::llround(std::sqrt(16.0 * (double)nmax)));
    const long long wave = slots / units;
    if (s > wave && !(batch >= 8 && capacity >= 4096)) s = wave;
    if (s < 1) s = 1;
    per = (capacity + s - 1) / s;
  } else {
    // Otherwise about 8 waves of work items over the worst case (every
    // length = capacity); such grids run the balanced schedule, where the
    // split count only bounds the pieces of a row.
    const long long target_ctas = 8LL * slots;
    per = (units * capacity + target_ctas - 1) / target_ctas;
  }
  per = (per + tile - 1) / tile * tile;
  // at least two tiles per split: a one-tile split costs more in fixed
  // prologue/epilogue than it streams (measured on the 1 x 1024 fp16 case)
  // (e2m1: from 4 tiles on a row a one-tile split pays; 256 tokens take 3.4 us in
  // one split, 3.7 in two)
  const long long least = kv_format == kKvE2M1 && nmax >= 4 ? tile : 2 * tile;
  if (per < least) per = least;
  long long s = (capacity + per - 1) / per;
  if (s < 1) s = 1;
  if (s > GQA_MAX_SPLITS) s = GQA_MAX_SPLITS;
  return (int)s;
}

// ---------------------------------------------------------------- launches

template <int QF>
cudaError_t launch_combine_t(const CombineParams& cp, int batch_rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kHkv, batch_rows, 1);
  cfg.blockDim = dim3(kGroup * 32 * cp.warps_per_head, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  // programmatic dependent launch: may be scheduled while stage 1 drains; the
  // kernel waits (griddepcontrol.wait) before it reads the partials
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (cp.warps_per_head) {
    case 1: return cudaLaunchKernelEx(&cfg, combine_kernel<QF, 1>, cp);
    case 2: return cudaLaunchKernelEx(&cfg, combine_kernel<QF, 2>, cp);
    default: return cudaLaunchKernelEx(&cfg, combine_kernel<QF, 4>, cp);
  }
}

struct Layout {
  float* part_o;
  float* part_m;
  float* part_l;
  uint32_t* flags;
};

Layout layout_of(void* ws, int batch, int splits) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  Layout l;
  l.flags = reinterpret_cast<uint32_t*>(base);
  uint8_t* p = base + GQA_WORKSPACE_HEADER_BYTES;
  l.part_o = reinterpret_cast<float*>(p);
  p += partial_o_bytes(batch, splits);
  l.part_m = reinterpret_cast<float*>(p);
  p += partial_ml_bytes(batch, splits);
  l.part_l = reinterpret_cast<float*>(p);
  return l;
}

// Checked builds: how far the extents given to the split kernel's range
// checks are cut short (gqa_decode_debug_cut_extents), so a test can make
// the checks fire while every redirected access stays in the real buffers.
std::atomic<uint64_t> g_cut_kv_bytes{0}, g_cut_scales_bytes{0};

// The balanced schedule serves decode and verify windows of batches up to
// kBalMaxBatch whose rows can be split (two or more tiles of capacity) and
// whose one-piece-per-CTA grid would take more than one wave, as long as the
// global stream (n + kBalRowCost positions for a row of n tiles, the first
// ones standing for the piece's fixed cost) fits an int.  q_min keeps every
// row within the workspace's split slots: a row of n <= nmax tiles meets at
// most ceil(n / q) + 1 <= num_splits CTAs.  Measured on GB300 (us per call,
// back to back): fp16 32 x U[1,8192] 96.4 -> 89.9, e4m3 64 x U[16k,32k]
// 459.4 -> 443.7, bf16 8 x 131072 589.4 -> 584.3.
struct BalPlan {
  int ctas = 0;  // 0: the one-piece-per-CTA grid
  int q_min = 0;
};

BalPlan bal_plan(const Call& c) {
  BalPlan bp;
  const int tile = tile_tokens(c.kv_format);
  const long long nmax = ((long long)c.capacity + tile - 1) / tile;
  if (c.batch > kBalMaxBatch || c.num_splits < 2 || c.sms < 1) return bp;
  const int splits_eff = split_count(c.capacity, c.num_splits, c.kv_format);
  if (splits_eff < 2) return bp;
  if ((long long)kHkv * c.batch * (nmax + kBalRowCost) > 0x7fffffffLL) return bp;
  const long long slots = (long long)mma_ctas_per_sm(c.kv_format, c.q_len) * c.sms;
  // one wave of pieces or less: nothing to balance, the plain grid starts sooner
  if ((long long)kHkv * c.batch * splits_eff <= slots) return bp;
  // One CTA per resident slot for a contiguous cache.  A paged 16-bit cache
  // runs 4 waves of smaller runs: its per-CTA rates vary more (pages
  // scattered over HBM), and the later waves let the hardware even them out
  // (bf16 8 x 131072 in shuffled 256-token pages, GB300: 586 us back to back
  // with one wave, 580 with four).  A paged 8-bit cache keeps one wave: at 3
  // CTAs per SM its issue-heavier CTAs pay more for the extra prologues and
  // pieces (64 x U[16k, 32k] in 256-token pages: int8 461 us with one wave,
  // 469 with four; e4m3 444 against 451).
  const bool waves4 = c.block_table != nullptr && !is_narrow(c.kv_format);
  bp.ctas = (int)((waves4 ? 4 : 1) * slots);
  bp.q_min = (int)((nmax + c.num_splits - 2) / (c.num_splits - 1));
  return bp;
}

// The one-piece grid merges on chip when its 2..8 splits that hold slots fit
// one portable thread-block cluster (distributed shared memory) and the grid
// is one wave at most: latency-bound launches, where the combine launch and
// the partials' round trip through HBM are a large share of the time.
// Measured on GB300: clusters of 9..16 (a non-portable size) were slower when
// warm (e4m3 1 x 8192 in a graph 10.3 -> 12.2 us, a 4-token window at
// 1 x 4096 9.6 -> 13.7), and so were multi-wave grids of clusters (int8
// 64 x U[16k, 32k] with a 2-token window, 8 splits, 4096 CTAs: 530 -> 760 us).
// The clusters must also all be resident at once (the device's occupancy
// table): a cluster's CTAs share one GPC, and near full occupancy clusters
// of some sizes pack into fewer than the slots allow, leaving the rest for a
// second wave.  Measured on GB300: e4m3 8 x 4096 (7 splits, 448 CTAs in
// clusters of 7, 456 slots) took 24.8 us per cold call, against 18.4 with 6
// splits.  Such a grid runs as the plain grid with the combine kernel.
// Returns the cluster size, or 0 for the combine kernel.
int cluster_fit(const Call& c, int s) {
  // the current device's table, once it has been set up with this SM count
  // (0: unknown, e.g. host-only planning without a device)
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();  // (no device here: clear the error)
    return 0;
  }
  const DeviceState& st = g_devices[dev];
  if (st.state.load(std::memory_order_acquire) != 1 || st.sm_count != c.sms) return 0;
  const auto& row = st.cluster_fit[c.kv_format];
  const int nq = c.q_len - 1;
  if (!is_narrow(c.kv_format)) return row[c.kv_format == kKvF16 ? kQF16 : kQBF16][nq][s];
  // an 8- or 4-bit cache with either q format when the call does not say which
  if (c.q_dtype == GQA_F16 || c.q_dtype == GQA_BF16) return row[c.q_dtype][nq][s];
  return std::min(row[kQF16][nq][s], row[kQBF16][nq][s]);
}

int cluster_splits(const Call& c) {
  if (bal_plan(c).ctas > 0 || c.sms < 1) return 0;
  const int s = split_count(c.capacity, c.num_splits, c.kv_format);
  if (s < 2 || s > kClusterMaxSplits) return 0;
  const long long slots = (long long)mma_ctas_per_sm(c.kv_format, c.q_len) * c.sms;
  if ((long long)kHkv * c.batch * s > slots) return 0;
  const int fit = cluster_fit(c, s);
  return fit > 0 && (long long)kHkv * c.batch > fit ? 0 : s;
}

gqa_status_t run_split(const Call& c) {
  const Layout lay = layout_of(c.workspace, c.batch * c.q_len, c.num_splits);
  SplitParams sp;
  sp.q = c.q;
  sp.kv = c.kv;
  sp.lens = c.lens;
  sp.out = c.out;
  sp.part_o = lay.part_o;
  sp.part_m = lay.part_m;
  sp.part_l = lay.part_l;
  sp.flags = lay.flags;
  sp.batch = c.batch;
  sp.capacity = c.capacity;
  sp.num_splits = c.num_splits;
  sp.chunk = split_chunk(c.capacity, c.num_splits, c.kv_format);
  sp.splits_eff = split_count(c.capacity, c.num_splits, c.kv_format);
  // log2(e) / sqrt(128): the softmax runs in the exp2 domain
  sp.scale_log2 = (float)((double)c.q_scale * (double)c.k_scale * 1.4426950408889634 / std::sqrt(128.0));
  sp.v_scale = c.v_scale;
  sp.wait_budget_ns = c.wait_budget_ns;
  sp.skip_tile = c.skip_tile;
  sp.kv_scales = c.kv_scales;
  sp.block_table = c.block_table;
  sp.page_log2 = c.page_log2;
  sp.max_pages = c.max_pages;
  sp.num_pages = c.num_pages;
  const BalPlan bp = bal_plan(c);
  sp.bal_q_min = bp.q_min;
  const size_t page_rows = c.block_table ? ((size_t)1 << c.page_log2) : (size_t)c.capacity;
  const size_t units = c.block_table ? (size_t)c.num_pages : (size_t)c.batch;
  sp.kv_bytes = units * 2 * kHkv * page_rows * kv_row_bytes(c.kv_format);
  sp.scales_bytes = units * 2 * kHkv * page_rows * scale_row_bytes(c.kv_format);
  if (kChecked) {
    sp.kv_bytes -= std::min<size_t>(sp.kv_bytes, g_cut_kv_bytes.load());
    sp.scales_bytes -= std::min<size_t>(sp.scales_bytes, g_cut_scales_bytes.load());
  }
  cudaError_t e;
  const int ql = c.q_len, nb = bp.ctas, cl = cluster_splits(c);
  if (c.kv_format == kKvF16) e = launch_split_t<kKvF16, kQF16>(sp, ql, nb, cl, c.stream);
  else if (c.kv_format == kKvBF16) e = launch_split_t<kKvBF16, kQBF16>(sp, ql, nb, cl, c.stream);
  else if (c.kv_format == kKvE4M3)
    e = c.q_dtype == GQA_BF16 ? launch_split_t<kKvE4M3, kQBF16>(sp, ql, nb, cl, c.stream)
                              : launch_split_t<kKvE4M3, kQF16>(sp, ql, nb, cl, c.stream);
  else if (c.kv_format == kKvI8)
    e = c.q_dtype == GQA_BF16 ? launch_split_t<kKvI8, kQBF16>(sp, ql, nb, cl, c.stream)
                              : launch_split_t<kKvI8, kQF16>(sp, ql, nb, cl, c.stream);
  else
    e = e2m1_launch_split(sp, c.q_dtype, ql, nb, cl, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "split kernel launch");
  return GQA_OK;
}

gqa_status_t run_combine(const Call& c) {
  const int splits_eff = split_count(c.capacity, c.num_splits, c.kv_format);
  if (splits_eff == 1 || cluster_splits(c) > 0) return GQA_OK;  // merged by stage 1
  const Layout lay = layout_of(c.workspace, c.batch * c.q_len, c.num_splits);
  CombineParams cp;
  cp.lens = c.lens;
  cp.out = c.out;
  cp.part_o = lay.part_o;
  cp.part_m = lay.part_m;
  cp.part_l = lay.part_l;
  cp.capacity = c.capacity;
  cp.num_splits = c.num_splits;
  cp.chunk = split_chunk(c.capacity, c.num_splits, c.kv_format);
  cp.q_len = c.q_len;
  cp.v_scale = c.v_scale;
  const BalPlan bp = bal_plan(c);
  cp.bal_ctas = bp.ctas;
  cp.bal_q_min = bp.q_min;
  cp.tile = tile_tokens(c.kv_format);
  cp.batch = c.batch;
  cp.flags = lay.flags;
  // Warps per query head: enough that each merges at most about 8 pieces of
  // its row in one round of loads (up to 4).  Pieces per row: the splits
  // that hold slots, or under the balanced schedule about CTAs / rows + 2 (a
  // row meets that many runs, plus the partial ones at its ends).
  const long long expected =
      bp.ctas > 0 ? std::min<long long>(c.num_splits, bp.ctas / (kHkv * (long long)c.batch) + 2) : splits_eff;
  int W = 1;
  while (W < kCombineMaxWarpsPerHead && expected > 8LL * W) W *= 2;
  cp.warps_per_head = W;
  cudaError_t e = c.q_dtype == GQA_F16 ? launch_combine_t<kQF16>(cp, c.batch * c.q_len, c.stream)
                                       : launch_combine_t<kQBF16>(cp, c.batch * c.q_len, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "combine kernel launch");
  return GQA_OK;
}

// Resolve num_splits = 0 (auto) and validate; then the device check.
gqa_status_t prepare_call(Call& c, bool q_scale_positive, bool need_q) {
  int sms = 0;
  if (c.num_splits == 0) {
    // validate everything that does not depend on the split count first
    Call probe = c;
    probe.num_splits = 1;
    probe.workspace_bytes = (size_t)-1;
    gqa_status_t st = validate(probe, q_scale_positive, need_q);
    if (st != GQA_OK) return st;
    st = current_device_ready(&sms);
    if (st != GQA_OK) return st;
    c.num_splits = plan_splits(c.batch, c.capacity, c.kv_format, sms);
  }
  gqa_status_t st = validate(c, q_scale_positive, need_q);
  if (st != GQA_OK) return st;
  st = current_device_ready(&sms);
  c.sms = sms;
  return st;
}

// A cache as the write and read-back calls take it: contiguous (block_table =
// nullptr; units = batch rows) or paged (units = num_pages).
struct CacheArgs {
  void* kv;
  int format;
  void* scales;
  int batch, capacity;  // capacity: slots a row holds (paged: max_pages * page size)
  const int32_t* block_table;
  int max_pages, num_pages, page_log2;
  float k_scale, v_scale;
  size_t rows() const {
    return (block_table ? (size_t)num_pages << page_log2 : (size_t)batch * capacity) * 2 * kHkv;
  }
  size_t kv_bytes() const { return rows() * kv_row_bytes(format); }
  size_t scale_bytes() const { return rows() * scale_row_bytes(format); }
  size_t table_bytes() const { return block_table ? (size_t)batch * max_pages * 4 : 0; }
};

// Rows of 128 that the checked build's write and read-back kernels may touch (cut
// short by gqa_decode_debug_cut_extents).
size_t checked_rows(const CacheArgs& c) {
  size_t cut = 0;
  if (kChecked) {
    const auto whole = [](uint64_t bytes, int row) -> size_t { return row ? bytes / row + (bytes % row != 0) : 0; };
    cut = std::max(whole(g_cut_kv_bytes.load(), kv_row_bytes(c.format)),
                   whole(g_cut_scales_bytes.load(), scale_row_bytes(c.format)));
  }
  return c.rows() - std::min(c.rows(), cut);
}

gqa_status_t paged_args(CacheArgs& c, const int32_t* block_table, int max_pages_per_seq, int num_pages,
                        int page_size) {
  if (!block_table) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table is null");
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(GQA_ERR_INVALID_ARGUMENT, "page_size %d is not a power of two in [16, 65536]", page_size);
  if (num_pages < 1 || max_pages_per_seq < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_pages and max_pages_per_seq must be >= 1");
  const long long cap = (long long)max_pages_per_seq * page_size;
  if (cap > (1LL << 30)) return fail(GQA_ERR_INVALID_ARGUMENT, "max_pages_per_seq * page_size exceeds 2^30");
  if (!aligned(block_table, 4)) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table must be 4-byte aligned");
  c.block_table = block_table;
  c.max_pages = max_pages_per_seq;
  c.num_pages = num_pages;
  c.capacity = (int)cap;
  c.page_log2 = 0;
  while ((1 << c.page_log2) < page_size) ++c.page_log2;
  return GQA_OK;
}

gqa_status_t validate_cache(const CacheArgs& c, const void* workspace, size_t workspace_bytes) {
  gqa_status_t st = validate_shape(c.batch, c.capacity);
  if (st != GQA_OK) return st;
  if (!known_format(c.format)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", c.format);
  if (!c.kv || !aligned(c.kv, 16)) return fail(GQA_ERR_INVALID_ARGUMENT, "kv must be non-null and 16-byte aligned");
  if (scale_row_bytes(c.format) > 0 && (!c.scales || !aligned(c.scales, 2)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "an int8 or e2m1 cache needs its 2-byte aligned row scales");
  if (!std::isfinite(c.k_scale) || c.k_scale <= 0.f || !std::isfinite(c.v_scale) || c.v_scale <= 0.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be finite and > 0");
  if (workspace && workspace_bytes < GQA_WORKSPACE_HEADER_BYTES)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than its %d-byte header", GQA_WORKSPACE_HEADER_BYTES);
  if (workspace && !aligned(workspace, 4)) return fail(GQA_ERR_INVALID_ARGUMENT, "workspace must be 4-byte aligned");
  return GQA_OK;
}

// What a write call takes besides the cache.
struct WriteArgs {
  const void *q_proj, *k_proj, *v_proj;
  long long q_stride, k_stride, v_stride;  // elements from one token to the next
  const void *q_norm_w, *k_norm_w;
  int dtype;
  const int32_t* positions;
  const int* section;  // host: three counts, or null
  int interleaved;
  const int32_t *rows, *slots;
  int tokens;
  void* q_out;
  float eps, rope_theta;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
};

// theta^(-i/64) / (2 pi) modulo 1 as a 64-bit fraction: the FP64 frequency's
// product with 1 / (2 pi), itself held as two doubles, to about 2^-64.
uint64_t turn_fraction(double inv_freq) {
  constexpr double kInvHi = 0x1.45f306dc9c883p-3;    // the double nearest to 1 / (2 pi)
  constexpr double kInvLo = -0x1.6b01ec5417056p-57;  // the rest
  const double hi = inv_freq * kInvHi;
  const double lo = std::fma(inv_freq, kInvHi, -hi) + inv_freq * kInvLo;
  const double whole = std::floor(hi);
  return (uint64_t)std::ldexp(hi - whole, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(lo, 64));
}

// The fractions of the 64 rotary frequencies of `theta`, kept by the calling
// thread for its next call with the same theta (64 pow cost a few us).
const uint64_t* turn_fractions(float theta) {
  thread_local float known = -1.f;
  thread_local uint64_t turns[kD / 2];
  if (known != theta) {
    for (int i = 0; i < kD / 2; ++i) turns[i] = turn_fraction(std::pow((double)theta, -(double)i / (kD / 2)));
    known = theta;
  }
  return turns;
}

gqa_status_t write_kv(const CacheArgs& c, const WriteArgs& a) {
  if (a.tokens == 0) return GQA_OK;
  if (a.tokens < 0 || a.tokens > (1 << 27)) return fail(GQA_ERR_INVALID_ARGUMENT, "tokens %d outside [0, 2^27]", a.tokens);
  if (!a.q_proj || !a.k_proj || !a.v_proj || !a.positions || !a.slots || !a.q_out)
    return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  if ((a.q_norm_w == nullptr) != (a.k_norm_w == nullptr))
    return fail(GQA_ERR_INVALID_ARGUMENT, "q_norm_w and k_norm_w are given together or not at all");
  if (a.dtype != GQA_F16 && a.dtype != GQA_BF16) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown dtype %d", a.dtype);
  gqa_status_t st = validate_cache(c, a.workspace, a.workspace_bytes);
  if (st != GQA_OK) return st;
  if (!is_narrow(c.format) && c.format != a.dtype)
    return fail(GQA_ERR_INVALID_ARGUMENT, "fp16/bf16 KV must have the dtype of the projections");
  // (the e2m1 scales' products and reciprocals stay normal FP32 numbers)
  if (c.format == kKvE2M1 && (c.k_scale < 0x1p-100f || c.k_scale > 0x1p100f || c.v_scale < 0x1p-100f || c.v_scale > 0x1p100f))
    return fail(GQA_ERR_INVALID_ARGUMENT, "the tensor scales of an e2m1 cache must lie in [2^-100, 2^100]");
  // (an e4m3 write multiplies with the reciprocals: infinite ones would make zeros NaN)
  if (c.format == kKvE4M3 && (c.k_scale < 0x1p-126f || c.k_scale > 0x1p126f || c.v_scale < 0x1p-126f || c.v_scale > 0x1p126f))
    return fail(GQA_ERR_INVALID_ARGUMENT, "the scales of an e4m3 cache must lie in [2^-126, 2^126]");
  if (!std::isfinite(a.eps) || a.eps < 0.f) return fail(GQA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (!std::isfinite(a.rope_theta) || a.rope_theta < 1.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "rope_theta must be finite and >= 1");
  if (a.section) {
    const int* s = a.section;
    if (s[0] < 0 || s[1] < 0 || s[2] < 0 || s[0] > 64 || s[1] > 64 || s[2] > 64 || s[0] + s[1] + s[2] != kD / 2)
      return fail(GQA_ERR_INVALID_ARGUMENT, "the three rotary sections must be >= 0 and sum to 64");
    if (a.interleaved && (s[1] > 21 || s[2] > 21))
      return fail(GQA_ERR_INVALID_ARGUMENT, "interleaved sections hold at most 21 of height and of width");
  }
  const void* vec[] = {a.q_proj, a.k_proj, a.v_proj, a.q_out, a.q_norm_w, a.k_norm_w};
  for (const void* ptr : vec)
    if (!aligned(ptr, 16)) return fail(GQA_ERR_INVALID_ARGUMENT, "projections, weights and q_out must be 16-byte aligned");
  const long long stride[] = {a.q_stride, a.k_stride, a.v_stride};
  const long long width[] = {kHq * kD, kHkv * kD, kHkv * kD};
  for (int i = 0; i < 3; ++i)
    if (stride[i] < width[i] || stride[i] % 8 != 0 || stride[i] > (1LL << 32))
      return fail(GQA_ERR_INVALID_ARGUMENT, "a token stride must be a multiple of 8 elements and hold the token's heads");
  if (!aligned(a.positions, 4) || !aligned(a.slots, 4) || !aligned(a.rows, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "positions, rows and slots must be 4-byte aligned");
  // nothing that is written overlaps anything else
  const size_t n = (size_t)a.tokens;
  const struct { const void* p; size_t bytes; } ins[] = {
      {a.q_proj, ((n - 1) * a.q_stride + width[0]) * 2}, {a.k_proj, ((n - 1) * a.k_stride + width[1]) * 2},
      {a.v_proj, ((n - 1) * a.v_stride + width[2]) * 2}, {a.q_norm_w, a.q_norm_w ? (size_t)kD * 2 : 0},
      {a.k_norm_w, a.k_norm_w ? (size_t)kD * 2 : 0},     {a.positions, n * 4 * (a.section ? 3 : 1)},
      {a.rows, a.rows ? n * 4 : 0},                      {a.slots, n * 4},
      {c.block_table, c.table_bytes()}};
  const struct { const void* p; size_t bytes; } outs[] = {
      {a.q_out, n * kHq * kD * 2}, {c.kv, c.kv_bytes()}, {c.scales, c.scale_bytes()},
      {a.workspace, a.workspace ? (size_t)GQA_WORKSPACE_HEADER_BYTES : 0}};
  for (size_t i = 0; i < sizeof outs / sizeof outs[0]; ++i) {
    if (!outs[i].bytes) continue;
    for (const auto& in : ins)
      if (in.bytes && overlap(outs[i].p, outs[i].bytes, in.p, in.bytes))
        return fail(GQA_ERR_ALIASING, "q_out, the cache, its scales or the workspace overlaps an input");
    for (size_t k = i + 1; k < sizeof outs / sizeof outs[0]; ++k)
      if (outs[k].bytes && overlap(outs[i].p, outs[i].bytes, outs[k].p, outs[k].bytes))
        return fail(GQA_ERR_ALIASING, "q_out, the cache, its scales and the workspace overlap one another");
  }
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  WriteParams w = {};
  w.q_proj = static_cast<const uint16_t*>(a.q_proj);
  w.k_proj = static_cast<const uint16_t*>(a.k_proj);
  w.v_proj = static_cast<const uint16_t*>(a.v_proj);
  w.q_stride = a.q_stride;
  w.k_stride = a.k_stride;
  w.v_stride = a.v_stride;
  w.q_norm_w = static_cast<const uint16_t*>(a.q_norm_w);
  w.k_norm_w = static_cast<const uint16_t*>(a.k_norm_w);
  w.positions = a.positions;
  w.rows = a.rows;
  w.slots = a.slots;
  w.q_out = static_cast<uint16_t*>(a.q_out);
  w.kv = c.kv;
  w.kv_scales = c.scales;
  w.flags = static_cast<uint32_t*>(a.workspace);
  w.tokens = a.tokens;
  w.batch = c.batch;
  w.capacity = c.capacity;
  w.block_table = c.block_table;
  w.max_pages = c.max_pages;
  w.num_pages = c.num_pages;
  w.page_log2 = c.page_log2;
  w.eps = a.eps;
  w.k_scale = c.k_scale;
  w.v_scale = c.v_scale;
  w.k_inv_scale = 1.f / c.k_scale;
  w.v_inv_scale = 1.f / c.v_scale;
  std::memcpy(w.turns, turn_fractions(a.rope_theta), sizeof w.turns);
  for (int i = 0; i < kD / 2; ++i) {
    int axis = 0;
    if (a.section && a.interleaved) axis = i % 3 == 1 && i < 3 * a.section[1] ? 1 : (i % 3 == 2 && i < 3 * a.section[2] ? 2 : 0);
    else if (a.section) axis = (i >= a.section[0]) + (i >= a.section[0] + a.section[1]);
    w.axis[i] = (uint8_t)axis;
  }
  w.kv_rows = checked_rows(c);
  w.q_bytes = ins[0].bytes;
  w.k_bytes = ins[1].bytes;
  w.v_bytes = ins[2].bytes;
  w.pos_bytes = n * 4 * (a.section ? 3 : 1);
  const cudaError_t e = launch_write_kv(w, c.format, a.dtype == GQA_BF16 ? kQBF16 : kQF16, sms, a.stream);
  if (e != cudaSuccess) return cuda_fail(e, "write kernel launch");
  return GQA_OK;
}

gqa_status_t read_kv(const CacheArgs& c, const int32_t* lens, const int32_t* starts, void* out, int out_dtype,
                     int out_capacity, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!lens || !out) return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (out_dtype != GQA_F16 && out_dtype != GQA_BF16) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown out dtype %d", out_dtype);
  if (out_capacity < 1 || out_capacity > (1 << 30))
    return fail(GQA_ERR_INVALID_ARGUMENT, "out_capacity %d outside [1, 2^30]", out_capacity);
  gqa_status_t st = validate_cache(c, workspace, workspace_bytes);
  if (st != GQA_OK) return st;
  if (!aligned(out, 16) || !aligned(lens, 4) || !aligned(starts, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "out must be 16-byte aligned, lens and starts 4-byte");
  // nothing that is written (out, the status word) overlaps anything else
  const size_t out_bytes = (size_t)c.batch * 2 * kHkv * out_capacity * kD * 2, b4 = (size_t)c.batch * 4;
  const size_t ws_bytes = workspace ? (size_t)GQA_WORKSPACE_HEADER_BYTES : 0;
  const struct { const void* p; size_t bytes; } ins[] = {
      {c.kv, c.kv_bytes()}, {c.scales, c.scale_bytes()}, {lens, b4}, {starts, starts ? b4 : 0},
      {c.block_table, c.table_bytes()}};
  for (const auto& in : ins)
    if (in.bytes && (overlap(out, out_bytes, in.p, in.bytes) || (ws_bytes && overlap(workspace, ws_bytes, in.p, in.bytes))))
      return fail(GQA_ERR_ALIASING, "out or the workspace overlaps the cache, its scales, the lengths or the block table");
  if (ws_bytes && overlap(out, out_bytes, workspace, ws_bytes))
    return fail(GQA_ERR_ALIASING, "out overlaps the workspace");
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  ReadParams r = {};
  r.kv = c.kv;
  r.kv_scales = c.scales;
  r.lens = lens;
  r.starts = starts;
  r.out = out;
  r.flags = static_cast<uint32_t*>(workspace);
  r.batch = c.batch;
  r.capacity = c.capacity;
  r.out_capacity = out_capacity;
  r.block_table = c.block_table;
  r.max_pages = c.max_pages;
  r.num_pages = c.num_pages;
  r.page_log2 = c.page_log2;
  r.k_scale = c.k_scale;
  r.v_scale = c.v_scale;
  r.kv_rows = checked_rows(c);
  const cudaError_t e = launch_read_kv(r, c.format, out_dtype == GQA_BF16 ? kQBF16 : kQF16, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "read kernel launch");
  return GQA_OK;
}

// A range of memory that a call reads or writes.
struct Range { const void* p; size_t bytes; };

bool meet(const Range& a, const Range& b) { return a.p && b.p && a.bytes && b.bytes && overlap(a.p, a.bytes, b.p, b.bytes); }

// Nothing that is written overlaps anything else.
template <size_t I, size_t O>
gqa_status_t no_aliasing(const Range (&ins)[I], const Range (&outs)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Range& in : ins)
      if (meet(outs[i], in)) return fail(GQA_ERR_ALIASING, "an output or the workspace overlaps an input");
    for (size_t k = i + 1; k < O; ++k)
      if (meet(outs[i], outs[k])) return fail(GQA_ERR_ALIASING, "two of the outputs and the workspace overlap");
  }
  return GQA_OK;
}

// The cache, and a workspace that a call needs, of the serving calls.
gqa_status_t validate_serving(const CacheArgs& c, const void* workspace, size_t workspace_bytes, size_t need) {
  gqa_status_t st = validate_cache(c, nullptr, 0);
  if (st != GQA_OK) return st;
  if (c.format == kKvE2M1 && !aligned(c.scales, 8))
    return fail(GQA_ERR_INVALID_ARGUMENT, "an e2m1 cache's scales must be 8-byte aligned");
  if (!workspace || !aligned(workspace, 16))
    return fail(GQA_ERR_INVALID_ARGUMENT, "workspace must be non-null and 16-byte aligned");
  if (workspace_bytes < need)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  return GQA_OK;
}

gqa_status_t validate_query(const CacheArgs& c, const void* q, int q_dtype, float q_scale) {
  if (!q || !aligned(q, 16)) return fail(GQA_ERR_INVALID_ARGUMENT, "q must be non-null and 16-byte aligned");
  if (q_dtype != GQA_F16 && q_dtype != GQA_BF16) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown dtype %d", q_dtype);
  if (!is_narrow(c.format) && c.format != q_dtype)
    return fail(GQA_ERR_INVALID_ARGUMENT, "fp16/bf16 KV must have the dtype of q");
  if (!std::isfinite(q_scale) || q_scale < 0.f) return fail(GQA_ERR_INVALID_ARGUMENT, "q_scale must be finite and >= 0");
  return GQA_OK;
}

CacheView view_of(const CacheArgs& c, void* workspace) {
  CacheView v = {};
  v.kv = c.kv;
  v.scales = c.scales;
  v.block_table = c.block_table;
  v.flags = static_cast<uint32_t*>(workspace);
  v.batch = c.batch;
  v.capacity = c.capacity;
  v.max_pages = c.max_pages;
  v.num_pages = c.num_pages;
  v.page_log2 = c.page_log2;
  v.rows = checked_rows(c);
  return v;
}

// log2(e) / sqrt(128): the softmax runs in the exp2 domain
float softmax_scale_log2(float q_scale, float k_scale) {
  return (float)((double)q_scale * (double)k_scale * 1.4426950408889634 / std::sqrt(128.0));
}

// Partials of the prompt attention: two pieces a CTA.
constexpr size_t kPrefillMlBytes = (size_t)2 * kPfMaxCtas * 2 * kPfRows * sizeof(float2);
constexpr size_t kPrefillOBytes = (size_t)2 * kPfMaxCtas * 2 * kPfRows * kD * sizeof(float);

gqa_status_t prefill(const CacheArgs& c, const void* q, int q_dtype, const int32_t* chunk_starts, const int32_t* lens,
                     void* out, int tokens, float q_scale, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  if (tokens == 0) return GQA_OK;
  if (tokens < 0 || tokens > (1 << 27)) return fail(GQA_ERR_INVALID_ARGUMENT, "tokens %d outside [0, 2^27]", tokens);
  if (!chunk_starts || !lens || !out) return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  const size_t need = gqa_prefill_workspace_size();
  gqa_status_t st = validate_serving(c, workspace, workspace_bytes, need);
  if (st != GQA_OK) return st;
  st = validate_query(c, q, q_dtype, q_scale);
  if (st != GQA_OK) return st;
  if (c.rows() > 0x7fffffff) return fail(GQA_ERR_INVALID_ARGUMENT, "the cache has more than 2^31 - 1 rows");
  if (!aligned(out, 16) || !aligned(chunk_starts, 4) || !aligned(lens, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "out must be 16-byte aligned, chunk_starts and lens 4-byte");
  const size_t qb = (size_t)tokens * kHq * kD * 2;
  const Range ins[] = {{q, qb}, {c.kv, c.kv_bytes()}, {c.scales, c.scale_bytes()},
                       {chunk_starts, ((size_t)c.batch + 1) * 4}, {lens, (size_t)c.batch * 4},
                       {c.block_table, c.table_bytes()}};
  const Range outs[] = {{out, qb}, {workspace, need}};
  st = no_aliasing(ins, outs);
  if (st != GQA_OK) return st;
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  PrefillParams p = {};
  p.c = view_of(c, workspace);
  p.q = q;
  p.out = out;
  p.chunk_starts = chunk_starts;
  p.lens = lens;
  p.tokens = tokens;
  char* ws = static_cast<char*>(workspace) + GQA_WORKSPACE_HEADER_BYTES;
  p.part_ml = reinterpret_cast<float2*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + kPrefillMlBytes);
  p.ctas = std::min(sms, kPfMaxCtas);
  p.scale_log2 = softmax_scale_log2(q_scale, c.k_scale);
  p.v_scale = c.v_scale;
  const cudaError_t e = launch_prefill(p, c.format, q_dtype == GQA_BF16 ? kQBF16 : kQF16, stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefill kernel launch");
  return GQA_OK;
}

// How the score kernel cuts a row: chunks of whole slab rounds, about 8 CTAs an SM in
// all where the capacity gives as many, 1024 chunks a row at most.
constexpr int kScoreRound = kScoreWarps * kSlab;
int max_score_chunks(int capacity) { return (int)std::min(1024LL, ((long long)capacity + kScoreRound - 1) / kScoreRound); }

size_t score_bytes(int batch, int capacity, int q_len) {
  return align_up((size_t)batch * kHkv * capacity * 4 * q_len * sizeof(float), 256);
}

gqa_status_t accumulate(const CacheArgs& c, const void* q, int q_dtype, const int32_t* lens, float* weights, int q_len,
                        float q_scale, int add, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (q_len < 1 || q_len > 4) return fail(GQA_ERR_INVALID_ARGUMENT, "q_len %d outside [1, 4]", q_len);
  if (!lens || !weights) return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  const size_t need = gqa_weights_workspace_size(c.batch, c.capacity, q_len);
  gqa_status_t st = validate_serving(c, workspace, workspace_bytes, need);
  if (st != GQA_OK) return st;
  st = validate_query(c, q, q_dtype, q_scale);
  if (st != GQA_OK) return st;
  if (!aligned(weights, 16) || !aligned(lens, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "weights must be 16-byte aligned, lens 4-byte");
  const Range ins[] = {{q, (size_t)c.batch * q_len * kHq * kD * 2}, {c.kv, c.kv_bytes()}, {c.scales, c.scale_bytes()},
                       {lens, (size_t)c.batch * 4}, {c.block_table, c.table_bytes()}};
  const Range outs[] = {{weights, (size_t)c.batch * kHkv * c.capacity * 4}, {workspace, need}};
  st = no_aliasing(ins, outs);
  if (st != GQA_OK) return st;
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  WeightParams p = {};
  p.c = view_of(c, workspace);
  p.q = q;
  p.lens = lens;
  p.weights = weights;
  char* ws = static_cast<char*>(workspace) + GQA_WORKSPACE_HEADER_BYTES;
  p.scores = reinterpret_cast<float*>(ws);
  p.stats = reinterpret_cast<float2*>(ws + score_bytes(c.batch, c.capacity, q_len));
  p.scale_log2 = softmax_scale_log2(q_scale, c.k_scale);
  const long long want = std::max(1LL, std::min<long long>(max_score_chunks(c.capacity), (8LL * sms + kHkv * c.batch - 1) / (kHkv * (long long)c.batch)));
  p.chunk = (int)(((c.capacity + want - 1) / want + kScoreRound - 1) / kScoreRound * kScoreRound);
  p.chunks = (c.capacity + p.chunk - 1) / p.chunk;
  p.add = add != 0;
  const cudaError_t e = launch_sum_weights(p, c.format, q_dtype == GQA_BF16 ? kQBF16 : kQF16, q_len, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "weight sum kernel launch");
  return GQA_OK;
}

size_t evict_chunks(int keep) {  // of the narrowest rows' moves the fewest, of 16-bit rows the most
  return ((size_t)keep + move_rows(kKvF16) - 1) / move_rows(kKvF16);
}

// What an eviction takes besides the cache; out and out_table null: in place.
struct EvictArgs {
  int32_t* lens;
  float* weights;
  void *out, *out_scales;
  const int32_t* out_table;
  int out_capacity, out_max_pages;
  int32_t* out_lens;
  float* out_weights;
  int32_t* kept;
  int weights_capacity, keep, recent, first;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
};

gqa_status_t evict(const CacheArgs& c, const EvictArgs& a) {
  if (a.keep < 1 || a.keep > (1 << 30)) return fail(GQA_ERR_INVALID_ARGUMENT, "keep %d outside [1, 2^30]", a.keep);
  if (a.first < 0 || a.recent < 0 || (long long)a.first + a.recent > a.keep)
    return fail(GQA_ERR_INVALID_ARGUMENT, "first and recent must be >= 0 and no more than keep together");
  if (!a.lens || !a.weights || !a.kept) return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  const size_t need = gqa_evict_workspace_size(c.batch, a.keep);
  gqa_status_t st = validate_serving(c, a.workspace, a.workspace_bytes, need);
  if (st != GQA_OK) return st;
  const bool in_place = !a.out && !a.out_table;
  if (in_place && (a.out_scales || a.out_lens || a.out_weights))
    return fail(GQA_ERR_INVALID_ARGUMENT, "an eviction in place has no out_scales, out_lens or out_weights");
  if (!in_place) {
    if (!a.out_lens) return fail(GQA_ERR_INVALID_ARGUMENT, "out_lens is null");
    if (!c.block_table && scale_row_bytes(c.format) && !a.out_scales) return fail(GQA_ERR_INVALID_ARGUMENT, "out_scales is null");
    const long long room = c.block_table ? (long long)a.out_max_pages << c.page_log2 : a.out_capacity;
    if (a.out_max_pages < 0 || room < a.keep || room > (1LL << 30))
      return fail(GQA_ERR_INVALID_ARGUMENT, "the output holds %lld slots a row, fewer than keep or more than 2^30", room);
    if (a.out_weights && (a.weights_capacity < a.keep || a.weights_capacity > (1 << 30)))
      return fail(GQA_ERR_INVALID_ARGUMENT, "weights_capacity %d below keep or above 2^30", a.weights_capacity);
  }
  if (!aligned(a.weights, 16) || !aligned(a.out, 16) || !aligned(a.out_scales, c.format == kKvE2M1 ? 8 : 2) ||
      !aligned(a.lens, 4) || !aligned(a.out_lens, 4) || !aligned(a.out_weights, 4) || !aligned(a.kept, 4) ||
      !aligned(a.out_table, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "misaligned argument");
  if ((long long)c.batch * kHkv * 2 * (long long)evict_chunks(a.keep) > 0x7fffffffLL)
    return fail(GQA_ERR_INVALID_ARGUMENT, "batch * keep is too large");
  CacheArgs to = c;
  if (!in_place && c.block_table) {
    to.block_table = a.out_table;
    to.max_pages = a.out_max_pages;
    to.capacity = a.out_max_pages << c.page_log2;
  } else if (!in_place) {
    to.kv = a.out;
    to.scales = a.out_scales;
    to.capacity = a.out_capacity;
  }
  const size_t b4 = (size_t)c.batch * 4;
  const Range lens{a.lens, b4}, weights{a.weights, (size_t)c.batch * kHkv * c.capacity * 4};
  const Range cache{c.kv, c.kv_bytes()}, scales{c.scales, c.scale_bytes()}, table{c.block_table, c.table_bytes()};
  const Range kept{a.kept, (size_t)c.batch * kHkv * a.keep * 4}, ws{a.workspace, need}, none{nullptr, 0};
  if (in_place || c.block_table) {
    const Range ins[] = {table, {a.out_table, to.table_bytes()}, in_place ? none : lens, in_place ? none : weights};
    const Range outs[] = {cache, scales, in_place ? lens : Range{a.out_lens, b4},
                          in_place ? weights : Range{a.out_weights, (size_t)c.batch * kHkv * a.weights_capacity * 4}, kept, ws};
    st = no_aliasing(ins, outs);
  } else {
    const Range ins[] = {cache, scales, lens, weights};
    const Range outs[] = {{to.kv, to.kv_bytes()}, {to.scales, to.scale_bytes()}, {a.out_lens, b4},
                          {a.out_weights, (size_t)c.batch * kHkv * a.weights_capacity * 4}, kept, ws};
    st = no_aliasing(ins, outs);
  }
  if (st != GQA_OK) return st;
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  EvictParams p = {};
  p.src = view_of(c, a.workspace);
  p.dst = view_of(to, a.workspace);
  p.lens = a.lens;
  p.out_lens = in_place ? a.lens : a.out_lens;
  p.weights = a.weights;
  p.out_weights = in_place ? a.weights : a.out_weights;
  p.kept = a.kept;
  char* at = static_cast<char*>(a.workspace) + GQA_WORKSPACE_HEADER_BYTES;
  p.old_lens = reinterpret_cast<int32_t*>(at);
  at += align_up(b4, 256);
  p.ticket = reinterpret_cast<uint32_t*>(at);
  p.read_flags = reinterpret_cast<uint32_t*>(at + 256);
  p.flags = static_cast<uint32_t*>(a.workspace);
  p.batch = c.batch;
  p.keep = a.keep;
  p.recent = a.recent;
  p.first = a.first;
  p.weights_capacity = in_place ? c.capacity : a.weights_capacity;
  p.chunks = (int)(((size_t)a.keep + move_rows(c.format) - 1) / move_rows(c.format));
  p.in_place = in_place;
  const cudaError_t e = launch_evict(p, c.format, sms, a.stream);
  if (e != cudaSuccess) return cuda_fail(e, "eviction kernel launch");
  return GQA_OK;
}

// The append step on a contiguous cache (block_table = nullptr; `units` =
// batch, `unit_rows` = capacity) or a paged one (units = num_pages, unit_rows
// = page size, capacity = max_pages * page size).
gqa_status_t append_kv(const void* q_proj, const void* k_proj, const void* v_proj, const void* q_norm_w,
                       const void* k_norm_w, gqa_dtype_t dtype, const int32_t* positions, const int32_t* slots,
                       int batch, void* q_out, void* kv, gqa_kv_format_t kv_format, void* kv_scales,
                       int capacity, const int32_t* block_table, int max_pages, int num_pages, int page_log2,
                       size_t units, size_t unit_rows, float eps, float rope_theta, float k_scale, float v_scale,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!q_proj || !k_proj || !v_proj || !q_norm_w || !k_norm_w || !positions || !slots || !q_out || !kv)
    return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  gqa_status_t st = validate_shape(batch, capacity);
  if (st != GQA_OK) return st;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)dtype);
  const int fmt = (int)kv_format;
  if (!known_format(fmt)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", fmt);
  if (fmt == kKvE2M1) {  // one token a row of the many-token write
    const CacheArgs c{kv, fmt, kv_scales, batch, capacity, block_table, max_pages, num_pages, page_log2, k_scale, v_scale};
    const WriteArgs a{q_proj, k_proj, v_proj, kHq * kD, kHkv * kD, kHkv * kD, q_norm_w, k_norm_w, (int)dtype, positions,
                      nullptr, 0, nullptr, slots, batch, q_out, eps, rope_theta, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream)};
    return write_kv(c, a);
  }
  if (!is_8bit(fmt) && fmt != (int)dtype)
    return fail(GQA_ERR_INVALID_ARGUMENT, "fp16/bf16 KV must have the dtype of the projections");
  if (fmt == kKvI8 && !kv_scales) return fail(GQA_ERR_INVALID_ARGUMENT, "an int8 cache needs its bf16 row scales");
  if (!std::isfinite(eps) || eps < 0.f) return fail(GQA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (!std::isfinite(rope_theta) || rope_theta <= 0.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "rope_theta must be finite and > 0");
  if (!std::isfinite(k_scale) || k_scale <= 0.f || !std::isfinite(v_scale) || v_scale <= 0.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be finite and > 0");
  if (workspace && workspace_bytes < GQA_WORKSPACE_HEADER_BYTES)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than its %d-byte header", GQA_WORKSPACE_HEADER_BYTES);
  const void* h16[] = {q_proj, k_proj, v_proj, q_norm_w, k_norm_w, q_out};
  for (const void* ptr : h16)
    if (!aligned(ptr, 2)) return fail(GQA_ERR_INVALID_ARGUMENT, "16-bit arrays must be 2-byte aligned");
  if (!aligned(positions, 4) || !aligned(slots, 4) || (workspace && !aligned(workspace, 4)) ||
      (!is_8bit(fmt) && !aligned(kv, 2)) || (kv_scales && !aligned(kv_scales, 2)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "misaligned argument");
  const size_t qb = (size_t)batch * kHq * kD * 2, kvb_in = (size_t)batch * kHkv * kD * 2;
  const size_t cache = units * 2 * kHkv * unit_rows * kv_row_bytes(fmt);
  const void* ins[] = {q_proj, k_proj, v_proj};
  const size_t in_bytes[] = {qb, kvb_in, kvb_in};
  for (int i = 0; i < 3; ++i)
    if (overlap(q_out, qb, ins[i], in_bytes[i]) || overlap(kv, cache, ins[i], in_bytes[i]))
      return fail(GQA_ERR_ALIASING, "q_out or kv overlaps an input projection");
  if (overlap(q_out, qb, kv, cache)) return fail(GQA_ERR_ALIASING, "q_out overlaps kv");
  int dev_sms = 0;
  st = current_device_ready(&dev_sms);
  if (st != GQA_OK) return st;
  AppendParams ap;
  ap.q_proj = q_proj;
  ap.k_proj = k_proj;
  ap.v_proj = v_proj;
  ap.q_norm_w = q_norm_w;
  ap.k_norm_w = k_norm_w;
  ap.positions = positions;
  ap.slots = slots;
  ap.q_out = q_out;
  ap.kv = kv;
  ap.kv_scales = static_cast<uint16_t*>(kv_scales);
  ap.flags = static_cast<uint32_t*>(workspace);
  ap.batch = batch;
  ap.capacity = capacity;
  ap.block_table = block_table;
  ap.max_pages = max_pages;
  ap.num_pages = num_pages;
  ap.page_log2 = page_log2;
  ap.eps = eps;
  ap.k_inv_scale = 1.f / k_scale;
  ap.v_inv_scale = 1.f / v_scale;
  for (int i = 0; i < kD / 2; ++i) ap.inv_freq[i] = std::pow((double)rope_theta, -(double)i / (kD / 2));
  ap.kv_rows = units * 2 * kHkv * unit_rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch, 1, 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  // programmatic dependent launch, as the split kernel: the kernel waits for
  // the previous grid before its first read
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  const bool bf = dtype == GQA_BF16;
  if (fmt == kKvF16) e = cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvF16, kQF16>, ap);
  else if (fmt == kKvBF16) e = cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvBF16, kQBF16>, ap);
  else if (fmt == kKvE4M3)
    e = bf ? cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvE4M3, kQBF16>, ap)
           : cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvE4M3, kQF16>, ap);
  else
    e = bf ? cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvI8, kQBF16>, ap)
           : cudaLaunchKernelEx(&cfg, append_kv_kernel<kKvI8, kQF16>, ap);
  if (e != cudaSuccess) return cuda_fail(e, "append kernel launch");
  return GQA_OK;
}

}  // namespace

extern "C" {

const char* gqa_status_string(gqa_status_t status) {
  switch (status) {
    case GQA_OK: return "GQA_OK";
    case GQA_ERR_INVALID_ARGUMENT: return "GQA_ERR_INVALID_ARGUMENT";
    case GQA_ERR_UNSUPPORTED_DEVICE: return "GQA_ERR_UNSUPPORTED_DEVICE";
    case GQA_ERR_WORKSPACE_TOO_SMALL: return "GQA_ERR_WORKSPACE_TOO_SMALL";
    case GQA_ERR_ALIASING: return "GQA_ERR_ALIASING";
    case GQA_ERR_CUDA: return "GQA_ERR_CUDA";
  }
  return "GQA_ERR_UNKNOWN";
}

const char* gqa_last_error(void) { return g_last_error.c_str(); }

// GQA_INTERFACE: a token that the build forms from the header's digest
#define GQA_TEXT_OF(x) #x
#define GQA_TEXT(x) GQA_TEXT_OF(x)
#ifndef GQA_INTERFACE
#define GQA_INTERFACE
#endif
const char* gqa_interface(void) { return GQA_TEXT(GQA_INTERFACE); }

size_t gqa_decode_workspace_size(int batch, int capacity, int num_splits) {
  if (batch < 1 || capacity < 1 || num_splits < 1 || num_splits > GQA_MAX_SPLITS) return 0;
  return workspace_bytes_for(batch, num_splits);
}

gqa_status_t gqa_decode_plan(int batch, int capacity, gqa_kv_format_t kv_format, int device,
                             int* num_splits_out) {
  if (!num_splits_out) return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits_out is null");
  gqa_status_t st = validate_shape(batch, capacity);
  if (st != GQA_OK) return st;
  if (!known_format((int)kv_format)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", (int)kv_format);
  int sms = 0;
  st = device_ready(device, &sms);
  if (st != GQA_OK) return st;
  *num_splits_out = plan_splits(batch, capacity, kv_format, sms);
  return GQA_OK;
}

gqa_status_t gqa_decode_plan_for(int batch, int capacity, gqa_kv_format_t kv_format, int sm_count,
                                 int* num_splits_out) {
  if (!num_splits_out) return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits_out is null");
  gqa_status_t st = validate_shape(batch, capacity);
  if (st != GQA_OK) return st;
  if (!known_format((int)kv_format)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", (int)kv_format);
  if (sm_count < 1) return fail(GQA_ERR_INVALID_ARGUMENT, "sm_count %d < 1", sm_count);
  *num_splits_out = plan_splits(batch, capacity, kv_format, sm_count);
  return GQA_OK;
}

gqa_status_t gqa_decode_split_geometry(int capacity, int num_splits, gqa_kv_format_t kv_format,
                                       int* chunk_tokens_out, int* splits_effective_out) {
  if (!chunk_tokens_out || !splits_effective_out) return fail(GQA_ERR_INVALID_ARGUMENT, "null output pointer");
  gqa_status_t st = validate_shape(1, capacity);
  if (st != GQA_OK) return st;
  if (!known_format((int)kv_format)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", (int)kv_format);
  if (num_splits < 1 || num_splits > GQA_MAX_SPLITS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits %d outside [1, %d]", num_splits, GQA_MAX_SPLITS);
  *chunk_tokens_out = split_chunk(capacity, num_splits, (int)kv_format);
  *splits_effective_out = split_count(capacity, num_splits, (int)kv_format);
  return GQA_OK;
}

gqa_status_t gqa_decode_launch_count_for(int batch, int capacity, gqa_kv_format_t kv_format, int q_len,
                                        int num_splits, int sm_count, int* launches_out) {
  if (!launches_out) return fail(GQA_ERR_INVALID_ARGUMENT, "launches_out is null");
  gqa_status_t st = validate_shape(batch, capacity);
  if (st != GQA_OK) return st;
  if (!known_format((int)kv_format)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", (int)kv_format);
  if (q_len < 1 || q_len > kMaxQLen) return fail(GQA_ERR_INVALID_ARGUMENT, "q_len %d outside [1, %d]", q_len, kMaxQLen);
  if (num_splits < 1 || num_splits > GQA_MAX_SPLITS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits %d outside [1, %d]", num_splits, GQA_MAX_SPLITS);
  if (sm_count < 1) return fail(GQA_ERR_INVALID_ARGUMENT, "sm_count %d < 1", sm_count);
  // the same rules run_split / run_combine apply to a launch of these sizes
  Call c{};
  c.kv_format = (int)kv_format;
  c.q_dtype = -1;  // (either q format)
  c.batch = batch;
  c.capacity = capacity;
  c.num_splits = num_splits;
  c.q_len = q_len;
  c.sms = sm_count;
  const bool merged = split_count(capacity, num_splits, (int)kv_format) == 1 || cluster_splits(c) > 0;
  *launches_out = merged ? 1 : 2;
  return GQA_OK;
}

gqa_status_t gqa_decode_prepared(const void* q, const void* kv, const int32_t* lens, void* out, int batch,
                                 int capacity, gqa_dtype_t dtype, float q_scale, int num_splits,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  Call c{q, (int)dtype, kv, (int)dtype, lens, out, batch, capacity, q_scale, 1.f, 1.f, num_splits,
         workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  gqa_status_t st = prepare_call(c, /*q_scale_positive=*/true, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_fp8kv(const void* q_bf16, const uint8_t* kv_e4m3, const int32_t* lens, void* out_bf16,
                              int batch, int capacity, float q_scale, float k_scale, float v_scale,
                              int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
  Call c{q_bf16, GQA_BF16, kv_e4m3, kKvE4M3, lens, out_bf16, batch, capacity, q_scale, k_scale, v_scale,
         num_splits, workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_int8kv(const void* q, const int8_t* kv_i8, const uint16_t* kv_scales_bf16,
                               const int32_t* lens, void* out, int batch, int capacity, gqa_dtype_t dtype,
                               float q_scale, int num_splits, void* workspace, size_t workspace_bytes,
                               void* stream) {
  Call c{q, (int)dtype, kv_i8, kKvI8, lens, out, batch, capacity, q_scale, 1.f, 1.f, num_splits, workspace,
         workspace_bytes, static_cast<cudaStream_t>(stream)};
  c.kv_scales = kv_scales_bf16;
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_fp4kv(const void* q, const uint8_t* kv_e2m1, const uint8_t* kv_scales_e4m3,
                              const int32_t* lens, void* out, int batch, int capacity, gqa_dtype_t dtype,
                              float q_scale, float k_scale, float v_scale, int num_splits, void* workspace,
                              size_t workspace_bytes, void* stream) {
  Call c{q, (int)dtype, kv_e2m1, kKvE2M1, lens, out, batch, capacity, q_scale, k_scale, v_scale, num_splits,
         workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  c.kv_scales = kv_scales_e4m3;
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages, gqa_kv_format_t kv_format,
                              const void* kv_scales_pages, const int32_t* block_table, int max_pages_per_seq,
                              int num_pages, int page_size, const int32_t* lens, void* out, int batch, int q_len,
                              float q_scale, float k_scale, float v_scale, int num_splits, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!block_table) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table is null");
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(GQA_ERR_INVALID_ARGUMENT, "page_size %d is not a power of two in [16, 65536]", page_size);
  if (num_pages < 1 || max_pages_per_seq < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_pages and max_pages_per_seq must be >= 1");
  if (q_len < 1 || q_len > kMaxQLen)
    return fail(GQA_ERR_INVALID_ARGUMENT, "q_len %d outside [1, %d]", q_len, kMaxQLen);
  const long long cap = (long long)max_pages_per_seq * page_size;
  if (cap > (1LL << 30)) return fail(GQA_ERR_INVALID_ARGUMENT, "max_pages_per_seq * page_size exceeds 2^30");
  if (!aligned(block_table, 4)) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table must be 4-byte aligned");
  if (kv_format == GQA_KV_I8) {
    if (!kv_scales_pages) return fail(GQA_ERR_INVALID_ARGUMENT, "an int8 cache needs its row scales");
    if (!aligned(kv_scales_pages, 16))
      return fail(GQA_ERR_INVALID_ARGUMENT, "the int8 scale pool must be 16-byte aligned");
  }
  // (validate checks an e2m1 cache's scales)
  Call c{q, (int)q_dtype, kv_pages, (int)kv_format, lens, out, batch, (int)cap, q_scale, k_scale, v_scale,
         num_splits, workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  c.block_table = block_table;
  c.max_pages = max_pages_per_seq;
  c.num_pages = num_pages;
  c.q_len = q_len;
  if (scale_row_bytes((int)kv_format) > 0) c.kv_scales = kv_scales_pages;
  int lg = 0;
  while ((1 << lg) < page_size) ++lg;
  c.page_log2 = lg;
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_verify(const void* q, gqa_dtype_t q_dtype, const void* kv, gqa_kv_format_t kv_format,
                               const void* kv_scales, const int32_t* lens, void* out, int batch,
                               int capacity, int q_len, float q_scale, float k_scale, float v_scale,
                               int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
  if (q_len < 1 || q_len > kMaxQLen)
    return fail(GQA_ERR_INVALID_ARGUMENT, "q_len %d outside [1, %d]", q_len, kMaxQLen);
  Call c{q, (int)q_dtype, kv, (int)kv_format, lens, out, batch, capacity, q_scale, k_scale, v_scale,
         num_splits, workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  c.q_len = q_len;
  c.kv_scales = kv_scales;
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}


gqa_status_t gqa_append_kv(const void* q_proj, const void* k_proj, const void* v_proj, const void* q_norm_w,
                           const void* k_norm_w, gqa_dtype_t dtype, const int32_t* positions, const int32_t* slots,
                           int batch, void* q_out, void* kv, gqa_kv_format_t kv_format, void* kv_scales,
                           int capacity, float eps, float rope_theta, float k_scale, float v_scale, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (capacity < 1) return fail(GQA_ERR_INVALID_ARGUMENT, "capacity %d < 1", capacity);
  return append_kv(q_proj, k_proj, v_proj, q_norm_w, k_norm_w, dtype, positions, slots, batch, q_out, kv, kv_format,
                   kv_scales, capacity, nullptr, 0, 0, 0, batch > 0 ? (size_t)batch : 0, (size_t)capacity,
                   eps, rope_theta, k_scale, v_scale, workspace, workspace_bytes, stream);
}

gqa_status_t gqa_append_kv_paged(const void* q_proj, const void* k_proj, const void* v_proj,
                                 const void* q_norm_w, const void* k_norm_w, gqa_dtype_t dtype,
                                 const int32_t* positions, const int32_t* slots, int batch, void* q_out,
                                 void* kv_pages, gqa_kv_format_t kv_format, void* kv_scales_pages,
                                 const int32_t* block_table, int max_pages_per_seq, int num_pages, int page_size,
                                 float eps, float rope_theta, float k_scale, float v_scale, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!block_table) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table is null");
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(GQA_ERR_INVALID_ARGUMENT, "page_size %d is not a power of two in [16, 65536]", page_size);
  if (num_pages < 1 || max_pages_per_seq < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_pages and max_pages_per_seq must be >= 1");
  const long long cap = (long long)max_pages_per_seq * page_size;
  if (cap > (1LL << 30)) return fail(GQA_ERR_INVALID_ARGUMENT, "max_pages_per_seq * page_size exceeds 2^30");
  if (!aligned(block_table, 4)) return fail(GQA_ERR_INVALID_ARGUMENT, "block_table must be 4-byte aligned");
  int lg = 0;
  while ((1 << lg) < page_size) ++lg;
  return append_kv(q_proj, k_proj, v_proj, q_norm_w, k_norm_w, dtype, positions, slots, batch, q_out, kv_pages,
                   kv_format, kv_scales_pages, (int)cap, block_table, max_pages_per_seq, num_pages, lg,
                   (size_t)num_pages, (size_t)page_size, eps, rope_theta, k_scale, v_scale, workspace,
                   workspace_bytes, stream);
}

gqa_status_t gqa_write_kv(const void* q_proj, const void* k_proj, const void* v_proj, long long q_stride,
                          long long k_stride, long long v_stride, const void* q_norm_w, const void* k_norm_w,
                          gqa_dtype_t dtype, const int32_t* positions, const int* mrope_section,
                          int mrope_interleaved, const int32_t* rows, const int32_t* slots, int tokens, void* q_out,
                          void* kv, gqa_kv_format_t kv_format, void* kv_scales, int batch, int capacity, float eps,
                          float rope_theta, float k_scale, float v_scale, void* workspace, size_t workspace_bytes,
                          void* stream) {
  const CacheArgs c{kv, (int)kv_format, kv_scales, batch, capacity, nullptr, 0, 0, 0, k_scale, v_scale};
  if (!rows) return fail(GQA_ERR_INVALID_ARGUMENT, "rows is null");
  return write_kv(c, {q_proj, k_proj, v_proj, q_stride, k_stride, v_stride, q_norm_w, k_norm_w, (int)dtype, positions,
                      mrope_section, mrope_interleaved, rows, slots, tokens, q_out, eps, rope_theta, workspace,
                      workspace_bytes, static_cast<cudaStream_t>(stream)});
}

gqa_status_t gqa_write_kv_paged(const void* q_proj, const void* k_proj, const void* v_proj, long long q_stride,
                                long long k_stride, long long v_stride, const void* q_norm_w, const void* k_norm_w,
                                gqa_dtype_t dtype, const int32_t* positions, const int* mrope_section,
                                int mrope_interleaved, const int32_t* rows, const int32_t* slots, int tokens,
                                void* q_out, void* kv_pages, gqa_kv_format_t kv_format, void* kv_scales_pages,
                                const int32_t* block_table, int batch, int max_pages_per_seq, int num_pages,
                                int page_size, float eps, float rope_theta, float k_scale, float v_scale,
                                void* workspace, size_t workspace_bytes, void* stream) {
  CacheArgs c{kv_pages, (int)kv_format, kv_scales_pages, batch, 0, nullptr, 0, 0, 0, k_scale, v_scale};
  gqa_status_t st = paged_args(c, block_table, max_pages_per_seq, num_pages, page_size);
  if (st != GQA_OK) return st;
  if (!rows) return fail(GQA_ERR_INVALID_ARGUMENT, "rows is null");
  return write_kv(c, {q_proj, k_proj, v_proj, q_stride, k_stride, v_stride, q_norm_w, k_norm_w, (int)dtype, positions,
                      mrope_section, mrope_interleaved, rows, slots, tokens, q_out, eps, rope_theta, workspace,
                      workspace_bytes, static_cast<cudaStream_t>(stream)});
}

gqa_status_t gqa_read_kv(const void* kv, gqa_kv_format_t kv_format, const void* kv_scales, const int32_t* lens,
                         const int32_t* starts, void* out, gqa_dtype_t out_dtype, int batch, int capacity,
                         int out_capacity, float k_scale, float v_scale, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const CacheArgs c{const_cast<void*>(kv), (int)kv_format, const_cast<void*>(kv_scales), batch, capacity, nullptr,
                    0, 0, 0, k_scale, v_scale};
  return read_kv(c, lens, starts, out, (int)out_dtype, out_capacity, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_read_kv_paged(const void* kv_pages, gqa_kv_format_t kv_format, const void* kv_scales_pages,
                               const int32_t* block_table, int max_pages_per_seq, int num_pages, int page_size,
                               const int32_t* lens, const int32_t* starts, void* out, gqa_dtype_t out_dtype,
                               int batch, int out_capacity, float k_scale, float v_scale, void* workspace,
                               size_t workspace_bytes, void* stream) {
  CacheArgs c{const_cast<void*>(kv_pages), (int)kv_format, const_cast<void*>(kv_scales_pages), batch, 0, nullptr,
              0, 0, 0, k_scale, v_scale};
  gqa_status_t st = paged_args(c, block_table, max_pages_per_seq, num_pages, page_size);
  if (st != GQA_OK) return st;
  return read_kv(c, lens, starts, out, (int)out_dtype, out_capacity, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}

size_t gqa_prefill_workspace_size(void) { return GQA_WORKSPACE_HEADER_BYTES + kPrefillMlBytes + kPrefillOBytes; }

gqa_status_t gqa_prefill(const void* q, gqa_dtype_t q_dtype, const void* kv, gqa_kv_format_t kv_format,
                         const void* kv_scales, const int32_t* chunk_starts, const int32_t* lens, void* out,
                         int tokens, int batch, int capacity, float q_scale, float k_scale, float v_scale,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const CacheArgs c{const_cast<void*>(kv), (int)kv_format, const_cast<void*>(kv_scales), batch, capacity, nullptr,
                    0, 0, 0, k_scale, v_scale};
  return prefill(c, q, (int)q_dtype, chunk_starts, lens, out, tokens, q_scale, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_prefill_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages, gqa_kv_format_t kv_format,
                               const void* kv_scales_pages, const int32_t* block_table, int max_pages_per_seq,
                               int num_pages, int page_size, const int32_t* chunk_starts, const int32_t* lens,
                               void* out, int tokens, int batch, float q_scale, float k_scale, float v_scale,
                               void* workspace, size_t workspace_bytes, void* stream) {
  CacheArgs c{const_cast<void*>(kv_pages), (int)kv_format, const_cast<void*>(kv_scales_pages), batch, 0, nullptr,
              0, 0, 0, k_scale, v_scale};
  gqa_status_t st = paged_args(c, block_table, max_pages_per_seq, num_pages, page_size);
  if (st != GQA_OK) return st;
  return prefill(c, q, (int)q_dtype, chunk_starts, lens, out, tokens, q_scale, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_verify_drafts(const void* probs, long long probs_batch_stride, long long probs_token_stride,
                               const void* draft_probs, long long draft_batch_stride, long long draft_token_stride,
                               gqa_prob_t prob_type, const int32_t* drafts, const float* uniforms,
                               const int32_t* lens, int32_t* out_lens, int32_t* tokens, int32_t* accepted,
                               int batch, int window, int vocab, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_INVALID_ARGUMENT, "batch %d outside [1, 65535]", batch);
  if (window < 1 || window > kMaxWindow) return fail(GQA_ERR_INVALID_ARGUMENT, "window %d outside [1, %d]", window, kMaxWindow);
  // (2^24 terms of up to 2^38 units: the sum stays below 2^63)
  if (vocab < 1 || vocab > (1 << 24)) return fail(GQA_ERR_INVALID_ARGUMENT, "vocab %d outside [1, 2^24]", vocab);
  if (!probs || !uniforms || !tokens || !accepted || (window > 1 && !drafts))
    return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  if ((lens == nullptr) != (out_lens == nullptr))
    return fail(GQA_ERR_INVALID_ARGUMENT, "lens and out_lens are given together or not at all");
  if (prob_type != GQA_PROB_F16 && prob_type != GQA_PROB_BF16 && prob_type != GQA_PROB_F32)
    return fail(GQA_ERR_INVALID_ARGUMENT, "unknown prob_type %d", (int)prob_type);
  const size_t width = prob_type == GQA_PROB_F32 ? 4 : 2;
  const bool with_q = draft_probs != nullptr && window > 1;
  const auto strides_fit = [&](long long bs, long long ts, long long rows) {
    return ts >= vocab && ts <= (1LL << 40) / rows && bs >= rows * ts - (ts - vocab) && bs <= (1LL << 40);
  };
  if (!strides_fit(probs_batch_stride, probs_token_stride, window) ||
      (with_q && !strides_fit(draft_batch_stride, draft_token_stride, window - 1)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "strides must hold the rows without overlap and be at most 2^40 elements");
  if (!aligned(probs, width) || !aligned(draft_probs, width) || !aligned(drafts, 4) || !aligned(uniforms, 4) ||
      !aligned(lens, 4) || !aligned(out_lens, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) || !aligned(workspace, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "misaligned argument");
  if (workspace && workspace_bytes < GQA_WORKSPACE_HEADER_BYTES)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than its %d-byte header", GQA_WORKSPACE_HEADER_BYTES);
  const size_t B = (size_t)batch;
  const size_t p_bytes = ((B - 1) * probs_batch_stride + (window - 1) * probs_token_stride + vocab) * width;
  const size_t q_bytes = with_q ? ((B - 1) * draft_batch_stride + (window - 2) * draft_token_stride + vocab) * width : 0;
  const Range ins[] = {{probs, p_bytes}, {draft_probs, q_bytes}, {drafts, B * (window - 1) * 4}, {uniforms, B * window * 4},
                       {lens == out_lens ? nullptr : lens, B * 4}};
  const Range outs[] = {{out_lens, B * 4}, {tokens, B * window * 4}, {accepted, B * 4},
                        {workspace, (size_t)GQA_WORKSPACE_HEADER_BYTES}};
  gqa_status_t st = no_aliasing(ins, outs);
  if (st != GQA_OK) return st;
  st = current_device_ready(nullptr);
  if (st != GQA_OK) return st;
  DraftParams p = {};
  p.probs = probs;
  p.draft_probs = with_q ? draft_probs : nullptr;
  p.p_batch = probs_batch_stride;
  p.p_token = probs_token_stride;
  p.q_batch = draft_batch_stride;
  p.q_token = draft_token_stride;
  p.drafts = drafts;
  p.uniforms = uniforms;
  p.lens = lens;
  p.out_lens = out_lens;
  p.tokens = tokens;
  p.accepted = accepted;
  p.flags = static_cast<uint32_t*>(workspace);
  p.batch = batch;
  p.window = window;
  p.vocab = vocab;
  p.p_bytes = p_bytes;
  p.q_bytes = q_bytes;
  const int pf = prob_type == GQA_PROB_F32 ? kPF32 : (prob_type == GQA_PROB_BF16 ? kPBF16 : kPF16);
  const cudaError_t e = launch_verify_drafts(p, pf, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "draft verification kernel launch");
  return GQA_OK;
}

size_t gqa_weights_workspace_size(int batch, int capacity, int q_len) {
  if (batch < 1 || batch > 65535 || capacity < 1 || capacity > (1 << 30) || q_len < 1 || q_len > 4) return 0;
  return GQA_WORKSPACE_HEADER_BYTES + score_bytes(batch, capacity, q_len) +
         align_up((size_t)batch * kHkv * max_score_chunks(capacity) * 4 * q_len * sizeof(float2), 256);
}

gqa_status_t gqa_accumulate_weights(const void* q, gqa_dtype_t q_dtype, const void* kv, gqa_kv_format_t kv_format,
                                    const void* kv_scales, const int32_t* lens, float* weights, int batch,
                                    int capacity, int q_len, float q_scale, float k_scale, int add, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const CacheArgs c{const_cast<void*>(kv), (int)kv_format, const_cast<void*>(kv_scales), batch, capacity, nullptr,
                    0, 0, 0, k_scale, 1.f};
  return accumulate(c, q, (int)q_dtype, lens, weights, q_len, q_scale, add, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_accumulate_weights_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages,
                                          gqa_kv_format_t kv_format, const void* kv_scales_pages,
                                          const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                          int page_size, const int32_t* lens, float* weights, int batch, int q_len,
                                          float q_scale, float k_scale, int add, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  CacheArgs c{const_cast<void*>(kv_pages), (int)kv_format, const_cast<void*>(kv_scales_pages), batch, 0, nullptr,
              0, 0, 0, k_scale, 1.f};
  gqa_status_t st = paged_args(c, block_table, max_pages_per_seq, num_pages, page_size);
  if (st != GQA_OK) return st;
  return accumulate(c, q, (int)q_dtype, lens, weights, q_len, q_scale, add, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream));
}

size_t gqa_evict_workspace_size(int batch, int keep) {
  if (batch < 1 || batch > 65535 || keep < 1 || keep > (1 << 30)) return 0;
  return GQA_WORKSPACE_HEADER_BYTES + align_up((size_t)batch * 4, 256) + 256 +
         align_up((size_t)batch * kHkv * 2 * evict_chunks(keep) * 4, 256);
}

gqa_status_t gqa_evict_kv(void* kv, gqa_kv_format_t kv_format, void* kv_scales, int32_t* lens, float* weights,
                          void* out, void* out_scales, int32_t* out_lens, float* out_weights, int32_t* kept,
                          int batch, int capacity, int out_capacity, int weights_capacity, int keep, int recent,
                          int first, void* workspace, size_t workspace_bytes, void* stream) {
  const CacheArgs c{kv, (int)kv_format, kv_scales, batch, capacity, nullptr, 0, 0, 0, 1.f, 1.f};
  const EvictArgs a{lens, weights, out, out_scales, nullptr, out_capacity, 0, out_lens, out_weights, kept,
                    weights_capacity, keep, recent, first, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream)};
  return evict(c, a);
}

gqa_status_t gqa_evict_kv_paged(void* kv_pages, gqa_kv_format_t kv_format, void* kv_scales_pages,
                                const int32_t* block_table, int max_pages_per_seq, int num_pages, int page_size,
                                int32_t* lens, float* weights, const int32_t* out_table, int out_max_pages,
                                int32_t* out_lens, float* out_weights, int32_t* kept, int batch,
                                int weights_capacity, int keep, int recent, int first, void* workspace,
                                size_t workspace_bytes, void* stream) {
  CacheArgs c{kv_pages, (int)kv_format, kv_scales_pages, batch, 0, nullptr, 0, 0, 0, 1.f, 1.f};
  gqa_status_t st = paged_args(c, block_table, max_pages_per_seq, num_pages, page_size);
  if (st != GQA_OK) return st;
  const EvictArgs a{lens, weights, nullptr, nullptr, out_table, 0, out_max_pages, out_lens, out_weights, kept,
                    weights_capacity, keep, recent, first, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream)};
  return evict(c, a);
}

gqa_status_t gqa_decode_split_stage(const void* q, gqa_dtype_t q_dtype, const void* kv,
                                    gqa_kv_format_t kv_format, const int32_t* lens, void* out, int batch,
                                    int capacity, float q_scale, float k_scale, float v_scale, int num_splits,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (kv_format == GQA_KV_I8)
    return fail(GQA_ERR_INVALID_ARGUMENT, "an int8 cache needs its scales: use gqa_decode_int8kv");
  if (kv_format == GQA_KV_E2M1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "an e2m1 cache needs its scales: use gqa_decode_fp4kv");
  Call c{q, (int)q_dtype, kv, (int)kv_format, lens, out, batch, capacity, q_scale, k_scale, v_scale,
         num_splits, workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  return run_split(c);
}

gqa_status_t gqa_decode_debug_skip_tile(const void* q, gqa_dtype_t q_dtype, const void* kv,
                                        gqa_kv_format_t kv_format, const int32_t* lens, void* out, int batch,
                                        int capacity, float q_scale, float k_scale, float v_scale,
                                        int num_splits, void* workspace, size_t workspace_bytes,
                                        int skip_tile, uint64_t wait_budget_ns, void* stream) {
  Call c{q, (int)q_dtype, kv, (int)kv_format, lens, out, batch, capacity, q_scale, k_scale, v_scale,
         num_splits, workspace, workspace_bytes, static_cast<cudaStream_t>(stream)};
  if (skip_tile < 0) return fail(GQA_ERR_INVALID_ARGUMENT, "skip_tile must be >= 0");
  if (wait_budget_ns < 1000000ull || wait_budget_ns > kWaitBudgetNs)
    return fail(GQA_ERR_INVALID_ARGUMENT, "wait_budget_ns must be in [1 ms, 4 s]");
  c.skip_tile = skip_tile;
  c.wait_budget_ns = wait_budget_ns;
  gqa_status_t st = prepare_call(c, false, true);
  if (st != GQA_OK) return st;
  return run_split(c);
}

gqa_status_t gqa_decode_combine_stage(const int32_t* lens, void* out, gqa_dtype_t out_dtype,
                                      gqa_kv_format_t kv_format, int batch, int capacity, float v_scale,
                                      int num_splits, const void* workspace, size_t workspace_bytes,
                                      void* stream) {
  // kv and q are not read by stage 2; stand in a dummy aligned address for
  // the checks (a null kv would be rejected) and skip the q checks.
  static const uint4 dummy = {0, 0, 0, 0};
  const int fmt = (int)kv_format;
  Call c{nullptr, (int)out_dtype, &dummy, is_narrow(fmt) ? fmt : (int)out_dtype, lens, out, batch,
         capacity, 1.f, 1.f, v_scale, num_splits, const_cast<void*>(workspace), workspace_bytes,
         static_cast<cudaStream_t>(stream)};
  if (!known_format(fmt)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown KV format %d", fmt);
  c.kv_format = fmt;
  if (!is_narrow(fmt) && fmt != (int)out_dtype)
    return fail(GQA_ERR_INVALID_ARGUMENT, "fp16/bf16 KV must have the dtype of out");
  // the dummy kv range (batch*capacity*...) would spuriously overlap out; check
  // only what stage 2 touches
  if (!lens || !out || !workspace) return fail(GQA_ERR_INVALID_ARGUMENT, "null pointer argument");
  gqa_status_t st = validate_shape(batch, capacity);
  if (st != GQA_OK) return st;
  if (out_dtype != GQA_F16 && out_dtype != GQA_BF16)
    return fail(GQA_ERR_INVALID_ARGUMENT, "unknown out dtype %d", (int)out_dtype);
  if (!std::isfinite(v_scale) || v_scale <= 0.f)
    return fail(GQA_ERR_INVALID_ARGUMENT, "v_scale must be finite and > 0");
  if (num_splits < 1 || num_splits > GQA_MAX_SPLITS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits %d outside [1, %d]", num_splits, GQA_MAX_SPLITS);
  if (!aligned(out, 16) || !aligned(workspace, 16) || !aligned(lens, 4))
    return fail(GQA_ERR_INVALID_ARGUMENT, "out, workspace must be 16-byte aligned, lens 4-byte");
  const size_t need = workspace_bytes_for(batch, num_splits);
  if (workspace_bytes < need)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  if (overlap(out, (size_t)batch * kHq * kD * 2, workspace, need))
    return fail(GQA_ERR_ALIASING, "out overlaps the workspace");
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  c.sms = sms;
  return run_combine(c);
}

gqa_status_t gqa_decode(const void* q, const void* kv, const int32_t* lens, void* out, int batch, int capacity,
                        gqa_dtype_t dtype, float q_scale, void* stream) {
  static const uint4 dummy_ws = {0, 0, 0, 0};
  Call c{q, (int)dtype, kv, (int)dtype, lens, out, batch, capacity, q_scale, 1.f, 1.f, 0,
         const_cast<uint4*>(&dummy_ws), (size_t)-1, static_cast<cudaStream_t>(stream)};
  // validate with a stand-in workspace, then allocate the real one
  Call probe = c;
  probe.num_splits = 1;
  gqa_status_t st = validate(probe, false, true);
  if (st != GQA_OK) return st;
  int sms = 0;
  st = current_device_ready(&sms);
  if (st != GQA_OK) return st;
  c.num_splits = plan_splits(batch, capacity, (int)dtype, sms);
  c.sms = sms;
  const size_t bytes = workspace_bytes_for(batch, c.num_splits);
  void* ws = nullptr;
  cudaError_t e = cudaMallocAsync(&ws, bytes, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocAsync(workspace)");
  c.workspace = ws;
  c.workspace_bytes = bytes;
  e = cudaMemsetAsync(ws, 0, GQA_WORKSPACE_HEADER_BYTES, c.stream);
  if (e != cudaSuccess) st = cuda_fail(e, "cudaMemsetAsync(workspace header)");
  if (st == GQA_OK) st = validate(c, false, true);
  if (st == GQA_OK) st = run_split(c);
  if (st == GQA_OK) st = run_combine(c);
  e = cudaFreeAsync(ws, c.stream);
  if (st == GQA_OK && e != cudaSuccess) st = cuda_fail(e, "cudaFreeAsync(workspace)");
  return st;
}

gqa_status_t gqa_decode_noalloc(const void* q, const void* kv, const int32_t* lens, void* out, int batch,
                                int capacity, gqa_dtype_t dtype, float q_scale, int num_splits, void* stream) {
  static const uint4 dummy_ws = {0, 0, 0, 0};
  Call c{q, (int)dtype, kv, (int)dtype, lens, out, batch, capacity, q_scale, 1.f, 1.f, 1,
         const_cast<uint4*>(&dummy_ws), (size_t)-1, static_cast<cudaStream_t>(stream)};
  gqa_status_t st = validate(c, false, true);  // everything but the split count and scratch
  if (st != GQA_OK) return st;
  if (num_splits < 0 || num_splits > GQA_MAX_SPLITS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_splits %d outside [0, %d]", num_splits, GQA_MAX_SPLITS);
  if (num_splits > 0 && workspace_bytes_for(batch, num_splits) > kStaticWorkspaceBytes)
    return fail(GQA_ERR_WORKSPACE_TOO_SMALL,
                "batch %d with %d splits needs %zu bytes of scratch; the static scratch holds %zu",
                batch, num_splits, workspace_bytes_for(batch, num_splits), kStaticWorkspaceBytes);
  int dev = -1, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  st = device_ready(dev, &sms);
  if (st != GQA_OK) return st;
  void* ws = nullptr;
  st = static_workspace(dev, c.stream, &ws);
  if (st != GQA_OK) return st;
  int S = num_splits;
  if (S == 0) {
    S = plan_splits(batch, capacity, (int)dtype, sms);
    while (S > 1 && workspace_bytes_for(batch, S) > kStaticWorkspaceBytes) --S;
  }
  c.num_splits = S;
  c.sms = sms;
  c.workspace = ws;
  c.workspace_bytes = kStaticWorkspaceBytes;
  st = validate(c, false, true);
  if (st != GQA_OK) return st;
  // the status word (zeroed at set-up) accumulates over calls until
  // gqa_decode_noalloc_get_status reads and clears it
  st = run_split(c);
  if (st != GQA_OK) return st;
  return run_combine(c);
}

gqa_status_t gqa_decode_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace || workspace_bytes < GQA_WORKSPACE_HEADER_BYTES)
    return fail(GQA_ERR_INVALID_ARGUMENT, "workspace must be non-null and hold the %d-byte header",
                GQA_WORKSPACE_HEADER_BYTES);
  cudaError_t e = cudaMemsetAsync(workspace, 0, GQA_WORKSPACE_HEADER_BYTES, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace header)");
  return GQA_OK;
}

gqa_status_t gqa_decode_get_status(void* workspace, size_t workspace_bytes, void* stream, uint32_t* flags) {
  if (!workspace || !flags || workspace_bytes < GQA_WORKSPACE_HEADER_BYTES)
    return fail(GQA_ERR_INVALID_ARGUMENT, "workspace and flags must be non-null; workspace >= header");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, workspace, sizeof host, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reading the workspace status word");
  *flags = host;
  return GQA_OK;
}

gqa_status_t gqa_decode_debug_cut_extents(uint64_t kv_cut_bytes, uint64_t scales_cut_bytes) {
  if (!kChecked && (kv_cut_bytes || scales_cut_bytes))
    return fail(GQA_ERR_INVALID_ARGUMENT, "extent cuts exist only in the range-checked build (GQA_CHECKED)");
  g_cut_kv_bytes = kv_cut_bytes;
  g_cut_scales_bytes = scales_cut_bytes;
  return GQA_OK;
}

gqa_status_t gqa_decode_noalloc_get_status(void* stream, uint32_t* flags) {
  if (!flags) return fail(GQA_ERR_INVALID_ARGUMENT, "flags must be non-null");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  gqa_status_t st = device_ready(dev, nullptr);
  if (st != GQA_OK) return st;
  void* ws = nullptr;
  st = static_workspace(dev, static_cast<cudaStream_t>(stream), &ws);
  if (st != GQA_OK) return st;
  return gqa_decode_get_status(ws, GQA_WORKSPACE_HEADER_BYTES, stream, flags);
}

}  // extern "C"
