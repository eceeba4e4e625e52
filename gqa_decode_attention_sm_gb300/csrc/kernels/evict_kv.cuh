// Making a cache smaller: of the slots [0, L) of a row the first `first`, the last
// `recent` and, of those between, the ones of the largest weights stay, `keep` in
// all, each KV head choosing for itself; they move in their order to slots 0, 1, ...
//
// A head's threshold is its k-th largest weight, of the weights' order-preserving
// integers.  select_few_kernel (up to 8192 slots) holds a head's weights in one CTA's
// registers and finds the threshold bit by bit, counting the weights that are no
// smaller, from the first bit in which the least and the largest differ, of all of them
// until 2048 are left and then of those.  (Histograms' atomics meet in the few bins that
// softmax weights lie in: 32 x 8192 took 25 us with them; 8 x 32768, a head in one CTA's
// registers, 36 us against 22 by a cluster of two.)
// select_kv_kernel takes more: 11, 11 and 10 bits at a time, a histogram each, by a
// cluster of CTAs that hold their parts of the weights in shared memory; histograms and
// counts meet in distributed shared memory.  Both then write the kept slots in ascending
// order by a prefix sum of "above the threshold, or equal to it and among the first
// such".  Everything counted is whole numbers, so the result does not depend on any order.
//
// move_kv_kernel gathers the rows (and their scales and weights), 8 KB a CTA (both
// kernels, 8 x U[16k, 32k] to 8192 bf16 tokens: 112 us; 16 KB 119, 128 threads 116).
// Bound by HBM: 537 MB moved, 0.80 of the copy rate.  In place a CTA may overwrite rows that another has yet to read: the CTAs
// take their chunks by ticket in ascending order, say when theirs is read and write
// once all chunks before it have been read.  Reading waits for nothing and a later
// chunk's rows lie behind every row that an earlier one writes, so no wait can last
// longer than the loads of CTAs that run already.
#pragma once

#include "cache_rows.cuh"

namespace gqa {

constexpr int kFewThreads = 512;
constexpr int kFewSlots = 16 * kFewThreads;
constexpr int kFewList = 2048;
constexpr int kSelectBins = 2048;
constexpr int kSelectKeys = 48 * 1024;  // weights that a CTA holds in shared memory (192 KB)
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 8192;  // of rows that a CTA moves

__host__ __device__ constexpr int move_rows(int kv_format) { return kMoveBytes / kv_row_bytes(kv_format); }

struct EvictParams {
  CacheView src, dst;  // dst: the same cache in place
  const int32_t* lens;
  int32_t* out_lens;
  const float* weights;  // [B, 8, capacity]
  float* out_weights;    // [B, 8, weights_capacity] or null; in place: weights
  int32_t* kept;         // [B, 8, keep]
  int32_t* old_lens;     // [B], workspace: the clamped lengths
  uint32_t* ticket;      // workspace, in place
  uint32_t* read_flags;  // [B, 8, 2, chunks], workspace, in place
  uint32_t* flags;
  int batch, keep, recent, first, weights_capacity, chunks;
  int in_place;
  int cluster;  // CTAs that share a head
  int held;  // weights a CTA of the select kernel holds in shared memory (0: reads them each time)
  __device__ __forceinline__ int32_t* kept_at(int32_t* row, int i) const {  // row: kept + unit * keep
    return cell(row, i, (size_t)keep, kept, (size_t)batch * kHkv, flags);
  }
  __device__ __forceinline__ float* out_weight(int unit, int i) const {
    return cell(out_weights + (size_t)unit * weights_capacity, i, (size_t)weights_capacity, out_weights, (size_t)batch * kHkv, flags);
  }
  __device__ __forceinline__ uint32_t* read_flag(int up, int i) const {  // up: unit * 2 + plane
    return cell(read_flags + (size_t)up * chunks, i, (size_t)chunks, read_flags, (size_t)batch * kHkv * 2, flags);
  }
  __device__ __forceinline__ int32_t* old_len(int b) const { return item(old_lens, b, batch, flags); }
};

// Integers in the order of the weights; NaN below everything, both zeros one.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// A head's CTAs: the cluster's, or one CTA launched without a cluster, which has no
// use for the cluster's barrier and shared memory.
__device__ __forceinline__ void head_sync(int S) {
  if (S > 1) cluster_sync_all();
  else __syncthreads();
}
__device__ __forceinline__ uint32_t head_ld(const uint32_t* p, int S, int rank) {
  if (S == 1) return *p;
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map(smem_addr(p), (uint32_t)rank)) : "memory");
  return v;
}

// What both kernels do besides choosing: the row's saved length, the in-place move's
// flags cleared, the slots that are kept anyway.  Returns the slots held; `keep` or
// fewer need no choice.
__device__ __forceinline__ int select_begin(const EvictParams& p, int unit, int first, int step) {
  const int b = unit / kHkv;
  const int L = clamp_length(__ldg(item(p.lens, b, p.batch, p.flags)), p.src.capacity, p.flags,
                             unit % kHkv == 0 && first == 0);
  int32_t* const kept = p.kept + (size_t)unit * p.keep;
  if (first == 0 && unit % kHkv == 0) *p.old_len(b) = L;
  if (p.in_place) {
    for (int i = first; i < 2 * p.chunks; i += step)
      *cell(p.read_flags + (size_t)unit * 2 * p.chunks, i, (size_t)2 * p.chunks, p.read_flags, (size_t)p.batch * kHkv, p.flags) = 0u;
    if (unit == 0 && first == 0) *p.ticket = 0u;
  }
  if (L <= p.keep) {
    for (int i = first; i < p.keep; i += step) *p.kept_at(kept, i) = i < L ? i : -1;
  } else {  // first + recent <= keep < L
    for (int i = first; i < p.first + p.recent; i += step)
      *p.kept_at(kept, i < p.first ? i : p.keep - p.recent + (i - p.first)) = i < p.first ? i : L - p.recent + (i - p.first);
  }
  return L;
}

// K weights a thread: warp w has K * 32 consecutive slots, 32 at a time.
template <int K>
__global__ void __launch_bounds__(kFewThreads, 2) select_few_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = kFewThreads / 32;
  static_assert(kWarps <= 32, "a lane adds a warp's count");
  __shared__ uint32_t s_count[2][kWarps], s_above[kWarps], s_equal[kWarps], s_list[kFewList], s_listed;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int unit = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int L = select_begin(p, unit, tid, kFewThreads);
  if (L <= p.keep) return;
  const int lo = p.first, hi = L - p.recent;
  const float* w = p.weights + (size_t)unit * p.src.capacity;
  const size_t extent = (size_t)p.batch * kHkv * p.src.capacity * 4;
  uint32_t x[K];  // 0 (no weight but NaN) where there is no slot: never counted, its index is looked at
  const int at = lo + warp * 32 * K + lane;
  if (!kChecked && lo + (warp + 1) * 32 * K <= hi) {  // the warp's slots are all there: one address, loads side by side
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = __float_as_uint(__ldg(w + at + 32 * i));
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = weight_key(__uint_as_float(x[i]));
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i)
      x[i] = at + 32 * i < hi ? weight_key(__ldg(in_buffer(w + at + 32 * i, 4, p.weights, extent, p.flags))) : 0u;
  }
  if (tid == 0) s_listed = 0u;
  __syncthreads();
  // The sum of the threads' numbers, by two buffers in turn (one is read before the
  // barrier after which it is written again).
  int turn = 0;
  const auto total = [&](uint32_t n) {
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_count[turn][warp] = n;
    __syncthreads();
    n = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_count[turn][lane] : 0u);
    turn ^= 1;
    return n;
  };
  const auto count = [&](uint32_t least) {  // weights at or above it, which is not 0
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) n += x[i] >= least;
    return total(n);
  };
  // kept: above `threshold`, and the first `need` equal to it
  uint32_t need = (uint32_t)(p.keep - p.first - p.recent), threshold = 0xffffffffu;  // (no weight's key)
  if (need > 0) {
    // the least and the largest weight: the bits before they differ are known
    uint32_t most = 0u, least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      most = max(most, x[i]);
      least = min(least, x[i] == 0u ? 0xffffffffu : x[i]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      s_above[warp] = most;
      s_equal[warp] = least;
    }
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, s_above[lane % kWarps]);
    least = __reduce_min_sync(0xffffffffu, s_equal[lane % kWarps]);
    __syncthreads();
    uint32_t upto = most == 0u ? 0u : count(least);  // weights at or above t
    if (upto < need) {                               // NaN among the kept
      threshold = 0u;
      need -= upto;
    } else {
      int bit = least == most ? -1 : 31 - __clz(least ^ most);
      // weights of the interval [t, t + 2^(bit + 1)), which holds the threshold, lie below
      // `upto` and above `over` in order
      uint32_t t = bit < 0 ? least : least & ~((2u << bit) - 1u), over = 0u;
      bool exact = upto == need;
      while (bit >= 0 && !exact && upto - over > kFewList) {
        const uint32_t middle = t | 1u << bit;
        const uint32_t n = count(middle);
        if (n >= need) {
          t = middle;
          upto = n;
        } else {
          over = n;
        }
        exact = n == need;
        --bit;
      }
      if (bit >= 0 && !exact) {
        // few are left in it: listed, two a thread
        const uint32_t width = (2u << bit) - 1u;
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (x[i] != 0u && x[i] - t <= width) {
            const uint32_t to = atomicAdd(&s_listed, 1u);
            if (to < kFewList) s_list[to] = x[i];
          }
        __syncthreads();
        // by the first eight warps, whose barrier is shorter
        constexpr int kListThreads = 256, kEach = kFewList / kListThreads;
        if (tid < kListThreads) {
          const uint32_t listed = min(s_listed, (uint32_t)kFewList), outside = over;
          uint32_t y[kEach];
#pragma unroll
          for (int i = 0; i < kEach; ++i) y[i] = tid + kListThreads * i < listed ? s_list[tid + kListThreads * i] : 0u;
          for (; bit >= 0 && !exact; --bit) {
            const uint32_t middle = t | 1u << bit;
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) n += y[i] >= middle;
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) s_count[turn][warp] = n;
            named_barrier_sync(1, kListThreads);
            n = outside + __reduce_add_sync(0xffffffffu, lane < kListThreads / 32 ? s_count[turn][lane] : 0u);
            turn ^= 1;
            if (n >= need) t = middle;
            else over = n;
            exact = n == need;
          }
          if (tid == 0) {
            s_above[0] = t;
            s_above[1] = over;
            s_above[2] = exact;
          }
        }
        __syncthreads();
        t = s_above[0];
        over = s_above[1];
        exact = s_above[2] != 0u;
        __syncthreads();
      }
      // exact: as many as needed at or above t, which is 0 where the least and the largest
      // weight differ in their first bit and every number is kept: all but key 0, which is NaN's
      threshold = exact ? max(t, 1u) - 1u : t;
      need = exact ? 0u : need - over;
    }
  }
  // how many lie above and on the threshold before each warp's slots (where there is no
  // slot x is 0, which is on a threshold of 0 only)
  uint32_t above = 0, equal = 0;
#pragma unroll
  for (int i = 0; i < K; ++i) above += x[i] > threshold;
  above = __reduce_add_sync(0xffffffffu, above);
  if (need > 0) {
#pragma unroll
    for (int i = 0; i < K; ++i) equal += x[i] == threshold && at + 32 * i < hi;
    equal = __reduce_add_sync(0xffffffffu, equal);
  }
  if (lane == 0) {
    s_above[warp] = above;
    s_equal[warp] = equal;
  }
  __syncthreads();
  // before this warp: lane k has warp k's
  above = __reduce_add_sync(0xffffffffu, lane < warp ? s_above[lane % kWarps] : 0u);
  equal = __reduce_add_sync(0xffffffffu, lane < warp ? s_equal[lane % kWarps] : 0u);
  above += min(equal, need);  // those on the threshold that the warps before keep
  int32_t* const kept = p.kept + (size_t)unit * p.keep;
  const uint32_t before = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    uint32_t chosen = __ballot_sync(0xffffffffu, x[i] > threshold);
    if (need > 0) {  // and of those on the threshold the first ones
      const uint32_t eq = __ballot_sync(0xffffffffu, x[i] == threshold && at + 32 * i < hi);
      chosen |= __ballot_sync(0xffffffffu, (eq >> lane & 1) && equal + __popc(eq & before) < need);
      equal += __popc(eq);
    }
    if (chosen >> lane & 1) {
      const uint32_t to = (uint32_t)p.first + above + __popc(chosen & before);
      if (kChecked || to < (uint32_t)p.keep) *p.kept_at(kept, (int)to) = at + 32 * i;  // (always; held in bounds)
    }
    above += __popc(chosen);
  }
}

template <int kSelectThreads>
__global__ void __launch_bounds__(kSelectThreads) select_kv_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kSelectWarps = kSelectThreads / 32;
  static_assert(2 * kSelectThreads == kSelectBins, "a thread counts two bins");
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t s_hist[2][kSelectBins];
  __shared__ uint32_t s_part[kSelectWarps], s_part2[kSelectWarps];
  __shared__ uint32_t s_bin, s_above, s_count[2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int S = p.cluster, rank = (int)blockIdx.x % S;
  const int unit = blockIdx.x / S;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int C = p.src.capacity;
  const int L = select_begin(p, unit, rank * kSelectThreads + tid, S * kSelectThreads);
  if (L <= p.keep) return;  // (the same in every CTA of the cluster)
  int32_t* const kept = p.kept + (size_t)unit * p.keep;
  const int lo = p.first, hi = L - p.recent;
  const float* w = p.weights + (size_t)unit * C;
  const size_t w_extent = (size_t)p.batch * kHkv * C * 4;
  const auto load_key = [&](int t) { return weight_key(__ldg(in_buffer(w + t, 4, p.weights, w_extent, p.flags))); };
  // the CTA's candidates, and the warps': consecutive slots
  const int all = hi - lo;
  const int seg = ((all + S - 1) / S + 31) / 32 * 32;
  const int c0 = (int)min((long long)all, (long long)rank * seg), c1 = min(all - c0, seg) + c0;
  const bool held = c1 - c0 <= p.held;
  if (held)
    for (int i = c0 + tid; i < c1; i += kSelectThreads) s_keys[i - c0] = load_key(lo + i);
  const auto key = [&](int i) { return held ? s_keys[i - c0] : load_key(lo + i); };
  uint32_t need = (uint32_t)(p.keep - p.first - p.recent);  // to be found, of those equal so far
  uint32_t threshold = 0xffffffffu;                         // (no weight's key)
  if (need > 0) {
    threshold = 0;
    constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const int shift = kShift[d], bits = d == 2 ? 10 : 11;
      const uint32_t mask = (1u << bits) - 1;
      uint32_t* hist = s_hist[d & 1];
      for (int i = tid; i < kSelectBins; i += kSelectThreads) hist[i] = 0u;
      __syncthreads();
      for (int i = c0 + tid; i < c1; i += kSelectThreads) {
        const uint32_t x = key(i);
        if (d == 0 || (x >> (shift + bits)) == (threshold >> (shift + bits))) atomicAdd(&hist[x >> shift & mask], 1u);
      }
      // (a histogram is cleared again two digits later, after the other's cluster
      // barrier, when every CTA has read it)
      head_sync(S);
      uint32_t mine[2] = {0, 0};  // bins 2 tid, 2 tid + 1 counted from the top
      const int top = kSelectBins - 1 - 2 * tid;
      uint32_t theirs[8][2];  // (all on their way before the first is added)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        theirs[k][0] = k < S ? head_ld(hist + top, S, k) : 0u;
        theirs[k][1] = k < S ? head_ld(hist + top - 1, S, k) : 0u;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        mine[0] += theirs[k][0];
        mine[1] += theirs[k][1];
      }
      uint32_t upto = mine[0] + mine[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) s_part[warp] = upto;
      __syncthreads();
      uint32_t above = upto - mine[0] - mine[1];
      for (int k = 0; k < warp; ++k) above += s_part[k];
      if (above < need && need <= above + mine[0]) {
        s_bin = (uint32_t)top;
        s_above = above;
      } else if (above + mine[0] < need && need <= above + mine[0] + mine[1]) {
        s_bin = (uint32_t)(top - 1);
        s_above = above + mine[0];
      }
      __syncthreads();
      threshold |= s_bin << shift;
      need -= s_above;
    }
  }
  // how many lie above and on the threshold before each warp's slots
  const int per = ((c1 - c0 + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int w0 = min(c1, c0 + warp * per), w1 = min(c1, w0 + per);
  uint32_t above = 0, equal = 0;
  for (int i = w0; i < w1; i += 32) {
    const uint32_t x = i + lane < w1 ? key(i + lane) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && x > threshold));
    equal += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && x == threshold));
  }
  __syncthreads();  // (s_part is done with)
  if (lane == 0) {
    s_part[warp] = above;
    s_part2[warp] = equal;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0, y = 0;
    for (int k = 0; k < kSelectWarps; ++k) {
      x += s_part[k];
      y += s_part2[k];
    }
    s_count[0] = x;
    s_count[1] = y;
  }
  head_sync(S);
  above = equal = 0;
  uint32_t theirs[8][2];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    theirs[k][0] = k < rank ? head_ld(s_count, S, k) : 0u;
    theirs[k][1] = k < rank ? head_ld(s_count + 1, S, k) : 0u;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    above += theirs[k][0];
    equal += theirs[k][1];
  }
  head_sync(S);  // (nobody's shared memory is left while it is read)
  for (int k = 0; k < warp; ++k) {
    above += s_part[k];
    equal += s_part2[k];
  }
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t x = in ? key(i + lane) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, in && x > threshold);
    const uint32_t eq = __ballot_sync(0xffffffffu, in && x == threshold);
    const uint32_t before = (1u << lane) - 1;
    const uint32_t rank_eq = equal + __popc(eq & before);
    if (in && (x > threshold || (x == threshold && rank_eq < need))) {
      const uint32_t at = (uint32_t)p.first + above + __popc(gt & before) + min(rank_eq, need);
      if (kChecked || at < (uint32_t)p.keep) *p.kept_at(kept, (int)at) = lo + i + lane;  // (always; held in bounds)
    }
    above += __popc(gt);
    equal += __popc(eq);
  }
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

template <int KVF>
__global__ void __launch_bounds__(kMoveThreads) move_kv_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kRow = kv_row_bytes(KVF), kPer = kRow / 16;     // threads a row
  constexpr int kRows = move_rows(KVF), kStep = kMoveThreads / kPer;  // rows a CTA has, and takes at once
  constexpr int kIter = kRows / kStep;
  __shared__ uint32_t s_ticket;
  __shared__ int s_late;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  uint32_t job = blockIdx.x;
  if (p.in_place) {
    if (threadIdx.x == 0) {
      s_ticket = atomicAdd(p.ticket, 1u);
      s_late = 0;
    }
    __syncthreads();
    job = s_ticket;
  }
  const int chunk = (int)(job % (uint32_t)p.chunks);
  const int up = (int)(job / (uint32_t)p.chunks), plane = up & 1, unit = up >> 1, b = unit / kHkv;
  const int L = min(max(*p.old_len(b), 0), p.src.capacity), n = min(L, p.keep);
  const int pg = plane * kHkv + unit % kHkv;
  if (unit % kHkv == 0 && plane == 0 && chunk == 0 && threadIdx.x == 0)
    *item(p.out_lens, b, p.batch, p.flags) = n;
  if (p.in_place && L <= p.keep) return;  // nothing moves
  const int lane = threadIdx.x % kPer, first = chunk * kRows;
  int32_t* const kept = p.kept + (size_t)unit * p.keep;
  const float* w = p.weights + (size_t)unit * p.src.capacity;
  bool strayed = false;
  uint4 x[kIter];
  uint2 sc[kIter];
  float wt[kIter];
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const int at = first + k * kStep + threadIdx.x / kPer;
    if (at >= n) continue;
    // a slot of the row, as the select kernel wrote it; another one (the caller's other
    // work, or a mistake here) is left inside the row and told
    const int said = *p.kept_at(kept, at);
    const int t = min(max(said, 0), L - 1);
    strayed |= t != said;
    const size_t row = cache_row(p.src, b, pg, t);
    x[k] = *(reinterpret_cast<const uint4*>(p.src.kv) + row * kPer + lane);
    if (lane == 0) {
      if constexpr (KVF == kKvI8) sc[k].x = static_cast<const uint16_t*>(p.src.scales)[row];
      if constexpr (KVF == kKvE2M1) sc[k] = static_cast<const uint2*>(p.src.scales)[row];
      if (plane == 0 && p.out_weights)
        wt[k] = *cell(w, t, (size_t)p.src.capacity, p.weights, (size_t)p.batch * kHkv, p.flags);
    }
  }
  if (p.in_place) {
    __threadfence();  // this thread's reads come before the flag
    __syncthreads();
    if (threadIdx.x == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.read_flag(up, chunk)), "r"(1u) : "memory");
    const uint64_t deadline = global_timer_ns() + kWaitBudgetNs;
    for (int c = threadIdx.x; c < chunk; c += kMoveThreads)
      while (load_acquire(p.read_flag(up, c)) == 0u)
        if (global_timer_ns() > deadline) {
          s_late = 1;
          break;
        }
    __syncthreads();
    if (s_late) {
      if (threadIdx.x == 0 && p.flags) atomicOr(p.flags, GQA_FLAG_WAIT_TIMEOUT);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const int at = first + k * kStep + threadIdx.x / kPer;
    if (at >= n) continue;
    bool known = true;
    const size_t row = cache_row(p.dst, b, pg, at, &known);
    if (!known) continue;
    *(reinterpret_cast<uint4*>(const_cast<void*>(p.dst.kv)) + row * kPer + lane) = x[k];
    if (lane == 0) {
      if constexpr (KVF == kKvI8) static_cast<uint16_t*>(const_cast<void*>(p.dst.scales))[row] = (uint16_t)sc[k].x;
      if constexpr (KVF == kKvE2M1) static_cast<uint2*>(const_cast<void*>(p.dst.scales))[row] = sc[k];
      if (plane == 0 && p.out_weights) *p.out_weight(unit, at) = wt[k];
    }
  }
  if (strayed && p.flags) atomicOr(p.flags, GQA_FLAG_BOUNDS);
  // slots behind the kept ones start their sums at zero (in place: those that held tokens)
  if (plane == 0 && p.out_weights) {
    const int end = chunk < p.chunks - 1 ? first + kRows : (p.in_place ? L : p.weights_capacity);
    for (int at = max(first, n) + threadIdx.x; at < end; at += kMoveThreads)
      *p.out_weight(unit, at) = 0.f;
  }
  // (kept[] of a row shorter than `keep` ends in -1, written by the select kernel)
}

}  // namespace gqa
