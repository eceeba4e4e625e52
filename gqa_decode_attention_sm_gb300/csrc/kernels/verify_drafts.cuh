// Drafted tokens against the target's probabilities.
//
// Draft j of a row (token d_j, drawn with probability q_j(d_j)) is taken while
// u_j q_j(d_j) < p_j(d_j), which is a probability of min(1, p / q); after n of them
// the next token is drawn from max(p_n - q_n, 0) if draft n was refused, from p_n if
// none is left.  A token drawn so has the target's distribution.
//
// The draw is the inverse of the running sum over the vocabulary.  Its terms are
// rounded to whole units of 2^-38 first (of a vocabulary of 2^18 tokens these
// roundings are 2^-21 of the sum at most), so that the sum is one of 64-bit
// integers: whatever order the threads add in, the same number picks the same token.
//
// Only the rows that the draw needs are read, one of p (and one of q) a request, and
// once: a cluster of CTAs holds a request's row, a warp a run of consecutive tokens;
// the runs' sums meet in distributed shared memory, and the one warp whose run holds
// the target reads its run again (4 KB of L2).  Bound by HBM for many requests, by
// the latency of draft -> probability -> row -> cluster for few.
#pragma once

#include "common.cuh"

namespace gqa {

constexpr int kDraftThreads = 256;  // (four CTAs an SM at 64 registers: 64 requests are one wave)
constexpr int kDraftCluster = 8;  // CTAs a request
constexpr int kDraftWarps = kDraftThreads / 32;
constexpr int kMaxWindow = 32;  // a warp's lanes judge a window's drafts at once

enum ProbFormat : int { kPF16 = 0, kPBF16 = 1, kPF32 = 2 };

struct DraftParams {
  const void* probs;        // [B, T, V]
  const void* draft_probs;  // [B, T - 1, V], or null: a draft has probability one
  long long p_batch, p_token, q_batch, q_token;  // strides in elements
  const int32_t* drafts;    // [B, T - 1]
  const float* uniforms;    // [B, T]
  const int32_t* lens;      // [B] or null
  int32_t* out_lens;        // [B] or null; may be lens
  int32_t* tokens;          // [B, T]
  int32_t* accepted;        // [B]
  uint32_t* flags;
  int batch, window, vocab;
  size_t p_bytes, q_bytes;  // extents, for checked builds
  __device__ __forceinline__ const int32_t* draft(int b, int j) const {
    return cell(drafts + (long long)b * (window - 1), j, (size_t)window - 1, drafts, (size_t)batch, flags);
  }
  __device__ __forceinline__ const float* uniform(int b, int j) const {
    return cell(uniforms + (long long)b * window, j, (size_t)window, uniforms, (size_t)batch, flags);
  }
  __device__ __forceinline__ int32_t* token(int b, int j) const {
    return cell(tokens + (long long)b * window, j, (size_t)window, tokens, (size_t)batch, flags);
  }
};

template <int PF>
struct ProbTraits {
  static constexpr int kBytes = PF == kPF32 ? 4 : 2;
  static constexpr int kVec = 16 / kBytes;  // elements of 16 bytes
};

template <int PF>
__device__ __forceinline__ float prob_at(const void* base, long long i, const DraftParams& p, size_t extent) {
  if constexpr (PF == kPF32) {
    return __ldg(in_buffer(static_cast<const float*>(base) + i, 4, static_cast<const float*>(base), extent, p.flags));
  } else {
    const uint16_t* b = static_cast<const uint16_t*>(base);
    const uint16_t x = __ldg(in_buffer(b + i, 2, b, extent, p.flags));
    return PF == kPBF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
  }
}

// 16 bytes as floats
template <int PF>
__device__ __forceinline__ void prob_vec(uint4 v, float (&x)[ProbTraits<PF>::kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PF == kPF32) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = PF == kPF16 ? f16x2_to_f32x2(w[i]) : bf16x2_to_f32x2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// The weight of a token with probability p where the draft's was q, in units of 2^-38
// (NaN and negative values none; p - q is rounded once, in FP32), as 2^22 hi + lo.
// Whole numbers come from adding 2^23, which costs an FP32 operation where the 64-bit
// conversion has a sixteenth of its rate (64 x 131072 tokens: 38 us with that, 17
// so): hi the 2^16 x rounded down, lo the exact rest in units of 2^-22, to the nearest
// (ties to even: 2^22 hi is even).
struct DraftWeight {
  uint32_t hi, lo;
};
__device__ __forceinline__ DraftWeight draft_weight(float p, float q) {
  const float x = __saturatef(p - q);
  const float whole = __fmaf_rz(x, 0x1p16f, 0x1p23f);
  const float rest = fmaf(x, 0x1p16f, -(whole - 0x1p23f));
  const float part = __fmaf_rn(rest, 0x1p22f, 0x1p23f);
  return {__float_as_uint(whole) - 0x4b000000u, __float_as_uint(part) - 0x4b000000u};
}
__device__ __forceinline__ unsigned long long units_of(uint32_t hi, uint32_t lo) {
  return ((unsigned long long)hi << 22) + lo;
}

// How a request's row is weighed: the row of p, the row of q or none, and the token
// that has no weight (a refused draft that had probability one) or -1.
struct DraftRow {
  long long p0, q0;
  int without;
  bool q;
};

template <int PF>
__device__ __forceinline__ unsigned long long token_weight(const DraftParams& p, const DraftRow& r, int i) {
  const float a = prob_at<PF>(p.probs, r.p0 + i, p, p.p_bytes);
  const float b = r.q ? prob_at<PF>(p.draft_probs, r.q0 + i, p, p.q_bytes) : 0.f;
  const DraftWeight w = draft_weight(a, b);
  return i == r.without ? 0ull : units_of(w.hi, w.lo);
}

// The sum of tokens [lo, hi) over the warp, in every lane.
template <int PF>
__device__ __forceinline__ unsigned long long run_sum(const DraftParams& p, const DraftRow& r, int lo, int hi) {
  constexpr int kVec = ProbTraits<PF>::kVec, kBytes = ProbTraits<PF>::kBytes;
  const int lane = threadIdx.x & 31;
  unsigned long long sum = 0;
  const char* a = static_cast<const char*>(p.probs) + (r.p0 + lo) * kBytes;
  const char* b = r.q ? static_cast<const char*>(p.draft_probs) + (r.q0 + lo) * kBytes : a;
  // whole 16-byte groups where both rows have the same place in one (a vocabulary
  // whose rows do not start on 16 bytes: an element a lane)
  const int off = (int)((uintptr_t)a & 15);
  int i = lo;
  if (off == (int)((uintptr_t)b & 15)) {
    const int head = min(hi - lo, off ? (16 - off) / kBytes : 0);
    if (lane < head) sum += token_weight<PF>(p, r, lo + lane);
    i += head;
    const int groups = (hi - i) / kVec;
    const uint4* va = reinterpret_cast<const uint4*>(a + (long long)head * kBytes);
    const uint4* vb = reinterpret_cast<const uint4*>(b + (long long)head * kBytes);
    const int skip = r.without - i;  // (in this run's groups, or not)
    constexpr int kDeep = 4;  // loads of each row in flight
    for (int g = lane; g < groups; g += 32 * kDeep) {
      uint4 x[kDeep], y[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        if (g + 32 * k < groups) {
          x[k] = __ldg(in_buffer(va + g + 32 * k, 16, reinterpret_cast<const uint4*>(p.probs), p.p_bytes, p.flags));
          if (r.q)
            y[k] = __ldg(in_buffer(vb + g + 32 * k, 16, reinterpret_cast<const uint4*>(p.draft_probs), p.q_bytes, p.flags));
        }
      }
      uint32_t hi = 0, lo = 0;  // (kDeep * kVec <= 32 terms: below 2^22 and 2^28)
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        float s[kVec], t[kVec];
        prob_vec<PF>(x[k], s);
        prob_vec<PF>(y[k], t);
        const int at = (g + 32 * k) * kVec;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const DraftWeight w = draft_weight(at + e == skip ? 0.f : s[e], t[e]);
          hi += w.hi;
          lo += w.lo;
        }
      }
      sum += units_of(hi, lo);
    }
    i += groups * kVec;
  }
  for (int j = i + lane; j < hi; j += 32) sum += token_weight<PF>(p, r, j);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The first token of [lo, hi) whose running sum passes `target` (the warp's; one is
// there): the 32 tokens that hold it by their sums, then the token among them.
template <int PF>
__device__ __forceinline__ int find_token(const DraftParams& p, const DraftRow& r, int lo, int hi,
                                          unsigned long long target) {
  const int lane = threadIdx.x & 31;
  unsigned long long before = 0;
  constexpr int kDeep = 8;
  for (int i = lo; i < hi; i += 32 * kDeep) {
    DraftWeight w[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int at = min(i + 32 * k + lane, hi - 1);
      const float a = prob_at<PF>(p.probs, r.p0 + at, p, p.p_bytes);
      const float b = r.q ? prob_at<PF>(p.draft_probs, r.q0 + at, p, p.q_bytes) : 0.f;
      w[k] = draft_weight(at == r.without || i + 32 * k + lane >= hi ? 0.f : a, b);
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const unsigned long long all = units_of(__reduce_add_sync(0xffffffffu, w[k].hi), __reduce_add_sync(0xffffffffu, w[k].lo));
      if (before + all > target) {
        unsigned long long upto = units_of(w[k].hi, w[k].lo);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        return i + 32 * k + __ffs(__ballot_sync(0xffffffffu, before + upto > target)) - 1;
      }
      before += all;
    }
  }
  return -1;
}

template <int PF>
__global__ void __launch_bounds__(kDraftThreads, 4) verify_drafts_kernel(const __grid_constant__ DraftParams p) {
  __shared__ unsigned long long s_warp[kDraftWarps], s_total;
  __shared__ int s_n, s_refused;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  constexpr int S = kDraftCluster;
  const int rank = (int)cluster_rank();
  const int b = blockIdx.x / S, T = p.window, V = p.vocab;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const long long pb = (long long)b * p.p_batch, qb = (long long)b * p.q_batch;
  if (warp == 0) {
    // every CTA of the cluster judges the drafts; lane j draft j
    const int d = lane < T - 1 ? __ldg(p.draft(b, lane)) : -1;
    const bool given = d >= 0 && d < V;
    if (lane < T - 1 && d >= V && rank == 0 && p.flags) atomicOr(p.flags, GQA_FLAG_SLOT_CLAMPED);
    bool taken = false;
    if (given) {
      const float u = __ldg(p.uniform(b, lane));
      const float pd = prob_at<PF>(p.probs, pb + lane * p.p_token + d, p, p.p_bytes);
      const float qd = p.draft_probs ? prob_at<PF>(p.draft_probs, qb + lane * p.q_token + d, p, p.q_bytes) : 1.f;
      taken = (double)u * (double)qd < (double)pd;  // (the product of two floats is exact)
    }
    const uint32_t all_given = __ballot_sync(0xffffffffu, given), all_taken = __ballot_sync(0xffffffffu, taken);
    const int n = __ffs(~all_taken) - 1;  // (lane T - 1 takes none)
    if (lane == 0) {
      s_n = n;
      s_refused = n < T - 1 && (all_given >> n & 1);
    }
    if (rank == 0) {
      if (lane < T && lane != n) *p.token(b, lane) = lane < n ? d : -1;
      if (lane == 0) {
        *item(p.accepted, b, p.batch, p.flags) = n;
        if (p.out_lens)
          *item(p.out_lens, b, p.batch, p.flags) = max(max(*item(p.lens, b, p.batch, p.flags), 0) - (T - 1) + n, 0);  // (no overflow)
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  const float u = __ldg(p.uniform(b, T - 1));
  DraftRow r;
  r.p0 = pb + n * p.p_token;
  r.q0 = qb + n * p.q_token;
  r.q = s_refused && p.draft_probs != nullptr;
  r.without = s_refused && p.draft_probs == nullptr ? __ldg(p.draft(b, n)) : -1;
  // the warps' runs: consecutive tokens, in whole groups of 32 * 16 bytes
  const int runs = S * kDraftWarps, unit = 32 * ProbTraits<PF>::kVec;
  const int per = ((V + runs - 1) / runs + unit - 1) / unit * unit;
  const int run = rank * kDraftWarps + warp;
  const int lo = (int)min((long long)V, (long long)run * per), hi = min(V - lo, per) + lo;
  for (int attempt = 0;; ++attempt) {
    const unsigned long long mine = run_sum<PF>(p, r, lo, hi);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    unsigned long long before = 0, here = 0;  // runs of this CTA before the warp's, and all of them
#pragma unroll
    for (int w = 0; w < kDraftWarps; ++w) {
      const unsigned long long x = s_warp[w];
      before += w < warp ? x : 0ull;
      here += x;
    }
    if (threadIdx.x == 0) s_total = here;
    cluster_sync_all();
    unsigned long long total = 0, theirs[kDraftCluster];  // (all on their way before the first is added)
    const uint32_t at = smem_addr(&s_total);
#pragma unroll
    for (int k = 0; k < kDraftCluster; ++k)
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(theirs[k]) : "r"(cluster_map(at, (uint32_t)k)) : "memory");
#pragma unroll
    for (int k = 0; k < kDraftCluster; ++k) {
      before += k < rank ? theirs[k] : 0ull;
      total += theirs[k];
    }
    cluster_sync_all();  // (nobody's shared memory is left or written while it is read)
    if (total == 0 && attempt == 0 && (r.q || r.without >= 0)) {
      // nothing is left of p beside q: from p itself
      r.q = false;
      r.without = -1;
      continue;
    }
    if (total == 0) {  // no weight at all (zeros, NaN): no token
      if (rank == 0 && threadIdx.x == 0) *p.token(b, n) = -1;
      return;
    }
    // floor(total * u), u in units of 2^-24; 128-bit product
    const unsigned long long k = (unsigned long long)fminf(fmaxf(floorf(u * 0x1p24f), 0.f), 0x1p24f - 1.f);
    const unsigned long long target = (total * k) >> 24 | __umul64hi(total, k) << 40;
    if (target >= before && target - before < mine) {
      const int pick = find_token<PF>(p, r, lo, hi, target - before);
      if (lane == 0) *p.token(b, n) = pick;
    }
    return;
  }
}

}  // namespace gqa
