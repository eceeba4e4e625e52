// The softmax weights that a step's queries give the slots of a cache, summed over
// the four heads of each KV head and the window's tokens:
//   weights[b, g, t] (+)= sum over j < T, h in g of exp(s_t - m) / sum_u exp(s_u - m)
//
// The weight of a slot needs the sum over all of them, so a score is formed, kept, and
// turned into a weight when the row's maximum and sum are known.
//
// fused_weights_kernel keeps them on chip: the CTAs of a cluster share a row of one KV
// head and hold its scores in shared memory; their maxima and sums meet in distributed
// shared memory.  For rows whose scores fit and batches that fill the GPU so.
// Otherwise two launches: score_kv_kernel writes the scores (FP32, log2 domain) and
// each chunk's maximum and sum, sum_weights_kernel merges those of a row and turns
// scores into weights.  A score costs 4 bytes to write and 4 to read for each head and
// token, where the key costs 256 bytes (4 bits: 72) for all of them; reading the keys
// twice instead would cost less only for 3- and 4-token windows over 4- and 8-bit caches.
//
// Scores come from mma.sync m16n8k16 with 16 slots as rows and the (token, head)
// pairs as columns.  The order of the dims in a dot product is free: each lane loads
// 16-byte pieces of its two rows and multiplies them as they come, with q arranged
// alike, so no shared memory and no transposition is needed.  Narrow keys are widened
// to fp16 (exact), which takes a third of the instructions that bf16 takes; a bf16 q is
// then scaled by a power of two a column into fp16's range.  Bound by HBM.
#pragma once

#include "cache_rows.cuh"

namespace gqa {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kSlab = 16;  // slots a warp takes at once
constexpr int kSumThreads = 256;
constexpr int kSumSlots = 1024;  // slots a CTA of the second launch takes
constexpr int kRowCluster = 8;           // CTAs of the fused kernel a row
constexpr int kScoreBytes = 96 * 1024;  // of scores that a CTA of the fused kernel holds (two CTAs an SM)

struct WeightParams {
  CacheView c;
  const void* q;        // [B, T, 32, 128]
  const int32_t* lens;
  float* weights;       // [B, 8, capacity]
  float* scores;        // [B, 8, capacity, 4 T]
  float2* stats;        // [B, 8, chunks, 4 T]: maximum, sum
  float scale_log2;
  int chunk, chunks, add;  // slots a CTA of the first launch takes, and how many such
  int held;                // slots whose scores a CTA of the fused kernel holds
};

__device__ __forceinline__ void mma_16816_f32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, bool bf16) {
  if (bf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's part of a row: pieces of 16 bytes, 4 lanes a row.
template <int KVF>
struct RowPart {
  static constexpr int kPieces = kv_row_bytes(KVF) / 64;  // 16-bit 4, 8-bit 2, 4-bit 1
  static constexpr int kRun = 32 / kPieces;               // dims of a piece
  uint4 v[kPieces];
  uint32_t scale;  // int8: the row's bf16; e2m1: the e4m3 of the piece's two groups
  __device__ __forceinline__ void load(const CacheView& c, size_t row, int part) {
    const uint4* src = reinterpret_cast<const uint4*>(c.kv) + row * (kv_row_bytes(KVF) / 16) + part;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) v[i] = __ldg(src + 4 * i);
    if constexpr (KVF == kKvI8) scale = __ldg(static_cast<const uint16_t*>(c.scales) + row);
    if constexpr (KVF == kKvE2M1) scale = __ldg(static_cast<const uint16_t*>(c.scales) + row * 4 + part);
  }
  // its 16 pairs, a narrow row's in fp16
  __device__ __forceinline__ void pairs(uint32_t (&d)[16]) const {
    if constexpr (!is_narrow(KVF)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[4 * i] = v[i].x;
        d[4 * i + 1] = v[i].y;
        d[4 * i + 2] = v[i].z;
        d[4 * i + 3] = v[i].w;
      }
    } else {
      constexpr int kW = KVF == kKvE2M1 ? 2 : 4;  // words of 16 elements
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = v[KVF == kKvE2M1 ? 0 : i];
        const uint32_t all[4] = {x.x, x.y, x.z, x.w};
        uint32_t w[kW], o[8];
#pragma unroll
        for (int j = 0; j < kW; ++j) w[j] = all[KVF == kKvE2M1 ? 2 * i + j : j];
        widen16<KVF>(w, KVF == kKvE2M1 ? (scale >> (8 * i)) & 0xff : 0u, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[8 * i + j] = o[j];
      }
    }
  }
};

__device__ __forceinline__ void merge_stats(float& m0, float& l0, float m1, float l1) {
  const float top = fmaxf(m0, m1);
  l0 = (l0 == 0.f ? 0.f : l0 * ex2(m0 - top)) + (l1 == 0.f ? 0.f : l1 * ex2(m1 - top));  // (a NaN sum is not 0)
  m0 = top;
}

// Scores of slots [begin, end) of batch row b and KV head g, each pair of columns given
// to `store`(slot, first column, scores); their maxima and sums in s_stats[0][column].
template <int KVF, int QF, int NT, class Store>
__device__ __forceinline__ void score_rows(const WeightParams& p, int q_len, int b, int g, int len, int begin, int end,
                                           float2 (*s_stats)[8 * NT], const Store& store) {
  constexpr int MF = is_narrow(KVF) ? (int)kQF16 : QF;  // type of the products' operands
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int cols = 4 * q_len;
  // q of column 8 nt + r, its dims in the order of a row's pieces
  uint32_t q[NT][16];
  float scale[NT][2];  // of columns 8 nt + 2 c, + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = 8 * nt + r;
    constexpr int kRun = RowPart<KVF>::kRun;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (((size_t)b * q_len + col / 4) * kHq + 4 * g + col % 4) * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (col < cols)
        x = __ldg(in_buffer(reinterpret_cast<const uint4*>(src + (8 * i / kRun) * 4 * kRun + c * kRun + 8 * i % kRun), 16, p.q,
                            (size_t)p.c.batch * q_len * kHq * kD * 2, p.c.flags));
      q[nt][4 * i] = x.x;
      q[nt][4 * i + 1] = x.y;
      q[nt][4 * i + 2] = x.z;
      q[nt][4 * i + 3] = x.w;
    }
    float down = 1.f;
    if constexpr (MF != QF) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, max(q[nt][i] & 0x7fffu, q[nt][i] >> 16 & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest |q| into [2^14, 2^15) (its exponent -100 at least, so that the
      // scale's stays a normal number)
      const int e = min(max((int)(top >> 7) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = bf16x2_to_f32x2(q[nt][i]);
        q[nt][i] = round2<kQF16>(f.x * up, f.y * up);
      }
    }
    scale[nt][0] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * c);
    scale[nt][1] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * c + 4);
  }
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[nt][k] = -INFINITY;
      l[nt][k] = 0.f;
    }
  // A narrow row has few bytes: two slabs in flight a warp.  Their rows (a paged cache's
  // block table) are looked up a step earlier.
  constexpr int kSub = is_narrow(KVF) ? 2 : 1, kStep = kScoreWarps * kSlab * kSub;
  RowPart<KVF> next[kSub][2];
  size_t rows[kSub][2];
  const auto look = [&](int t0) {
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k)  // (a slot at or past the end: the last one, whose scores are not used)
        rows[u][k] = cache_row(p.c, b, g, min(t0 + kSlab * u + r + 8 * k, end - 1));
  };
  int t0 = begin + warp * kSlab * kSub;
  if (t0 < end) {
    look(t0);
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) next[u][k].load(p.c, rows[u][k], c);
    if (t0 + kStep < end) look(t0 + kStep);
  }
  for (; t0 < end; t0 += kStep) {
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      uint32_t a[2][16];
      float row_scale[2] = {1.f, 1.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        next[u][k].pairs(a[k]);
        if constexpr (KVF == kKvI8) row_scale[k] = bf16_bits_to_f32((uint16_t)next[u][k].scale);
      }
      if (t0 + kStep < end) {
#pragma unroll
        for (int k = 0; k < 2; ++k) next[u][k].load(p.c, rows[u][k], c);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 8; ++s)
          mma_16816_f32(d, a[0][2 * s], a[1][2 * s], a[0][2 * s + 1], a[1][2 * s + 1], q[nt][2 * s], q[nt][2 * s + 1],
                        MF == kQBF16);
        const int col = 8 * nt + 2 * c;
        // query j sees slots up to len - T + j
        const int seen = len - q_len + col / 4;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = t0 + kSlab * u + r + 8 * k;
          float2 s = make_float2(d[2 * k] * row_scale[k] * scale[nt][0], d[2 * k + 1] * row_scale[k] * scale[nt][1]);
          if (t > seen || t >= end) s = make_float2(-INFINITY, -INFINITY);
          if (col < cols && t < end) store(t, col, s);
          const float sv[2] = {s.x, s.y};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = fmaxf(m[nt][e], sv[e]);
            if (top > m[nt][e]) {
              l[nt][e] *= ex2(m[nt][e] - top);
              m[nt][e] = top;
            }
            // (-inf: a hidden slot, or a score of no weight wherever it lies, also where the
            // maximum is -inf still; a NaN score makes a NaN sum)
            if (sv[e] != -INFINITY) l[nt][e] += ex2(sv[e] - m[nt][e]);
          }
        }
      }
    }
    if (t0 + 2 * kStep < end) look(t0 + 2 * kStep);
  }
  // over the lanes of a column, then the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m[nt][e], o), lo = __shfl_xor_sync(0xffffffffu, l[nt][e], o);
        merge_stats(m[nt][e], l[nt][e], mo, lo);
      }
      if (r == 0) s_stats[warp][8 * nt + 2 * c + e] = make_float2(m[nt][e], l[nt][e]);
    }
  __syncthreads();
  if (threadIdx.x < 8 * NT) {
    float2 x = s_stats[0][threadIdx.x];
    for (int w = 1; w < kScoreWarps; ++w) merge_stats(x.x, x.y, s_stats[w][threadIdx.x].x, s_stats[w][threadIdx.x].y);
    s_stats[0][threadIdx.x] = x;
  }
  __syncthreads();
}

template <int KVF, int QF, int NT>
__global__ void __launch_bounds__(kScoreThreads) score_kv_kernel(const __grid_constant__ WeightParams p, int q_len) {
  __shared__ float2 s_stats[kScoreWarps][8 * NT];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, g = blockIdx.y, C = p.c.capacity, cols = 4 * q_len;
  const bool tell = blockIdx.x == 0 && g == 0 && threadIdx.x == 0;
  const int len = clamp_length(__ldg(item(p.lens, b, p.c.batch, p.c.flags)), C, p.c.flags, tell);
  if (len < q_len && tell && p.c.flags) atomicOr(p.c.flags, GQA_FLAG_LENGTH_CLAMPED);
  const int begin = blockIdx.x * p.chunk, end = min(len, begin + p.chunk);
  if (begin >= len) return;
  const size_t unit = (size_t)b * kHkv + g;
  float* out = p.scores + unit * C * cols;
  const size_t extent = (size_t)p.c.batch * kHkv * C * cols * 4;
  score_rows<KVF, QF, NT>(p, q_len, b, g, len, begin, end, s_stats, [&](int t, int col, float2 s) {
    *reinterpret_cast<float2*>(in_buffer(out + (size_t)t * cols + col, 8, p.scores, extent, p.c.flags)) = s;
  });
  if (threadIdx.x < cols)
    *cell(p.stats + (unit * p.chunks + blockIdx.x) * cols, (int)threadIdx.x, (size_t)cols, p.stats,
          (size_t)p.c.batch * kHkv * p.chunks, p.c.flags) = s_stats[0][threadIdx.x];
}

// A cluster of CTAs a (row, KV head); a CTA's slots are an equal part of the
// row's, p.held at most.
template <int KVF, int QF, int NT>
__global__ void __launch_bounds__(kScoreThreads) fused_weights_kernel(const __grid_constant__ WeightParams p, int q_len) {
  extern __shared__ float s_scores[];  // [slot][column]
  __shared__ float2 s_stats[kScoreWarps][8 * NT];
  __shared__ float s_m[8 * NT], s_r[8 * NT];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  constexpr int S = kRowCluster;
  const int rank = (int)blockIdx.x % S;
  const size_t unit = blockIdx.x / S;
  const int b = (int)(unit / kHkv), g = (int)(unit % kHkv), C = p.c.capacity, cols = 4 * q_len;
  const bool tell = rank == 0 && g == 0 && threadIdx.x == 0;
  const int len = clamp_length(__ldg(item(p.lens, b, p.c.batch, p.c.flags)), C, p.c.flags, tell);
  if (len < q_len && tell && p.c.flags) atomicOr(p.c.flags, GQA_FLAG_LENGTH_CLAMPED);
  if (len == 0) return;  // (all of the cluster)
  const int part = ((len + S - 1) / S + kSlab - 1) / kSlab * kSlab;
  const int begin = min(len, rank * part), end = min(len, begin + part);
  score_rows<KVF, QF, NT>(p, q_len, b, g, len, begin, end, s_stats, [&](int t, int col, float2 s) {
    *reinterpret_cast<float2*>(s_scores + (size_t)min(t - begin, p.held - 1) * cols + col) = s;
  });
  cluster_sync_all();
  if (threadIdx.x < 8 * NT) {
    const uint32_t at = smem_addr(&s_stats[0][threadIdx.x]);
    float2 y[S];  // (all on their way before the first is merged)
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const uint32_t theirs = cluster_map(at, (uint32_t)k);
      y[k] = make_float2(cluster_ld(theirs), cluster_ld(theirs + 4));
    }
    float2 x = y[0];
#pragma unroll
    for (int k = 1; k < S; ++k) merge_stats(x.x, x.y, y[k].x, y[k].y);
    s_m[threadIdx.x] = x.x;
    s_r[threadIdx.x] = x.y == 0.f ? 0.f : 1.f / x.y;  // (a query that sees no slot gives no weight)
  }
  cluster_sync_all();  // (nobody's shared memory is left while it is read)
  const size_t extent = (size_t)p.c.batch * kHkv * C * 4;
  for (int t = begin + threadIdx.x; t < end; t += kScoreThreads) {
    const float4* src = reinterpret_cast<const float4*>(s_scores + (size_t)(t - begin) * cols);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      if (j >= q_len) break;
      const float4 x = src[j];
      const float s[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (s[h] != -INFINITY) sum += ex2(s[h] - s_m[4 * j + h]) * s_r[4 * j + h];
    }
    float* dst = in_buffer(p.weights + unit * C + t, 4, p.weights, extent, p.c.flags);
    *dst = p.add ? *dst + sum : sum;
  }
}

// COLS = 4 T: a thread's scores of a slot are COLS / 4 loads of 16 bytes.
template <int COLS>
__global__ void __launch_bounds__(kSumThreads) sum_weights_kernel(const __grid_constant__ WeightParams p) {
  __shared__ float s_m[COLS], s_r[COLS];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, g = blockIdx.y, C = p.c.capacity;
  const int len = min(max(__ldg(item(p.lens, b, p.c.batch, p.c.flags)), 0), C);
  const int begin = blockIdx.x * kSumSlots, end = min(len, begin + kSumSlots);
  if (begin >= len) return;
  const size_t unit = (size_t)b * kHkv + g;
  const int used = (len + p.chunk - 1) / p.chunk;
  float2* const stats = p.stats + unit * p.chunks * COLS;
  const auto stat = [&](int k, int col) {
    return cell(stats + (size_t)k * COLS, col, COLS, p.stats, (size_t)p.c.batch * kHkv * p.chunks, p.c.flags);
  };
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int col = warp; col < COLS; col += kSumThreads / 32) {
    float m = -INFINITY;
    for (int k = lane; k < used; k += 32) m = fmaxf(m, stat(k, col)->x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int k = lane; k < used; k += 32) {
      const float2 x = *stat(k, col);
      if (x.y != 0.f) l += x.y * ex2(x.x - m);  // (a NaN sum is not 0)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      s_m[col] = m;
      s_r[col] = l == 0.f ? 0.f : 1.f / l;  // (a query that sees no slot gives no weight)
    }
  }
  __syncthreads();
  const size_t extent = (size_t)p.c.batch * kHkv * C * 4;
  for (int t = begin + threadIdx.x; t < end; t += kSumThreads) {
    const float4* src = reinterpret_cast<const float4*>(
        in_buffer(p.scores + (unit * C + t) * COLS, COLS * 4, p.scores, (size_t)p.c.batch * kHkv * C * COLS * 4, p.c.flags));
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < COLS / 4; ++j) {
      const float4 x = __ldcs(src + j);
      const float s[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int h = 0; h < 4; ++h)  // (a hidden slot's score is -inf: no weight, whatever the row's sum is)
        if (s[h] != -INFINITY) sum += ex2(s[h] - s_m[4 * j + h]) * s_r[4 * j + h];
    }
    float* dst = in_buffer(p.weights + unit * C + t, 4, p.weights, extent, p.c.flags);
    *dst = p.add ? *dst + sum : sum;
  }
}

}  // namespace gqa
