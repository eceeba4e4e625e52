// The softmax weights that a step's queries give the slots of a cache, summed over
// the four heads of each KV head and the window's tokens:
//   weights[b, g, t] (+)= sum over j < T, h in g of exp(s_t - m) / sum_u exp(s_u - m)
//
// The weight of a slot needs the sum over all of them.  Two launches: the first
// reads the keys once and writes every score (FP32, log2 domain) and each chunk's
// maximum and sum; the second merges those of a row and turns scores into weights.
// A score costs 4 bytes to write and 4 to read for each head and token, where the key
// costs 256 bytes (4 bits: 72) for all of them, so keeping the scores beats reading the
// keys twice except for 3- and 4-token windows over 4- and 8-bit caches.
//
// Scores come from mma.sync m16n8k16 with 16 slots as rows and the (token, head)
// pairs as columns.  The order of the dims in a dot product is free: each lane loads
// 16-byte pieces of its two rows and multiplies them as they come, with q arranged
// alike, so no shared memory and no transposition is needed.  Bound by HBM.
#pragma once

#include "cache_rows.cuh"

namespace gqa {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kSlab = 16;  // slots a warp takes at once
constexpr int kSumThreads = 256;
constexpr int kSumSlots = 1024;  // slots a CTA of the second launch takes
constexpr int kMaxScoreCols = 16;

struct WeightParams {
  CacheView c;
  const void* q;        // [B, T, 32, 128]
  const int32_t* lens;
  float* weights;       // [B, 8, capacity]
  float* scores;        // [B, 8, capacity, 4 T]
  float2* stats;        // [B, 8, chunks, 4 T]: maximum, sum
  float scale_log2;
  int chunk, chunks, add;  // slots a CTA of the first launch takes, and how many such
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
  // its 16 pairs
  template <int QF>
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
        widen16<KVF, QF>(w, KVF == kKvE2M1 ? (scale >> (8 * i)) & 0xff : 0u, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[8 * i + j] = o[j];
      }
    }
  }
};

template <int KVF, int QF, int NT>
__global__ void __launch_bounds__(kScoreThreads) score_kv_kernel(const __grid_constant__ WeightParams p, int q_len) {
  __shared__ float2 s_stats[kScoreWarps][8 * NT];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, g = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int C = p.c.capacity, cols = 4 * q_len;
  const int raw = __ldg(p.lens + b);
  const int len = clamp_length(raw, C, p.c.flags, blockIdx.x == 0 && g == 0 && threadIdx.x == 0);
  if (len < q_len && blockIdx.x == 0 && g == 0 && threadIdx.x == 0 && p.c.flags) atomicOr(p.c.flags, GQA_FLAG_LENGTH_CLAMPED);
  const int begin = blockIdx.x * p.chunk, end = min(len, begin + p.chunk);
  if (begin >= len) return;
  // q of column 8 nt + r, its dims in the order of a row's pieces
  uint32_t q[NT][16];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = 8 * nt + r;
    constexpr int kRun = RowPart<KVF>::kRun;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (((size_t)b * q_len + col / 4) * kHq + 4 * g + col % 4) * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (col < cols)
        x = __ldg(reinterpret_cast<const uint4*>(src + (8 * i / kRun) * 4 * kRun + c * kRun + 8 * i % kRun));
      q[nt][4 * i] = x.x;
      q[nt][4 * i + 1] = x.y;
      q[nt][4 * i + 2] = x.z;
      q[nt][4 * i + 3] = x.w;
    }
  }
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[nt][k] = -INFINITY;
      l[nt][k] = 0.f;
    }
  const size_t unit = (size_t)b * kHkv + g;
  float* out = p.scores + unit * C * cols;
  const size_t out_extent = (size_t)p.c.batch * kHkv * C * cols * 4;
  RowPart<KVF> next[2];
  const auto fetch = [&](int t0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // (a slot at or past the end: the chunk's last one, whose scores are not used)
      const int t = min(t0 + r + 8 * k, end - 1);
      next[k].load(p.c, cache_row(p.c, b, g, t), c);
    }
  };
  int t0 = begin + warp * kSlab;
  if (t0 < end) fetch(t0);
  for (; t0 < end; t0 += kScoreWarps * kSlab) {
    uint32_t a[2][16];
    float row_scale[2] = {p.scale_log2, p.scale_log2};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      next[k].template pairs<QF>(a[k]);
      if constexpr (KVF == kKvI8) row_scale[k] *= bf16_bits_to_f32((uint16_t)next[k].scale);
    }
    if (t0 + kScoreWarps * kSlab < end) fetch(t0 + kScoreWarps * kSlab);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_16816_f32(d, a[0][2 * s], a[1][2 * s], a[0][2 * s + 1], a[1][2 * s + 1], q[nt][2 * s], q[nt][2 * s + 1],
                      QF == kQBF16);
      const int col = 8 * nt + 2 * c;
      // query j sees slots up to len - T + j
      const int seen = len - q_len + col / 4;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = t0 + r + 8 * k;
        float2 s = make_float2(d[2 * k] * row_scale[k], d[2 * k + 1] * row_scale[k]);
        if (t > seen || t >= end) s = make_float2(-INFINITY, -INFINITY);
        if (col < cols && t < end)
          *reinterpret_cast<float2*>(in_buffer(out + (size_t)t * cols + col, 8, p.scores, out_extent, p.c.flags)) = s;
        const float sv[2] = {s.x, s.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float top = fmaxf(m[nt][e], sv[e]);
          if (top > m[nt][e]) {
            l[nt][e] *= ex2(m[nt][e] - top);
            m[nt][e] = top;
          }
          if (t <= seen && t < end) l[nt][e] += ex2(sv[e] - m[nt][e]);  // (a NaN score makes a NaN sum)
        }
      }
    }
  }
  // the chunk's maximum and sum of each column: over the lanes of a column, then the warps
  const auto merge = [](float& m0, float& l0, float m1, float l1) {
    const float top = fmaxf(m0, m1);
    l0 = (l0 == 0.f ? 0.f : l0 * ex2(m0 - top)) + (l1 == 0.f ? 0.f : l1 * ex2(m1 - top));
    m0 = top;
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m[nt][e], o), lo = __shfl_xor_sync(0xffffffffu, l[nt][e], o);
        merge(m[nt][e], l[nt][e], mo, lo);
      }
      if (r == 0) s_stats[warp][8 * nt + 2 * c + e] = make_float2(m[nt][e], l[nt][e]);
    }
  __syncthreads();
  if (threadIdx.x < cols) {
    float2 x = s_stats[0][threadIdx.x];
    for (int w = 1; w < kScoreWarps; ++w) merge(x.x, x.y, s_stats[w][threadIdx.x].x, s_stats[w][threadIdx.x].y);
    p.stats[(unit * p.chunks + blockIdx.x) * cols + threadIdx.x] = x;
  }
}

// COLS = 4 T: a thread's scores of a slot are COLS / 4 loads of 16 bytes.
template <int COLS>
__global__ void __launch_bounds__(kSumThreads) sum_weights_kernel(const __grid_constant__ WeightParams p) {
  __shared__ float s_m[COLS], s_r[COLS];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, g = blockIdx.y, C = p.c.capacity;
  const int len = min(max(__ldg(p.lens + b), 0), C);
  const int begin = blockIdx.x * kSumSlots, end = min(len, begin + kSumSlots);
  if (begin >= len) return;
  const size_t unit = (size_t)b * kHkv + g;
  const int used = (len + p.chunk - 1) / p.chunk;
  const float2* stats = p.stats + unit * p.chunks * COLS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int col = warp; col < COLS; col += kSumThreads / 32) {
    float m = -INFINITY;
    for (int k = lane; k < used; k += 32) m = fmaxf(m, stats[(size_t)k * COLS + col].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int k = lane; k < used; k += 32) {
      const float2 x = stats[(size_t)k * COLS + col];
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
    const float4* src = reinterpret_cast<const float4*>(p.scores + (unit * C + t) * COLS);
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
