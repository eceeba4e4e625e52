// Attention of chunks of new tokens over a cache: the simplest form, a warp for a
// token and a KV head.
#pragma once

#include "cache_rows.cuh"

namespace gqa {

struct PrefillParams {
  CacheView c;
  const void* q;               // [tokens, 32, 128]
  void* out;                   // [tokens, 32, 128]
  const int32_t* chunk_starts;  // [B + 1]
  const int32_t* lens;         // [B]
  int tokens;
  float scale_log2, v_scale;
};

// Eight consecutive elements of a row as floats, scales included.
template <int KVF>
__device__ __forceinline__ void row8(const CacheView& c, size_t row, int i, float (&x)[8]) {
  if constexpr (!is_narrow(KVF)) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(c.kv) + row * 16 + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = KVF == kKvF16 ? f16x2_to_f32x2(w[k]) : bf16x2_to_f32x2(w[k]);
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  } else {
    uint32_t w[4] = {}, d[8];
    float s = 1.f;
    uint32_t group = 0;
    if constexpr (KVF == kKvE2M1) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(c.kv) + row * 16 + i);
      group = __ldg(static_cast<const uint8_t*>(c.scales) + row * 8 + i / 2);
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(c.kv) + row * 16 + i);
      w[0] = v.x;
      w[1] = v.y;
      if constexpr (KVF == kKvI8) s = bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(c.scales) + row));
    }
    widen16<KVF, kQF16>(w, group, d);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = f16x2_to_f32x2(d[k]);
      x[2 * k] = f.x * s;
      x[2 * k + 1] = f.y * s;
    }
  }
}

template <int KVF, int QF>
__global__ void __launch_bounds__(128) prefill_kernel(const __grid_constant__ PrefillParams p) {
  __shared__ float s_q[4][4][kD];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = blockIdx.y;
  const int i = blockIdx.x * 4 + warp;
  if (i >= p.tokens) return;
  int b = 0, at = 0, n = 0;
  for (; b < p.c.batch; ++b) {
    at = min(max(__ldg(p.chunk_starts + b), 0), p.tokens);
    n = min(max(__ldg(p.chunk_starts + b + 1), at), p.tokens) - at;
    if (i >= at && i < at + n) break;
  }
  if (b == p.c.batch) return;
  const int len = clamp_length(__ldg(p.lens + b), p.c.capacity, p.c.flags, lane == 0);
  const int end = len - n + (i - at) + 1;  // slots seen
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + ((size_t)i * kHq + 4 * g) * kD;
  for (int k = lane; k < 2 * kD; k += 32) {
    const float2 f = pair_to_f32x2<QF>(reinterpret_cast<const uint32_t*>(q)[k]);
    s_q[warp][k / 64][2 * (k % 64)] = f.x;
    s_q[warp][k / 64][2 * (k % 64) + 1] = f.y;
  }
  __syncwarp();
  float m[4], l[4], o[4][4];
  for (int h = 0; h < 4; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int k = 0; k < 4; ++k) o[h][k] = 0.f;
  }
  for (int t0 = 0; t0 < end; t0 += 32) {
    const int t = min(t0 + lane, end - 1);
    const size_t krow = cache_row(p.c, b, g, t);
    float s[4] = {};
    for (int k = 0; k < 16; ++k) {
      float x[8];
      row8<KVF>(p.c, krow, k, x);
      for (int h = 0; h < 4; ++h)
        for (int e = 0; e < 8; ++e) s[h] += x[e] * s_q[warp][h][8 * k + e];
    }
    for (int h = 0; h < 4; ++h) {
      const bool in = t0 + lane < end;
      s[h] = in ? s[h] * p.scale_log2 : -INFINITY;
      float top = fmaxf(m[h], s[h]);
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float f = m[h] == -INFINITY ? 0.f : ex2(m[h] - top);
      m[h] = top;
      s[h] = in ? ex2(s[h] - (top == -INFINITY ? 0.f : top)) : 0.f;
      float sum = s[h];
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[h] = l[h] * f + sum;
      for (int k = 0; k < 4; ++k) o[h][k] *= f;
    }
    for (int j = 0; j < min(32, end - t0); ++j) {
      const size_t vrow = cache_row(p.c, b, kHkv + g, t0 + j);
      float x[8];
      row8<KVF>(p.c, vrow, lane / 2, x);
      for (int h = 0; h < 4; ++h) {
        const float w = __shfl_sync(0xffffffffu, s[h], j);
        for (int k = 0; k < 4; ++k) o[h][k] += w * (lane & 1 ? x[4 + k] : x[k]);
      }
    }
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + ((size_t)i * kHq + 4 * g) * kD) + 2 * lane;
  for (int h = 0; h < 4; ++h) {
    const float f = l[h] == 0.f ? 0.f : p.v_scale / l[h];
    out[64 * h] = round2<QF>(o[h][0] * f, o[h][1] * f);
    out[64 * h + 1] = round2<QF>(o[h][2] * f, o[h][3] * f);
  }
}

}  // namespace gqa
