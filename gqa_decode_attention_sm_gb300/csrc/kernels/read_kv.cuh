// Reading a cache back: slots [start, len) of every batch row, from a cache of
// any format, contiguous or paged, into a dense fp16 or bf16 cache from its
// slot 0 on ([B, 2, 8, out_capacity, 128]).
//
// Each value is code * scale (* the tensor scale) in FP32, exact but for the
// tensor scale's product, and rounded once.  Eight threads hold a row, sixteen
// elements each (one e2m1 scale group), and a thread has kReadRows rows in
// flight; a CTA reads kReadChunk slots of one (row, plane, KV head).
#pragma once

#include "common.cuh"

namespace gqa {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;                                // rows a thread has in flight
constexpr int kReadChunk = kReadRows * kReadThreads / 8;    // slots a CTA reads

struct ReadParams {
  const void* kv;
  const void* kv_scales;
  const int32_t* lens;    // [B]
  const int32_t* starts;  // [B] or null (0)
  void* out;              // [B, 2, 8, out_capacity, 128]
  uint32_t* flags;        // optional status word
  int batch, capacity, out_capacity;
  const int32_t* block_table;
  int max_pages, num_pages, page_log2;
  float k_scale, v_scale;
  size_t kv_rows;  // rows of 128 in the cache, for checked builds
};

template <int OF>
__device__ __forceinline__ uint32_t read_round2(float lo, float hi) {
  if constexpr (OF == kQF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int KVF, int OF>
__global__ void __launch_bounds__(kReadThreads) read_kv_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, pg = blockIdx.y;  // pg = plane * 8 + KV head
  const int len_raw = __ldg(p.lens + b), start_raw = p.starts ? __ldg(p.starts + b) : 0;
  const int len = min(max(len_raw, 0), p.capacity), start = min(max(start_raw, 0), len);
  if ((len != len_raw || start != start_raw) && p.flags && pg == 0 && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.flags, GQA_FLAG_LENGTH_CLAMPED);
  const int n = min(len - start, p.out_capacity);
  const int j0 = blockIdx.x * kReadChunk + (threadIdx.x >> 3), e = threadIdx.x & 7;
  constexpr int kWords = kv_row_bytes(KVF) / 32;  // 32-bit words of a thread's 16 elements
  uint32_t w[kReadRows][kWords];
  float sc[kReadRows];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    const int j = j0 + k * (kReadThreads / 8);
    if (j >= n) continue;
    const int t = start + j;
    size_t unit = (size_t)b, rows = (size_t)p.capacity, in = (size_t)t;
    if (p.block_table != nullptr) {
      int id = __ldg(p.block_table + (size_t)b * p.max_pages + (t >> p.page_log2));
      if (id < 0 || id >= p.num_pages) {  // out-of-contract page id: clamp, flag, never fault
        if (p.flags) atomicOr(p.flags, GQA_FLAG_PAGE_CLAMPED);
        id = min(max(id, 0), p.num_pages - 1);
      }
      unit = (size_t)id;
      rows = (size_t)1 << p.page_log2;
      in = (size_t)(t & ((1 << p.page_log2) - 1));
    }
    size_t row = (unit * 2 * kHkv + pg) * rows + in;
    if constexpr (kChecked) {
      if (row >= p.kv_rows) {
        if (p.flags) atomicOr(p.flags, GQA_FLAG_BOUNDS);
        row = 0;
      }
    }
    const uint32_t* src = static_cast<const uint32_t*>(p.kv) + row * (kv_row_bytes(KVF) / 4) + e * kWords;
    if constexpr (kWords == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
      w[k][0] = v.x;
      w[k][1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
        w[k][4 * i] = v.x;
        w[k][4 * i + 1] = v.y;
        w[k][4 * i + 2] = v.z;
        w[k][4 * i + 3] = v.w;
      }
    }
    if constexpr (KVF == kKvE2M1) {
      const uint32_t s = __ldg(static_cast<const uint8_t*>(p.kv_scales) + row * 8 + e);
      sc[k] = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)s)).x;
    } else if constexpr (KVF == kKvI8) {
      sc[k] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.kv_scales) + row) << 16);
    } else {
      sc[k] = 1.f;
    }
  }
  const float all = pg < kHkv ? p.k_scale : p.v_scale;
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    const int j = j0 + k * (kReadThreads / 8);
    if (j >= n) continue;
    uint32_t o[8];
    if constexpr (KVF == kKvF16 || KVF == kKvBF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr ((KVF == kKvF16) == (OF == kQF16)) {
          o[i] = w[k][i];
        } else {
          const float2 f = KVF == kKvF16 ? f16x2_to_f32x2(w[k][i]) : bf16x2_to_f32x2(w[k][i]);
          o[i] = read_round2<OF>(f.x, f.y);
        }
      }
    } else {
      float x[16];
      if constexpr (KVF == kKvE2M1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t d[4];
          e2m1x8_to_f16(w[k][i], d);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float2 f = f16x2_to_f32x2(d[m]);
            x[8 * i + 2 * m] = f.x;
            x[8 * i + 2 * m + 1] = f.y;
          }
        }
      } else if constexpr (KVF == kKvE4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[k][i >> 1] >> (16 * (i & 1)))));
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = (float)(int8_t)(w[k][i >> 2] >> (8 * (i & 3)));
      }
      // code * scale is exact; then the tensor scale (1 for int8), rounded once in FP32
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = read_round2<OF>(x[2 * i] * sc[k] * all, x[2 * i + 1] * sc[k] * all);
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                          (((size_t)b * 2 * kHkv + pg) * p.out_capacity + j) * kD) + 2 * e;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace gqa
