// Reading a cache back: slots [start, len) of every batch row, from a cache of
// any format, contiguous or paged, into a dense fp16 or bf16 cache from its
// slot 0 on ([B, 2, 8, out_capacity, 128]).
//
// Each value is code * scale (* the tensor scale) in FP32, exact but for the
// tensor scale's product, and rounded once.  Eight threads hold a row, 16
// elements each (an e2m1 scale group); a CTA takes every gridDim.x-th chunk of 32
// slots of one (row, plane, KV head).
//
// Bound by HBM, most of it the output's writes.  One row in flight a thread and
// many CTAs keep the writes of a CTA close together: 8 x U[16k, 32k] e2m1 tokens
// (328 bytes a row moved) take 148 us, 1.03 of the copy peak, with 4 rows in
// flight 197; 16 threads a row 175.
#pragma once

#include "common.cuh"

namespace gqa {

constexpr int kReadThreads = 256;
constexpr int kReadRowThreads = 8;                           // threads a row
constexpr int kReadElems = kD / kReadRowThreads;             // elements of a thread
constexpr int kReadChunk = kReadThreads / kReadRowThreads;   // slots a CTA takes at once
static_assert(kReadElems == kE2M1Group, "a thread's elements have one e2m1 scale");

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

template <int KVF, int OF>
__global__ void __launch_bounds__(kReadThreads) read_kv_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.z, pg = blockIdx.y;  // pg = plane * 8 + KV head
  const size_t list = (size_t)p.batch * 4;
  const int len_raw = __ldg(in_buffer(p.lens + b, 4, p.lens, list, p.flags));
  const int start_raw = p.starts ? __ldg(in_buffer(p.starts + b, 4, p.starts, list, p.flags)) : 0;
  const int len = min(max(len_raw, 0), p.capacity), start = min(max(start_raw, 0), len);
  if ((len != len_raw || start != start_raw) && p.flags && pg == 0 && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.flags, GQA_FLAG_LENGTH_CLAMPED);
  const int n = min(len - start, p.out_capacity);
  constexpr int kWords = kv_row_bytes(KVF) / (4 * kReadRowThreads);  // 32-bit words of a thread's elements
  const int e = threadIdx.x % kReadRowThreads;
  const float all = pg < kHkv ? p.k_scale : p.v_scale;
  for (int j = blockIdx.x * kReadChunk + threadIdx.x / kReadRowThreads; j < n; j += gridDim.x * kReadChunk) {
    const int t = start + j;
    size_t unit = (size_t)b, rows = (size_t)p.capacity, in = (size_t)t;
    if (p.block_table != nullptr) {
      int id = __ldg(in_buffer(p.block_table + (size_t)b * p.max_pages + (t >> p.page_log2), 4, p.block_table,
                               (size_t)p.batch * p.max_pages * 4, p.flags));
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
    uint32_t w[kWords], o[kReadElems / 2];
    if constexpr (kWords == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    }
    if constexpr (KVF == kKvF16 || KVF == kKvBF16) {
#pragma unroll
      for (int i = 0; i < kReadElems / 2; ++i) {
        if constexpr ((KVF == kKvF16) == (OF == kQF16)) {
          o[i] = w[i];
        } else {
          const float2 f = KVF == kKvF16 ? f16x2_to_f32x2(w[i]) : bf16x2_to_f32x2(w[i]);
          o[i] = round2<OF>(f.x, f.y);
        }
      }
    } else {
      float x[kReadElems], sc = 1.f;
      if constexpr (KVF == kKvE2M1) {
        const uint32_t s = __ldg(static_cast<const uint8_t*>(p.kv_scales) + row * (kD / kE2M1Group) + e);
        sc = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)s)).x;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint32_t d[4];
          e2m1x8_to_f16(w[i], d);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float2 f = f16x2_to_f32x2(d[m]);
            x[8 * i + 2 * m] = f.x;
            x[8 * i + 2 * m + 1] = f.y;
          }
        }
      } else if constexpr (KVF == kKvE4M3) {
#pragma unroll
        for (int i = 0; i < kReadElems / 2; ++i) {
          const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
      } else {
        sc = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.kv_scales) + row) << 16);
#pragma unroll
        for (int i = 0; i < kReadElems; ++i) x[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
      // code * scale is exact; then the tensor scale, rounded once in FP32
#pragma unroll
      for (int i = 0; i < kReadElems / 2; ++i) o[i] = round2<OF>(x[2 * i] * sc * all, x[2 * i + 1] * sc * all);
    }
    uint16_t* out = static_cast<uint16_t*>(p.out);
    const size_t at = (((size_t)b * 2 * kHkv + pg) * p.out_capacity + j) * kD + e * kReadElems;
    uint4* dst = reinterpret_cast<uint4*>(in_buffer(out + at, kReadElems * 2, out,
                                                    (size_t)p.batch * 2 * kHkv * p.out_capacity * kD * 2, p.flags));
#pragma unroll
    for (int i = 0; i < kReadElems / 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
}

}  // namespace gqa
