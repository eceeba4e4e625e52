// The rows of a cache, contiguous or paged, as the kernels that take a prompt's
// chunk, sum softmax weights or move rows address them, and a narrow row's elements
// widened to fp16.
#pragma once

#include "common.cuh"

namespace gqa {

struct CacheView {
  const void* kv;
  const void* scales;          // int8: bf16, e2m1: e4m3 bytes, else null
  const int32_t* block_table;  // null: contiguous
  uint32_t* flags;             // status word, or null
  int batch, capacity;         // slots a row holds (paged: max_pages * page size)
  int max_pages, num_pages, page_log2;
  size_t rows;  // rows of 128 in the cache (checked builds compare with it)
};

// Row (of 128 elements) of slot t < capacity of batch row b, plane and KV head pg =
// plane * 8 + head.  A page id outside the pool is clamped and flagged, and *known
// (where rows are written, which are then left out) set to false.
__device__ __forceinline__ size_t cache_row(const CacheView& c, int b, int pg, int t, bool* known = nullptr) {
  size_t unit = (size_t)b, rows = (size_t)c.capacity, in = (size_t)t;
  if (c.block_table != nullptr) {
    int id = __ldg(in_buffer(c.block_table + (size_t)b * c.max_pages + (t >> c.page_log2), 4, c.block_table,
                             (size_t)c.batch * c.max_pages * 4, c.flags));
    if (id < 0 || id >= c.num_pages) {
      if (c.flags) atomicOr(c.flags, GQA_FLAG_PAGE_CLAMPED);
      if (known) *known = false;
      id = min(max(id, 0), c.num_pages - 1);
    }
    unit = (size_t)id;
    rows = (size_t)1 << c.page_log2;
    in = (size_t)(t & ((1 << c.page_log2) - 1));
  }
  size_t row = (unit * 2 * kHkv + pg) * rows + in;
  if constexpr (kChecked) {
    if (row >= c.rows) {
      if (c.flags) atomicOr(c.flags, GQA_FLAG_BOUNDS);
      if (known) *known = false;
      row = 0;
    }
  }
  return row;
}

// A length as the contract has it, flagged once where it is not.
__device__ __forceinline__ int clamp_length(int raw, int capacity, uint32_t* flags, bool report) {
  const int len = min(max(raw, 0), capacity);
  if (report && len != raw && flags) atomicOr(flags, GQA_FLAG_LENGTH_CLAMPED);
  return len;
}

// Sixteen consecutive elements of a narrow row as pairs of fp16, exactly: e4m3 values and
// int8 codes (16 bytes), or e2m1 codes times their e4m3 scale (8 bytes; 2 + 4 significand
// bits and exponents -10..11).
template <int KVF>
__device__ __forceinline__ void widen16(const uint32_t* w, uint32_t scale, uint32_t (&d)[8]) {
  if constexpr (KVF == kKvE4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
  } else if constexpr (KVF == kKvI8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) i8x4_to_f16x2x2(w[i], d[2 * i], d[2 * i + 1]);
  } else {
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(scale | scale << 8));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x[4];
      e2m1x8_to_f16(w[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x[j]), *reinterpret_cast<const __half2*>(&s2));
        d[4 * i + j] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
  }
}

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

}  // namespace gqa
