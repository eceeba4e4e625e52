// Writing many tokens at once: normalise and rotate their query and key heads
// (rotary positions of one axis, or of time, height and width) and write keys
// and values into the cache in its format, contiguous or paged.
//
// For token n, every head vector x of 128 of q and k:
//   y_d = x_d / sqrt(mean(x^2) + eps) * w_d      (no weights: y = x)
//   z_i = y_i cos a_i - y_{i+64} sin a_i,  z_{i+64} = y_{i+64} cos a_i + y_i sin a_i,
//   a_i = positions[axis(i)][n] * theta^(-i/64)
// q -> q_out (one rounding); k and v -> row rows[n], slot slots[n] of the cache:
//   fp16/bf16  one rounding
//   e4m3       x / scale, to the nearest, saturating
//   int8       bf16 scale amax / 127 of the row, code = round(x / scale)
//   e2m1       e4m3 scale amax / (6 * tensor scale) of each 16 dims, code = the
//              e2m1 level nearest to x / (scale * tensor scale)
//
// A warp takes a whole token (or, for few tokens, one of its 12 units of 4
// heads: 8 of q, 2 of k, 2 of v).  A quarter of the warp holds one head, a lane
// dims 8i..8i+7 and 64+8i..: every rotary pair stays in a lane, a load or a
// store is 16 bytes and the norm takes three shuffles for four heads.  The 64
// angles of a token are spread over the lanes, two each, and handed round by
// shuffles.
//
// Angles without FP64 (slow on sm_103a): the host holds theta^(-i/64) / (2 pi)
// as a 64-bit binary fraction of a turn, so that position * fraction modulo
// 2^64 is the angle in turns with the whole turns gone, for any 32-bit position
// within 2^-33 of a turn.  The top two bits (after adding an eighth of a turn)
// are the quadrant; sin and cos of the rest, |x| <= pi/4, are the Taylor series
// to x^9 and x^10 (first terms left out below 2^-28), within about 2^-23.
//
// e2m1 keys are rounded as the exact z would be.  The FP32 z is off by at most
// kKeyError of the head's largest magnitude; where that could turn a group's
// scale or a code (the two ends of the interval round apart), the warp computes
// those heads again in FP64 (about one unit in a hundred).  Values are exact
// inputs: their quotients are brought to the tie or off it by the sign of the
// exact remainder.
#pragma once

#include "append_kv.cuh"

namespace gqa {

constexpr int kWriteThreads = 256;
constexpr int kWriteWarps = kWriteThreads / 32;
constexpr int kWriteUnits = 12;  // units of 4 heads in a token: q 0..7, k 8..9, v 10..11
constexpr int kWriteQUnits = kHq / 4, kWriteKUnits = kHkv / 4;

struct WriteParams {
  const uint16_t *q_proj, *k_proj, *v_proj;  // [tokens, heads, 128], rows `stride` elements apart
  long long q_stride, k_stride, v_stride;
  const uint16_t *q_norm_w, *k_norm_w;  // [128], or both null
  const int32_t* positions;             // [tokens], or [3, tokens] by axis
  const int32_t* rows;                  // [tokens] batch rows (null: token n is row n)
  const int32_t* slots;                 // [tokens]
  uint16_t* q_out;                      // [tokens, 32, 128]
  void* kv;
  void* kv_scales;                      // int8: bf16 a row; e2m1: 8 e4m3 a row
  uint32_t* flags;                      // optional status word
  int tokens, batch, capacity;
  int parts;                            // warps per token: 1, or kWriteUnits
  const int32_t* block_table;           // paged cache, else null
  int max_pages, num_pages, page_log2;
  float eps, k_scale, v_scale, k_inv_scale, v_inv_scale;
  uint64_t turns[kD / 2];    // theta^(-i/64) / (2 pi) modulo 1, in units of 2^-64
  uint8_t axis[kD / 2];      // which row of positions
  size_t kv_rows;            // rows of 128 in the cache, for checked builds
};

// sin and cos of `turn` * 2 pi / 2^64
__device__ __forceinline__ void sincos_turn(uint64_t turn, float& s, float& c) {
  const uint32_t h = (uint32_t)(turn >> 32);
  const uint32_t quad = (h + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(h - (quad << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float sp = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
  sp = fmaf(x2, sp, 8.33333333e-3f);
  sp = fmaf(x2, sp, -1.66666667e-1f);
  const float sx = fmaf(x * x2, sp, x);
  float cp = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
  cp = fmaf(x2, cp, -1.38888889e-3f);
  cp = fmaf(x2, cp, 4.16666667e-2f);
  cp = fmaf(x2, cp, -0.5f);
  const float cx = fmaf(x2, cp, 1.f);
  s = quad & 1u ? cx : sx;
  c = quad & 1u ? sx : cx;
  if (quad & 2u) s = -s;
  if ((quad + 1u) & 2u) c = -c;
}

template <int QF>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = QF == kQF16 ? f16x2_to_f32x2(u[i]) : bf16x2_to_f32x2(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <int QF>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  if constexpr (QF == kQF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int QF>
__device__ __forceinline__ uint4 round8(const float (&z)[8]) {
  return make_uint4(round2<QF>(z[0], z[1]), round2<QF>(z[2], z[3]), round2<QF>(z[4], z[5]), round2<QF>(z[6], z[7]));
}

// Two FP32 values to e4m3 bytes (lo in the low byte), to the nearest, saturating.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Eight FP32 values to e2m1 nibbles (x[0] lowest), to the nearest, ties to the
// even code, saturating at 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(byte & 0xffu));
  return f16x2_to_f32x2(h2).x;
}

// x / S for S = sh + sl > 0 (inv near 1 / S), as an FP32 number that rounds to
// any format of at most 5 significant bits as the exact quotient does: if the
// quotient is within 2^-17 of such a format's midpoint m it becomes m itself
// (the exact remainder x - m S is 0) or m (1 +- 2^-20), else a number within
// 2^-16 of it.  x has at most 11 significant bits and m at most 6, so x - m sh
// is exact and the remainder's sign is.
__device__ __forceinline__ float quotient_to_round(float x, float inv, float sh, float sl) {
  const float q = x * inv;
  const float m = __uint_as_float((__float_as_uint(q) + 0x40u) & ~0x7fu);
  const float d = fmaf(-m, sl, fmaf(-m, sh, x)) * (inv * 4096.f);
  const float t = fabsf(m) * 0x1p-20f;
  return m + fminf(fmaxf(d, -t), t);
}

// A double as the FP32 number that rounds to any narrower format as the double
// does: cut off, with the last bit set where something was lost (rounding to
// odd; a narrow format's ties end in zeros).
__device__ __forceinline__ float double_to_round(double t) {
  const float f = __double2float_rz(t);
  return (double)f != t ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// The bound of |FP32 z - z| as a share of the head's largest |z|: sums of 16
// squares in a lane and 8 lanes (19 roundings of the sum, half of that in its
// root), rsqrt, a coefficient w * cos with cos within 2^-23, and the products:
// below 2^-20.2 of |y_i| + |y_{i+64}|, itself at most twice the largest |z|.
constexpr float kKeyError = 0x1p-19f;

struct KeyCodes {
  uint32_t lo, hi;  // codes of dims 8i..8i+7 and 64+8i..
  uint32_t slo, shi;  // the scale bytes of their groups
};

// One unit of four key heads in FP64: this lane's 16 dims of its quarter's head.
template <int QF>
__device__ __noinline__ void key_codes_f64(const WriteParams& p, int n, const uint4& wlo, const uint4& whi,
                                           KeyCodes& out) {
  const int idx = threadIdx.x & 7;
  float xl[8], xh[8], wl[8], wh[8];
  unpack8<QF>(wlo, xl);
  unpack8<QF>(whi, xh);
  double r = 1.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) wl[i] = wh[i] = 1.f;
  if (p.k_norm_w) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)xl[i], (double)xl[i], fma((double)xh[i], (double)xh[i], ss));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r = 1.0 / sqrt(ss / kD + (double)p.eps);
    unpack8<QF>(*reinterpret_cast<const uint4*>(p.k_norm_w + 8 * idx), wl);
    unpack8<QF>(*reinterpret_cast<const uint4*>(p.k_norm_w + 64 + 8 * idx), wh);
  }
  double zl[8], zh[8], al = 0.0, ah = 0.0;
  for (int i = 0; i < 8; ++i) {
    const int a = 8 * idx + i;
    const int64_t pos = __ldg(p.positions + (size_t)p.axis[a] * p.tokens + n);
    Float2 sv, cv;  // the angle's part of a turn, in [-pi, pi)
    sincos_series((double)(int64_t)((uint64_t)pos * p.turns[a]) * 3.4061215800865545e-19, sv, cv);  // 2 pi / 2^64
    const double s = (double)sv.hi + (double)sv.lo, c = (double)cv.hi + (double)cv.lo;
    const double yl = (double)xl[i] * (double)wl[i] * r, yh = (double)xh[i] * (double)wh[i] * r;
    zl[i] = yl * c - yh * s;
    zh[i] = yh * c + yl * s;
    al = fmax(al, fabs(zl[i]));
    ah = fmax(ah, fabs(zh[i]));
  }
  al = fmax(al, __shfl_xor_sync(0xffffffffu, al, 1));
  ah = fmax(ah, __shfl_xor_sync(0xffffffffu, ah, 1));
  const double ks = (double)p.k_scale;
  out.slo = to_e4m3x2(double_to_round(al / (6.0 * ks)), 0.f) & 0xffu;
  out.shi = to_e4m3x2(double_to_round(ah / (6.0 * ks)), 0.f) & 0xffu;
  const double sl = (double)e4m3_value(out.slo) * ks, sh = (double)e4m3_value(out.shi) * ks;
  float ql[8], qh[8];
  for (int i = 0; i < 8; ++i) {
    ql[i] = sl > 0.0 ? double_to_round(zl[i] / sl) : 0.f;
    qh[i] = sh > 0.0 ? double_to_round(zh[i] / sh) : 0.f;
  }
  out.lo = to_e2m1x8(ql);
  out.hi = to_e2m1x8(qh);
}

// Scale byte and codes of one group half from FP32 z within `e` of the exact
// ones (amax: the group's); false if the exact ones could differ.
__device__ __forceinline__ bool key_group(const float (&z)[8], float amax, float e, float k_scale, float inv6,
                                          uint32_t& codes, uint32_t& scale) {
  // (e covers the roundings of inv6, inv and the products too: 2^-22 of amax)
  const uint32_t two = to_e4m3x2((amax + e) * inv6, fmaxf(amax - e, 0.f) * inv6);
  scale = two & 0xffu;
  const float s = e4m3_value(scale) * k_scale;
  const float inv = s > 0.f ? 1.f / s : 0.f;
  const float ei = e * inv;
  float up[8], down[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    up[i] = fmaf(z[i], inv, ei);
    down[i] = fmaf(z[i], inv, -ei);
  }
  codes = to_e2m1x8(up);
  // (a zero of either sign is the same value)
  return scale == (two >> 8) && ((codes ^ to_e2m1x8(down)) & 0x77777777u) == 0u;
}

// Where the cache rows of a token go: row index of (plane 0, head 0), and how
// far a plane and a head are apart; ok is false where nothing is to be written.
struct RowAt {
  size_t base, head;
  bool ok;
};
__device__ __forceinline__ RowAt locate(const WriteParams& p, int n) {
  const int b = p.rows ? __ldg(p.rows + n) : n;
  const int slot = __ldg(p.slots + n);
  RowAt at;
  at.ok = b >= 0 && b < p.batch && slot >= 0 && slot < p.capacity;
  uint32_t flag = at.ok ? 0u : GQA_FLAG_SLOT_CLAMPED;
  size_t unit = at.ok ? (size_t)b : 0, rows = (size_t)p.capacity, in = at.ok ? (size_t)slot : 0;
  if (p.block_table != nullptr && at.ok) {
    const int id = __ldg(p.block_table + (size_t)b * p.max_pages + (slot >> p.page_log2));
    if (id < 0 || id >= p.num_pages) {  // never write through an out-of-range entry
      at.ok = false;
      flag = GQA_FLAG_PAGE_CLAMPED;
    }
    unit = (size_t)max(id, 0);
    in = (size_t)(slot & ((1 << p.page_log2) - 1));
  }
  if (p.block_table != nullptr) rows = (size_t)1 << p.page_log2;
  at.base = unit * 2 * kHkv * rows + in;
  at.head = rows;
  if constexpr (kChecked) {
    if (at.ok && at.base + (2 * kHkv - 1) * rows >= p.kv_rows) {
      at.ok = false;
      flag = GQA_FLAG_BOUNDS;
    }
  }
  if (flag && p.flags && (threadIdx.x & 31) == 0) atomicOr(p.flags, flag);
  return at;
}

// Coefficients of the rotation with the norm weights folded in:
// z_lo = r (x_lo * a - x_hi * b), z_hi = r (x_hi * c + x_lo * d).
struct Coefs {
  float a[8], b[8], c[8], d[8];
};
template <int QF>
__device__ __forceinline__ void make_coefs(const uint16_t* w, int idx, const float (&cs)[8], const float (&sn)[8],
                                           Coefs& k) {
  float wl[8], wh[8];
  if (w) {
    unpack8<QF>(__ldg(reinterpret_cast<const uint4*>(w + 8 * idx)), wl);
    unpack8<QF>(__ldg(reinterpret_cast<const uint4*>(w + 64 + 8 * idx)), wh);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) wl[i] = wh[i] = 1.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    k.a[i] = wl[i] * cs[i];
    k.b[i] = wh[i] * sn[i];
    k.c[i] = wh[i] * cs[i];
    k.d[i] = wl[i] * sn[i];
  }
}
template <int QF>
__device__ __forceinline__ void rotate_unit(const uint4& wlo, const uint4& whi, const Coefs& k, bool norm, float eps,
                                            float (&zl)[8], float (&zh)[8]) {
  float xl[8], xh[8];
  unpack8<QF>(wlo, xl);
  unpack8<QF>(whi, xh);
  float r = 1.f;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(xl[i], xl[i], fmaf(xh[i], xh[i], ss));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r = rsqrtf(fmaf(ss, 1.f / kD, eps));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    zl[i] = r * fmaf(xl[i], k.a[i], -(xh[i] * k.b[i]));
    zh[i] = r * fmaf(xh[i], k.c[i], xl[i] * k.d[i]);
  }
}

// int8: the row's bf16 scale and codes (as an append step writes them).
__device__ __forceinline__ void int8_row(const float (&xl)[8], const float (&xh)[8], uint2& lo, uint2& hi,
                                         uint16_t& scale) {
  float amax = fmaxf(amax8(xl), amax8(xh));
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  scale = __bfloat16_as_ushort(__float2bfloat16_rn(amax / 127.f));
  if (scale == 0) scale = 0x3f80;  // an all-zero row keeps scale 1
  const float s = __uint_as_float((uint32_t)scale << 16);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i >> 2] |= (uint32_t)(uint8_t)(int8_t)max(-127, min(127, __float2int_rn(xl[i] / s))) << (8 * (i & 3));
    w[2 + (i >> 2)] |= (uint32_t)(uint8_t)(int8_t)max(-127, min(127, __float2int_rn(xh[i] / s))) << (8 * (i & 3));
  }
  lo = make_uint2(w[0], w[1]);
  hi = make_uint2(w[2], w[3]);
}

__device__ __forceinline__ uint2 e4m3_8(const float (&x)[8], float inv) {
  return make_uint2(to_e4m3x2(x[0] * inv, x[1] * inv) | (to_e4m3x2(x[2] * inv, x[3] * inv) << 16),
                    to_e4m3x2(x[4] * inv, x[5] * inv) | (to_e4m3x2(x[6] * inv, x[7] * inv) << 16));
}

// One unit of four cache rows (KV heads 4u .. 4u + 3 of `plane`) to row `row`.
template <int KVF, int QF>
__device__ __forceinline__ void store_unit(const WriteParams& p, int n, int plane, size_t row, int idx, bool ok,
                                           const uint4& wlo, const uint4& whi, const float (&xl)[8],
                                           const float (&xh)[8]) {
  uint8_t* dst = static_cast<uint8_t*>(p.kv) + row * kv_row_bytes(KVF);
  if constexpr (KVF == kKvE2M1) {
    KeyCodes k;
    if (plane == 0) {
      const float al = amax8(xl), ah = amax8(xh);
      const float gl = fmaxf(al, __shfl_xor_sync(0xffffffffu, al, 1));
      const float gh = fmaxf(ah, __shfl_xor_sync(0xffffffffu, ah, 1));
      float e = fmaxf(gl, gh);
      e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 2));
      e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 4)) * (1.25f * kKeyError);
      const float inv6 = 1.f / (6.f * p.k_scale);
      bool sure = key_group(xl, gl, e, p.k_scale, inv6, k.lo, k.slo);
      sure &= key_group(xh, gh, e, p.k_scale, inv6, k.hi, k.shi);
      if (!__all_sync(0xffffffffu, sure)) key_codes_f64<QF>(p, n, wlo, whi, k);
    } else {
      // values are the inputs themselves: exact
      const float al = amax8(xl), ah = amax8(xh);
      const float gl = fmaxf(al, __shfl_xor_sync(0xffffffffu, al, 1));
      const float gh = fmaxf(ah, __shfl_xor_sync(0xffffffffu, ah, 1));
      const float vs = p.v_scale, d6 = 6.f * vs, d6l = fmaf(6.f, vs, -d6), inv6 = 1.f / d6;
      const uint32_t two = to_e4m3x2(quotient_to_round(gl, inv6, d6, d6l), quotient_to_round(gh, inv6, d6, d6l));
      k.slo = two & 0xffu;
      k.shi = two >> 8;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float s = e4m3_value(half ? k.shi : k.slo), sh = s * vs, sl = fmaf(s, vs, -sh);
        const float inv = sh > 0.f ? 1.f / sh : 0.f;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient_to_round(half ? xh[i] : xl[i], inv, sh, sl);
        (half ? k.hi : k.lo) = to_e2m1x8(q);
      }
    }
    if (!ok) return;
    *reinterpret_cast<uint32_t*>(dst + 4 * idx) = k.lo;
    *reinterpret_cast<uint32_t*>(dst + 32 + 4 * idx) = k.hi;
    if ((idx & 1) == 0) {
      uint8_t* sc = static_cast<uint8_t*>(p.kv_scales) + row * scale_row_bytes(KVF) + (idx >> 1);
      sc[0] = (uint8_t)k.slo;
      sc[4] = (uint8_t)k.shi;
    }
  } else if constexpr (KVF == kKvI8) {
    uint2 lo, hi;
    uint16_t scale;
    int8_row(xl, xh, lo, hi, scale);
    if (!ok) return;
    *reinterpret_cast<uint2*>(dst + 8 * idx) = lo;
    *reinterpret_cast<uint2*>(dst + 64 + 8 * idx) = hi;
    if (idx == 0) static_cast<uint16_t*>(p.kv_scales)[row] = scale;
  } else if constexpr (KVF == kKvE4M3) {
    if (!ok) return;
    const float inv = plane == 0 ? p.k_inv_scale : p.v_inv_scale;
    *reinterpret_cast<uint2*>(dst + 8 * idx) = e4m3_8(xl, inv);
    *reinterpret_cast<uint2*>(dst + 64 + 8 * idx) = e4m3_8(xh, inv);
  } else {
    if (!ok) return;
    *reinterpret_cast<uint4*>(dst + 16 * idx) = plane == 0 ? round8<QF>(xl) : wlo;
    *reinterpret_cast<uint4*>(dst + 128 + 16 * idx) = plane == 0 ? round8<QF>(xh) : whi;
  }
}

template <int KVF, int QF>
__global__ void __launch_bounds__(kWriteThreads, 2) write_kv_kernel(const __grid_constant__ WriteParams p) {
  __shared__ uint64_t turns[kD / 2];
  __shared__ uint8_t axis[kD / 2];
  pdl_launch_dependents();
  if (threadIdx.x < kD / 2) {
    turns[threadIdx.x] = p.turns[threadIdx.x];
    axis[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, quarter = lane >> 3, idx = lane & 7;
  const long long items = (long long)p.tokens * p.parts;
  const int step = gridDim.x * kWriteWarps;
  for (long long it = (long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int n = p.parts == 1 ? (int)it : (int)(it / kWriteUnits);
    const int u0 = p.parts == 1 ? 0 : (int)(it - (long long)n * kWriteUnits);
    const int u1 = p.parts == 1 ? kWriteUnits : u0 + 1;
    const bool does_kv = u1 > kWriteQUnits;
    RowAt at{0, 0, false};
    if (does_kv) at = locate(p, n);

    // the token's angles (not needed by its values)
    float cs[8], sn[8];
    if (u0 < kWriteQUnits + kWriteKUnits) {
      float c2[2], s2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int a = 8 * idx + 2 * quarter + j;
        const int pos = __ldg(p.positions + (size_t)axis[a] * p.tokens + n);
        sincos_turn((uint64_t)(int64_t)pos * turns[a], s2[j], c2[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cs[j] = __shfl_sync(0xffffffffu, c2[j & 1], (j >> 1) * 8 + idx);
        sn[j] = __shfl_sync(0xffffffffu, s2[j & 1], (j >> 1) * 8 + idx);
      }
    }

    // keys
    const int k0 = max(u0, kWriteQUnits), k1 = min(u1, kWriteQUnits + kWriteKUnits);
    if (k0 < k1) {
      Coefs kc;
      make_coefs<QF>(p.k_norm_w, idx, cs, sn, kc);
      for (int u = k0; u < k1; ++u) {
        const int g = 4 * (u - kWriteQUnits) + quarter;
        const uint4* src = reinterpret_cast<const uint4*>(p.k_proj + n * p.k_stride + g * kD + 8 * idx);
        const uint4 wlo = __ldg(src), whi = __ldg(src + 8);
        float zl[8], zh[8];
        rotate_unit<QF>(wlo, whi, kc, p.k_norm_w != nullptr, p.eps, zl, zh);
        store_unit<KVF, QF>(p, n, 0, at.base + g * at.head, idx, at.ok, wlo, whi, zl, zh);
      }
    }
    // values
    const int v0 = max(u0, kWriteQUnits + kWriteKUnits);
    for (int u = v0; u < u1; ++u) {
      const int g = 4 * (u - kWriteQUnits - kWriteKUnits) + quarter;
      const uint4* src = reinterpret_cast<const uint4*>(p.v_proj + n * p.v_stride + g * kD + 8 * idx);
      const uint4 wlo = __ldg(src), whi = __ldg(src + 8);
      float xl[8], xh[8];
      unpack8<QF>(wlo, xl);
      unpack8<QF>(whi, xh);
      store_unit<KVF, QF>(p, n, 1, at.base + (kHkv + g) * at.head, idx, at.ok, wlo, whi, xl, xh);
    }
    // queries
    if (u0 < kWriteQUnits) {
      Coefs qc;
      make_coefs<QF>(p.q_norm_w, idx, cs, sn, qc);
      const uint16_t* src = p.q_proj + n * p.q_stride + quarter * kD + 8 * idx;
      uint16_t* dst = p.q_out + (size_t)n * kHq * kD + quarter * kD + 8 * idx;
      for (int u = u0; u < min(u1, kWriteQUnits); ++u) {
        const uint4* s4 = reinterpret_cast<const uint4*>(src + u * 4 * kD);
        const uint4 wlo = __ldg(s4), whi = __ldg(s4 + 8);
        float zl[8], zh[8];
        rotate_unit<QF>(wlo, whi, qc, p.q_norm_w != nullptr, p.eps, zl, zh);
        uint4* d4 = reinterpret_cast<uint4*>(dst + u * 4 * kD);
        d4[0] = round8<QF>(zl);
        d4[8] = round8<QF>(zh);
      }
    }
  }
}

}  // namespace gqa
