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
//   e4m3       x * (1 / scale) in FP32, to the nearest, saturating: the append step's
//              codes, next to a tie (2^-23) the other neighbour of x / scale's
//   int8       bf16 scale amax / 127 of the row, code = round(x / scale)
//   e2m1       e4m3 scale amax / (6 * tensor scale) of each 16 dims, code = the
//              e2m1 level nearest to x / (scale * tensor scale)
//
// A token is 12 units of 4 heads (8 of q, 2 of k, 2 of v).  A warp takes 4 units
// at a time (16 q heads, or k and v), or for few tokens one, and issues all their
// loads before anything else.  A quarter of the warp holds one head, a lane dims
// 8i..8i+7 and 64+8i..: every rotary pair stays in a lane, a load or a store is
// 16 bytes and the norm takes three shuffles for four heads.  The 64 angles of a
// token are spread over the lanes, two each (the same two for every token), and
// handed round by shuffles.
//
// Angles without FP64 (slow on sm_103a): the host holds theta^(-i/64) / (2 pi)
// as a 64-bit binary fraction of a turn, so that position * fraction modulo
// 2^64 is the angle in turns with the whole turns gone, for any 32-bit position
// within 2^-33 of a turn.  The top two bits (after adding an eighth of a turn)
// are the quadrant; sin and cos of the rest, |x| <= pi/4, are the Taylor series
// to x^9 and x^10 (first terms left out below 2^-28) at the FP32 next to x, and
// one step along the derivative to x itself: within 1.5 * 2^-24 (a CPU test goes
// through the same operations).
//
// e2m1 keys are rounded as the exact z would be.  The FP32 z is off by at most
// kKeyError of the head's largest magnitude; where that could turn a group's
// scale or a code (the two ends of the interval round apart), the unit goes on the
// warp's list (about one unit of four heads in 45), and the warp forms its
// elements in doubt again, exactly enough, when its tokens are done.  (Called
// where the doubt arises, that code cost every unit its registers: 4096 tokens
// into an fp4 cache and back 55 us, without any of it 39.)  Values are exact
// inputs: their quotients are brought to the tie or off it by the sign of the
// exact remainder.
#pragma once

#include <type_traits>

#include "append_kv.cuh"

namespace gqa {

constexpr int kWriteThreads = 256;
constexpr int kWriteWarps = kWriteThreads / 32;
constexpr int kWriteUnits = 12;  // units of 4 heads in a token: q 0..7, k 8..9, v 10..11
constexpr int kWriteDoubts = 32;  // units a warp's list holds
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
  const int32_t* block_table;           // paged cache, else null
  int max_pages, num_pages, page_log2;
  float eps, k_scale, v_scale, k_inv_scale, v_inv_scale;
  uint64_t turns[kD / 2];    // theta^(-i/64) / (2 pi) modulo 1, in units of 2^-64
  uint8_t axis[kD / 2];      // which row of positions
  // for checked builds: rows of 128 in the cache, bytes of the projections and positions
  size_t kv_rows, q_bytes, k_bytes, v_bytes, pos_bytes;
};

__device__ __forceinline__ int position(const WriteParams& p, int axis, int n) {
  return __ldg(in_buffer(p.positions + (size_t)axis * p.tokens + n, 4, p.positions, p.pos_bytes, p.flags));
}
// 8 elements at `at`, in a projection or a norm weight `base` of `bytes`.
__device__ __forceinline__ uint4 load8(const WriteParams& p, const uint16_t* at, const uint16_t* base, size_t bytes) {
  return __ldg(reinterpret_cast<const uint4*>(in_buffer(at, 16, base, bytes, p.flags)));
}
// ... of q_out
__device__ __forceinline__ void store8(const WriteParams& p, uint16_t* at, const uint4& v) {
  *reinterpret_cast<uint4*>(in_buffer(at, 16, p.q_out, (size_t)p.tokens * kHq * kD * 2, p.flags)) = v;
}

// sin and cos of `turn` * 2 pi / 2^64
__device__ __forceinline__ void sincos_turn(uint64_t turn, float& s, float& c) {
  const uint32_t h = (uint32_t)(turn >> 32);
  const uint32_t quad = (h + 0x20000000u) >> 30;
  const int32_t r = (int32_t)(h - (quad << 30));
  constexpr float kUnit = 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float rf = (float)r;
  const float x = rf * kUnit;
  // what the two roundings of x left out (and 2 pi / 2^32 itself, to a second term)
  const float rest = fmaf((float)(r - (int32_t)rf), kUnit, fmaf(rf, kUnit, -x) + rf * -4.0709404e-17f);
  const float x2 = x * x;
  float sp = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
  sp = fmaf(x2, sp, 8.33333333e-3f);
  sp = fmaf(x2, sp, -1.66666667e-1f);
  float sx = fmaf(x * x2, sp, x);
  float cp = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
  cp = fmaf(x2, cp, -1.38888889e-3f);
  cp = fmaf(x2, cp, 4.16666667e-2f);
  cp = fmaf(x2, cp, -0.5f);
  float cx = fmaf(x2, cp, 1.f);
  const float s0 = sx;
  sx = fmaf(cx, rest, sx);
  cx = fmaf(-s0, rest, cx);
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
  // (past 2^127, where m may be infinite, every format saturates; a NaN stays one)
  return fabsf(q) < 0x1p127f ? m + fminf(fmaxf(d, -t), t) : q;
}

// The same for x and S known as double-float pairs (x to about 2^-44 of itself):
// at a midpoint the sign of the remainder decides.
__device__ __forceinline__ float quotient_to_round(Float2 x, float inv, Float2 S) {
  const float q = x.hi * inv;
  const float m = __uint_as_float((__float_as_uint(q) + 0x40u) & ~0x7fu);
  const Float2 ms = df_mul(Float2{m, 0.f}, S);
  const float d = df_add(x, Float2{-ms.hi, -ms.lo}).hi;
  const float t = fabsf(m) * 0x1p-20f;
  return d > 0.f ? m + t : (d < 0.f ? m - t : m);
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}
// The larger of two, NaN if either is (fmaxf drops a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float amax8_nan(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
  return m;
}

// mean(x^2) + eps of a head whose lane holds xl and xh (the same in its 8 lanes).
__device__ __forceinline__ float mean_square(const float (&xl)[8], const float (&xh)[8], float eps) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    t[i] = fmaf(xl[i], xl[i], xh[i] * xh[i]) + fmaf(xl[i + 4], xl[i + 4], xh[i + 4] * xh[i + 4]);
  float ss = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  return fmaf(ss, 1.f / kD, eps);
}
// FP32 holds the squares of such a head, and a sum of them, well inside its range:
// so it is for fp16 at any size, for bf16 from about 2^-30 (with a smaller eps) to
// 2^30.  (A NaN stays one either way: padding often holds some.)
__device__ __forceinline__ bool squares_fit(float ss) { return !(ss <= 0x1p-60f || ss >= 0x1p60f); }
// A head whose squares do not fit is scaled by the power of two k that brings its
// largest element, or the root of eps, to [1, 2), and eps by k^2: the normalised
// head is the same.  A head of zeros without eps, and one with an infinite element,
// stay as they are.
__device__ __forceinline__ void scale_head(float (&xl)[8], float (&xh)[8], float& eps) {
  float m = fmaxf(amax8(xl), amax8(xh));
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  m = fmaxf(m, sqrtf(eps));
  if (squares_fit(mean_square(xl, xh, eps)) || m == 0.f || !(m < INFINITY)) return;
  const int exponent = (int)(__float_as_uint(m) >> 23);  // 0 for a subnormal m: k = 2^127 will do
  const float k = __uint_as_float((uint32_t)max(254 - exponent, 1) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xl[i] *= k;
    xh[i] *= k;
  }
  eps = eps * k * k;
}

// The bound of |FP32 z - z| as a share of the head's largest |z|, A, in units of
// 2^-24 (a rounding is one of what it rounds, at most; P is the pair's length, at
// most sqrt(2) A; |y_i| + |y_j| <= sqrt(2) P and |y_i cos| + |y_j sin| <= P):
//   cos and sin off by 1.5, whatever their size: 1.5 (|y_i| + |y_j|)     2.2 P
//   their products with a weight: |y_i cos| + |y_j sin|                    1 P
//   the rotation's one rounded product: |y_j sin|                          1 P
//   (4.2 P: 5.9 A) the rotation's sum and the product with r               2 A
//   r: 9 roundings of mean(x^2) + eps (5 in a lane, 3 over the lanes, eps), half of
//   them in the root, and 1.5 of the Newton step                           6 A
// together 13.9; 4 more where a quotient is formed from z (amax +- e, 6 k_scale, its
// reciprocal, the product).  The constant is 22, which also covers an eps past 2^60
// (no Newton step: 4 instead of 1.5).
constexpr float kKeyError = 0x1.6p-20f;

struct KeyCodes {
  uint32_t lo, hi;  // codes of dims 8i..8i+7 and 64+8i..
  uint32_t slo, shi;  // the scale bytes of their groups
};

// Scale byte of a group whose largest FP32 |z| is `amax`, within `e` of the exact
// one; false if the exact one could round to another.  (An infinite amax gives 448,
// a NaN the NaN.)
__device__ __forceinline__ bool key_scale(float amax, float e, float inv6, uint32_t& scale) {
  const uint32_t two = to_e4m3x2((amax + e) * inv6, max_nan(amax - e, 0.f) * inv6);
  scale = two & 0xffu;
  return scale == (two >> 8);
}
// Codes of eight of its z; the nibbles of `unsure` that are not 0 could be others.
__device__ __forceinline__ void key_codes(const float (&z)[8], float e, uint32_t scale, float k_scale, uint32_t& codes,
                                          uint32_t& unsure) {
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
  const uint32_t low = to_e2m1x8(down);
  // a zero of either sign is the same value; every other magnitude counts with its
  // sign (an interval about zero may reach the same code on both sides)
  const uint32_t nonzero = ((codes | low) & 0x77777777u) + 0x77777777u;  // bit 3 of each nibble
  unsure = (codes ^ low) & (nonzero | 0x77777777u);
}

// sin and cos of `turn` * 2 pi / 2^64 as double-float pairs, within about 2^-46.
__device__ __forceinline__ void sincos_turn_exact(uint64_t turn, Float2& s, Float2& c) {
  const uint32_t quad = (uint32_t)((turn + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(turn - ((uint64_t)quad << 62));
  const float hi = (float)(int32_t)(r >> 32);
  const float lo = (float)(r - ((int64_t)(int32_t)hi << 32)) * 0x1p-32f;
  constexpr Float2 kUnit = df_const(1.4629180792671596e-09);  // 2 pi / 2^32
  Float2 sx, cx;
  sincos_reduced(df_mul(fast_two_sum(hi, lo), kUnit), sx, cx);
  s = quad & 1u ? cx : sx;
  c = quad & 1u ? sx : cx;
  if (quad & 2u) s = Float2{-s.hi, -s.lo};
  if ((quad + 1u) & 2u) c = Float2{-c.hi, -c.lo};
}
__device__ __forceinline__ Float2 df_scale(float a, Float2 b) { return df_mul(Float2{a, 0.f}, b); }

// One unit of four key heads whose rounding FP32 could not decide: the elements
// in doubt, and nothing else, are formed again in double-float arithmetic, to
// about 2^-43 of the head's largest.  (FP64 would do, at many times the latency.)
template <int QF, bool ANY>
__device__ __forceinline__ void key_codes_exact(const WriteParams& p, int n, const uint4& wlo, const uint4& whi,
                                             const float (&zl)[8], const float (&zh)[8], float gl, float gh, float e,
                                             KeyCodes& out) {
  const int idx = threadIdx.x & 7;
  float yl[8], yh[8];
  unpack8<QF>(wlo, yl);
  unpack8<QF>(whi, yh);
  Float2 r = {1.f, 0.f};
  if (p.k_norm_w) {
    float eps = p.eps;
    if constexpr (ANY) scale_head(yl, yh, eps);
    Float2 acc[4] = {};  // (squares of 16-bit elements are exact)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[i & 3] = df_add(acc[i & 3], Float2{yl[i] * yl[i], 0.f});
      acc[i & 3] = df_add(acc[i & 3], Float2{yh[i] * yh[i], 0.f});
    }
    Float2 ss = df_add(df_add(acc[0], acc[1]), df_add(acc[2], acc[3]));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
      ss = df_add(ss, Float2{__shfl_xor_sync(0xffffffffu, ss.hi, off), __shfl_xor_sync(0xffffffffu, ss.lo, off)});
    ss = df_add(Float2{ss.hi * (1.f / kD), ss.lo * (1.f / kD)}, Float2{eps, 0.f});
    // 1 / sqrt(ss) = r0 (1 - h)^(-1/2), h = 1 - ss r0^2 about 2^-21: to h^2
    const float r0 = rsqrtf(ss.hi);
    const float rr = r0 * r0;
    const Float2 t = df_mul(ss, Float2{rr, fmaf(r0, r0, -rr)});
    const float h = (1.f - t.hi) - t.lo;
    r = fast_two_sum(r0, r0 * fmaf(0.375f * h, h, 0.5f * h));
    float wl[8], wh[8];
    unpack8<QF>(load8(p, p.k_norm_w + 8 * idx, p.k_norm_w, 2 * kD), wl);
    unpack8<QF>(load8(p, p.k_norm_w + 64 + 8 * idx, p.k_norm_w, 2 * kD), wh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (exact)
      yl[i] *= wl[i];
      yh[i] *= wh[i];
    }
  }
  const auto exact = [&](int i, Float2& lo, Float2& hi) {
    const int a = 8 * idx + i;
    const int64_t pos = position(p, p.axis[a], n);
    Float2 s, c;
    sincos_turn_exact((uint64_t)pos * p.turns[a], s, c);
    const Float2 us = df_scale(yl[i], s), vs = df_scale(yh[i], s);
    lo = df_mul(r, df_add(df_scale(yl[i], c), Float2{-vs.hi, -vs.lo}));
    hi = df_mul(r, df_add(df_scale(yh[i], c), us));
  };
  const auto larger = [](Float2 a, Float2 b) {  // the larger magnitude, as a pair >= 0
    if (b.hi < 0.f) b = Float2{-b.hi, -b.lo};
    return b.hi > a.hi || (b.hi == a.hi && b.lo > a.lo) ? b : a;
  };
  const auto of_pair = [&](Float2 a) {  // the larger of the two lanes that share a group
    return larger(a, Float2{__shfl_xor_sync(0xffffffffu, a.hi, 1), __shfl_xor_sync(0xffffffffu, a.lo, 1)});
  };
  const float ks = p.k_scale, k6 = 6.f * ks, inv6 = 1.f / k6;
  // scales in doubt: from the exact values of the elements that could be the largest
  const bool sure_l = key_scale(gl, e, inv6, out.slo), sure_h = key_scale(gh, e, inv6, out.shi);
  if (!__all_sync(0xffffffffu, sure_l && sure_h)) {
    Float2 al = {0.f, 0.f}, ah = {0.f, 0.f};
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const bool nl = !sure_l && fabsf(zl[i]) >= gl - 2.f * e, nh = !sure_h && fabsf(zh[i]) >= gh - 2.f * e;
      if (!__any_sync(0xffffffffu, nl || nh)) continue;
      Float2 lo, hi;
      exact(i, lo, hi);
      if (nl) al = larger(al, lo);
      if (nh) ah = larger(ah, hi);
    }
    al = of_pair(al);
    ah = of_pair(ah);
    const Float2 S = {k6, fmaf(6.f, ks, -k6)};
    const uint32_t two = to_e4m3x2(quotient_to_round(al, inv6, S), quotient_to_round(ah, inv6, S));
    if (!sure_l) out.slo = two & 0xffu;
    if (!sure_h) out.shi = two >> 8;
  }
  uint32_t ul, uh;
  key_codes(zl, e, out.slo, ks, out.lo, ul);
  key_codes(zh, e, out.shi, ks, out.hi, uh);
  const float vl = e4m3_value(out.slo), vh = e4m3_value(out.shi), sl = vl * ks, sh = vh * ks;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t mask = 0xfu << (4 * i);
    if (!__any_sync(0xffffffffu, ((ul | uh) & mask) != 0u)) continue;
    Float2 lo, hi;
    exact(i, lo, hi);
    float q[8] = {};
    if (sl > 0.f) q[0] = quotient_to_round(lo, 1.f / sl, Float2{sl, fmaf(vl, ks, -sl)});
    if (sh > 0.f) q[1] = quotient_to_round(hi, 1.f / sh, Float2{sh, fmaf(vh, ks, -sh)});
    const uint32_t c = to_e2m1x8(q);
    // (only what is in doubt: an infinite element has no exact pair)
    if (ul & mask) out.lo = (out.lo & ~mask) | ((c & 0xfu) << (4 * i));
    if (uh & mask) out.hi = (out.hi & ~mask) | (((c >> 4) & 0xfu) << (4 * i));
  }
}

// Where the cache rows of a token go: row index of (plane 0, head 0), and how
// far a plane and a head are apart; ok is false where nothing is to be written.
struct RowAt {
  size_t base, head;
  bool ok;
};
__device__ __forceinline__ RowAt locate(const WriteParams& p, int n) {
  const size_t list = (size_t)p.tokens * 4;
  const int b = p.rows ? __ldg(in_buffer(p.rows + n, 4, p.rows, list, p.flags)) : n;
  const int slot = __ldg(in_buffer(p.slots + n, 4, p.slots, list, p.flags));
  RowAt at;
  at.ok = b >= 0 && b < p.batch && slot >= 0 && slot < p.capacity;
  uint32_t flag = at.ok ? 0u : GQA_FLAG_SLOT_CLAMPED;
  size_t unit = at.ok ? (size_t)b : 0, rows = (size_t)p.capacity, in = at.ok ? (size_t)slot : 0;
  if (p.block_table != nullptr && at.ok) {
    const int id = __ldg(in_buffer(p.block_table + (size_t)b * p.max_pages + (slot >> p.page_log2), 4, p.block_table,
                                   (size_t)p.batch * p.max_pages * 4, p.flags));
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
__device__ __forceinline__ void make_coefs(const WriteParams& p, const uint16_t* w, int idx, const float (&cs)[8], const float (&sn)[8],
                                           Coefs& k) {
  float wl[8], wh[8];
  if (w) {
    unpack8<QF>(load8(p, w + 8 * idx, w, 2 * kD), wl);
    unpack8<QF>(load8(p, w + 64 + 8 * idx, w, 2 * kD), wh);
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
// The result says whether the squares fit; ANY (elsewhere too) takes heads whose
// squares do not.
template <int QF, bool ANY = false>
__device__ __forceinline__ bool rotate_unit(const uint4& wlo, const uint4& whi, const Coefs& k, bool norm, float eps,
                                            float (&zl)[8], float (&zh)[8]) {
  float xl[8], xh[8];
  unpack8<QF>(wlo, xl);
  unpack8<QF>(whi, xh);
  float r = 1.f;
  bool fit = true;
  if (norm) {
    if constexpr (ANY) scale_head(xl, xh, eps);
    const float ss = mean_square(xl, xh, eps);
    fit = squares_fit(ss);
    r = rsqrtf(ss);
    if (fit) r = fmaf(0.5f * r, fmaf(-ss * r, r, 1.f), r);  // (a Newton step)
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    zl[i] = r * fmaf(xl[i], k.a[i], -(xh[i] * k.b[i]));
    zh[i] = r * fmaf(xh[i], k.c[i], xl[i] * k.d[i]);
  }
  return fit;
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

// The largest |z| of a lane's two groups (NaN with one in them), and the bound of
// the error of its head's z (not finite where some z is not: see finite_bound).
__device__ __forceinline__ void key_bounds(const float (&zl)[8], const float (&zh)[8], float& gl, float& gh, float& e) {
  gl = amax8_nan(zl);
  gh = amax8_nan(zh);
  gl = max_nan(gl, __shfl_xor_sync(0xffffffffu, gl, 1));
  gh = max_nan(gh, __shfl_xor_sync(0xffffffffu, gh, 1));
  e = max_nan(gl, gh);
  e = max_nan(e, __shfl_xor_sync(0xffffffffu, e, 2));
  e = max_nan(e, __shfl_xor_sync(0xffffffffu, e, 4)) * kKeyError;
}
// The bound of the finite z of a head, from the largest of them: a pair is finite
// only where both its elements are, and its error comes from them alone.
__device__ __forceinline__ float finite_bound(const float (&zl)[8], const float (&zh)[8]) {
  float e = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(zl[i]), b = fabsf(zh[i]);
    e = fmaxf(e, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, off));
  return e * kKeyError;
}

__device__ __forceinline__ void store_e2m1(const WriteParams& p, size_t row, int idx, const KeyCodes& k) {
  uint8_t* dst = static_cast<uint8_t*>(p.kv) + row * kv_row_bytes(kKvE2M1);
  *reinterpret_cast<uint32_t*>(dst + 4 * idx) = k.lo;
  *reinterpret_cast<uint32_t*>(dst + 32 + 4 * idx) = k.hi;
  if ((idx & 1) == 0) {
    uint8_t* sc = static_cast<uint8_t*>(p.kv_scales) + row * scale_row_bytes(kKvE2M1) + (idx >> 1);
    sc[0] = (uint8_t)k.slo;
    sc[4] = (uint8_t)k.shi;
  }
}

// One unit of four cache rows (KV heads 4u .. 4u + 3 of `plane`) to row `row`;
// true if it holds an e2m1 key in doubt.
template <int KVF, int QF>
__device__ __forceinline__ bool store_unit(const WriteParams& p, int plane, size_t row, int idx, bool ok,
                                           const uint4& wlo, const uint4& whi, const float (&xl)[8],
                                           const float (&xh)[8]) {
  bool doubt = false;  // (warp-uniform)
  uint8_t* dst = static_cast<uint8_t*>(p.kv) + row * kv_row_bytes(KVF);
  if constexpr (KVF == kKvE2M1) {
    KeyCodes k;
    if (plane == 0) {
      float gl, gh, e;
      key_bounds(xl, xh, gl, gh, e);
      const float inv6 = 1.f / (6.f * p.k_scale);
      bool sure = key_scale(gl, e, inv6, k.slo);
      sure &= key_scale(gh, e, inv6, k.shi);
      sure &= e < INFINITY;  // (infinite and NaN keys are settled as those in doubt)
      uint32_t ul, uh;
      key_codes(xl, e, k.slo, p.k_scale, k.lo, ul);
      key_codes(xh, e, k.shi, p.k_scale, k.hi, uh);
      doubt = ok && !__all_sync(0xffffffffu, sure && (ul | uh) == 0u);  // (ok is the token's, the warp's)
    } else {
      // values are the inputs themselves: exact
      const float al = amax8_nan(xl), ah = amax8_nan(xh);
      const float gl = max_nan(al, __shfl_xor_sync(0xffffffffu, al, 1));
      const float gh = max_nan(ah, __shfl_xor_sync(0xffffffffu, ah, 1));
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
    if (ok) store_e2m1(p, row, idx, k);
  } else if constexpr (KVF == kKvI8) {
    uint2 lo, hi;
    uint16_t scale;
    int8_row(xl, xh, lo, hi, scale);
    if (!ok) return false;
    *reinterpret_cast<uint2*>(dst + 8 * idx) = lo;
    *reinterpret_cast<uint2*>(dst + 64 + 8 * idx) = hi;
    if (idx == 0) static_cast<uint16_t*>(p.kv_scales)[row] = scale;
  } else if constexpr (KVF == kKvE4M3) {
    if (!ok) return false;
    const float inv = plane == 0 ? p.k_inv_scale : p.v_inv_scale;
    *reinterpret_cast<uint2*>(dst + 8 * idx) = e4m3_8(xl, inv);
    *reinterpret_cast<uint2*>(dst + 64 + 8 * idx) = e4m3_8(xh, inv);
  } else {
    if (!ok) return false;
    *reinterpret_cast<uint4*>(dst + 16 * idx) = plane == 0 ? round8<QF>(xl) : wlo;
    *reinterpret_cast<uint4*>(dst + 128 + 16 * idx) = plane == 0 ? round8<QF>(xh) : whi;
  }
  return doubt;
}

// This lane's eight cosines and sines of token n; turn and axis: its own two
// angles'.
__device__ __forceinline__ void token_angles(const WriteParams& p, int n, const uint64_t (&turn)[2], const int (&axis)[2],
                                             float (&cs)[8], float (&sn)[8]) {
  float c2[2], s2[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int pos = position(p, axis[j], n);
    sincos_turn((uint64_t)(int64_t)pos * turn[j], s2[j], c2[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int from = (j >> 1) * 8 + (threadIdx.x & 7);
    cs[j] = __shfl_sync(0xffffffffu, c2[j & 1], from);
    sn[j] = __shfl_sync(0xffffffffu, s2[j & 1], from);
  }
}

// U: units a warp takes at a time, 4 (parts of a token: q 0..3, q 4..7, k and v)
// or 1.  The grid is the CTAs resident at once (2 an SM).
//
// Bound by HBM for the 16-bit cache (24 KB a token moved): 8192 tokens take 33.3
// us, 0.89 of the copy peak; one warp a token with a load at a time took 50, two
// units at a time 38.6.  An e2m1 cache adds the rounding of keys and values, half
// as much arithmetic again.
template <int KVF, int QF, int U>
__global__ void __launch_bounds__(kWriteThreads, 2) write_kv_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kParts = kWriteUnits / U;
  constexpr bool kList = KVF == kKvE2M1 && U > 1;
  __shared__ int2 lists[kList ? kWriteWarps : 1][kList ? kWriteDoubts : 1];
  [[maybe_unused]] int2* list = lists[kList ? threadIdx.x >> 5 : 0];
  static_assert(kWriteQUnits % U == 0 && (U == 1 || U == kWriteUnits - kWriteQUnits), "whole parts");
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, quarter = lane >> 3, idx = lane & 7;
  // this lane's two angles, by way of shared memory (lanes that read different
  // words of the parameters are served one by one)
  __shared__ uint64_t turns[kD / 2];
  __shared__ uint8_t axes[kD / 2];
  if (threadIdx.x < kD / 2) {
    turns[threadIdx.x] = p.turns[threadIdx.x];
    axes[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  uint64_t turn[2];
  int axis[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    turn[j] = turns[8 * idx + 2 * quarter + j];
    axis[j] = axes[8 * idx + 2 * quarter + j];
  }
  pdl_wait_prior_grid();
  const long long items = (long long)p.tokens * kParts;
  const int step = gridDim.x * kWriteWarps;
  long long it = (long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  [[maybe_unused]] int doubts = 0;  // units on this warp's list
  // Heads whose squares do not fit FP32 are looked for on the way, and a warp that
  // met one writes its units again after its tokens.  (4096 bf16 tokens into an
  // e2m1 cache 24.8 us, 24.1 without any of it; a branch in each unit, which keeps
  // the loads and shuffles of four from overlapping, 25.5.)
  constexpr bool kWide = QF == kQBF16;
  bool fit = true;
  // the same lanes write the bytes of a unit in doubt again
  [[maybe_unused]] const auto settle = [&](auto any, int n, const RowAt& at, int g, const uint4& wlo, const uint4& whi,
                                           const float(&zl)[8], const float(&zh)[8]) {
    float gl, gh, e;
    key_bounds(zl, zh, gl, gh, e);
    if (!__all_sync(0xffffffffu, e < INFINITY)) e = finite_bound(zl, zh);  // (the same where all are finite)
    KeyCodes k;
    key_codes_exact<QF, any.value>(p, n, wlo, whi, zl, zh, gl, gh, e, k);
    if (at.ok) store_e2m1(p, at.base + g * at.head, idx, k);
  };
  do {
    for (; it < items && (!kList || doubts <= kWriteDoubts - kWriteKUnits); it += step) {
      const int n = (int)(it / kParts), u0 = (int)(it - (long long)n * kParts) * U;
      uint4 wlo[U], whi[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + i;
        const bool q = u < kWriteQUnits, k = u < kWriteQUnits + kWriteKUnits;
        const uint16_t* src = q   ? p.q_proj + n * p.q_stride + u * 4 * kD
                              : k ? p.k_proj + n * p.k_stride + (u - kWriteQUnits) * 4 * kD
                                  : p.v_proj + n * p.v_stride + (u - kWriteQUnits - kWriteKUnits) * 4 * kD;
        src += quarter * kD + 8 * idx;
        const uint16_t* base = q ? p.q_proj : (k ? p.k_proj : p.v_proj);
        const size_t bytes = q ? p.q_bytes : (k ? p.k_bytes : p.v_bytes);
        wlo[i] = load8(p, src, base, bytes);
        whi[i] = load8(p, src + 64, base, bytes);
      }
      RowAt at{0, 0, false};
      if (u0 + U > kWriteQUnits) at = locate(p, n);

      // the token's angles (not needed by its values)
      float cs[8], sn[8];
      if (u0 < kWriteQUnits + kWriteKUnits) token_angles(p, n, turn, axis, cs, sn);
      if (u0 < kWriteQUnits) {
        Coefs qc;
        make_coefs<QF>(p, p.q_norm_w, idx, cs, sn, qc);
        uint16_t* dst = p.q_out + ((size_t)n * kHq + 4 * u0 + quarter) * kD + 8 * idx;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float zl[8], zh[8];
          fit &= rotate_unit<QF>(wlo[i], whi[i], qc, p.q_norm_w != nullptr, p.eps, zl, zh);
          store8(p, dst + i * 4 * kD, round8<QF>(zl));
          store8(p, dst + i * 4 * kD + 64, round8<QF>(zh));
        }
        continue;
      }
      if (u0 < kWriteQUnits + kWriteKUnits) {
        Coefs kc;
        make_coefs<QF>(p, p.k_norm_w, idx, cs, sn, kc);
#pragma unroll
        for (int i = 0; i < (U == 1 ? 1 : kWriteKUnits); ++i) {
          const int g = 4 * (u0 + i - kWriteQUnits) + quarter;
          float zl[8], zh[8];
          fit &= rotate_unit<QF>(wlo[i], whi[i], kc, p.k_norm_w != nullptr, p.eps, zl, zh);
          if (store_unit<KVF, QF>(p, 0, at.base + g * at.head, idx, at.ok, wlo[i], whi[i], zl, zh)) {
            if constexpr (U == 1) {  // (a call of few tokens is as long as its longest unit)
              settle(std::false_type(), n, at, g, wlo[i], whi[i], zl, zh);
            } else {
              if (lane == 0) list[doubts] = make_int2(n, u0 + i - kWriteQUnits);
              ++doubts;
            }
          }
        }
      }
      if (u0 + U > kWriteQUnits + kWriteKUnits) {
#pragma unroll
        for (int i = U == 1 ? 0 : kWriteKUnits; i < U; ++i) {
          const int g = 4 * (u0 + i - kWriteQUnits - kWriteKUnits) + quarter;
          float xl[8], xh[8];
          unpack8<QF>(wlo[i], xl);
          unpack8<QF>(whi[i], xh);
          store_unit<KVF, QF>(p, 1, at.base + (kHkv + g) * at.head, idx, at.ok, wlo[i], whi[i], xl, xh);
        }
      }
    }
    if constexpr (kList) {
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < doubts; ++i) {
        const int n = list[i].x, g = 4 * list[i].y + quarter;
        const RowAt at = locate(p, n);
        const uint16_t* src = p.k_proj + n * p.k_stride + g * kD + 8 * idx;
        const uint4 wlo = load8(p, src, p.k_proj, p.k_bytes), whi = load8(p, src + 64, p.k_proj, p.k_bytes);
        float cs[8], sn[8], zl[8], zh[8];
        token_angles(p, n, turn, axis, cs, sn);
        Coefs kc;
        make_coefs<QF>(p, p.k_norm_w, idx, cs, sn, kc);
        rotate_unit<QF>(wlo, whi, kc, p.k_norm_w != nullptr, p.eps, zl, zh);
        settle(std::false_type(), n, at, g, wlo, whi, zl, zh);
      }
      doubts = 0;
      __syncwarp();
    }
  } while (it < items);
  if constexpr (kWide) {
    if (__all_sync(0xffffffffu, fit)) return;
#pragma unroll 1
    for (it = (long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5); it < items; it += step) {
#pragma unroll 1
      for (int i = 0; i < U; ++i) {
        const int n = (int)(it / kParts), u = (int)(it - (long long)n * kParts) * U + i;
        if (u >= kWriteQUnits + kWriteKUnits) break;  // (values have no norm)
        const bool q = u < kWriteQUnits;
        const int g = 4 * (q ? u : u - kWriteQUnits) + quarter;
        const uint16_t *base = q ? p.q_proj : p.k_proj, *w = q ? p.q_norm_w : p.k_norm_w;
        const size_t bytes = q ? p.q_bytes : p.k_bytes;
        const uint16_t* src = base + n * (q ? p.q_stride : p.k_stride) + g * kD + 8 * idx;
        const uint4 wlo = load8(p, src, base, bytes), whi = load8(p, src + 64, base, bytes);
        float cs[8], sn[8], zl[8], zh[8];
        token_angles(p, n, turn, axis, cs, sn);
        Coefs kc;
        make_coefs<QF>(p, w, idx, cs, sn, kc);
        rotate_unit<QF, true>(wlo, whi, kc, true, p.eps, zl, zh);
        if (q) {
          uint16_t* dst = p.q_out + ((size_t)n * kHq + g) * kD + 8 * idx;
          store8(p, dst, round8<QF>(zl));
          store8(p, dst + 64, round8<QF>(zh));
        } else {
          const RowAt at = locate(p, n);
          if (store_unit<KVF, QF>(p, 0, at.base + g * at.head, idx, at.ok, wlo, whi, zl, zh))
            settle(std::true_type(), n, at, g, wlo, whi, zl, zh);
        }
      }
    }
  }
}

}  // namespace gqa
