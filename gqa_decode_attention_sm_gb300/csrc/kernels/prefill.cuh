// Attention of chunks of new tokens over a cache, on the tcgen05 tensor cores.
//
// A unit is 64 tokens of a row with the 4 query heads of one KV head: two tiles of 128
// rows (row = token * 4 + head) that share every K and V tile.  For each 128 slots
//   S = Q K^T      tcgen05.mma 128x128x128, both operands in shared memory, S in TMEM
//   P = 2^(S - m)  a warpgroup a tile, a thread a row: no exchange between threads for
//                  the maximum and the sum; P goes back over S in TMEM, in 16 bits
//   O += P V       tcgen05.mma, P from TMEM, V as it lies in the cache (MN-major)
// One thread issues the products in the order S0 S1 | O0 S0' O1 S1' | ...: while one
// tile's softmax runs the tensor cores work on the other.  The products of one thread
// run in order, so "S0' is there" says that O0 is complete, and a row's O may be
// rescaled then without another barrier.  It is rescaled only when its maximum grows
// by more than 8 (weights of an fp16 P up to 2^15: with a maximum at 2^7, small ones stay
// normal numbers down to 2^-21 of the largest; of a bf16 P up to 1).
//
// K and V tiles go through a ring of five 32 KB slots in the 128-byte swizzled layout.
// 16-bit caches come by TMA (a box of 128 rows, or of a page's), and two warps look at
// the V tiles that hold slots which some query of the unit does not see: a zero weight
// times an infinity or NaN there would be NaN, so rows past the length become zeros and
// other values that are not finite zeros too, to be put into the rows that do see
// them in the epilogue (rarely: then straight from the cache).  Narrow caches come by
// TMA as they are and those two warps widen them to fp16 (exact); a bf16 q is then scaled by a power of two a
// row into fp16's range, so these calls have fp16 products whatever q's type is.
// int8 scales multiply the columns of S and of P.
//
// Measured (GB300, calls back to back; ranges are GPUs and the clock that the power limit
// leaves): 8192 bf16 tokens 350 to 385 us, 1430 to 1573 TFLOP/s, 0.73 to 0.81 of the
// library GEMM's burst rate; 512 tokens over 131072 slots in pages 740 to 866 us.  A tile
// pair takes 4 products of 512 tensor clocks; the rest is the chain S -> maximum -> 2^x ->
// P of a row (1380 clocks), the issuing warp's steps and the latency between the two, of
// which the other tile covers a part.  152 CTAs ask for 64 KB each tile: of one long row's K and V most comes
// from L2; 16 rows' units lie too far apart for it (1.65 GB from HBM in 390 us, 4.2
// TB/s), which costs no more than 5 %: the same chunks over one row's pages take 374 and
// 376 us or, of longer rows, 596 and 626.  Narrow caches are bound by the two widening
// warps: of 2260 clocks a K or V tile of e2m1 they widen for 1690 and wait for 390, of
// e4m3's 2090 for 1560 and 380 (raw codes read one step ahead: 729 us before and after; a
// third warp: 1108 us, its registers are the softmax's).  int8's softmax threads have two
// scale products more a column, and its raw tiles (two, each told only when the next
// one's copies are issued) keep the widening warps waiting for 1050 of 3440 clocks.
//
// All rows' tiles form one stream that the resident CTAs (one an SM) cut into equal
// runs, whatever the lengths are; a unit cut by a run's end leaves FP32 partials (two a
// CTA at most) that a second kernel merges.
#pragma once

#include <cuda.h>

#include "cache_rows.cuh"

namespace gqa {

constexpr int kPfThreads = 384;      // two softmax warpgroups, one of issue and load warps
constexpr int kPfTokens = 64;        // tokens of a unit
constexpr int kPfRows = 128;         // rows of a tile
constexpr int kPfTile = 128;         // slots of a K or V tile
constexpr int kPfTileBytes = kPfTile * kD * 2;
constexpr int kPfSlots = 5;
constexpr int kPfMaxCtas = 160;
// Balancing, measured on prompts of 8192 tokens, 16 ragged chunks over 8192 and 512 tokens
// over 131072 slots: a unit counted as 1, 2, 3, 4, 5 tiles more than it has 401 / 449 / 776,
// 375 / 426 / 787, 354 / 400 / 781, 350 / 375 / 740, 352 / 381 / 729 us; 17 tokens over
// 1024 slots in runs of 1, 2, 3 tiles at least 28, 19, 22 us (with an earlier merge).
constexpr int kPfMinRun = 2;         // K/V tiles a CTA takes at least
constexpr int kPfUnitCost = 4;       // what a unit costs besides its tiles (q, the first product, the output), in tiles
constexpr int kPfFewTiles = 4;       // tiles a CTA up to which that is not counted (every CTA then has about one piece)
constexpr float kPfGrow = 8.f;       // growth of the maximum that a row is rescaled for
// log2 of the weight of a row's maximum.  fp16: 7, so that weights down to 2^-21 of the
// largest are normal numbers, and 2^(7 + 8) is one too.  bf16 has FP32's range: -8, so that
// no weight is above 1 and a row's sum of weight * |V| no larger than with the exact
// maximum (V may be as large as the type's largest).
__host__ __device__ constexpr float pf_lift(bool bf16) { return bf16 ? -kPfGrow : 7.f; }

constexpr size_t kPfTokenBytes = kHq * kD * 2;  // of a token of q or out

struct PrefillParams {
  CacheView c;
  const void* q;                // [tokens, 32, 128]
  void* out;                    // [tokens, 32, 128]
  const int32_t* chunk_starts;  // [B + 1]
  const int32_t* lens;          // [B]
  float* part_o;                // [2 * ctas][128 dims][256 rows]
  float2* part_ml;              // [2 * ctas][256 rows]: maximum, sum
  int tokens, ctas;
  int box;                      // rows loaded together: a tile's, or a page's if it is smaller
  float scale_log2, v_scale;
};

// Checked: a piece's partial output, and a row's maximum and sum.
__device__ __forceinline__ float* pf_part(const PrefillParams& p, float* at) {
  return in_buffer(at, 4, p.part_o, (size_t)2 * p.ctas * kD * 2 * kPfRows * 4, p.c.flags);
}
__device__ __forceinline__ float2* pf_part_ml(const PrefillParams& p, float2* at) {
  return in_buffer(at, 8, p.part_ml, (size_t)2 * p.ctas * 2 * kPfRows * 8, p.c.flags);
}
// The cache's row that a box starts at.  (A contiguous cache's last boxes may reach past its
// last row, and past a row's length start behind it: the copy fills those with zeros.)
__device__ __forceinline__ int pf_box_row(const PrefillParams& p, size_t row, bool held) {
  if constexpr (kChecked) {
    if (held && row >= p.c.rows) {
      if (p.c.flags) atomicOr(p.c.flags, GQA_FLAG_BOUNDS);
      return 0;
    }
  }
  return (int)row;
}

// ---- the schedule ----------------------------------------------------------

// A batch row's chunk.
struct PfRow {
  int at, n, len, base;  // first token, tokens, length, length - tokens
  __device__ __forceinline__ int units() const { return (n + kPfTokens - 1) / kPfTokens; }
  // K/V tiles of unit m: up to what its last token sees (a row shorter than its chunk
  // counts as if it were as long, so that every unit has a tile)
  __device__ __forceinline__ int tiles(int m) const {
    return (max(base, 0) + min(n, (m + 1) * kPfTokens) + kPfTile - 1) / kPfTile;
  }
  // Positions of the stream before unit m: `cost` and its tiles for each unit k < m, m <=
  // units().  tiles(k) = floor((q + k) / 2)
  // for full units, q = floor((base + 64 + 127) / 64), and sums of floor(j / 2) are squares.
  __device__ __forceinline__ long long before(int m, int cost) const {
    const int u = units();
    const long long q = (max(base, 0) + kPfTokens + kPfTile - 1) / kPfTokens;
    const auto f = [](long long x) { return (x - 1) * (x - 1) / 4; };
    const long long full = min(m, u - 1);
    return m <= 0 ? 0 : f(q + full) - f(q) + (m == u ? tiles(u - 1) : 0) + (long long)m * cost;
  }
  __device__ __forceinline__ long long positions(int cost) const { return n > 0 ? kHkv * before(units(), cost) : 0; }
};

__device__ __forceinline__ PfRow pf_row(const PrefillParams& p, int b) {
  PfRow r;
  const auto start = [&](int i) { return __ldg(item(p.chunk_starts, i, p.c.batch + 1, p.c.flags)); };
  r.at = min(max(start(b), 0), p.tokens);
  r.n = min(max(start(b + 1), r.at), p.tokens) - r.at;
  r.len = min(max(__ldg(item(p.lens, b, p.c.batch, p.c.flags)), 0), p.c.capacity);
  r.base = r.len - r.n;
  return r;
}

// Where a position of the stream lies, position `rem` of row r's: tile j of unit m, or
// (j < 0) in the unit's cost, -j positions before its first tile.
__device__ __forceinline__ void pf_locate(const PfRow& r, long long rem, int cost, int& g, int& m, int& j) {
  const int u = r.units();
  const long long head = r.before(u, cost);
  g = (int)(rem / head);
  rem -= g * head;
  int lo = 0, hi = u - 1;  // the last unit that begins at or before rem
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (r.before(mid, cost) <= rem) lo = mid;
    else hi = mid - 1;
  }
  m = lo;
  j = (int)(rem - r.before(lo, cost)) - cost;
}

// A CTA's run, walked by each warp by itself: the part of a unit that it is at, K/V
// tiles [j0, j1) of `all`.  Kept in shared memory, one for each warp: a row of S leaves
// a softmax thread no registers for it, and it is looked at once a unit.
struct PfCursor {
  long long left;  // positions of the run from tile j0 on
  PfRow row;
  int b, g, m, j0, j1, all, begun, cost;
  // The next part, by one lane.
  __device__ __forceinline__ void step(const PrefillParams& p) {
    if (begun) {
      left -= j1 - j0;
      j0 = 0;
      if (++m == row.units()) {
        m = 0;
        if (++g == kHkv) {
          g = 0;
          while (left > 0 && ++b < p.c.batch) {
            row = pf_row(p, b);
            if (row.n > 0) break;
          }
          if (b >= p.c.batch) left = 0;
        }
      }
      left -= cost;
    } else if (j0 < 0) {
      left += j0;
      j0 = 0;
    }
    begun = 1;
    if (left > 0) {
      all = row.tiles(m);
      j1 = (int)min((long long)all, j0 + left);
    }
  }
  // The same by a warp; false at the run's end.
  __device__ __forceinline__ bool next(const PrefillParams& p) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) step(p);
    __syncwarp();
    return left > 0;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == all; }
  __device__ __forceinline__ int rows_of_q() const { return row.n - m * kPfTokens > kPfTokens / 2 ? 2 : 1; }
  // the last slot that every token of the unit sees
  __device__ __forceinline__ int first_seen() const { return row.base + m * kPfTokens; }
};

struct PfPlan {
  long long total, run;  // positions in all and a CTA's
  int cost;              // a unit's besides its tiles
  int b;                 // run c begins at position `rem` of row b's (if it begins before `total`)
  long long rem;
};
struct PfScan {
  long long tiles[32], units[32], rem;
  int b;
};

// The plan, and where run c begins.  Every thread of the block calls it; each has an
// equal part of the rows.
__device__ __forceinline__ PfPlan pf_plan(const PrefillParams& p, int c, PfScan& s) {
  const int warps = (int)blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int per = (p.c.batch + (int)blockDim.x - 1) / (int)blockDim.x;
  const int b0 = min(p.c.batch, (int)threadIdx.x * per), b1 = min(p.c.batch, b0 + per);
  long long tiles = 0, units = 0;
  for (int b = b0; b < b1; ++b) {
    const PfRow r = pf_row(p, b);
    tiles += r.positions(0);
    units += kHkv * r.units();
  }
  const long long my_tiles = tiles, my_units = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {  // up to this lane
    const long long x = __shfl_up_sync(0xffffffffu, tiles, o), y = __shfl_up_sync(0xffffffffu, units, o);
    if (lane >= o) {
      tiles += x;
      units += y;
    }
  }
  if (lane == 31) {
    s.tiles[warp] = tiles;
    s.units[warp] = units;
  }
  __syncthreads();
  long long all_tiles = 0, all_units = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) {
      tiles += all_tiles;
      units += all_units;
    }
    all_tiles += s.tiles[w];
    all_units += s.units[w];
  }
  PfPlan plan;
  plan.cost = all_tiles > (long long)kPfFewTiles * p.ctas ? kPfUnitCost : 0;
  plan.total = all_tiles + plan.cost * all_units;
  plan.run = max((plan.total + p.ctas - 1) / p.ctas, (long long)kPfMinRun);
  // the thread whose rows hold the position says which it is
  const long long at = c * plan.run, upto = tiles + plan.cost * units, before = upto - my_tiles - plan.cost * my_units;
  if (before <= at && at < upto) {
    long long rem = at - before;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long n = pf_row(p, b).positions(plan.cost);
      if (rem < n) break;
      rem -= n;
    }
    s.b = b;
    s.rem = rem;
  }
  __syncthreads();
  plan.b = s.b;
  plan.rem = s.rem;
  return plan;
}

// ---- tcgen05 ---------------------------------------------------------------

// Shared-memory descriptor of a 128-byte swizzled operand: K-major (lead unused) or
// MN-major (lead: bytes from 64 elements of M or N to the next); 1024 bytes from eight
// rows to the next.
__device__ __forceinline__ uint64_t tc_desc(uint32_t address, uint32_t lead) {
  return (uint64_t)((address & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// FP32 accumulators, 128 x 128, fp16 or bf16 operands; B MN-major for P V.
__host__ __device__ constexpr uint32_t tc_idesc(bool bf16, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn ? 1u << 16 : 0u) | (128u >> 3) << 17 | (128u >> 4) << 24;
}
// The products are issued by a converged warp: its elected lane (always the same one)
// issues them, and the operands, the same in every lane, stay in uniform registers.  A
// step's products are one block of code: the warp shares its scheduler with two softmax
// warps, and every instruction between two products costs it some ten cycles.
//
// S = Q K^T over 128 dims: eight products of 16 dims, four to a 64-dim half.
__device__ __forceinline__ void tc_qk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, no, yes;\n\t.reg .b64 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, no;\n\t"
      "add.u64 x, %1, 2;\n\tadd.u64 y, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 4;\n\tadd.u64 y, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 6;\n\tadd.u64 y, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 1024;\n\tadd.u64 y, %2, 1024;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 1026;\n\tadd.u64 y, %2, 1026;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 1028;\n\tadd.u64 y, %2, 1028;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t"
      "add.u64 x, %1, 1030;\n\tadd.u64 y, %2, 1030;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, yes;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
// O += P V over 64 slots: four products of 16 slots, P in TMEM; `add` 0: the first one
// writes O.
__device__ __forceinline__ void tc_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred e, first, yes;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 first, %4, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, first;\n\t"
      "add.u32 x, %1, 8;\n\tadd.u64 y, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, yes;\n\t"
      "add.u32 x, %1, 16;\n\tadd.u64 y, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, yes;\n\t"
      "add.u32 x, %1, 24;\n\tadd.u64 y, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, yes;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// The barrier is arrived at when every product issued so far by the elected lane is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#define GQA_R8(a, i) "=r"((a)[i]), "=r"((a)[(i) + 1]), "=r"((a)[(i) + 2]), "=r"((a)[(i) + 3]), "=r"((a)[(i) + 4]), \
                     "=r"((a)[(i) + 5]), "=r"((a)[(i) + 6]), "=r"((a)[(i) + 7])
#define GQA_W8(a, i) "r"((a)[i]), "r"((a)[(i) + 1]), "r"((a)[(i) + 2]), "r"((a)[(i) + 3]), "r"((a)[(i) + 4]), \
                     "r"((a)[(i) + 5]), "r"((a)[(i) + 6]), "r"((a)[(i) + 7])
// 32 columns of the warp's 32 TMEM lanes.
__device__ __forceinline__ void tc_ld32(uint32_t* x, uint32_t address) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : GQA_R8(x, 0), GQA_R8(x, 8), GQA_R8(x, 16), GQA_R8(x, 24)
      : "r"(address)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t address, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(address),
      GQA_W8(x, 0), GQA_W8(x, 8), GQA_W8(x, 16), GQA_W8(x, 24)
      : "memory");
}
#undef GQA_R8
#undef GQA_W8
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// A box of the cache, 64 elements wide, to shared memory.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(row), "r"(smem_addr(bar))
      : "memory");
}

// ---- shared memory ---------------------------------------------------------

struct PfShared {
  uint8_t q[2][kPfTileBytes];         // [tile][64-dim half][row][128 bytes]
  uint8_t kv[kPfSlots][kPfTileBytes];  // [64-dim half][slot][128 bytes]
  // int8: a tile's K and V row scales (bf16 bits).  Four tiles' are enough: they are
  // loaded once item i - 2 (two to a tile) has been widened, which had to wait until
  // item i - 6 was used, and so for the softmax of four tiles before.
  uint16_t scales[4][2][kPfTile];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], done;  // (P in halves of 64 slots)
  // Of a tile: K there, V there, V looked through (tile & 3 each; at most three tiles
  // are between a load and its product).  A barrier is waited on in every one of its
  // phases by whoever waits on it: a parity says nothing about a phase further on.
  uint64_t k_full[4], v_full[4], v_fixed[4];
  // A tile's K and the V of the tile before were used (tile & 3).
  uint64_t used[4], raw_full[3], raw_empty[3];
  PfCursor cursor[kPfThreads / 32];
  uint32_t tmem;
  uint16_t odd[8];  // a part's number + 1 where a value was taken out of V (a stale one only costs time)
};

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Waits for a phase, two seconds at most (32 bits of the nanosecond timer keep the
// registers of the waiting roles free).
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const auto now = [] {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
  };
  const uint32_t begun = now();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (now() - begun > 2000000000u) return false;
  }
}

// Position of a 16-byte piece of a row in a swizzled tile.
__device__ __forceinline__ uint32_t pf_piece(int row, int piece) {
  return (uint32_t)((piece >> 3) * (kPfTileBytes / 2) + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void st_shared16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}
// Neither infinite nor NaN, of two 16-bit numbers.
template <int QF>
__device__ __forceinline__ bool pair_finite(uint32_t w) {
  constexpr uint32_t kExp = QF == kQF16 ? 0x7c00u : 0x7f80u;
  return (w & kExp) != kExp && (w >> 16 & kExp) != kExp;
}

// Eight elements of a row as floats, the tensor scale left out.
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
    uint32_t group = 0;
    if constexpr (KVF == kKvE2M1) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(c.kv) + row * 16 + i);
      group = __ldg(static_cast<const uint8_t*>(c.scales) + row * 8 + i / 2);
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(c.kv) + row * 16 + i);
      w[0] = v.x;
      w[1] = v.y;
    }
    widen16<KVF>(w, group, d);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = f16x2_to_f32x2(d[k]);
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  }
}

// ---- the kernel ------------------------------------------------------------

// KVF: cache format, QF: q's and out's type.  The products' type is a 16-bit cache's,
// else fp16.
template <int KVF, int QF>
__global__ void __launch_bounds__(kPfThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap map) {
  constexpr bool kNarrow = is_narrow(KVF), kI8 = KVF == kKvI8;
  constexpr int MF = kNarrow ? (int)kQF16 : QF;  // type of the products' operands
  // Slots of K and V tiles.  A narrow cache gives the fifth to tiles as they lie in
  // memory, with an e2m1 cache's scales behind the codes.
  constexpr int kSlots = kNarrow ? kPfSlots - 1 : kPfSlots;
  constexpr int kRawBytes = kPfTile * (kv_row_bytes(KVF) + (KVF == kKvE2M1 ? 8 : 0));
  constexpr int kRaws = kNarrow ? kPfTileBytes / kRawBytes : 1;
  static_assert(kRaws <= 3, "barriers of raw tiles");
  extern __shared__ __align__(1024) uint8_t s_raw[];
  PfShared& sm = *reinterpret_cast<PfShared*>(s_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  pdl_launch_dependents();
  if (smem_addr(s_raw) % 1024 != 0) {  // (the swizzled tiles need it; it is so)
    if (tid == 0 && p.c.flags) atomicOr(p.c.flags, GQA_FLAG_BOUNDS);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], kPfRows);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], kPfRows);
      mbar_init(&sm.p_full[i][1], kPfRows);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.k_full[i], kNarrow ? 2 : 1);
      mbar_init(&sm.v_full[i], kNarrow ? 2 : 1);
      mbar_init(&sm.v_fixed[i], 2);
      mbar_init(&sm.used[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sm.raw_full[i], scale_row_bytes(KVF) > 0 ? 2 : 1);
      mbar_init(&sm.raw_empty[i], 2);
    }
    mbar_init(&sm.done, 1);
    for (int i = 0; i < 8; ++i) sm.odd[i] = 0;
    fence_barrier_init();
  }
  pdl_wait_prior_grid();
  const PfPlan plan = pf_plan(p, (int)blockIdx.x, *reinterpret_cast<PfScan*>(sm.q[0]));
  // lengths and starts that are out of order are told once, also where no row has a token
  if (blockIdx.x == 0 && p.c.flags) {
    for (int b = tid; b < p.c.batch; b += kPfThreads) {
      const int at = __ldg(p.chunk_starts + b), end = __ldg(p.chunk_starts + b + 1), len = __ldg(p.lens + b);
      if (at < 0 || end < at || end > p.tokens || len < 0 || len > p.c.capacity || len < end - at)
        atomicOr(p.c.flags, GQA_FLAG_LENGTH_CLAMPED);
    }
  }
  const long long begin = (long long)blockIdx.x * plan.run;
  if (begin >= plan.total) return;  // (all of the block)
  if (warp == 0) {
    if (lane < kPfThreads / 32) {
      PfCursor& c = sm.cursor[lane];
      c.b = plan.b;
      c.row = pf_row(p, plan.b);
      c.left = min(plan.run, plan.total - begin);
      c.begun = 0;
      c.cost = plan.cost;
      pf_locate(c.row, plan.rem, c.cost, c.g, c.m, c.j0);
    }
  } else if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  PfCursor& sg = sm.cursor[warp];
  bool ok = true;
  // a bounded wait of a warp, whose lanes go on or give up together
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!pf_wait(bar, parity)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };

  // Registers: 168 a thread at launch, 504 over the three warpgroups' like threads;
  // 208 for each softmax thread (a row of S is 128) and 88 for the others use as many.
  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int t = warp / 4, r = tid & (kPfRows - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 TMEM lanes
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * 128;
    uint32_t s_phase = 0;
    uint32_t seg = 0, o_phase = 0;
    int tile_no = 0;  // of the CTA's K/V tiles, for the scales' ring
    float scale = 0.f;
    // the run's next part that has rows for this warpgroup, and its q into shared memory
    const auto find = [&]() {
      bool there = sg.next(p);
      for (; there && t >= sg.rows_of_q(); there = sg.next(p), ++seg) tile_no += sg.j1 - sg.j0;
      return there;
    };
    const auto load_q = [&]() {
      scale = p.scale_log2;
      // the warp's 32 rows, two at a time: 16 lanes hold a row's 256 bytes
      const int piece = lane & 15;
      uint4 x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = (warp & 3) * 32 + 2 * i + (lane >> 4), tok = sg.m * kPfTokens + t * 32 + row / 4;
        x[i] = make_uint4(0, 0, 0, 0);
        if (tok < sg.row.n)
          x[i] = __ldg(in_buffer(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                                ((size_t)(sg.row.at + tok) * kHq + 4 * sg.g + (row & 3)) * kD) + piece,
                                 16, p.q, p.tokens * kPfTokenBytes, p.c.flags));
      }
      if constexpr (kNarrow && QF == kQBF16) {
        // by a power of two into fp16's range: a row's largest |q| into [2^14, 2^15)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // (its exponent -100 at least, so that the scale's stays a normal number)
          const int e = min(max((int)(top >> 7) - 127, -100), 127);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          const int mine = __shfl_sync(0xffffffffu, e, (lane & 1) << 4);  // (row 2 i + (lane & 1)'s)
          if (lane >> 1 == i) scale *= __uint_as_float((uint32_t)(127 - 14 + mine) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = bf16x2_to_f32x2(w[k]);
            w[k] = round2<kQF16>(f.x * up, f.y * up);
          }
          x[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<uint4*>(sm.q[t] + pf_piece((warp & 3) * 32 + 2 * i + (lane >> 4), piece)) = x[i];
      // (a q_scale of 0: the least normal number, so that a hidden slot's -inf stays one)
      scale = fmaxf(scale, 0x1p-126f);
      proxy_fence();
      mbar_arrive(&sm.q_full[t]);
    };
    bool more = find();
    if (more) load_q();
    while (ok && more) {
      const int token = sg.m * kPfTokens + t * 32 + r / 4;
      const bool live = token < sg.row.n;
      // slots that the row sees: up to `seen` (none: a row without a token, or without a slot)
      const int seen = live ? sg.row.base + token : -1;
      float m = -INFINITY, l = 0.f;
      const int j0 = sg.j0, j1 = sg.j1;
      for (int j = j0; ok && j < j1; ++j, ++tile_no) {
        if (!wait(&sm.s_full[t], s_phase)) break;
        s_phase ^= 1;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_ld32(x + 32 * k, s_at + 32 * k);
        tc_wait_ld();
        float* s = reinterpret_cast<float*>(x);
        const uint16_t(*scales)[kPfTile] = sm.scales[tile_no & 3];
        if constexpr (kI8) {
          // (the scales of V are there with V)
          if (!wait(&sm.v_full[tile_no & 3], tile_no >> 2 & 1)) break;
#pragma unroll
          for (int k = 0; k < 128; k += 2) {
            const float2 f = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(scales[0] + k));
            s[k] *= f.x;
            s[k + 1] *= f.y;
          }
        }
        const int visible = seen - j * kPfTile + 1;  // columns of this tile that the row sees
        const bool masked = __any_sync(0xffffffffu, visible < kPfTile);
        uint32_t big = 0;  // int8: the largest V scale that the row sees in this tile, a pair's in 15 bits each
        if (masked) {
#pragma unroll
          for (int k = 0; k < 128; ++k) s[k] = k < visible ? s[k] : -INFINITY;
          if constexpr (kI8) {
#pragma unroll
            for (int k = 0; k < 128; k += 2) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(scales[1] + k) & 0x7fff7fffu;
              big = __vmaxu2(big, k + 1 < visible ? w : (k < visible ? w & 0xffffu : 0u));
            }
          }
        } else if constexpr (kI8) {
#pragma unroll
          for (int k = 0; k < 128; k += 2) big = __vmaxu2(big, *reinterpret_cast<const uint32_t*>(scales[1] + k) & 0x7fff7fffu);
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) top4[i] = fmaxf(top4[i], fmaxf(s[k + i], s[k + i + 4]));
        }
        float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * scale;
        if constexpr (kI8) {
          // int8: P holds weights times V scales, so the largest of these counts too, by
          // its exponent (-60 at least: the weights' sum stays in range).  Of the slots that
          // the row sees only: a later token's scale may be anything.
          const int lg = (int)(max(big & 0xffffu, big >> 16) >> 7) - 126;
          top += (float)max(lg, -60);
        }
        if (__any_sync(0xffffffffu, top > m + kPfGrow)) {
          const float grown = fmaxf(m, top);
          const float f = m == grown ? 1.f : ex2(m - grown);  // (0 from -inf)
          m = grown;
          l *= f;
          if (j > j0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t o[32];
              tc_ld32(o, o_at + 32 * k);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tc_st32(o_at + 32 * k, o);
            }
          }
        }
        const float minus = pf_lift(MF == kQBF16) - (m == -INFINITY ? 0.f : m);
        const float2 scale2 = make_float2(scale, scale), minus2 = make_float2(minus, minus);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int k = 0; k < 128; k += 4) {
          float2 a = fma2(make_float2(s[k], s[k + 1]), scale2, minus2), b = fma2(make_float2(s[k + 2], s[k + 3]), scale2, minus2);
          a = make_float2(ex2(a.x), ex2(a.y));
          b = make_float2(ex2(b.x), ex2(b.y));
          sum0 = add2(sum0, a);
          sum1 = add2(sum1, b);
          if constexpr (kI8) {
            const float2 f = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(scales[1] + k));
            const float2 g = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(scales[1] + k + 2));
            // (a hidden slot's weight stays zero whatever its scale is)
            a.x = masked && k >= visible ? 0.f : a.x * f.x;
            a.y = masked && k + 1 >= visible ? 0.f : a.y * f.y;
            b.x = masked && k + 2 >= visible ? 0.f : b.x * g.x;
            b.y = masked && k + 3 >= visible ? 0.f : b.y * g.y;
          }
          x[k / 2] = round2<MF>(a.x, a.y);
          x[k / 2 + 1] = round2<MF>(b.x, b.y);
          if (k == 60) {  // the first half of P: its product starts
            tc_st32(s_at, x);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&sm.p_full[t][0]);
          }
        }
        sum0 = add2(sum0, sum1);
        l += sum0.x + sum0.y;
        tc_st32(s_at + 32, x + 32);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[t][1]);
      }
      if (!ok) break;
      // Q is free once its last product is there, so the next part's goes there now, and
      // its first S is formed while this part's output is written
      const bool whole = sg.whole();
      const int g = sg.g, b = sg.b, hidden = max(sg.first_seen() + 1, j0 * kPfTile), part = (int)seg;
      const int tokens = sg.row.n - sg.m * kPfTokens - t * 32;  // of the tile
      const size_t out_at = ((size_t)(sg.row.at + sg.m * kPfTokens + t * 32) * kHq + 4 * g) * kD;
      ++seg;
      more = find();
      if (more) load_q();
      if (!wait(&sm.o_full[t], o_phase)) break;
      o_phase ^= 1;
      tc_fence_after();
      const bool odd = !kI8 && sm.odd[part & 7] == (uint16_t)(part + 1);  // (a code of int8 is a number)
      const int slot = 2 * (int)blockIdx.x + (j0 > 0 ? 0 : 1);
      const float f = l == 0.f ? 0.f : p.v_scale / l;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t o[32];
        __syncwarp();
        tc_ld32(o, o_at + 32 * k);
        tc_wait_ld();
        if constexpr (!kI8) {
          if (odd) {
            // values taken out of V: into the rows that see their slots
            for (int u = hidden; u <= min(seen, j1 * kPfTile - 1); ++u) {
              const size_t vrow = cache_row(p.c, b, kHkv + g, u);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float y[8];
                row8<KVF>(p.c, vrow, 4 * k + i, y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!(fabsf(y[e]) <= 3.4e38f)) o[8 * i + e] = __float_as_uint(__uint_as_float(o[8 * i + e]) + y[e]);
              }
            }
            __syncwarp();
          }
        }
        if (whole) {
          // four lanes hold a token's four heads: turned about, so that they store 64
          // bytes of one head after another
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = round2<QF>(__uint_as_float(o[8 * i + 2 * e]) * f, __uint_as_float(o[8 * i + 2 * e + 1]) * f);
            c[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
#pragma unroll
          for (int step = 1; step < 4; step *= 2)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((i & step) == 0) {
                const bool up = (lane & step) != 0;
                const uint4 give = up ? c[i] : c[i + step];
                const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, step), __shfl_xor_sync(0xffffffffu, give.y, step),
                                             __shfl_xor_sync(0xffffffffu, give.z, step), __shfl_xor_sync(0xffffffffu, give.w, step));
                c[i] = up ? got : c[i];
                c[i + step] = up ? c[i + step] : got;
              }
          if (r / 4 < tokens) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_at + (size_t)(r / 4) * kHq * kD) + 4 * k + (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) *in_buffer(dst + i * (kD / 8), 16, p.out, p.tokens * kPfTokenBytes, p.c.flags) = c[i];
          }
        } else {
          float* dst = p.part_o + ((size_t)slot * kD + 32 * k) * (2 * kPfRows) + t * kPfRows + r;
#pragma unroll
          for (int i = 0; i < 32; ++i) *pf_part(p, dst + i * (2 * kPfRows)) = __uint_as_float(o[i]);
        }
      }
      if (!whole) *pf_part_ml(p, p.part_ml + (size_t)slot * (2 * kPfRows) + t * kPfRows + r) = make_float2(m, l);
    }
  } else if (warp == 8) {
    // ----------------------------------------------------------- products
    {
      constexpr uint32_t kQk = tc_idesc(MF == kQBF16, false), kPv = tc_idesc(MF == kQBF16, true);
      const uint64_t q0 = tc_desc(smem_addr(sm.q[0]), 16), k0 = tc_desc(smem_addr(sm.kv[0]), 16),
                     v0 = tc_desc(smem_addr(sm.kv[0]), kPfTileBytes / 2);
      // (a descriptor's address counts 16 bytes in its lowest 14 bits; all of shared memory fits)
      constexpr uint32_t kTile = kPfTileBytes >> 4;
      // a lane that gives up a wait goes on with the others to the end of the tile
      const auto await = [&](uint64_t* bar, uint32_t parity) {
        if (!pf_wait(bar, parity)) ok = false;
      };
      uint32_t tile = 0, k_slot = 0, v_slot = 1;  // the tile whose K comes next; its slot, V's of the tile before
      uint32_t q_phase = 0, p_phase = 0;
      while (ok && sg.next(p)) {
        const int nq = sg.rows_of_q(), n = sg.j1 - sg.j0;
        for (int j = -1; ok && j < n; ++j) {
          if (j >= 0) {
            const uint32_t v_no = tile - 1;
            await(kNarrow ? &sm.v_full[v_no & 3] : &sm.v_fixed[v_no & 3], v_no >> 2 & 1);
          }
          const uint64_t kd = k0 + k_slot * kTile, vd = v0 + v_slot * kTile;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= nq) break;
            if (j >= 0) {
              const uint32_t parity = p_phase >> t & 1;
              await(&sm.p_full[t][0], parity);
              tc_fence_after();
              tc_pv(tmem + 256 + t * 128, tmem + t * 128, vd, kPv, j > 0);
              await(&sm.p_full[t][1], parity);
              tc_fence_after();
              tc_pv(tmem + 256 + t * 128, tmem + t * 128 + 32, vd + 512, kPv, 1);
              if (j == n - 1) tc_commit(&sm.o_full[t]);
            } else {
              await(&sm.q_full[t], q_phase >> t & 1);
              tc_fence_after();
            }
            if (j + 1 < n) {
              if (t == 0) await(&sm.k_full[tile & 3], tile >> 2 & 1);
              tc_qk(tmem + t * 128, q0 + t * kTile, kd, kQk);
              tc_commit(&sm.s_full[t]);
            }
          }
          if (j >= 0) {
            p_phase ^= (1u << nq) - 1;
            v_slot = v_slot + 2 >= kSlots ? v_slot + 2 - kSlots : v_slot + 2;
          } else {
            q_phase ^= (1u << nq) - 1;
          }
          if (j + 1 < n) {
            // K of this tile and V of the one before are done with
            tc_commit(&sm.used[tile & 3]);
            k_slot = k_slot + 2 >= kSlots ? k_slot + 2 - kSlots : k_slot + 2;
            ++tile;
          }
          ok = __all_sync(0xffffffffu, ok);
        }
      }
      if (!ok) {  // products in flight end before the block's memory is given up
        tc_commit(&sm.done);
        pf_wait(&sm.done, 0);
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------- K and V tiles
    uint32_t item = 0, seg = 0;
    int tile_no = 0;
    // The slot of item i (tile i / 2's K, or its V) held item i - kSlots, which is free
    // when the first product of tile (i - kSlots + 1) / 2 with its K is done.  (Every
    // tile's barrier is waited on, one after another.)
    uint32_t freed = 0;  // tiles whose barrier was waited on
    const auto slot_free = [&](uint32_t i) {
      while (ok && i >= (uint32_t)kSlots && freed <= (i - kSlots + 1) / 2) {
        wait(&sm.used[freed & 3], freed >> 2 & 1);
        ++freed;
      }
      return ok;
    };
    if constexpr (kNarrow) {
      // One warp has the tiles loaded as they lie; two widen them, four rows at a time, a
      // lane 16 elements, eight lanes a row.  (The first widening a quarter too was
      // slower: 1108 us against 730, fp4 4 x 1024 of 16384.  It then waits for the others
      // where it should run ahead of them.)
      PfCursor& la = sg;
      uint32_t l_item = 0;
      int lj = 0, l_end = 0, l_plane = 1, l_len = 0, l_row = -1, ids = 0, ids_next = 0;
      uint2 sc[4], sc_next[4];  // row scales of the item before the one being loaded, and of that
      const auto page_of = [&](int j) {  // of the lane's box
        const int t = j * kPfTile + lane * p.box;
        return lane < kPfTile / p.box && t < l_len
                   ? __ldg(cell(p.c.block_table + (size_t)la.b * p.c.max_pages, t >> p.c.page_log2, (size_t)p.c.max_pages,
                                p.c.block_table, (size_t)p.c.batch, p.c.flags))
                   : 0;
      };
      const auto load = [&]() {  // false: the run's end
        if (l_plane == 1 && ++lj >= l_end) {
          if (!la.next(p)) return false;
          lj = la.j0;
          l_end = la.j1;
          l_len = la.row.len;
          if (p.c.block_table) ids_next = page_of(lj);
        }
        l_plane ^= 1;
        const int raw = (int)(l_item % kRaws), t0 = lj * kPfTile, pg = l_plane * kHkv + la.g;
        uint8_t* bytes = sm.kv[kSlots] + raw * kRawBytes;
        if (l_plane == 0 && p.c.block_table) {
          ids = ids_next;
          if (lj + 1 < l_end) ids_next = page_of(lj + 1);
          if (ids < 0 || ids >= p.c.num_pages) {
            if (p.c.flags) atomicOr(p.c.flags, GQA_FLAG_PAGE_CLAMPED);
            ids = min(max(ids, 0), p.c.num_pages - 1);
          }
        }
        l_row = -1;
        if (p.c.block_table == nullptr) {
          if (lane == 0) l_row = pf_box_row(p, ((size_t)la.b * 2 * kHkv + pg) * p.c.capacity + t0, t0 < l_len);
        } else if (lane < kPfTile / p.box && t0 + lane * p.box < l_len) {
          l_row = pf_box_row(p, (((size_t)ids * 2 * kHkv + pg) << p.c.page_log2) + ((t0 + lane * p.box) & ((1 << p.c.page_log2) - 1)),
                             true);
        }
        if (!wait(&sm.raw_empty[raw], (l_item / kRaws & 1) ^ 1)) return false;
        const uint32_t some = __ballot_sync(0xffffffffu, l_row >= 0);
        if (lane == 0) {
          if (some) mbar_arrive_expect_tx(&sm.raw_full[raw], (uint32_t)(__popc(some) * p.box * kv_row_bytes(KVF)));
          else mbar_arrive(&sm.raw_full[raw]);
        }
        __syncwarp();
        if (l_row >= 0) tma_box(smem_addr(bytes) + lane * p.box * kv_row_bytes(KVF), &map, 0, l_row, &sm.raw_full[raw]);
        if constexpr (scale_row_bytes(KVF) > 0) {
          // the rows' scales, by plain loads; store_scales puts them behind the codes
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 32 * k + lane, first = __shfl_sync(0xffffffffu, l_row, r / p.box);
            sc_next[k] = make_uint2(0, 0);
            if (first >= 0 && t0 + r < l_len) {
              size_t at = (size_t)first + (r & (p.box - 1));
              if constexpr (kChecked) {
                if (at >= p.c.rows) {
                  if (p.c.flags) atomicOr(p.c.flags, GQA_FLAG_BOUNDS);
                  at = 0;
                }
              }
              if constexpr (kI8) sc_next[k].x = __ldg(static_cast<const uint16_t*>(p.c.scales) + at);
              else sc_next[k] = __ldg(static_cast<const uint2*>(p.c.scales) + at);
            }
          }
        }
        ++l_item;
        return true;
      };
      const auto store_scales = [&](uint32_t n) {
        const int raw = (int)(n % kRaws), tile = (int)(n >> 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 32 * k + lane;
          if constexpr (kI8) sm.scales[tile & 3][n & 1][r] = (uint16_t)sc[k].x;
          else reinterpret_cast<uint2*>(sm.kv[kSlots] + raw * kRawBytes + kPfTile * kv_row_bytes(KVF))[r] = sc[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.raw_full[raw]);
      };
      if (warp == 9) {
        // an item's scales are stored when the next one's are on their way
        for (bool more = true; ok && more;) {
          const uint32_t n = l_item;
          more = load();
          if constexpr (scale_row_bytes(KVF) > 0) {
            if (n > 0 && ok) store_scales(n - 1);
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[k] = sc_next[k];
          }
        }
        // copies in flight land before the block's shared memory is given up
        if (!ok)
          for (uint32_t k = l_item > kRaws ? l_item - kRaws : 0; k < l_item; ++k) pf_wait(&sm.raw_full[k % kRaws], k / kRaws & 1);
      } else {
        const int piece = lane & 7;
        for (; ok && sg.next(p); ++seg) {
          const int len = sg.row.len, first_seen = sg.first_seen(), j1 = sg.j1;
          for (int j = sg.j0; ok && j < j1; ++j, ++tile_no) {
            const int t0 = j * kPfTile;
            for (int plane = 0; ok && plane < 2; ++plane, ++item) {
              const int slot = (int)(item % kSlots), raw = (int)(item % kRaws);
              const uint8_t* bytes = sm.kv[kSlots] + raw * kRawBytes;
              uint8_t* dst = sm.kv[slot];
              if (!wait(&sm.raw_full[raw], item / kRaws & 1) || !slot_free(item)) break;
              // slots past the length, and values that some query does not see
              const bool tail = t0 + kPfTile > len, check = !kI8 && plane == 1 && t0 + kPfTile - 1 > first_seen;
              bool odd = false;
#pragma unroll 1
              for (int step = 0; step < 4; ++step) {
                const int row0 = 64 * (warp - 10) + 16 * step + (lane >> 3);
                uint32_t d[4][8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int row = row0 + 4 * i;
                  if constexpr (KVF == kKvE2M1) {
                    const uint2 v = *reinterpret_cast<const uint2*>(bytes + row * 64 + piece * 8);
                    const uint32_t w[2] = {v.x, v.y};
                    widen16<KVF>(w, bytes[kPfTile * 64 + row * 8 + piece], d[i]);
                  } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(bytes + row * 128 + piece * 16);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    widen16<KVF>(w, 0, d[i]);
                  }
                }
                if (tail || check) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int u = t0 + row0 + 4 * i;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      if (u >= len) d[i][e] = 0;
                      if (check && u > first_seen && !pair_finite<kQF16>(d[i][e])) {
                        odd = true;
                        if (!pair_finite<kQF16>(d[i][e] & 0xffffu)) d[i][e] &= 0xffff0000u;
                        if (!pair_finite<kQF16>(d[i][e] & 0xffff0000u)) d[i][e] &= 0xffffu;
                      }
                    }
                  }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int row = row0 + 4 * i;
                  st_shared16(dst + pf_piece(row, 2 * piece), d[i][0], d[i][1], d[i][2], d[i][3]);
                  st_shared16(dst + pf_piece(row, 2 * piece + 1), d[i][4], d[i][5], d[i][6], d[i][7]);
                }
              }
              if (odd) sm.odd[seg & 7] = (uint16_t)(seg + 1);
              proxy_fence();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&sm.raw_empty[raw]);
                mbar_arrive(plane == 0 ? &sm.k_full[tile_no & 3] : &sm.v_full[tile_no & 3]);
              }
            }
          }
        }
      }
    } else {
      for (; ok && sg.next(p); ++seg) {
        const int len = sg.row.len, first_seen = sg.first_seen(), j1 = sg.j1;
        for (int j = sg.j0; ok && j < j1; ++j, ++tile_no) {
          const int t0 = j * kPfTile;
          for (int plane = 0; ok && plane < 2; ++plane, ++item) {
            const int slot = (int)(item % kSlots);
            uint64_t* full = plane == 0 ? &sm.k_full[tile_no & 3] : &sm.v_full[tile_no & 3];
            uint8_t* dst = sm.kv[slot];
            if (warp == 9) {
              // by TMA, in boxes of `box` rows: one, or a page's each; pages past the
              // length are left out
              if (!slot_free(item)) break;
              const int pg = plane * kHkv + sg.g;
              int row = -1;
              if (p.c.block_table == nullptr) {
                if (lane == 0) row = pf_box_row(p, ((size_t)sg.b * 2 * kHkv + pg) * p.c.capacity + t0, t0 < len);
              } else if (lane < kPfTile / p.box && t0 + lane * p.box < len) {
                row = (int)cache_row(p.c, sg.b, pg, t0 + lane * p.box);
              }
              const uint32_t some = __ballot_sync(0xffffffffu, row >= 0);
              if (lane == 0) {
                if (some) mbar_arrive_expect_tx(full, (uint32_t)(__popc(some) * p.box * kD * 2));
                else mbar_arrive(full);
              }
              __syncwarp();
              if (row >= 0) {
                const uint32_t at = smem_addr(dst) + lane * p.box * 128;
                tma_box(at, &map, 0, row, full);
                tma_box(at + kPfTileBytes / 2, &map, 64, row, full);
              }
            } else if (plane == 1) {
              // the V tiles that hold slots which some query does not see
              if (!wait(full, tile_no >> 2 & 1)) break;
              if (t0 + kPfTile - 1 > first_seen) {
                bool odd = false;
                for (int i = tid - 320; i < kPfTile * 16; i += 64) {
                  const int row = i >> 4, u = t0 + row;
                  if (u <= first_seen) continue;
                  uint4* at = reinterpret_cast<uint4*>(dst + pf_piece(row, i & 15));
                  if (u >= len) {
                    *at = make_uint4(0, 0, 0, 0);
                    continue;
                  }
                  const uint4 v = *at;
                  uint32_t w[4] = {v.x, v.y, v.z, v.w};
                  bool bad = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if (!pair_finite<MF>(w[e] & 0xffffu)) w[e] &= 0xffff0000u, bad = true;
                    if (!pair_finite<MF>(w[e] & 0xffff0000u)) w[e] &= 0xffffu, bad = true;
                  }
                  if (bad) {
                    odd = true;
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                  }
                }
                if (odd) sm.odd[seg & 7] = (uint16_t)(seg + 1);
                proxy_fence();
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.v_fixed[tile_no & 3]);
            }
          }
        }
      }
      // copies in flight land before the block's shared memory is given up
      if (warp == 9 && !ok)
        for (uint32_t k = item > kSlots ? item - kSlots : 0; k < item; ++k)
          pf_wait(k & 1 ? &sm.v_full[k / 2 & 3] : &sm.k_full[k / 2 & 3], k / 8 & 1);
    }
  }
  if (!ok && lane == 0 && p.c.flags) atomicOr(p.c.flags, GQA_FLAG_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ---- merging a unit's pieces -----------------------------------------------

constexpr int kMergeThreads = 256;
constexpr int kMergeDims = kD / (kMergeThreads / 32);  // of a row that a thread merges

// CTA (c, k): rows [32 k, 32 k + 32) of the unit that run c begins inside of, if c is
// the first run that does.
template <int QF>
__global__ void __launch_bounds__(kMergeThreads) prefill_merge_kernel(const __grid_constant__ PrefillParams p) {
  __shared__ PfScan s_scan;
  __shared__ PfCursor s_unit;
  __shared__ int s_pieces;  // 0: nothing to do
  __shared__ long long s_begin;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int c = (int)blockIdx.x + 1;
  const PfPlan plan = pf_plan(p, c, s_scan);
  const long long at = c * plan.run;
  if (at >= plan.total) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    PfCursor u;
    u.b = plan.b;
    u.row = pf_row(p, plan.b);
    int j;
    pf_locate(u.row, plan.rem, plan.cost, u.g, u.m, j);
    u.all = u.row.tiles(u.m);
    const long long begin = at - j;  // the position of the unit's first tile
    s_begin = begin;
    // inside the unit, and no earlier run's begin is
    s_pieces = j > 0 && at - plan.run <= begin ? (int)((begin + u.all - 1) / plan.run - begin / plan.run) + 1 : 0;
    s_unit = u;
  }
  __syncthreads();
  if (s_pieces == 0) return;
  const PfCursor& u = s_unit;
  const int row = 32 * (int)blockIdx.y + lane, token = u.m * kPfTokens + row / 4;
  if (u.m * kPfTokens + 8 * (int)blockIdx.y >= u.row.n) return;
  const bool live = token < u.row.n;
  const int first = (int)(s_begin / plan.run);
  const auto slot_of = [&](int k) { return 2 * (first + k) + ((long long)(first + k) * plan.run > s_begin ? 0 : 1); };
  constexpr int kSide = 4;  // pieces whose loads are in flight together
  float m = -INFINITY;
  for (int k0 = 0; k0 < s_pieces; k0 += 2 * kSide) {
    float x[2 * kSide];
#pragma unroll
    for (int k = 0; k < 2 * kSide; ++k)
      x[k] = k0 + k < s_pieces ? pf_part_ml(p, p.part_ml + (size_t)slot_of(k0 + k) * (2 * kPfRows) + row)->x : -INFINITY;
#pragma unroll
    for (int k = 0; k < 2 * kSide; ++k) m = fmaxf(m, x[k]);
  }
  float l = 0.f, o[kMergeDims];
#pragma unroll
  for (int i = 0; i < kMergeDims; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 < s_pieces; k0 += kSide) {
    float2 ml[kSide];
    float y[kSide][kMergeDims];
#pragma unroll
    for (int k = 0; k < kSide; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (k0 + k < s_pieces) {
        const int slot = slot_of(k0 + k);
        ml[k] = *pf_part_ml(p, p.part_ml + (size_t)slot * (2 * kPfRows) + row);
        float* src = p.part_o + ((size_t)slot * kD + kMergeDims * warp) * (2 * kPfRows) + row;
#pragma unroll
        for (int i = 0; i < kMergeDims; ++i) y[k][i] = *pf_part(p, src + i * (2 * kPfRows));
      }
    }
#pragma unroll
    for (int k = 0; k < kSide; ++k) {
      if (k0 + k >= s_pieces) break;
      const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - m);
      if (ml[k].y != 0.f) l += ml[k].y * f;
#pragma unroll
      for (int i = 0; i < kMergeDims; ++i) o[i] = fmaf(y[k][i], f, o[i]);
    }
  }
  if (!live) return;
  const float f = l == 0.f ? 0.f : p.v_scale / l;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                        ((size_t)(u.row.at + token) * kHq + 4 * u.g + (row & 3)) * kD + kMergeDims * warp);
#pragma unroll
  for (int i = 0; i < kMergeDims / 8; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = round2<QF>(o[8 * i + 2 * e] * f, o[8 * i + 2 * e + 1] * f);
    *in_buffer(dst + i, 16, p.out, p.tokens * kPfTokenBytes, p.c.flags) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace gqa
