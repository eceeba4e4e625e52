/*
 * gqa_decode.h -- C ABI of libgqa_decode.so: single-token grouped-query decode
 * attention over a KV cache on NVIDIA GB300 (sm_103a).
 *
 * What is computed (restated from the "FlashInfer sm110_gqa_decode" article,
 * sections "Input contract", "Convenience API" and "Prepared continuous
 * decoding", and for FP8 from the "FP8 KV cache port on Jetson AGX Thor" blog,
 * section 1, patch 2):
 *
 *   Fixed geometry: 32 query heads, 8 KV heads, head_dim 128, one query token
 *   per request.  Query head h reads KV head g = h / 4 (the grouped view
 *   that splits the 32 heads into 8 groups of 4 consecutive heads).  For every batch row b and query head h:
 *     s_t   = q_scale * k_scale / sqrt(128) * dot(q[b,h,:], K[b,g,t,:]),  0 <= t < len[b]
 *     out[b,h,:] = v_scale * sum_t softmax(s)_t * V[b,g,t,:]
 *   k_scale = v_scale = 1 except for the e4m3 and e2m1 caches.  Slots t >= len[b]
 *   are never read.  Arithmetic is FP32 (exp2-domain online softmax); the
 *   output is rounded once to fp16/bf16, round-to-nearest-even.
 *
 * Layouts (all dense, row-major, contiguous; element offsets):
 *   q    [batch, 32, 128]              fp16 or bf16 (gqa_dtype_t)
 *   kv   [batch, 2, 8, capacity, 128]  plane 0 = K, plane 1 = V; same dtype
 *                                      as q, e4m3 bytes (fp8 entry), int8
 *                                      codes with bf16 row scales (int8 entry)
 *                                      or [..., 64] bytes of e2m1 pairs with
 *                                      e4m3 group scales (fp4 entry); a paged
 *                                      pool on the paged entries
 *   lens int32 [batch], device memory, read only by the kernels; the contract
 *        is 1 <= lens[b] <= capacity (see "Lengths" below)
 *   out  [batch, 32, 128]              same dtype as q (bf16 on the fp8 entry)
 *   q, kv, out and the workspace must be 16-byte aligned; lens 4-byte aligned.
 *
 * Pointers are device pointers unless stated.  `stream` is a cudaStream_t
 * (NULL = the legacy default stream).  Every launching call is asynchronous,
 * enqueues on `stream`, reads nothing back to the host and performs no host
 * synchronisation, except gqa_decode_get_status and
 * gqa_decode_noalloc_get_status (documented there).
 *
 * Ownership: the caller owns every buffer (q, kv, lens, out, workspace).  The
 * library never frees caller memory and keeps no pointer past the call.  The
 * only library-owned state is a per-device cache of the device check and of
 * kernel attributes, and the static scratch of gqa_decode_noalloc.
 *
 * Errors: every function validates its arguments before any CUDA call and
 * returns a gqa_status_t; no exception or abort crosses this ABI.  A
 * thread-local message with details of the last failure on the calling thread
 * is available from gqa_last_error().
 *
 * Lengths: read on the device only.  A length outside [1, capacity] is
 * clamped to [0, capacity] (0 produces a zero output row), never read out of
 * bounds, and flagged with GQA_FLAG_LENGTH_CLAMPED in the workspace header
 * (gqa_decode_get_status).
 *
 * Workspace (split-KV, the flash-decoding scheme of the article's
 * "num_splits" section): a caller-owned device buffer of
 * gqa_decode_workspace_size(batch, capacity, num_splits) bytes.  It holds a
 * 256-byte header (status flags) and FP32 partial results (unnormalised
 * output, running max in the log2 domain, softmax denominator) per
 * (b, query head, split slot).  How a row is cut is decided per call from the
 * sizes: into num_splits chunks of capacity (one CTA each), or, for grids of
 * more than one wave, into pieces of equal runs of one stream of all rows'
 * tiles (each row start weighs one more tile when some row is shorter than
 * a run) taken by the resident CTAs (lengths read on the device); either way
 * a row has at most num_splits pieces, and the results are deterministic.
 * With one piece per CTA, 2..8 splits that hold slots and a grid of one wave
 * at most, the splits of each (b, KV head) run as one thread-block cluster
 * and merge on chip through distributed shared memory: no partial is
 * written and stage 2 launches nothing.  Zero the header once before first use (gqa_decode_workspace_init).
 * Launches that may run concurrently (different streams or graphs) need
 * distinct workspaces; launches ordered on one stream may share one.
 */
#ifndef GQA_DECODE_H_
#define GQA_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_NUM_Q_HEADS 32
#define GQA_NUM_KV_HEADS 8
#define GQA_HEAD_DIM 128
#define GQA_MAX_SPLITS 256
#define GQA_WORKSPACE_HEADER_BYTES 256

typedef enum {
  GQA_OK = 0,
  GQA_ERR_INVALID_ARGUMENT = 1,   /* null pointer, size, dtype, scale, misalignment */
  GQA_ERR_UNSUPPORTED_DEVICE = 2, /* not a compute capability 10.3 (sm_103) device */
  GQA_ERR_WORKSPACE_TOO_SMALL = 3,
  GQA_ERR_ALIASING = 4,           /* out overlaps q, kv or lens */
  GQA_ERR_CUDA = 5                /* a CUDA runtime call failed (see gqa_last_error) */
} gqa_status_t;

typedef enum { GQA_F16 = 0, GQA_BF16 = 1 } gqa_dtype_t;

typedef enum {
  GQA_KV_F16 = 0,
  GQA_KV_BF16 = 1,
  GQA_KV_E4M3 = 2,
  GQA_KV_I8 = 3,
  GQA_KV_E2M1 = 4 /* 4 bits: see gqa_decode_fp4kv */
} gqa_kv_format_t;

/* Bits of the status word in the workspace header. */
#define GQA_FLAG_LENGTH_CLAMPED 0x1u  /* some lens[b] was outside [1, capacity] */
#define GQA_FLAG_WAIT_TIMEOUT 0x2u    /* a pipeline wait gave up; outputs are invalid */
#define GQA_FLAG_PAGE_CLAMPED 0x4u    /* a block-table entry was outside [0, num_pages) (decode: clamped; append: not written) */
#define GQA_FLAG_SLOT_CLAMPED 0x8u    /* gqa_append_kv: a slot outside [0, capacity), not written */
#define GQA_FLAG_BOUNDS 0x10u         /* checked builds (GQA_CHECKED): an access fell outside its buffer and was
                                         redirected inside it; the library has a bug.  Any build: an eviction's
                                         list of kept slots was no longer what the call had written */

/* Name of a status code (static string). */
const char* gqa_status_string(gqa_status_t status);

/* Details of the last failure on the calling thread ("" if none). */
const char* gqa_last_error(void);

/* Which interface the library was built with: a digest of this header (static
 * string, "" if the build gave none).  A binding that calls functions by address
 * compares it with that of the header it was compiled against. */
const char* gqa_interface(void);

/* Bytes of workspace needed for (batch, capacity, num_splits); 0 if the
 * arguments are invalid (batch, capacity < 1; num_splits outside
 * [1, GQA_MAX_SPLITS]).  num_splits = 1 needs only the 256-byte header. */
size_t gqa_decode_workspace_size(int batch, int capacity, int num_splits);

/* Host-only split planner (no CUDA call besides a cached SM-count query; safe
 * during stream capture once the device has been seen).  Picks the number of
 * KV splits from batch x capacity, the KV format and the SM count of `device`:
 * about 8 waves of (batch, KV head, split) work items over the worst case, or,
 * for latency-bound sizes (at most 16 tiles per resident CTA in all), about
 * sqrt(6 x tiles per row) (e2m1: sqrt(16 x tiles), 32 at most) capped at one wave.  Writes the chosen count
 * (1..GQA_MAX_SPLITS) to *num_splits_out. */
gqa_status_t gqa_decode_plan(int batch, int capacity, gqa_kv_format_t kv_format, int device,
                             int* num_splits_out);

/* The same planner with the SM count given: pure host arithmetic, no CUDA
 * call.  sm_count < 1 is invalid. */
gqa_status_t gqa_decode_plan_for(int batch, int capacity, gqa_kv_format_t kv_format, int sm_count,
                                 int* num_splits_out);

/* Split geometry (pure host arithmetic): tokens per split, rounded up to
 * whole 64-token (fp16/bf16) or 128-token (8- and 4-bit) tiles, and the number of
 * splits that hold slots, ceil(capacity / chunk) <= num_splits.  With one
 * piece per CTA, split s covers slots [s * chunk, min((s + 1) * chunk, len));
 * the balanced schedule cuts rows elsewhere but never into more pieces.
 * Stage 2 runs only when the effective count is above 1 and the splits do
 * not merge on chip (2..8 of them with one piece per CTA in a grid of one
 * wave whose clusters can all be resident at once do, in a thread-block
 * cluster). */
gqa_status_t gqa_decode_split_geometry(int capacity, int num_splits, gqa_kv_format_t kv_format,
                                       int* chunk_tokens_out, int* splits_effective_out);

/* Kernels one decode call of these sizes enqueues on its stream (host
 * arithmetic; no work is enqueued): 1 when a single split holds every slot
 * or the splits merge on chip in a thread-block cluster, else 2 (the split
 * kernel and the combine).  The on-chip merge also needs all its clusters
 * resident at once; once the current device has been set up by a call that
 * launches, and sm_count is its SM count, its cluster occupancy (queried at
 * set-up) decides that as the launches do, else only the SM count does.
 * The same for the contiguous and paged entries; q_len 1..4 as
 * gqa_decode_verify; num_splits 1..GQA_MAX_SPLITS after resolving 0;
 * sm_count < 1 is invalid.  Writes the count to *launches_out. */
gqa_status_t gqa_decode_launch_count_for(int batch, int capacity, gqa_kv_format_t kv_format, int q_len,
                                         int num_splits, int sm_count, int* launches_out);

/* Convenience call (the article's sm110_gqa_decode): plans the split count,
 * takes a stream-ordered workspace with cudaMallocAsync/cudaFreeAsync on
 * `stream`, and launches.  q_scale must be finite and >= 0 (0 gives the mean
 * of V).  Length-clamp flags are not observable through this call. */
gqa_status_t gqa_decode(const void* q, const void* kv, const int32_t* lens, void* out,
                        int batch, int capacity, gqa_dtype_t dtype, float q_scale,
                        void* stream);

/* Prepared call (the article's launch_sm110_gqa_decode_prepared): no
 * allocation and no host synchronisation, so it can be captured in a CUDA
 * graph.  q_scale must be finite and > 0 (as the article's prepare step
 * requires).  num_splits = 0 picks gqa_decode_plan's choice; otherwise
 * 1..GQA_MAX_SPLITS.  `workspace` must hold gqa_decode_workspace_size(batch,
 * capacity, num_splits) bytes (after resolving 0).  `out` must not overlap q,
 * kv or lens. */
gqa_status_t gqa_decode_prepared(const void* q, const void* kv, const int32_t* lens, void* out,
                                 int batch, int capacity, gqa_dtype_t dtype, float q_scale,
                                 int num_splits, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* FP8 KV cache (the blog's e4m3 port): kv holds float8 e4m3fn bytes (OCP FP8:
 * bias 7, no infinities, 0x7F/0xFF NaN), q and out are bf16.  k_scale
 * multiplies the scores, v_scale the normalised output; both finite and > 0.
 * q_scale finite and >= 0.  Other rules as gqa_decode_prepared. */
gqa_status_t gqa_decode_fp8kv(const void* q_bf16, const uint8_t* kv_e4m3, const int32_t* lens,
                              void* out_bf16, int batch, int capacity, float q_scale,
                              float k_scale, float v_scale, int num_splits, void* workspace,
                              size_t workspace_bytes, void* stream);

/* INT8 KV cache (the "Qwen3-VL official BF16 on Jetson Orin (SM87)" docs,
 * section "INT8 KV cache (kv_mode)": the cache kept as int8 codes, each
 * (position, KV head) row with its own bf16 scale).  kv_i8 holds int8 codes [batch, 2, 8,
 * capacity, 128]; kv_scales_bf16 holds bf16 scales [batch, 2, 8, capacity]
 * (plane 0 K rows, plane 1 V rows), 16-byte aligned, and capacity must be a
 * multiple of 8 (the scales are staged by 16-byte bulk copies); element (b, p, g, t, d)
 * of the cache is code * scale[b, p, g, t].  q and out are fp16 or bf16
 * (`dtype`).  The K row scale multiplies that slot's scores, the V row scale
 * its weight; scales of slots >= len[b] are never read.  q_scale finite and
 * >= 0.  Other rules as gqa_decode_prepared (no allocation, no host sync). */
gqa_status_t gqa_decode_int8kv(const void* q, const int8_t* kv_i8, const uint16_t* kv_scales_bf16,
                               const int32_t* lens, void* out, int batch, int capacity,
                               gqa_dtype_t dtype, float q_scale, int num_splits, void* workspace,
                               size_t workspace_bytes, void* stream);

/* FP4 KV cache: e2m1 codes in blocks of 16 with an e4m3 scale each, and one
 * FP32 scale for all keys and one for all values (the two-level scaling of
 * the FP4 tensor formats).  kv_e2m1 is [batch, 2, 8, capacity, 64] bytes: byte j of a row holds
 * dims 2j (low nibble) and 2j + 1 (high nibble), each a sign bit and one of
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6.  kv_scales_e4m3 is [batch, 2, 8, capacity, 8]
 * e4m3fn bytes, 16-byte aligned: byte j scales dims 16j .. 16j + 15.  Element
 * d of a key row is code[d] * scale[d / 16] * k_scale, of a value row the
 * same with v_scale.  capacity must be a multiple of 2 (the scales are staged
 * by 16-byte bulk copies).  q and out are fp16 or bf16 (`dtype`).  Each
 * softmax weight is rounded to fp16 where it meets V (by 2^-12 of itself down to
 * 2^-29 of the largest); everything else is FP32 or exact.  Codes and
 * scales of slots >= len[b] are never used.  k_scale and v_scale finite and
 * > 0, q_scale finite and >= 0.  Other rules as gqa_decode_prepared (no
 * allocation, no host sync).  The pages have no counterpart to this call. */
gqa_status_t gqa_decode_fp4kv(const void* q, const uint8_t* kv_e2m1, const uint8_t* kv_scales_e4m3,
                              const int32_t* lens, void* out, int batch, int capacity,
                              gqa_dtype_t dtype, float q_scale, float k_scale, float v_scale,
                              int num_splits, void* workspace, size_t workspace_bytes, void* stream);

/* Paged KV cache.  The pages only say that a paged cache is gathered into
 * one contiguous prefix matrix before attention; this entry reads the pages
 * in place instead, with the same result.  Layout (this library's reading):
 *   kv_pages        [num_pages, 2, 8, page_size, 128] in `kv_format` (fp16,
 *                   bf16, e4m3 or int8; e2m1: [..., page_size, 64] bytes),
 *                   each (page, plane, KV head) block contiguous
 *   kv_scales_pages int8: bf16 [num_pages, 2, 8, page_size]; e2m1: e4m3 bytes
 *                   [num_pages, 2, 8, page_size, 8]; the row scales of the
 *                   same page rows, 16-byte aligned (NULL otherwise)
 *   block_table     int32 [batch, max_pages_per_seq], device memory, read only
 *                   by the kernels: slot t of batch row b is row t % page_size
 *                   of page block_table[b][t / page_size]
 * page_size is a power of two in [16, 65536]; the capacity is
 * max_pages_per_seq * page_size (<= 2^30), and lengths follow the usual
 * contract against it.  Only the entries of pages holding slots < len[b] are
 * used; an entry outside [0, num_pages) is clamped and flagged with
 * GQA_FLAG_PAGE_CLAMPED, never dereferenced out of bounds.  q_len 1..4: q
 * and out are [batch, q_len, 32, 128] and query j attends slots
 * [0, len - q_len + j] (gqa_decode_verify); 1 is plain decode.  q/out dtype
 * `q_dtype` (must equal fp16/bf16 KV; either for 8- and 4-bit KV).  k_scale,
 * v_scale as gqa_decode_fp8kv (1 for the other formats but e2m1).  Both stages, no
 * allocation, no host sync; the workspace as gqa_decode_prepared for batch
 * * q_len rows and capacity max_pages_per_seq * page_size. */
gqa_status_t gqa_decode_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages,
                              gqa_kv_format_t kv_format, const void* kv_scales_pages,
                              const int32_t* block_table, int max_pages_per_seq, int num_pages,
                              int page_size, const int32_t* lens, void* out, int batch, int q_len,
                              float q_scale, float k_scale, float v_scale, int num_splits,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Verify window: q_len query tokens per request (1..4), the draft tokens of
 * speculative / multi-token-prediction decoding (the "FP8 KV cache port on
 * Jetson AGX Thor" blog, section 2, MTP).  The window's tokens are the last
 * q_len slots already written to the cache: query token j of row b sits at
 * slot len[b] - q_len + j and attends slots [0, len[b] - q_len + j] (causal
 * within the window).  q and out are [batch, q_len, 32, 128]; the workspace
 * holds gqa_decode_workspace_size(batch * q_len, capacity, num_splits) bytes.
 * Lengths must lie in [q_len, capacity]; a query with no slot (len below
 * q_len) gets a zero row and GQA_FLAG_LENGTH_CLAMPED.  kv_format: fp16 / bf16
 * (= q_dtype), e4m3, int8 (kv_scales as gqa_decode_int8kv) or e2m1 (kv_scales
 * as gqa_decode_fp4kv; NULL for the others).  k_scale, v_scale as
 * gqa_decode_fp8kv (1 unless e4m3 or e2m1).  q_scale finite and
 * >= 0.  Both stages, no allocation, no host sync. */
gqa_status_t gqa_decode_verify(const void* q, gqa_dtype_t q_dtype, const void* kv,
                               gqa_kv_format_t kv_format, const void* kv_scales,
                               const int32_t* lens, void* out, int batch, int capacity, int q_len,
                               float q_scale, float k_scale, float v_scale, int num_splits,
                               void* workspace, size_t workspace_bytes, void* stream);

/* The two stages of a prepared launch, for callers that schedule (or time)
 * them separately.  Stage 1 streams K/V once per (b, KV head, split) and
 * writes FP32 partials to the workspace, or the final output when
 * num_splits == 1 or when its 2..8 effective splits merge on chip (one
 * thread-block cluster per (b, KV head), one piece per CTA, one wave, every
 * cluster resident at once).  Stage 2 merges the partials of each (b, query
 * head) with a log-sum-exp combine and writes `out`; when stage 1 wrote the
 * output it launches nothing.  Both must be given the same geometry, scales
 * and workspace, in this order, on one stream, with the same device
 * current.  Validation as gqa_decode_prepared, except that
 * q_scale may be 0.  Stage 1 does not take an int8 or e2m1 cache (it has no
 * scale argument: use gqa_decode_int8kv or gqa_decode_fp4kv); stage 2 accepts
 * every format. */
gqa_status_t gqa_decode_split_stage(const void* q, gqa_dtype_t q_dtype, const void* kv,
                                    gqa_kv_format_t kv_format, const int32_t* lens, void* out,
                                    int batch, int capacity, float q_scale, float k_scale,
                                    float v_scale, int num_splits, void* workspace,
                                    size_t workspace_bytes, void* stream);
gqa_status_t gqa_decode_combine_stage(const int32_t* lens, void* out, gqa_dtype_t out_dtype,
                                      gqa_kv_format_t kv_format, int batch, int capacity,
                                      float v_scale, int num_splits, const void* workspace,
                                      size_t workspace_bytes, void* stream);

/* No-allocation variant of gqa_decode, for callers that cannot allocate
 * device memory at call time: code running inside a memory-budgeted runtime
 * or a custom allocator that forbids cudaMalloc on the decode path, plugins
 * handed only pre-existing buffers, or hosts that must not touch the
 * allocator between steps.  The pages have no counterpart to this call (their
 * convenience call allocates its workspace and their prepared call takes one
 * from the caller).
 *
 * The split-KV scratch lives in a file-scope static __device__ array of
 * GQA_STATIC_WORKSPACE_BYTES (16 MiB) that every GPU which loads this library
 * holds until the process exits.  The caller still passes q, kv, lens and out.
 * This call performs no cudaMalloc, cudaFree or other allocation; it launches
 * the two stages on `stream`.
 *
 * Set-up: the first call on a device (with that device current) looks up the
 * array's device address with cudaGetSymbolAddress, zeroes its 256-byte
 * header (the status word) with cudaMemsetAsync on `stream`, and caches the
 * address; make that first call before any stream capture.  A failed lookup
 * is reported (GQA_ERR_CUDA) and retried by the next call.  The cached
 * address belongs to the device's primary context: do not use this call (or
 * gqa_decode_noalloc_get_status) on a device after cudaDeviceReset.  Every
 * call on a device shares the one array, which keeps the last call's
 * contents: calls that may overlap on the GPU (different streams or graphs
 * without ordering) race and corrupt each other's results; order them on one
 * stream.  The partials need no clearing (each call writes before it reads);
 * the status flags (GQA_FLAG_LENGTH_CLAMPED, GQA_FLAG_WAIT_TIMEOUT) accumulate
 * over calls until gqa_decode_noalloc_get_status reads and clears them.
 *
 * num_splits = 0 takes gqa_decode_plan's choice, lowered if needed to the
 * largest split count whose scratch fits the array.  An explicit num_splits
 * whose scratch (gqa_decode_workspace_size) exceeds GQA_STATIC_WORKSPACE_BYTES
 * is rejected with GQA_ERR_WORKSPACE_TOO_SMALL.  q_scale finite and >= 0;
 * other rules as gqa_decode_prepared. */
#define GQA_STATIC_WORKSPACE_BYTES (16u << 20)
gqa_status_t gqa_decode_noalloc(const void* q, const void* kv, const int32_t* lens, void* out,
                                int batch, int capacity, gqa_dtype_t dtype, float q_scale,
                                int num_splits, void* stream);

/* The status word of the static scratch of gqa_decode_noalloc on the current
 * device (GQA_FLAG_* bits, accumulated since set-up or the last read): copies
 * it to *flags and clears it.  Like gqa_decode_get_status it synchronises
 * `stream`, so it is for checks outside the hot path, never inside a
 * capture.  Performs the static scratch's set-up if no call has yet (flags
 * are then 0).  The pages have no counterpart to this call. */
gqa_status_t gqa_decode_noalloc_get_status(void* stream, uint32_t* flags);

/* Test hook for the failure path (not for production use).  Launches stage 1
 * exactly as gqa_decode_split_stage does, except that the producer never
 * issues the copies of tile `skip_tile` (0-based, 64 tokens for fp16/bf16,
 * 128 for e4m3) of each split, so the consumers' wait on that tile runs out
 * after `wait_budget_ns` (1 ms .. 4 s).  Each affected CTA then sets
 * GQA_FLAG_WAIT_TIMEOUT in the workspace header, waits (bounded) for its own
 * copies in flight and returns; outputs and partials are invalid.  Lets a test
 * check that a stalled pipeline is reported to the host while the CUDA
 * context stays usable, without faulting or hanging the GPU. */
gqa_status_t gqa_decode_debug_skip_tile(const void* q, gqa_dtype_t q_dtype, const void* kv,
                                        gqa_kv_format_t kv_format, const int32_t* lens, void* out,
                                        int batch, int capacity, float q_scale, float k_scale,
                                        float v_scale, int num_splits, void* workspace,
                                        size_t workspace_bytes, int skip_tile,
                                        uint64_t wait_budget_ns, void* stream);

/* Test hook of the range-checked build (compiled with GQA_CHECKED; not for
 * production use).  From the next launch of this process on, the extents
 * that the range checks of the split, the many-token write and the read-back
 * kernels compare against are cut short: the
 * KV cache (or page pool) by `kv_cut_bytes` and the int8 or e2m1 row scales by
 * `scales_cut_bytes` (each to 0 at most).  A cache access past the cut extent
 * then sets GQA_FLAG_BOUNDS and is redirected to an address inside the
 * buffer (a write is left out), as a real out-of-range access would be, so a test can see the
 * checks fire without any access leaving the real buffers; outputs of such
 * launches are invalid.  0, 0 restores the true extents.  The product build
 * has no range checks: there it accepts 0, 0 and rejects anything else with
 * GQA_ERR_INVALID_ARGUMENT.  The pages have no counterpart to this call. */
gqa_status_t gqa_decode_debug_cut_extents(uint64_t kv_cut_bytes, uint64_t scales_cut_bytes);

/* The step before decode: one new token per batch row (the "Qwen3-VL
 * official BF16 on Jetson Thor (SM110)" docs, "Runtime architecture": fused
 * kernels that normalise Q and K, rotate them and write the cache; decode
 * graphs keyed by (cache_pos,
 * rope_pos)).  For each query head and each KV head vector x of 128:
 *   y_d = x_d / sqrt(mean(x^2) + eps) * w_d     (w = q_norm_w or k_norm_w, [128])
 *   z_i = y_i cos a_i - y_{i+64} sin a_i,  z_{i+64} = y_{i+64} cos a_i + y_i sin a_i,
 *   a_i = positions[b] * rope_theta^(-i/64)     (rotate-half RoPE, i = 0..63)
 * q_out[b] <- z of the 32 query heads (dtype, RNE); the K plane of `kv` at
 * slot slots[b] <- z of the 8 key heads; the V plane at that slot <- v_proj
 * unchanged.  q_proj [batch,32,128], k_proj and v_proj [batch,8,128] and the
 * weights are `dtype`.  The cache format decides the write: fp16/bf16 (must
 * equal dtype; RNE), e4m3 (value * (1 / k_scale) or * (1 / v_scale), quotient
 * and product in FP32, RNE, saturating: the code of value / scale but where that
 * lies within 2^-23 of itself of a tie, and either neighbour there) or
 * int8 (codes round-to-nearest-even of value / scale with a fresh bf16 row
 * scale amax/127 written to kv_scales, clipped to +-127; a NaN among other
 * numbers gets code 0) or e2m1 (as
 * gqa_write_kv, whose rules for alignment and rope_theta then hold too).  positions and
 * slots are int32 [batch] in device memory, read only by the kernel; a slot
 * outside [0, capacity) is not written and, when a workspace is given, sets
 * GQA_FLAG_SLOT_CLAMPED in its header (workspace may be NULL).  eps finite >= 0,
 * rope_theta finite > 0.  One launch, no allocation, no host sync.  A decode
 * that should see the new token uses len[b] = slots[b] + 1. */
gqa_status_t gqa_append_kv(const void* q_proj, const void* k_proj, const void* v_proj,
                           const void* q_norm_w, const void* k_norm_w, gqa_dtype_t dtype,
                           const int32_t* positions, const int32_t* slots, int batch, void* q_out,
                           void* kv, gqa_kv_format_t kv_format, void* kv_scales, int capacity,
                           float eps, float rope_theta, float k_scale, float v_scale, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The same step on a paged cache (the layout of gqa_decode_paged): slot
 * slots[b] of row b is row slots[b] % page_size of page
 * block_table[b][slots[b] / page_size]; an int8 cache writes its fresh row
 * scale into kv_scales_pages [num_pages, 2, 8, page_size].  A slot outside
 * [0, max_pages_per_seq * page_size) sets GQA_FLAG_SLOT_CLAMPED and a
 * block-table entry outside [0, num_pages) sets GQA_FLAG_PAGE_CLAMPED; in both
 * cases nothing of that row is written to the cache (q_out still is).  Other
 * arguments and rules as gqa_append_kv. */
gqa_status_t gqa_append_kv_paged(const void* q_proj, const void* k_proj, const void* v_proj,
                                 const void* q_norm_w, const void* k_norm_w, gqa_dtype_t dtype,
                                 const int32_t* positions, const int32_t* slots, int batch,
                                 void* q_out, void* kv_pages, gqa_kv_format_t kv_format,
                                 void* kv_scales_pages, const int32_t* block_table,
                                 int max_pages_per_seq, int num_pages, int page_size, float eps,
                                 float rope_theta, float k_scale, float v_scale, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Many tokens at once: the append step for the tokens of prompts, of chunks of
 * them or of verify windows (the "Qwen3-VL official BF16 on Jetson Thor
 * (SM110)" docs, "Runtime architecture": a batched norm + RoPE + cache write
 * for prefill), with rotary positions of one axis, or of the three axes of
 * image and video tokens.  Token n belongs to batch row rows[n] and goes to
 * its slot slots[n]; the tokens of a call come in any order, each (row, slot)
 * at most once.
 *   q_proj [tokens, 32, 128], k_proj and v_proj [tokens, 8, 128] of `dtype`:
 *     token n starts q_stride (k_stride, v_stride) elements after token n - 1
 *     (parts of a fused projection); strides are multiples of 8 and hold at
 *     least the token's heads
 *   q_norm_w, k_norm_w [128], or both NULL: no norm (y = x, eps unused)
 *   positions int32 [tokens], or [3, tokens] (time, height, width) with
 *     mrope_section, three counts in HOST memory that sum to 64: angle i turns
 *     with axis 0, 1 or 2.  In blocks (mrope_interleaved 0): the first
 *     section[0] angles are time, then section[1] height, then width.
 *     Interleaved: i is height if i % 3 == 1 and i < 3 section[1], width if
 *     i % 3 == 2 and i < 3 section[2], else time (at most 21 of each).
 *     mrope_section NULL: one axis.
 *   rows, slots int32 [tokens]
 *   q_out [tokens, 32, 128], dense
 * The arithmetic of y and z is gqa_append_kv's, in FP32 with angles exact to
 * 2^-33 of a turn: q_out and a 16-bit cache hold z within half a step plus
 * 2^-19 of the head's largest |z|.  Cache formats as gqa_append_kv, and e2m1
 * (kv_scales: e4m3 bytes, 8 a row): each 16 dims x of a row get the scale
 * s = e4m3(amax(|x|) / (6 k_scale)) (v_scale for values; to the nearest,
 * saturating at 448) and the codes nearest to x / (s k_scale), ties to the
 * even code, saturating at 6; s = 0 gives codes 0.  Scales and codes are those
 * of the exact v, and of the exact z (known to 2^-43 of the head's largest |z|
 * and an angle of 2^-64 of a turn a position: nearer to a tie than that, either
 * neighbour).  An infinite element saturates, and 16 dims with a NaN among them
 * get the NaN scale 0x7f (their codes are any): they read back as NaN.  kv as
 * gqa_decode's, [batch, 2, 8, capacity, 128] (e2m1: 64 bytes a row).  A row outside [0, batch) or a slot outside
 * [0, capacity) writes nothing to the cache (q_out is still written) and sets
 * GQA_FLAG_SLOT_CLAMPED in the workspace's header, if there is one: a padded
 * batch gives its padding slot -1.  tokens = 0 does nothing.  Pointers are
 * 16-byte aligned (int32 arrays and the workspace 4, scales 2).  eps finite
 * >= 0, rope_theta finite >= 1, k_scale and v_scale finite > 0 (e2m1: within
 * [2^-100, 2^100]; e4m3: [2^-126, 2^126], so that their reciprocals are normal
 * numbers; the other formats' writes do not use them).  Nothing written may overlap anything else
 * (GQA_ERR_ALIASING).  One launch, no allocation, no host sync. */
gqa_status_t gqa_write_kv(const void* q_proj, const void* k_proj, const void* v_proj,
                          long long q_stride, long long k_stride, long long v_stride,
                          const void* q_norm_w, const void* k_norm_w, gqa_dtype_t dtype,
                          const int32_t* positions, const int* mrope_section, int mrope_interleaved,
                          const int32_t* rows, const int32_t* slots, int tokens, void* q_out, void* kv,
                          gqa_kv_format_t kv_format, void* kv_scales, int batch, int capacity, float eps,
                          float rope_theta, float k_scale, float v_scale, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The same on a paged cache (the layout of gqa_decode_paged; block_table
 * [batch, max_pages_per_seq]): slot s of row b is row s % page_size of page
 * block_table[b][s / page_size] (two tokens of a call must not meet there
 * either, where rows share a page).  A block-table entry outside [0, num_pages)
 * sets GQA_FLAG_PAGE_CLAMPED and nothing of that token is written to the
 * cache. */
gqa_status_t gqa_write_kv_paged(const void* q_proj, const void* k_proj, const void* v_proj,
                                long long q_stride, long long k_stride, long long v_stride,
                                const void* q_norm_w, const void* k_norm_w, gqa_dtype_t dtype,
                                const int32_t* positions, const int* mrope_section, int mrope_interleaved,
                                const int32_t* rows, const int32_t* slots, int tokens, void* q_out,
                                void* kv_pages, gqa_kv_format_t kv_format, void* kv_scales_pages,
                                const int32_t* block_table, int batch, int max_pages_per_seq, int num_pages,
                                int page_size, float eps, float rope_theta, float k_scale, float v_scale,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Reading a cache back (the "FreeToken-Kai: Running on Turing (sm_75)" docs,
 * change 7: a paged prefix gathered into a contiguous matrix, quantised rows
 * decoded once): slots [starts[b], lens[b]) of every batch row, of a cache of
 * any format, into out [batch, 2, 8, out_capacity, 128] (`out_dtype`) from slot
 * 0 on, out_capacity slots at most; the rest of out keeps what it holds.  Each
 * element is code * scale * k_scale (v_scale for values) in FP32, rounded once;
 * a 16-bit cache's is the value itself (the scales are not used).  lens and starts int32 [batch], device memory;
 * starts may be NULL (0).  A length outside [0, capacity] or a start outside
 * [0, length] is clamped and sets GQA_FLAG_LENGTH_CLAMPED in the header of the
 * workspace, if one is given.  kv and out 16-byte aligned; neither out nor the
 * workspace overlaps anything else.  One launch, no allocation, no host sync. */
gqa_status_t gqa_read_kv(const void* kv, gqa_kv_format_t kv_format, const void* kv_scales,
                         const int32_t* lens, const int32_t* starts, void* out, gqa_dtype_t out_dtype,
                         int batch, int capacity, int out_capacity, float k_scale, float v_scale,
                         void* workspace, size_t workspace_bytes, void* stream);

/* The same from a paged cache (the layout of gqa_decode_paged).  A block-table
 * entry in use outside [0, num_pages) is clamped and sets
 * GQA_FLAG_PAGE_CLAMPED. */
gqa_status_t gqa_read_kv_paged(const void* kv_pages, gqa_kv_format_t kv_format, const void* kv_scales_pages,
                               const int32_t* block_table, int max_pages_per_seq, int num_pages,
                               int page_size, const int32_t* lens, const int32_t* starts, void* out,
                               gqa_dtype_t out_dtype, int batch, int out_capacity, float k_scale,
                               float v_scale, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of chunks of new tokens over the cache that they are already written
 * to (the "FreeToken-Kai: Running on Turing (sm_75)" docs, change 7: prefill
 * attention over the paged prefix; here the pages are read in place).  The chunks
 * of the rows lie one behind another: row b has tokens chunk_starts[b] ..
 * chunk_starts[b + 1] - 1 of q and out [tokens, 32, 128], n of them, and they are
 * the last n of the lens[b] slots of its cache: query j (from 0) attends slots
 * [0, lens[b] - n + j].  n may be 0 or the whole row.  chunk_starts int32
 * [batch + 1], never decreasing, within [0, tokens], and lens int32 [batch], are
 * device memory, read only by the kernels; tokens of q outside every chunk
 * (padding behind the last one) are not read, and out keeps what it holds there.
 * A length outside [0, capacity] or a start out of order is clamped and sets
 * GQA_FLAG_LENGTH_CLAMPED; a query with no slot (n above the length) gets a zero
 * row and sets it too.  Formats, scales and q_scale as gqa_decode_verify, but no
 * rule on the capacity of an int8 or e2m1 cache.  Scores, maximum and sum are
 * FP32 (the sum over the slots of weight * |V|, the largest weight being 1, has to be
 * below FP32's largest number); each softmax weight is rounded where it meets V, to
 * bf16 over a bf16 cache, else to fp16 (by 2^-11 of itself down to 2^-21 of the
 * largest, by 2^-32 of the largest below).  int8: what is rounded is the weight times
 * its slot's V scale, and the largest weight times the largest V scale that the query
 * sees (2^-61 at least; 2^100 at most, above it small weights are lost) takes the
 * largest's place: by 2^-11 of itself down to 2^-20 of that product, by 2^-31 of it
 * below.  A value, key or scale that a query does not see never reaches its output,
 * whatever it holds.
 * q, kv, out and the workspace 16-byte aligned (int8 scales 2, e2m1 scales 8);
 * nothing written overlaps anything else.  The workspace holds
 * gqa_prefill_workspace_size() bytes whatever the sizes; its header as
 * gqa_decode_prepared's.  tokens = 0 does nothing.  No allocation, no host sync. */
size_t gqa_prefill_workspace_size(void);
gqa_status_t gqa_prefill(const void* q, gqa_dtype_t q_dtype, const void* kv, gqa_kv_format_t kv_format,
                         const void* kv_scales, const int32_t* chunk_starts, const int32_t* lens,
                         void* out, int tokens, int batch, int capacity, float q_scale, float k_scale,
                         float v_scale, void* workspace, size_t workspace_bytes, void* stream);

/* The same over a paged cache (the layout and page rules of gqa_decode_paged). */
gqa_status_t gqa_prefill_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages,
                               gqa_kv_format_t kv_format, const void* kv_scales_pages,
                               const int32_t* block_table, int max_pages_per_seq, int num_pages,
                               int page_size, const int32_t* chunk_starts, const int32_t* lens,
                               void* out, int tokens, int batch, float q_scale, float k_scale,
                               float v_scale, void* workspace, size_t workspace_bytes, void* stream);

/* After a verify window: which of its drafted tokens stay, and the token that
 * follows them.  A window has T tokens, the last accepted one and T - 1 drafts.
 *   probs [batch, T, vocab] of `prob_type`: row j is the target's distribution
 *     behind token j of the window
 *   drafts int32 [batch, T - 1]: token j + 1 of the window; a row with fewer
 *     drafts ends in -1 (an id of vocab or above ends them too, and sets
 *     GQA_FLAG_SLOT_CLAMPED)
 *   draft_probs [batch, T - 1, vocab], the distributions that the drafts were drawn
 *     from, or NULL: each draft had probability one
 *   uniforms float [batch, T], random numbers in [0, 1)
 * Draft j is taken if all before it are and uniforms[j] * q_j(d_j) < p_j(d_j)
 * (exactly; p, q = probs, draft_probs; a NaN refuses).  With n taken, tokens[b]
 * holds those n, then one drawn from max(p_n - q_n, 0) if a draft was refused,
 * from p_n if none was left, then -1; accepted[b] = n.  The draw: each term,
 * rounded once to FP32, clipped to [0, 1] (NaN: 0), is taken to whole units of
 * 2^-38, and the token is the first whose running sum is above
 * floor(sum * floor(uniforms[T - 1] * 2^24) / 2^24).  If nothing is left of p
 * beside q, the draw is from p_n; if that has no weight either, the token is -1.
 * out_lens[b] = max(lens[b] - (T - 1) + n, 0), the length without the refused
 * drafts' slots (lens counts all T of the window); lens and out_lens may both be
 * NULL, or be the same array.  Strides are in elements; the vocab's are 1.  T
 * 1..32 (drafts may be NULL with T = 1).  Arrays aligned to their elements; the
 * workspace (optional) has the status flags; nothing written overlaps anything
 * else.  One launch, no allocation, no host sync. */
typedef enum { GQA_PROB_F16 = 0, GQA_PROB_BF16 = 1, GQA_PROB_F32 = 2 } gqa_prob_t;
gqa_status_t gqa_verify_drafts(const void* probs, long long probs_batch_stride,
                               long long probs_token_stride, const void* draft_probs,
                               long long draft_batch_stride, long long draft_token_stride,
                               gqa_prob_t prob_type, const int32_t* drafts, const float* uniforms,
                               const int32_t* lens, int32_t* out_lens, int32_t* tokens,
                               int32_t* accepted, int batch, int window, int vocab, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The softmax weights that a step gives the slots of a cache, summed over the 4
 * query heads of each KV head and the q_len tokens of the step (1..4, the last
 * slots as in gqa_decode_verify):
 *   w[b, g, t] = sum over j, h of softmax over [0, len - q_len + j] of
 *                q_scale * k_scale / sqrt(128) * dot(q[b, j, h], K[b, g, .]) at t
 * weights float [batch, 8, capacity]: for t < lens[b], w is added to it (add != 0)
 * or written (add = 0); slots at and past the length keep what they hold.  FP32
 * throughout.  Formats as gqa_decode_verify (no rule on the capacity), lengths too;
 * a score of minus infinity gives its slot none, and a query that sees no slot, or
 * none but such, gives no weight at all; a NaN score makes NaN of the weights that
 * its head's query gives.  Pointers 16-byte aligned (int8
 * scales 2, e2m1 scales 8, lens 4).  The workspace holds
 * gqa_weights_workspace_size(batch, capacity, q_len) bytes (0: invalid sizes), the
 * scores of the whole capacity among them, whichever way the call takes.
 * One launch where a row's scores fit on chip and the batch fills the GPU or the
 * capacity is at most 8192, else two; no allocation, no host sync. */
size_t gqa_weights_workspace_size(int batch, int capacity, int q_len);
gqa_status_t gqa_accumulate_weights(const void* q, gqa_dtype_t q_dtype, const void* kv,
                                    gqa_kv_format_t kv_format, const void* kv_scales, const int32_t* lens,
                                    float* weights, int batch, int capacity, int q_len, float q_scale,
                                    float k_scale, int add, void* workspace, size_t workspace_bytes,
                                    void* stream);
gqa_status_t gqa_accumulate_weights_paged(const void* q, gqa_dtype_t q_dtype, const void* kv_pages,
                                          gqa_kv_format_t kv_format, const void* kv_scales_pages,
                                          const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                          int page_size, const int32_t* lens, float* weights, int batch,
                                          int q_len, float q_scale, float k_scale, int add, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Making a cache smaller by such weights.  Of the lens[b] slots of a row, `keep`
 * stay (all, if there are no more): the first `first`, the last `recent`, and of
 * those between the ones with the largest weights, of equal ones the lowest slots
 * (both zeros are equal; NaN is below everything).  Each KV head chooses for itself.
 * The kept rows of K and V (and their scales) move, in their order, to slots 0, 1,
 * ... of `out`; kept int32 [batch, 8, keep] gets the slots they come from, -1
 * behind the last; out_lens[b] = min(lens[b], keep).  The keys keep the rotation of
 * their first positions.
 *   out NULL: in place.  lens and weights [batch, 8, capacity] are updated, the
 *     weights of slots that no longer hold a token set to 0; rows of no more than
 *     `keep` slots do not change.  out_scales, out_lens and out_weights are NULL.
 *   else out [batch, 2, 8, out_capacity, 128] of the cache's format, out_scales,
 *     out_lens [batch], out_weights [batch, 8, weights_capacity] (or NULL), whose
 *     slots behind the kept ones are set to 0; both capacities at least `keep`.
 * Slots of `out` past the new length keep what they hold.  keep in [1, 2^30],
 * first, recent >= 0, first + recent <= keep.  kv, out and weights 16-byte aligned
 * (int8 scales 2, e2m1 scales 8, int32 arrays 4); nothing written overlaps anything
 * else (but in place).  The workspace holds gqa_evict_workspace_size(batch, keep)
 * bytes (0: invalid sizes).  Two launches, no allocation, no host sync.  Should a
 * wait of an eviction in place run out (GQA_FLAG_WAIT_TIMEOUT), the cache is
 * invalid. */
size_t gqa_evict_workspace_size(int batch, int keep);
gqa_status_t gqa_evict_kv(void* kv, gqa_kv_format_t kv_format, void* kv_scales, int32_t* lens,
                          float* weights, void* out, void* out_scales, int32_t* out_lens,
                          float* out_weights, int32_t* kept, int batch, int capacity, int out_capacity,
                          int weights_capacity, int keep, int recent, int first, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The same on a paged cache: out_table int32 [batch, out_max_pages] names the pages
 * of the same pool that the kept rows move to (out_max_pages * page_size at least
 * `keep`), none of them a page of a block table's row in use; NULL: in place, where
 * no page may belong to two rows.  A block-table entry in use outside [0, num_pages)
 * is clamped and sets GQA_FLAG_PAGE_CLAMPED; where rows are written to, they are
 * left out instead. */
gqa_status_t gqa_evict_kv_paged(void* kv_pages, gqa_kv_format_t kv_format, void* kv_scales_pages,
                                const int32_t* block_table, int max_pages_per_seq, int num_pages,
                                int page_size, int32_t* lens, float* weights, const int32_t* out_table,
                                int out_max_pages, int32_t* out_lens, float* out_weights, int32_t* kept,
                                int batch, int weights_capacity, int keep, int recent, int first,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Zero the workspace header (status flags) on `stream`.  Asynchronous. */
gqa_status_t gqa_decode_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/* Debug only, never inside a capture: synchronises `stream`, copies the
 * status word of the workspace header to *flags (GQA_FLAG_* bits) and clears
 * it. */
gqa_status_t gqa_decode_get_status(void* workspace, size_t workspace_bytes, void* stream,
                                   uint32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* GQA_DECODE_H_ */
