/*
 * leank.h -- C ABI of a decode-attention library for a LeanK-pruned KV cache
 * on NVIDIA GB300 (sm_103a).
 *
 * The method (the passages each call follows):
 *   - "KV cache optimisation for LLMs and LeanK pruning" (framerc.cn),
 *     section 2.2 stage 2: a static binary mask beta per (layer, kv head) keeps
 *     a multiple of 32 K channels; section 3.1: heads are grouped by kept count,
 *     the K cache is split into a full-width part for the attention sinks and
 *     the local window and a pruned part K_prun for the middle tokens, and a
 *     fused FlashAttention reads both; section 3.2: a head with no kept channel
 *     drops its middle V as well.
 *   - "FastGen: profile-based adaptive KV compression" (mhpn.cn), section 2.1:
 *     each decode step appends K_t, V_t and then attends with Q_t over the
 *     whole cache; sections 3.1-3.2: per-head policies (local window only,
 *     special tokens only, full); section 5.1: the three integration points
 *     (per-head allocation, policy-aware append, a kernel reading per-head
 *     ranges).
 *
 * Conventions (all calls):
 *   - Every call returns lk_status.  On a non-OK status nothing was enqueued
 *     and lk_last_error() holds a message (per calling thread).
 *   - Device memory (cache buffer, workspace, q/k/v/o/ids) is owned by the
 *     caller and passed as raw device pointers.  The library never calls
 *     cudaMalloc or cudaFree; its handles are host objects.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Hot calls only enqueue work; they never synchronise.
 *   - Tensors are dense row-major: bf16 = 16-bit bfloat16 stored as uint16.
 *   - Errors found on the device (capacity overflow of a special-token head,
 *     an out-of-range token id, a bounded wait that ran out) set a sticky
 *     status word inside the cache; lk_check() reads and clears it.
 */
#ifndef LEANK_H
#define LEANK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lk_status {
  LK_OK = 0,
  LK_ERR_ARG = 1,         /* bad argument (null pointer, range, mask count, ...) */
  LK_ERR_ALIGN = 2,       /* a pointer is not aligned as required */
  LK_ERR_CAPACITY = 3,    /* token capacity or buffer size exceeded */
  LK_ERR_STATE = 4,       /* call not valid in the cache's current state */
  LK_ERR_CUDA = 5,        /* a CUDA runtime call failed (message has the CUDA error) */
  LK_ERR_TIMEOUT = 6,     /* a device-side bounded wait ran out (lk_check) */
  LK_ERR_UNSUPPORTED = 7  /* shape outside what the kernels implement */
} lk_status;

/* Per-(layer, kv head) cache policy (FastGen section 3.1). */
typedef enum lk_policy {
  LK_POLICY_FULL = 0,     /* LeanK layout: sinks + window at full width, middle on kept channels */
  LK_POLICY_LOCAL = 1,    /* last local_only_window tokens only, full width, no sinks */
  LK_POLICY_SPECIAL = 2   /* tokens whose id is special only, full width, in arrival order */
} lk_policy;

/* Model geometry and cache parameters. */
typedef struct lk_plan_desc {
  int32_t num_layers;         /* L >= 1 */
  int32_t num_q_heads;        /* Hq, a multiple of num_kv_heads */
  int32_t num_kv_heads;       /* Hkv >= 1; query head j reads kv head j / (Hq/Hkv) */
  int32_t head_dim;           /* d; must be 128 */
  int32_t sink;               /* S >= 0: attention-sink tokens of FULL heads */
  int32_t local;              /* W >= 1: local window of FULL heads */
  int32_t local_only_window;  /* W_loc >= 1 if any head is LOCAL */
  int32_t vocab;              /* entries of is_special (>= 1 if any head is SPECIAL) */
  int32_t special_capacity;   /* max rows of a SPECIAL head per sequence; 0 = token capacity */
} lk_plan_desc;

typedef struct lk_plan_s* lk_plan;    /* host object owned by the library */
typedef struct lk_cache_s* lk_cache;  /* host object; its device buffer is the caller's */

/* Where one (layer, sequence, kv head) lives inside the cache buffer (byte
 * offsets from the buffer start).  Region A is full width (sinks + window
 * ring, LOCAL ring, or SPECIAL rows); region B holds middle tokens on the
 * kept channels (FULL heads with n_kept > 0).
 *   Contiguous cache (page_rows = 0): middle row m is row m of region B.
 *   Paged cache (page_rows = 128): region B is the page area of the head's
 *   width class, shared by every head of that class; middle row m is row
 *   page_table[m / 128] * 128 + m % 128 of it, page_table being the head's
 *   int32 [max_pages] row at page_table_offset (-1: no page). */
typedef struct lk_region_info {
  int32_t policy;
  int32_t n_kept;             /* kept K channels (FULL), else 0 */
  int32_t rows_a;             /* row capacity of region A */
  int32_t rows_b;             /* rows of region B (paged: of the class's page area) */
  uint64_t k_a_offset;        /* bf16 [rows_a][128] */
  uint64_t v_a_offset;        /* bf16 [rows_a][128] */
  uint64_t k_b_offset;        /* bf16 [rows_b][n_kept], kept channels ascending */
  uint64_t v_b_offset;        /* bf16 [rows_b][128] */
  int32_t page_rows;          /* 0: contiguous region B; else rows per page */
  int32_t max_pages;          /* entries of the head's page-table row */
  uint64_t page_table_offset; /* int32 [max_pages] */
  int32_t kv_format;          /* lk_kv_format of region B */
  int32_t sealed_blocks;      /* quantised: complete 128-row blocks (read them with
                                 lk_cache_block); region B's offsets then give
                                 the bf16 tail: middle row m >= 128 * sealed_blocks
                                 is tail row m - 128 * sealed_blocks */
} lk_region_info;

/* Storage format of region B (the middle tokens).
 *   LK_KV_BF16  K_prun and V rows in bf16.
 *   LK_KV_INT8  KIVI-style quantisation applied after pruning and
 *               reorganisation (LeanK 4.2 and 5.2 problem 3; KIVI's
 *               per-channel K / per-token V, pruning white paper 5.2.1):
 *               every complete 128-row block of a head's middle is stored as
 *               INT8 codes with one fp32 scale per kept K channel and one per
 *               V token, scale = max|x| / 127 (fp32), code = x / scale
 *               rounded half to even, clipped to +-127; the last,
 *               incomplete block stays bf16.
 *   LK_KV_FP8   as LK_KV_INT8 with FP8 codes (one of the low-precision
 *               formats of the white paper's 5.2.1): OCP e4m3 (largest
 *               finite value 448), scale = max|x| / 448 (fp32), code = x /
 *               scale rounded to the nearest e4m3 value, ties to the even
 *               code, saturated at +-448; a zero code keeps the sign.
 *   LK_KV_FP8_BLOCK  as LK_KV_FP8 with two scales for a whole block: the
 *               largest |x| of the block's 128 tokens and kept K channels gives
 *               one, of its V rows the other, scale = max(max|x| / 448, 2^-64)
 *               (fp32).  A block is 4 (k + 124) bytes shorter; chunks attend over
 *               it in three quarters of the time; decode steps of many short
 *               sequences take nine tenths, of a few long ones the same (one of
 *               32768 tokens 4 % more).  e4m3 codes keep their relative precision
 *               2^-4 for values down to 2^-6 / 448 = 1 / 28672 of the block's
 *               largest.  Attention over it wants values below 2^80 in magnitude
 *               (beside blocks of next to no values, sums of larger ones may pass
 *               fp32's range). */
typedef enum { LK_KV_BF16 = 0, LK_KV_INT8 = 1, LK_KV_FP8 = 2, LK_KV_FP8_BLOCK = 3 } lk_kv_format;

/* Cache options for lk_cache_bytes_ex / lk_cache_init_ex. */
typedef struct lk_cache_options {
  int64_t middle_tokens;      /* < 0: contiguous region B; >= 0: paged, pools
                                 sized as in lk_cache_bytes_paged (quantised:
                                 sealed blocks are the pages,
                                 floor(middle_tokens/128) per head of a class) */
  int32_t kv_format;          /* lk_kv_format */
  int32_t reserved;           /* 0 */
} lk_cache_options;

/* Build a plan (host only; touches no GPU).
 *   masks      host uint8 [L][Hkv][128], 0/1: the static mask beta (LeanK 2.2).
 *              For FULL heads the kept count must be 0, 32, 64, 96 or 128;
 *              rows of other policies are ignored.
 *   policies   host int32 [L][Hkv] of lk_policy.
 *   is_special host uint8 [vocab] (1 = special id) or NULL if no SPECIAL head.
 * Heads are grouped by (policy, kept count) and each FULL head gets its kept
 * channel list (ascending), used to permute q.  Errors: LK_ERR_ARG,
 * LK_ERR_UNSUPPORTED (head_dim != 128 or Hq/Hkv > 8). */
lk_status lk_build_plan(const lk_plan_desc* desc, const uint8_t* masks, const int32_t* policies,
                        const uint8_t* is_special, lk_plan* out);
void lk_plan_destroy(lk_plan plan);

/* Build the static mask beta on the device from learned channel importances
 * (LeanK 2.2 stage 2):
 *   alpha     device fp32 [L][Hkv][128] importances
 *   eligible  device uint8 [L][Hkv], 1 for heads that take a mask (FULL
 *             policy), or NULL for all; other heads get all ones
 *   prune_pct s in [0, 100]: share of eligible channels pruned; a channel
 *             stays when alpha >= the s-th percentile of the eligible alphas
 *             (linear interpolation, computed in fp32)
 *   align     32, 64 or 128: per-head kept counts become multiples of it
 *   exact     0: counts rounded down; 1: then topped up by +align on the heads
 *             with the largest remainders (ties: lower head index) until the
 *             total is align * floor((1 - s/100) * heads * 128 / align + 1/2)
 *   masks     device uint8 [L][Hkv][128] out; a head keeps its channels of
 *             largest alpha, equal alphas to the lower channel index.
 * L * Hkv <= 8192.  Enqueued on `stream`; copy the masks to the host for
 * lk_build_plan. */
lk_status lk_build_masks(const float* alpha, const uint8_t* eligible, int32_t num_layers, int32_t num_kv_heads,
                         double prune_pct, int32_t align, int32_t exact, uint8_t* masks, void* stream);

/* Host-side query of one head's policy, kept count and kept channels
 * (kept_channels: host int16 [128] or NULL; first n_kept entries valid). */
lk_status lk_plan_head(lk_plan plan, int32_t layer, int32_t kv_head, int32_t* policy,
                       int32_t* n_kept, int16_t* kept_channels);

/* Bytes of the cache buffer for `batch` sequences of up to `capacity_tokens`
 * tokens each (LeanK 3.1 split cache, FastGen 5.1 per-head allocation). */
lk_status lk_cache_bytes(lk_plan plan, int32_t batch, int32_t capacity_tokens, size_t* bytes);

/* Paged variant (continuous batching; paged KV blocks as in the pruning
 * white paper, yyx235 blog, section 3.2 "granularity", with FastGen 5.1's
 * per-head variable allocation): region B of every FULL head with k > 0 is
 * held in 128-row pages of its width class instead of a contiguous
 * capacity-sized run.  Each class gets enough pages for `middle_tokens`
 * middle tokens (positions past the sinks and the window) summed over the
 * batch, plus one partly filled page per sequence; a sequence still holds at
 * most `capacity_tokens` tokens.  Pages are taken by appends and prefills on
 * the device and given back by lk_release_sequence.  Errors as
 * lk_cache_bytes; LK_ERR_ARG for middle_tokens < 0. */
lk_status lk_cache_bytes_paged(lk_plan plan, int32_t batch, int32_t capacity_tokens, int64_t middle_tokens,
                               size_t* bytes);

/* Bytes of the decode workspace (split partials and counters for every
 * layer's entries, staging of lk_step_host) for `batch` sequences. */
lk_status lk_workspace_bytes(lk_plan plan, int32_t batch, size_t* bytes);

/* Bind a cache to a caller-owned device buffer of at least lk_cache_bytes
 * bytes, 256-byte aligned.  Enqueues a zero fill of the buffer and the upload
 * of the plan's tables on `stream`; all layers start empty.  The plan must
 * outlive nothing: the cache copies what it needs.  Needs a CUDA device. */
lk_status lk_cache_init(lk_plan plan, void* dev_buf, size_t bytes, int32_t batch,
                        int32_t capacity_tokens, void* stream, lk_cache* out);
/* lk_cache_bytes / lk_cache_init with explicit options (paging and the
 * storage format of region B).  Errors as lk_cache_bytes; LK_ERR_ARG for a
 * null opt or an unknown kv_format. */
lk_status lk_cache_bytes_ex(lk_plan plan, int32_t batch, int32_t capacity_tokens,
                            const lk_cache_options* opt, size_t* bytes);
lk_status lk_cache_init_ex(lk_plan plan, void* dev_buf, size_t bytes, int32_t batch,
                           int32_t capacity_tokens, const lk_cache_options* opt, void* stream,
                           lk_cache* out);

/* Host copy of sealed block `block` of a quantised cache's (layer, b,
 * kv_head), in logical order: k_codes [128][n_kept] (kept channels
 * ascending), k_scales [n_kept], v_codes [128][128], v_scales [128]; any
 * pointer may be NULL.  Codes are one byte each: INT8 values, or e4m3 bit
 * patterns for FP8 and FP8_BLOCK (whose k_scales are all the same, and whose
 * v_scales are).  Synchronises `stream`.  Errors: LK_ERR_STATE (not a
 * quantised cache), LK_ERR_ARG (no such sealed block). */
lk_status lk_cache_block(lk_cache cache, int32_t layer, int32_t b, int32_t kv_head, int32_t block,
                         int8_t* k_codes, float* k_scales, int8_t* v_codes, float* v_scales, void* stream);

/* As lk_cache_init, for a paged cache of lk_cache_bytes_paged bytes. */
lk_status lk_cache_init_paged(lk_plan plan, void* dev_buf, size_t bytes, int32_t batch,
                              int32_t capacity_tokens, int64_t middle_tokens, void* stream, lk_cache* out);
void lk_cache_destroy(lk_cache cache);

/* Zero a caller-owned workspace of at least lk_workspace_bytes bytes
 * (256-byte aligned).  Needed once before the first lk_decode_attn with it,
 * and again after lk_check reported LK_ERR_TIMEOUT. */
lk_status lk_workspace_init(lk_cache cache, void* workspace, size_t ws_bytes, void* stream);

/* Build one empty layer from a dense history of n tokens (prefill, "white
 * paper" 2.3): equal, byte for byte, to n successive lk_append calls.
 *   k, v  device bf16 [B][n][Hkv][128];  ids device int32 [B][n] or NULL.
 * Errors: LK_ERR_STATE if the layer is not empty, LK_ERR_CAPACITY if n
 * exceeds the token capacity. */
lk_status lk_prefill(lk_cache cache, int32_t layer, const void* k, const void* v,
                     const int32_t* ids, int32_t n, void* stream);

/* lk_prefill with a length per sequence: sequence b gets the first lens[b]
 * tokens of its row of the padded inputs.
 *   k, v  device bf16 [B][n_max][Hkv][128];  ids device int32 [B][n_max] or NULL;
 *   lens  host int32 [B], each in [0, n_max].
 * Decode then handles each sequence at its own length (continuous batching). */
lk_status lk_prefill_ragged(lk_cache cache, int32_t layer, const void* k, const void* v,
                            const int32_t* ids, const int32_t* lens, int32_t n_max, void* stream);

/* Prefill one slot b of one layer while the other slots keep their tokens
 * (continuous batching: a new request takes a released slot).
 *   k, v  device bf16 [n][Hkv][128];  ids device int32 [n] or NULL.
 * Sequence b of `layer` must be empty (fresh or released); n = 0 is allowed.
 * The slot becomes active: lk_append writes to it again.  Paged caches take
 * the pages of its middle rows here.  Errors: LK_ERR_STATE (slot not empty),
 * LK_ERR_CAPACITY (n > capacity, or not enough free pages: nothing is
 * launched then). */
lk_status lk_prefill_sequence(lk_cache cache, int32_t layer, int32_t b, const void* k, const void* v,
                              const int32_t* ids, int32_t n, void* stream);

/* Release slot b in every layer: its pages (paged caches) go back to the
 * free stacks, its lengths and special counts become 0, and the slot turns
 * inactive: lk_append skips it (decode gives o = 0 for it) until
 * lk_prefill_sequence fills it again.  Enqueued on `stream`. */
lk_status lk_release_sequence(lk_cache cache, int32_t b, void* stream);

/* Pages of one width class (32, 64, 96 or 128 kept channels) of a paged
 * cache: total and currently free (host mirror, exact at every call
 * boundary).  A contiguous cache reports 0 and 0. */
lk_status lk_cache_pages(lk_cache cache, int32_t width, int64_t* total, int64_t* free_pages);

/* Append one token per sequence to a layer (FastGen 2.1, 3.2 stage 2).
 *   k, v  device bf16 [B][Hkv][128];  ids device int32 [B] or NULL.
 * FULL heads: token n < S goes to sink row n; later tokens go to window ring
 * row S + (n-S) mod W, and once the window is full the token n-W it replaces
 * first moves to the middle (K gathered to the kept channels into K_prun row
 * n-W-S, V copied; dropped when n_kept = 0).  LOCAL: ring row n mod W_loc.
 * SPECIAL: appended (row = count) only if is_special[id].  Bit-exact copies.
 * Released slots (lk_release_sequence) are skipped.  Paged caches take a
 * page from the class's free stack when a middle row starts a new page.
 * Errors: LK_ERR_CAPACITY when an active sequence of the layer already holds
 * capacity_tokens, or a paged cache has too few free pages (nothing is
 * launched then). */
lk_status lk_append(lk_cache cache, int32_t layer, const void* k, const void* v,
                    const int32_t* ids, void* stream);

/* Decode attention of one layer (LeanK 3.1 fused FlashAttention over the
 * split cache; FastGen 3.2 per-policy ranges).
 *   q  device bf16 [B][Hq][128];  o  device fp32 [B][Hq][128].
 * For query head j of sequence b (kv head h = j / G): scores q.k / sqrt(128)
 * over sinks + window at all channels and over the middle tokens at the kept
 * channels (q gathered to the kept channel list), one softmax over both,
 * o = sum p V.  Split over tokens across CTAs; partials are merged inside the
 * same launch.  A head with no resident token gives o = 0.
 * workspace: >= lk_workspace_bytes bytes, zeroed once by lk_workspace_init;
 * calls sharing one workspace must not overlap on the GPU. */
lk_status lk_decode_attn(lk_cache cache, int32_t layer, const void* q, float* o,
                         void* workspace, size_t ws_bytes, void* stream);

/* lk_decode_attn without a caller workspace.  The pages have no counterpart:
 * this is a library convenience.  Some callers cannot call cudaMalloc at all
 * -- a plugin running inside a host runtime that owns the device allocator
 * and its memory accounting, or a latency-critical loop where an allocation
 * would synchronise the device -- and so cannot provide the split workspace.
 * This entry point keeps the split counters and partials in a fixed 8 MiB
 * device array built into the library (a file-scope __device__ array that
 * every GPU loading the library holds until the process exits); it
 * allocates nothing.
 *   q, o  as for lk_decode_attn.
 * Limit: the split scratch of the cache (about (256 + B*Hkv) * G * 520
 * bytes) must fit in 8 MiB, else LK_ERR_CAPACITY and nothing is enqueued.
 * Every call looks up the array's device address in the current context
 * (cudaGetSymbolAddress, which allocates nothing); on the first call on a
 * device that lookup may load the library's device code into the context,
 * so make that first call before any stream capture.  Each call clears the
 * split counters on `stream` before its launch; the partials need no
 * clearing (each is written before it is read).  All calls share the one
 * array and it keeps the last call's contents: calls that overlap on the GPU
 * (other streams, other threads) race and give wrong results. */
lk_status lk_decode_attn_static(lk_cache cache, int32_t layer, const void* q, float* o, void* stream);

/* lk_append over layers layer0 .. layer0+nlayers-1 in one launch:
 *   k, v  device bf16 [nlayers][B][Hkv][128];  ids device int32 [B] or NULL
 *   (the same token enters every layer). */
lk_status lk_append_layers(lk_cache cache, int32_t layer0, int32_t nlayers, const void* k, const void* v,
                           const int32_t* ids, void* stream);

/* lk_decode_attn over layers layer0 .. layer0+nlayers-1 in one launch (the
 * work of all layers is split across the CTAs together):
 *   q  device bf16 [nlayers][B][Hq][128];  o  device fp32 [nlayers][B][Hq][128].
 * Useful when every layer's query is known up front (benchmarks, drafts). */
lk_status lk_decode_attn_layers(lk_cache cache, int32_t layer0, int32_t nlayers, const void* q, float* o,
                                void* workspace, size_t ws_bytes, void* stream);

/* One decode step of a layer: the append of the new token followed by
 * attention with the new query (FastGen 2.1: append K_t, V_t, then attend
 * with Q_t), in one launch.  Same arguments, results and errors as
 *   lk_append(cache, layer, k, v, ids, stream);
 *   lk_decode_attn(cache, layer, q, o, workspace, ws_bytes, stream);
 * and the cache is left as they leave it (byte for byte, except that a
 * paged cache may hand out its free pages in another order).  With a bf16
 * middle one kernel does both: the CTA that combines a head's split
 * partials adds the new token (and the token leaving a full window for the
 * middle) to the softmax from the inputs, then writes them into the cache;
 * the window slot being replaced is left out of the scores.  INT8 / FP8 / FP8_BLOCK caches
 * (where an append may seal a block, changing the values decode reads) run
 * the two launches.  Nothing is launched on an error. */
lk_status lk_step(lk_cache cache, int32_t layer, const void* q, const void* k, const void* v,
                  const int32_t* ids, float* o, void* workspace, size_t ws_bytes, void* stream);

/* lk_step over layers layer0 .. layer0+nlayers-1 in one launch: q, o as for
 * lk_decode_attn_layers, k, v, ids as for lk_append_layers. */
lk_status lk_step_layers(lk_cache cache, int32_t layer0, int32_t nlayers, const void* q, const void* k,
                         const void* v, const int32_t* ids, float* o, void* workspace, size_t ws_bytes,
                         void* stream);

/* One decode step end to end from host memory: q [B][Hq][128] bf16, k, v
 * [B][Hkv][128] bf16 and ids [B] int32 (NULL allowed) in, o [B][Hq][128]
 * fp32 out.  When every buffer is page-locked and mapped into the device's
 * address space (cudaHostAlloc / cudaMallocHost, cudaHostRegister with
 * mapping; torch's pin_memory), the append and decode kernels read the
 * inputs from host memory and write o there directly over the host link
 * (NVLink-C2C on Grace) -- no staging copies.  Otherwise the inputs are
 * copied into the workspace, lk_step runs, and o is copied back (pinned
 * buffers keep those copies asynchronous).  Read o only after synchronising
 * `stream`. */
lk_status lk_step_host(lk_cache cache, int32_t layer, const void* q_host, const void* k_host,
                       const void* v_host, const int32_t* ids_host, float* o_host,
                       void* workspace, size_t ws_bytes, void* stream);

/* lk_step_host with the step's inputs in one host block: host_in = q bf16
 * [B][Hq][128] | k bf16 [B][Hkv][128] | v bf16 [B][Hkv][128] | ids int32 [B]
 * (present iff has_ids != 0), back to back.  Read in place when the block
 * and o are mapped page-locked memory, else moved by a single copy each
 * way. */
lk_status lk_step_host_packed(lk_cache cache, int32_t layer, const void* host_in, int32_t has_ids,
                              float* o_host, void* workspace, size_t ws_bytes, void* stream);

/* A step of layers layer0 .. layer0+nlayers-1 from host memory, as
 * lk_append_layers + lk_decode_attn_layers: host_in = q bf16
 * [nlayers][B][Hq][128] | k bf16 [nlayers][B][Hkv][128] | v (as k) | ids
 * int32 [B] (present iff has_ids != 0; the same token for every layer),
 * back to back; o_host fp32 [nlayers][B][Hq][128] out.  Both must be
 * page-locked and mapped into the device's address space (the kernels read
 * and write them in place over the host link); otherwise LK_ERR_ARG and
 * nothing is launched.  Two launches whatever the step mode (the fused
 * kernel stages the new token with bulk copies, which are kept away from
 * host memory).  Errors as for lk_append_layers and lk_decode_attn_layers.
 * Read o only after synchronising `stream`. */
lk_status lk_step_layers_host_packed(lk_cache cache, int32_t layer0, int32_t nlayers, const void* host_in,
                                     int32_t has_ids, float* o_host, void* workspace, size_t ws_bytes,
                                     void* stream);

/* A chunk of new tokens for every sequence of a cache: the tokens of a prompt
 * that arrives in pieces, or drafted tokens to be verified.  Sequence b's token
 * i is row b * n_max + i of the tensors; its position is the number of tokens
 * that the sequence holds plus i.
 *   q          device bf16 [B][n_max][Hq][128] (lk_append_chunk ignores it)
 *   k, v       device bf16 [B][n_max][Hkv][128]
 *   ids        device int32 [B][n_max] or NULL (no token is special)
 *   lens       host int32 [B], each in [0, n_max], or NULL (n_max each); read
 *              before the call returns.  What rows past lens[b] hold
 *              never matters; in the output they are never written.
 *   n_max      tokens per sequence of the tensors, at most 2^28
 *   *_stride   elements between consecutive tokens of q, k and v: at least
 *              heads * 128 and a multiple of 8, or 0 for dense rows.  A row's
 *              heads are dense, so q, k and v may be views of one projection's
 *              rows.
 * Released slots take no tokens, as if their length here were 0. */
typedef struct lk_chunk {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* ids;
  const int32_t* lens;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  int32_t n_max;
  int32_t reserved;           /* 0 */
} lk_chunk;

/* Bytes of lk_chunk_attn's workspace for chunks of up to n_max tokens, over a
 * cache of any format.  It needs no initialisation and may be shared by calls
 * that do not overlap on the GPU. */
lk_status lk_chunk_workspace_bytes(lk_plan plan, int32_t batch, int32_t n_max, size_t* bytes);

/* Attention of a chunk's queries over the cache and the chunk itself (chunked
 * prefill and draft verification over the split cache of LeanK 3.1 with
 * FastGen 3.2's per-policy ranges).  The cache is only read: append the chunk,
 * or the part of it that was accepted, afterwards.
 *   o  device bf16 [B][n_max][Hq][128], dense.
 * Query i of sequence b, at position p, sees of the token at position t <= p
 * what a decode step at p would have seen had the chunk been appended token by
 * token: FULL heads score it at all channels if t < S or p - t < W, else at
 * the kept channels (not at all when none is kept); LOCAL heads see the last
 * local_only_window tokens; SPECIAL heads the special ones that they have rows
 * for.  One softmax runs over all of it; a query that sees nothing gives 0.
 * Scores and sums are fp32; the weights that multiply the values are rounded to
 * bf16 (over sealed blocks, with their values' scales, to 11 bits), and o to bf16:
 * its relative error is 2.3e-3 (1.75e-3 where sealed blocks weigh most), 1.7e-3 of
 * which is its own rounding.  (lk_decode_attn and lk_step hold both to more bits.)
 * Middle tokens are read as the cache holds them when the call runs: sealed
 * INT8 / FP8 blocks as their dequantised values (a key's scale and its product
 * with the code rounded to 11 bits; of FP8_BLOCK, exact codes and fp32 scales),
 * everything else, the chunk's own tokens included, in bf16.
 * k, v and the cache must hold finite values (v below 2^80 where it attends over
 * sealed blocks); o must not overlap the inputs.
 * workspace: >= lk_chunk_workspace_bytes bytes, 256-byte aligned.  Calls on one
 * cache may overlap on the GPU if each has its own workspace and nothing
 * appends to the layer meanwhile.  A captured call keeps the lens it was given;
 * the tokens held are those of the replay.  Errors: LK_ERR_ARG, LK_ERR_ALIGN (16
 * bytes for q, k, v, o; 4 for ids), LK_ERR_CAPACITY (workspace), LK_ERR_STATE
 * (the current device is not the cache's), LK_ERR_UNSUPPORTED (n_max, B n_max
 * or a position too large), LK_ERR_CUDA (a launch, or the driver's tensor maps). */
lk_status lk_chunk_attn(lk_cache cache, int32_t layer, const lk_chunk* chunk, void* o, void* workspace,
                        size_t ws_bytes, void* stream);

/* Append a chunk to a layer that may already hold tokens: sequence b takes the
 * chunk's first lens[b] tokens, and the layer is left, byte for byte, as that
 * many lk_append calls would leave it (a paged cache may hand out its free
 * pages in another order).  Errors as lk_chunk_attn; LK_ERR_CAPACITY when an
 * active sequence would exceed capacity_tokens or a paged cache has too few
 * free pages (nothing is launched then).  Appends to different layers of a
 * contiguous cache may overlap on the GPU; k and v must not be rows of the
 * cache. */
lk_status lk_append_chunk(lk_cache cache, int32_t layer, const lk_chunk* chunk, void* stream);

/* lk_chunk_attn, then lk_append_chunk of the same chunk: what lk_step does for
 * one token.  Nothing is launched on an error of either. */
lk_status lk_extend(lk_cache cache, int32_t layer, const lk_chunk* chunk, void* o, void* workspace,
                    size_t ws_bytes, void* stream);

/* Which channels of a head turn together: (i, i + rotary_dim / 2), or
 * (2 i, 2 i + 1). */
typedef enum lk_rope_layout { LK_ROPE_HALF = 0, LK_ROPE_INTERLEAVED = 1 } lk_rope_layout;

/* How the angle w_i = base^(-2 i / rotary_dim) that pair i turns per position
 * is stretched for contexts of `factor` times the trained length T:
 *   NONE    not at all
 *   LINEAR  w_i / factor
 *   NTK     base * factor^(d / (d - 2)) in the place of base, d = rotary_dim
 *   YARN    w_i (1 - r_i) + w_i / factor * r_i with r_i = clamp((i - lo) /
 *           (hi - lo), 0, 1); lo = floor(at(high_turns)) >= 0 and hi =
 *           ceil(at(low_turns)) <= d - 1 are the pairs that turn so often in T
 *           positions, at(n) = d ln(T / (2 pi n)) / (2 ln base)
 *   BANDS   w_i s_i + w_i / factor * (1 - s_i) with s_i = clamp((T w_i / 2 pi -
 *           low_turns) / (high_turns - low_turns), 0, 1) */
typedef enum lk_rope_scaling {
  LK_ROPE_SCALE_NONE = 0,
  LK_ROPE_SCALE_LINEAR = 1,
  LK_ROPE_SCALE_NTK = 2,
  LK_ROPE_SCALE_YARN = 3,
  LK_ROPE_SCALE_BANDS = 4
} lk_rope_scaling;

typedef struct lk_rope_desc {
  int32_t rotary_dim;         /* channels that turn, the first of each head: a multiple of 16 in [16, 128] */
  int32_t layout;             /* lk_rope_layout */
  int32_t scaling;            /* lk_rope_scaling */
  int32_t trained_positions;  /* T >= 1 (YARN, BANDS) */
  double base;                /* > 1 */
  double factor;              /* >= 1; ignored by NONE */
  double low_turns;           /* 0: 1 */
  double high_turns;          /* > low_turns; 0: 32 (YARN), 4 (BANDS) */
  double magnitude;           /* multiplies cosine and sine; 0: 0.1 ln(factor) + 1 (YARN), else 1 */
} lk_rope_desc;

typedef struct lk_rope_s* lk_rope;    /* host object owned by the library */

/* Rotary positions for heads of 128 channels (host only; touches no GPU). */
lk_status lk_build_rope(const lk_rope_desc* desc, lk_rope* out);
void lk_rope_destroy(lk_rope rope);

/* Which pairs belong to which axis, where a token has a position on each of
 * several axes (time, height and width of an image's or a video's patches): in
 * runs, axis after axis, or in turn: axis a >= 1 takes its pairs from i mod
 * num_axes = a, the lowest first, and axis 0 the rest. */
typedef enum lk_rope_order { LK_ROPE_AXES_BLOCKS = 0, LK_ROPE_AXES_CYCLIC = 1 } lk_rope_order;

/* Which angle w_i a pair turns per position on its axis: the pair i of the whole
 * head has it as without axes, or the j-th pair of its axis the j-th of a rope of
 * rotary_dim 2 pairs[axis] (scaling included). */
typedef enum lk_rope_spectrum { LK_ROPE_SPECTRUM_SHARED = 0, LK_ROPE_SPECTRUM_OWN = 1 } lk_rope_spectrum;

typedef struct lk_rope_axes {
  int32_t num_axes;           /* 1 .. 4 */
  int32_t pairs[4];           /* of each axis, >= 1; rotary_dim / 2 in all */
  int32_t order;              /* lk_rope_order */
  int32_t spectrum;           /* lk_rope_spectrum */
  int32_t reserved;           /* 0 */
} lk_rope_axes;

/* lk_build_rope for positions of several axes (host only; touches no GPU):
 * calls that take the rope read positions [num_axes][...], one axis after
 * another.  One axis is what lk_build_rope gives.  (A token of text has the same
 * position on every axis, and with LK_ROPE_SPECTRUM_SHARED turns as without
 * axes.) */
lk_status lk_build_rope_axes(const lk_rope_desc* desc, const lk_rope_axes* axes, lk_rope* out);

/* Turn the heads of q and k by their tokens' positions, before they enter
 * lk_prefill, lk_append, lk_step, lk_chunk_attn and so on:
 *   q [tokens][num_q_heads][128], k [tokens][num_kv_heads][128]  device bf16;
 *   positions  device int32 [tokens] ([num_axes][tokens] for a rope of
 *              several axes), any value (negative ones turn back);
 *   q_out, k_out  as q and k; may be q and k themselves (with the same
 *   stride), else must not overlap the inputs.
 * Strides are elements between consecutive tokens: at least heads * 128 and a
 * multiple of 8, or 0 for dense rows.  q or k may be left out with a head
 * count of 0.  Each result is rounded once to bf16 from fp32; the angle keeps
 * its fraction of a turn exactly, however far the position. */
lk_status lk_rope_apply(lk_rope rope, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const int32_t* positions, int64_t tokens, int32_t num_q_heads, int32_t num_kv_heads,
                        void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/* lk_append_chunk with the rotation on the way: the chunk's keys are turned by
 * their tokens' positions (lk_rope_apply) as they enter the layer, which is left as
 * lk_rope_apply and lk_append_chunk would leave it, byte for byte (a paged cache
 * may hand out its free pages in another order).
 *   positions  device int32 [B][n_max] ([num_axes][B][n_max] for a rope of several
 *              axes), any values; NULL: every token's own position in its sequence
 *              (the number of tokens before it), on every axis
 *   chunk->q, q_out  both NULL, or the chunk's queries and where they go turned:
 *              q_out device bf16 [B][n_max][Hq][128], tokens q_out_stride
 *              elements apart (as q_stride); it may be q itself with the same stride,
 *              else must not overlap the inputs.  Rows past a sequence's length,
 *              and of released slots, are left as they are.
 * With n_max = 1 (a decode step: lk_decode_attn with q_out follows) it is one launch,
 * which saves host time; on the GPU lk_rope_apply and lk_append take less (bf16, 8
 * sequences: 4.7 us instead of 6.2).
 * k must not be q_out.  Errors as lk_append_chunk and lk_rope_apply. */
lk_status lk_append_rope(lk_cache cache, int32_t layer, lk_rope rope, const lk_chunk* chunk, const int32_t* positions,
                         void* q_out, int64_t q_out_stride, void* stream);

/* One decode step of a layer whose queries and keys are not turned yet:
 * lk_append_rope of one token of every sequence (chunk->n_max 1, chunk->lens
 * NULL), then lk_decode_attn with the turned queries, which wait in the workspace.
 *   o  device fp32 [B][Hq][128].
 * workspace as for lk_decode_attn.  Nothing is launched on an error of either. */
lk_status lk_step_rope(lk_cache cache, int32_t layer, lk_rope rope, const lk_chunk* chunk, const int32_t* positions,
                       float* o, void* workspace, size_t ws_bytes, void* stream);

/* Host-tracked token count of a layer: the longest sequence's length. */
lk_status lk_cache_length(lk_cache cache, int32_t layer, int32_t* n);

/* Host-tracked token count of every sequence of a layer (lens: host int32 [B]). */
lk_status lk_cache_lengths(lk_cache cache, int32_t layer, int32_t* lens);

/* Location of one (layer, sequence, kv head) in the cache buffer. */
lk_status lk_cache_region(lk_cache cache, int32_t layer, int32_t b, int32_t kv_head,
                          lk_region_info* out);

/* K+V bytes one lk_decode_attn of `layer` reads from the resident cache
 * (synchronises `stream` to read the special-token counts). */
lk_status lk_resident_bytes(lk_cache cache, int32_t layer, void* stream, uint64_t* bytes);

/* How lk_step / lk_step_layers run a step on a bf16 middle:
 *   LK_STEP_AUTO   the library's choice (default): one fused launch when
 *                  the decode's CTAs each stream at least 256 KB and meet
 *                  at most 32 (layer, sequence, kv head) entries (e.g. a
 *                  32K-token layer: 26.6 -> 25.1 us per step), else the
 *                  append and decode launches (a 0.24 MB layer, or a
 *                  32-layer, 64-sequence step, are faster that way);
 *   LK_STEP_FUSED  always one launch;   LK_STEP_SPLIT  always two.
 * Results and cache contents do not depend on the mode.  INT8 / FP8 / FP8_BLOCK
 * middles always run two launches. */
typedef enum { LK_STEP_AUTO = 0, LK_STEP_FUSED = 1, LK_STEP_SPLIT = 2 } lk_step_mode;
lk_status lk_set_step_mode(lk_cache cache, int32_t mode);

/* Whether lk_step_layers(cache, layer0, nlayers, ...) would run as one fused
 * launch now (at the host's current lengths): *fused = 1 or 0. */
lk_status lk_step_is_fused(lk_cache cache, int32_t layer0, int32_t nlayers, int32_t* fused);

/* Override the number of CTAs of lk_decode_attn (0 = the library's choice:
 * one per SM, or 27/32 of the SMs for a bf16 launch over at most 64
 * (sequence, kv head) entries, where fewer, longer streams reach a higher
 * HBM rate); for tuning and split-invariance tests.  Must be <= 256. */
lk_status lk_set_decode_ctas(lk_cache cache, int32_t ctas);

/* Bound of the decode kernel's waits on its stage ring and on its warps'
 * segment barriers, and of chunk attention's waits, in ns (default 1 s; at
 * most 10 s).  A wait that runs out records LK_ERR_TIMEOUT for lk_check and the
 * launch's outputs are garbage; after it, call lk_workspace_init before the
 * next decode (chunk attention's workspace needs nothing).  0 makes every
 * wait that is not already complete run out at once: a way to exercise that
 * failure path without a fault.  The kernel's final wait for its own copies
 * to land keeps its 1 s bound whatever this is.  Errors: LK_ERR_ARG. */
lk_status lk_set_wait_limit(lk_cache cache, uint64_t ns);

/* Synchronise `stream`, read the device status word and, when a bit is set,
 * clear it on `stream` and synchronise again (the clear has landed when the
 * call returns).  Returns
 * LK_ERR_TIMEOUT, LK_ERR_CAPACITY or LK_ERR_ARG (bad token id) for a set
 * bit, LK_ERR_CUDA for a pending CUDA error, else LK_OK. */
lk_status lk_check(lk_cache cache, void* stream);

/* Message of the last non-OK status on the calling thread ("" if none). */
const char* lk_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* LEANK_H */
