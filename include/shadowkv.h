/*
 * shadowkv.h -- C ABI of the ShadowKV decode path for GB300 (sm_103a).
 *
 * The method is the one of "ShadowKV: KV Cache in Shadows for High-Throughput
 * Long-Context LLM Inference" as the xllm-io paper review page states it:
 *   - Algorithm 1 (Pre-filling): A, B <- SVD(K) over the pre-RoPE keys;
 *     landmarks L <- Reduce(K_RoPE) per chunk of c tokens; S <- cosine of
 *     each token to its chunk mean; outliers I <- ArgTopK(-Min(S), o);
 *     V offloaded to the CPU.
 *   - Algorithm 2 (Decoding): P <- MatMul(Q, L^T); I <- ArgTopK(S2, k);
 *     in parallel V_sparse <- Gather(V_CPU, I) and
 *     K_sparse <- MatMul(Gather(A, I), B); attention over
 *     [K_outlier; RoPE(K_sparse); K_local].
 *   - The temporal-locality cache (section 核心创新, and the Telegram explainer
 *     of ShadowKV): chunks selected at the previous step stay on the GPU and
 *     only the set difference is fetched from host memory.
 *
 * Conventions shared by every entry point
 *   - Tensors are dense, row-major, in the element type given by
 *     shadowkv_params.dtype (SKV_DTYPE_F32: float, SKV_DTYPE_BF16: bfloat16).
 *     Index tensors are int32.
 *   - "device" pointers are CUDA global-memory addresses on the context's
 *     device; "host" pointers are ordinary CPU addresses.  The caller owns
 *     every pointer it passes; the library never frees or keeps them past the
 *     call (prefill copies what it needs).
 *   - stream is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Work is enqueued on it in order; calls return before the GPU
 *     finishes unless stated otherwise.  With bf16, d = 128 contexts the
 *     decode step's kernels all run on `stream`, chained with programmatic
 *     dependent launch; other contexts also use one library-owned side
 *     stream, joined back to `stream` before the call returns.
 *   - Every entry point returns an skv_status; on failure
 *     shadowkv_last_error() (thread-local) describes the cause.  No entry point
 *     aborts the process, traps the GPU, or falls back to the CPU.
 *   - Shapes: n = (s - w) / c chunks form the compressed region [0, s - w);
 *     the last w prompt tokens and every appended token form the exact local
 *     window.  G = h_q / h_kv query heads share a KV head; query head g uses
 *     KV head g / G.
 */
#ifndef SHADOWKV_H
#define SHADOWKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum skv_status {
  SKV_OK = 0,
  SKV_ERR_INVALID_ARG = 1,   /* bad shape, pointer, option or size */
  SKV_ERR_OOM = 2,           /* device or pinned-host allocation failed */
  SKV_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  SKV_ERR_DEVICE_CHECK = 4,  /* a kernel found an out-of-range index (status word) */
  SKV_ERR_TIMEOUT = 5,       /* a bounded device wait gave up */
  SKV_ERR_STATE = 6,         /* call not valid in the context's state (e.g. max_new reached) */
  SKV_ERR_UNSUPPORTED = 7    /* a combination the kernels do not implement */
} skv_status;

enum { SKV_DTYPE_F32 = 0, SKV_DTYPE_BF16 = 1 };
/* How S2 combines the softmax scores of a KV head's query group (S2 is not
 * defined on the page): maximum over the group (default) or their sum. */
enum { SKV_GROUP_MAX = 0, SKV_GROUP_SUM = 1 };

/* Shapes and parameters of one attention layer.  Algorithm 1's r, c, o and
 * Algorithm 2's k follow the page's notation. */
typedef struct shadowkv_params {
  int b;            /* sequences in the batch */
  int h_q;          /* query heads (multiple of h_kv) */
  int h_kv;         /* key/value heads */
  int d;            /* head dimension: 64 or 128 */
  int s;            /* prompt tokens */
  int c;            /* chunk size (tokens per landmark) */
  int r;            /* SVD rank of the pre-RoPE key cache, <= min(s, h_kv*d), <= 256 */
  int k;            /* chunks selected per KV head per step, 1..min(n - o, 1024) */
  int o;            /* outlier chunks per KV head, 0..n - 1 */
  int w;            /* local-window prompt tokens; (s - w) must be a positive multiple of c */
  int max_new;      /* decode steps the context can append */
  float rope_theta; /* RoPE base; rotate-half pairing (i, i + d/2) */
  int dtype;        /* SKV_DTYPE_F32 or SKV_DTYPE_BF16 */
  int group_reduce; /* SKV_GROUP_MAX or SKV_GROUP_SUM */
  int svd_iters;    /* subspace iterations of the prefill SVD; 0 = default (3) */
  int reserved;     /* must be 0 */
  unsigned long long seed; /* seed of the SVD's random starting basis */
} shadowkv_params;

typedef struct shadowkv_ctx shadowkv_ctx;   /* opaque, library-owned */

/* Cumulative counters of a context. */
typedef struct shadowkv_stats {
  long long steps;       /* decode steps enqueued */
  long long hits;        /* selected chunks already resident in the cache */
  long long misses;      /* selected chunks fetched from host memory */
  long long link_bytes;  /* value bytes read over the host link by the fetch */
  long long launches;    /* kernels launched by this context */
} shadowkv_stats;

/* Checks the parameters without touching the GPU. */
skv_status shadowkv_validate_params(const shadowkv_params* p);

/* Bytes the context will hold on the device and in pinned host memory
 * (excluding the transient prefill workspace).  Host-only. */
skv_status shadowkv_footprint(const shadowkv_params* p, size_t* device_bytes,
                              size_t* host_bytes);

/*
 * Algorithm 1 (Pre-filling).
 *   k_pre : device, b x h_kv x s x d, pre-RoPE keys.
 *   v     : b x h_kv x s x d values; a host pointer if v_on_host != 0, else device.
 * Computes K_RoPE (position = token index), landmarks L (chunk means of
 * K_RoPE over [0, s - w)), the per-chunk minimum cosine, the o outlier chunks
 * per (sequence, KV head) by ArgTopK(-min cos) (ties to the lower index),
 * the rank-r factors A (b x s x r) and B (b x h_kv x r x d) of the pre-RoPE
 * keys of each sequence viewed as an s x (h_kv d) matrix, the post-RoPE keys
 * and values of the outlier chunks and of the local window, and copies V to
 * library-owned pinned host memory.  On success *out owns everything; k_pre
 * and v may be freed once the call returns (it synchronizes `stream`).  The
 * prefill's kernels are timed with CUDA events whatever SKV_OPT_TIMING says;
 * shadowkv_kernel_times reports them until shadowkv_reset_timers.
 */
skv_status shadowkv_prefill(const shadowkv_params* p, const void* k_pre, const void* v,
                            int v_on_host, void* stream, shadowkv_ctx** out);

/* A compressed layer state supplied by the caller instead of computed by
 * shadowkv_prefill (checkpoint restore, or a prefill done elsewhere).  All
 * device pointers, element type p->dtype, except V (see v_on_host). */
typedef struct shadowkv_state_in {
  const void* A;               /* b x s x r */
  const void* B;               /* b x h_kv x r x d */
  const void* L;               /* b x h_kv x n x d landmarks */
  const int32_t* outlier_ids;  /* b x h_kv x o, ascending, distinct, < n */
  const void* K_out;           /* b x h_kv x (o c) x d post-RoPE outlier keys, chunk order of outlier_ids */
  const void* V_out;           /* b x h_kv x (o c) x d outlier values */
  const void* K_loc;           /* b x h_kv x w x d post-RoPE local-window keys */
  const void* V_loc;           /* b x h_kv x w x d */
  const void* V;               /* b x h_kv x s x d values (host if v_on_host) */
  int v_on_host;
} shadowkv_state_in;

/* Builds a context from a given compressed state (no prefill).  Outlier ids
 * are checked on the device; a bad id makes the call return
 * SKV_ERR_DEVICE_CHECK.  Synchronizes `stream`. */
skv_status shadowkv_load_state(const shadowkv_params* p, const shadowkv_state_in* st,
                               void* stream, shadowkv_ctx** out);

/*
 * Algorithm 2 (Decoding), one token for every sequence.
 *   q     : device, b x h_q x d, post-RoPE queries of the new token.
 *   k_new : device, b x h_kv x d, post-RoPE key of the new token, or NULL.
 *   v_new : device, b x h_kv x d, its value (NULL iff k_new is NULL).
 *   out   : device, b x h_q x d, attention output; it may also be the device
 *           address of mapped pinned host memory (the result is then written
 *           over the host link, with no separate copy).
 * With k_new given, the token is appended to the local window first (at most
 * max_new times; then SKV_ERR_STATE).  Step t (0-based) scores
 * P = q L^T / sqrt(d) over the non-outlier chunks, forms S2 (group_reduce),
 * selects the top-k chunks per KV head (ties to the lower index), rebuilds
 * their keys as RoPE(Gather(A, I) B) at their token positions, takes their
 * values from the GPU chunk cache (hits of the previous step) or from pinned
 * host memory (misses, fetched while the rest is attended), and writes
 * softmax(q K^T / sqrt(d)) V over [outliers; rebuilt chunks; local window].
 * The kernels read q in place through tensor maps: q must be 16-byte aligned
 * (else SKV_ERR_INVALID_ARG before any work is enqueued) and must not change
 * before the step has completed on `stream`.  Asynchronous on `stream`.
 */
skv_status shadowkv_decode_step(shadowkv_ctx* ctx, const void* q, const void* k_new,
                                const void* v_new, void* out, void* stream);

/* The same step with the token's inputs and output in host memory (the call
 * a caller makes whose decode loop lives on the CPU side):
 *   q     : host, b x h_q x d (copied into a library-owned device buffer)
 *   k_new, v_new : host, b x h_kv x d, or NULL; read in place through their
 *           device mapping when they are pinned host memory, else copied
 *   out   : host, b x h_q x d; written in place by the attention when it is
 *           pinned host memory, else copied back after the step
 * Pinned (page-locked) buffers make every copy asynchronous on `stream`;
 * the result is in `out` once `stream` has passed the call.  Pageable
 * buffers work too, with the copies the CUDA runtime makes for them.  The
 * pinned-or-not answer is cached per address (the last 8 addresses). */
skv_status shadowkv_decode_step_host(shadowkv_ctx* ctx, const void* q, const void* k_new,
                                     const void* v_new, void* out, void* stream);

/* Returns the context to its state right after prefill / load_state: the
 * appended tokens are dropped (the local window holds the w prompt tokens
 * again) and the chunk cache is emptied.  Stream-ordered on `stream` after
 * every earlier decode step of this context. */
skv_status shadowkv_rewind(shadowkv_ctx* ctx, void* stream);

/* Releases everything the context owns (NULL-safe).  Synchronizes the device. */
void shadowkv_free(shadowkv_ctx* ctx);

/* Text of the last failure of this thread ("" if none). */
const char* shadowkv_last_error(void);

/* ---------------------------------------------------------------- options */
enum {
  SKV_OPT_CACHE = 0,        /* 1 (default): reuse the previous step's chunks; 0: fetch all k */
  SKV_OPT_TIMING = 1,       /* 1: time each kernel with CUDA events on its stream */
  SKV_OPT_SPLIT_TOKENS = 2, /* tokens per attention split (multiple of 32 in 32..256 whose K/V
                               rows fit in shared memory; default 128).  Setting it selects the
                               classic split-KV attention kernel.  By default bf16 contexts
                               with d = 128 and c a multiple of 8 dividing 128 use the
                               tensor-core attention over K/V records; other bf16 contexts
                               use the pipelined (TMA-fed, 64-token items) kernel */
  SKV_OPT_CUDA_CORES = 3,   /* 1: compute the landmark scores and rebuild the keys with the
                               CUDA-core kernels even where the tensor-core (tcgen05) kernels
                               apply (bf16; for the rebuild also c a multiple of 8 dividing 128
                               and r a multiple of 16), and run the classic split-KV attention
                               instead of the pipelined one; for cross-checking the paths */
  SKV_OPT_REBUILD_IN_ATTENTION = 4 /* 1: where the tensor-core attention moves the values itself
                               (shadowkv_layout.fetch_in_attention) and the rebuild runs on the
                               tensor cores over tiled A, the missed chunks' keys are rebuilt
                               inside the attention's launch: its first CTAs rebuild them
                               (Algorithm 2 step 3, key branch) into the cache slots before
                               they take attention items, and each missed chunk's item waits
                               for its own keys and values.  Three launches per step instead
                               of four.  0 (default): a rebuild launch of its own */
};
skv_status shadowkv_set_option(shadowkv_ctx* ctx, int option, long long value);

/* Synchronizes the context's streams and reads the cumulative counters. */
skv_status shadowkv_get_stats(shadowkv_ctx* ctx, shadowkv_stats* out);

/* Which storage layout and kernels the context uses; they follow from the
 * parameters (and SKV_OPT_CUDA_CORES / SKV_OPT_SPLIT_TOKENS).  Host-only. */
typedef struct shadowkv_layout {
  int kv_records;       /* keys and values of every 8-token group in one 4 KB record;
                           cache slots keep their rebuilt keys, so a step rebuilds
                           only the chunks it fetches */
  int a_tiled;          /* A's chunked region in 8-token core-matrix groups */
  int tc_score;         /* landmark scores on the tensor cores (tcgen05) */
  int tc_rebuild;       /* key rebuild on the tensor cores */
  int tc_attention;     /* attention on the tensor cores over K/V records */
  int fetch_in_rebuild; /* value fetch runs as CTAs of the rebuild launch (one stream) */
  int fetch_in_attention; /* value fetch runs as warps of the tensor-core attention's
                           launch; each missed chunk is attended as soon as its
                           values are in its cache slot */
  int rebuild_in_attention; /* SKV_OPT_REBUILD_IN_ATTENTION is on and applies: the missed
                           chunks' keys are rebuilt by the first CTAs of the attention's
                           launch (three launches per step) */
} shadowkv_layout;
skv_status shadowkv_get_layout(const shadowkv_ctx* ctx, shadowkv_layout* out);

/* Synchronizes and reads the device status word (kernel bounds checks);
 * SKV_ERR_DEVICE_CHECK if any kernel recorded a violation. */
skv_status shadowkv_check(shadowkv_ctx* ctx);

/* ----------------------------------------------- attention without allocation
 * (no counterpart in the paper: a service for callers that cannot allocate)
 *
 * Some callers cannot call cudaMalloc: an inference engine that hands every
 * byte of device memory to its own pool at start-up, or code that records a
 * decode loop into a CUDA graph and must not allocate inside it.  This entry
 * point runs the library's split-KV GQA attention kernel on keys and values
 * the caller already holds and allocates nothing: its scratch (the per-split
 * partial results and the per-head completion tickets) lives in one static
 * device array of SKV_NOALLOC_SCRATCH_BYTES that the library image carries,
 * so every GPU that loads the library holds that array until the process
 * exits.
 *   p        : b, h_q, h_kv, d and dtype are used (h_q / h_kv in {1,2,4,8},
 *              d in {64, 128}); the other fields are ignored.
 *   q        : device, b x h_q x d, post-RoPE queries.
 *   K, V     : device, b x h_kv x n_tokens x d, post-RoPE keys and values.
 *   out      : device, b x h_q x d; out = softmax(q K^T / sqrt(d)) V, query
 *              head g reading KV head g / G.
 * K and V must be 16-byte aligned (their rows are copied 16 bytes at a time)
 * and q and out aligned to their element size; otherwise SKV_ERR_INVALID_ARG
 * is returned before anything is enqueued.
 * Needs P = b * h_q * ceil(n_tokens / 128) * (d + 2) * 4 bytes of partials
 * and T = b * h_kv * 4 bytes of tickets, each rounded up to 256 bytes; when
 * P + T exceeds SKV_NOALLOC_SCRATCH_BYTES the call returns
 * SKV_ERR_UNSUPPORTED.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Every call shares the one array and clears the
 * tickets it needs, so calls whose GPU work overlaps (different streams, or
 * different host threads on the same device without ordering) race; order
 * them on one stream.  Asynchronous on `stream`. */
#define SKV_NOALLOC_SCRATCH_BYTES (8u << 20)
skv_status shadowkv_attention_noalloc(const shadowkv_params* p, const void* q, const void* K,
                                      const void* V, int n_tokens, void* out, void* stream);

/* -------------------------------------------- queries and keys for a step
 * A b x h x s x d tensor given by strides: element (i, g, t, j) lies at
 * ptr + i sb + g sh + t ss + j (strides in elements, not negative; the d
 * elements of a row are adjacent; the stride of an extent of 1 is not used).  A
 * projection's output b x s x (h d) read in place has sh = d. */
typedef struct shadowkv_rows {
  void* ptr;
  long long sb, sh, ss;
} shadowkv_rows;

typedef struct shadowkv_norm_rope_params {
  int b, s;           /* sequences, tokens of each */
  int h_q, h_kv;      /* query heads, key heads */
  int d;              /* head dimension: 64 or 128 */
  int rot;            /* rotated dimensions, the first of each head: a multiple of 8, 0..d */
  int dtype;          /* SKV_DTYPE_F32 or SKV_DTYPE_BF16: rows and weights */
  int norm;           /* 1: normalise each head's row before the rotation; 0: rotate only */
  int pos_per_token;  /* 0: pos holds b first positions, token t at pos[i] + t; 1: b x s positions */
  float eps;          /* added to the mean square (norm); > 0 */
  float theta;        /* base of the rotation's frequencies; > 0 */
} shadowkv_norm_rope_params;

/*
 * Norm of every query and key head, with the rotation to the token's
 * position in the same pass:
 *   y = x / sqrt(mean_j x_j^2 + eps) * w        (norm = 1; w = 1 where the weight is NULL)
 *   (y_i, y_{i + rot/2}) turned by the angle pos theta^(-2i/rot), i < rot/2,
 * the rotate-half pairing the rest of the library uses.  rot = 0 leaves the
 * rows normed but not turned: the pre-RoPE keys shadowkv_prefill takes.
 *   q, k           : device rows b x h_q x s x d and b x h_kv x s x d; either may be
 *                    NULL (then its weight and output are too).
 *   q_weight, k_weight : device, d elements each, or NULL; not used with norm = 0.
 *   pos            : device int32, b or b x s (pos_per_token), any value;
 *                    NULL: token t at position t.
 *   q_out, k_out   : device rows.  An output may be its own input (same pointer and
 *                    strides); otherwise no output overlaps an input or the other output.
 * Everything is computed in fp32 and rounded once (a row whose sum of squares
 * passes fp32's range, |x| above about 1e18, gives zeros); the angle is reduced in
 * 64-bit integers and is exact to 2^-30 of a turn at any position (theta >= 1).  Row
 * pointers and strides must be multiples of 4 elements, and pointers aligned
 * to 4 elements (SKV_ERR_INVALID_ARG).  b = 0 or s = 0 does nothing.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_qk_norm_rope(const shadowkv_norm_rope_params* p, const shadowkv_rows* q,
                                 const shadowkv_rows* k, const void* q_weight, const void* k_weight,
                                 const int32_t* pos, const shadowkv_rows* q_out,
                                 const shadowkv_rows* k_out, void* stream);

/* ------------------------------------------------ 8-bit block cache
 * A dense key/value cache for the sequences and layers a caller does not
 * compress: post-RoPE keys and values held in 8 bits (e4m3: sign, 4 exponent
 * and 3 mantissa bits), with one scale per block of `block` tokens of one KV
 * head.  All memory is the caller's and stays the caller's; the struct only
 * names it, and the calls allocate nothing.
 *
 * Blocks live in a pool.  Pair (i, g) = sequence i, KV head g holds
 * n_tok[i, g] tokens: token t is row t % block of the pool block
 * table[i, g, t / block].  Every table entry, also past the tokens held (there, in a pool that
 * sequences share, it may be -1: see below), must
 * name a pool block (0 <= id < n_pool) and no pool block that a pair appends to may be
 * named twice; entry c of pair p = p max_blocks + c does for a pool of
 * b h_kv max_blocks blocks.  Codes inside a pool block:
 *   k_codes : row t, dimension j at byte (t/8) 8 d + (j/16) 128 + (t%8) 16 + j%16
 *   v_codes : row t, dimension j at byte (t/16) 16 d + j 16 + t%16
 * (the tensor core's K-major operand order for K, and for V transposed).  The
 * value of a code is the e4m3 number times the block's k_scale or v_scale.
 * A scale written by the library is 2^e with the smallest e >= -100 for which
 * max |x| <= 448 2^e over the block's finite entries, those that shadowkv_cache_truncate has taken off
 * since the block's first token among them.
 *
 * A kernel that meets a table entry outside the pool or a token count outside
 * 0..max_blocks block records it in *status (see shadowkv_cache_check).  Attention reads
 * block 0 in such an entry's place; an append drops what belongs there (the tokens still
 * count as held) and writes to no other block; a count is clamped.  Calls that touch the same
 * cache must be ordered (one stream, or events), except that attention calls
 * that do not gather weights may overlap each other.  Host threads may call at
 * the same time: a call's kernels are enqueued together, so that calls of several
 * threads on one stream take effect one after the other. */
typedef struct shadowkv_cache {
  int b, h_kv;        /* sequences, KV heads */
  int d;              /* head dimension: 64 or 128 */
  int block;          /* tokens per block: 16, 32, 64 or 128 */
  int max_blocks;     /* table entries per pair, 1..16384 */
  int n_pool;         /* blocks in the pool */
  void* k_codes;      /* n_pool x block x d bytes, 32-byte aligned */
  void* v_codes;
  float* k_scale;     /* n_pool */
  float* v_scale;
  int32_t* table;     /* b x h_kv x max_blocks */
  int32_t* n_tok;     /* b x h_kv */
  float* weight;      /* b x h_kv x max_blocks: attention weight gathered per block; NULL: none kept */
  int32_t* status;    /* 1 int, 0 at the start */
} shadowkv_cache;

/* Checks the cache's sizes and pointers without touching the GPU. */
skv_status shadowkv_cache_validate(const shadowkv_cache* c);

/*
 * Appends tokens to every pair, quantising them.
 *   dtype : SKV_DTYPE_F32 or SKV_DTYPE_BF16, of k and v.
 *   k, v  : device rows b x h_kv x s x d (post-RoPE keys, values); pointers and
 *           strides multiples of 16 bytes.
 *   lens  : device int32, b: tokens of each sequence, 0..s (k and v are not read
 *           past them); NULL: s each.
 * A block's scale covers its tokens; where a later append needs a larger one, the
 * codes held are rescaled by the power of two between them (exact unless
 * they leave e4m3's normal range).  Infinities become the largest code, NaN
 * stays NaN.  Bytes of a block past its tokens are left as they were.  The weight of a
 * block that gets its first token is set to 0.  Tokens past max_blocks block are dropped and
 * recorded in *status, as is a length outside 0..s (clamped).
 * s = 0 does nothing.  Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_append(const shadowkv_cache* c, int dtype, const shadowkv_rows* k,
                                 const shadowkv_rows* v, int s, const int32_t* lens, void* stream);

/* Bytes of workspace shadowkv_cache_attend needs for h_q query heads on the
 * current device (0 if the arguments are not valid). */
size_t shadowkv_cache_attend_workspace(const shadowkv_cache* c, int h_q);

/*
 * Attention of one new token per sequence over the cache:
 *   out = sum_t p_t V_t,  p = softmax_t(scale q . K_t)  over the pair's tokens,
 * query head g reading KV head g / (h_q / h_kv); h_q / h_kv in {1, 2, 4, 8}.
 *   dtype : SKV_DTYPE_F32 or SKV_DTYPE_BF16, of q and out.
 *   q, out: device rows b x h_q x 1 x d (ss is not used), aligned to their elements;
 *           out may be q itself (same pointer and strides), else it does not overlap q.
 *   lse   : device f32, b x h_q: log sum_t exp(scale q . K_t), or NULL.
 *   gather, decay : with gather = 1 every block i that holds tokens gets
 *           weight[i] = decay weight[i] + sum over its tokens and the pair's query
 *           heads of p (decay = 0: the old weight is not read); needs weight.
 *   work  : device, 256-byte aligned, at least shadowkv_cache_attend_workspace bytes; its
 *           contents before and after the call mean nothing.  Calls on different
 *           streams that may run at the same time need workspaces of their own.
 * A pair without tokens gives zeros, an lse of -inf and no weight.
 * The products run on e4m3 operands: q and p are split into sums of e4m3 terms,
 * accumulated in fp32.  bf16: an entry of q exact from 2^-21 of its row's largest on and
 * to 2^-29 of that below, p times its V scale to 2^-16 of
 * itself and 2^-30 of the largest p times the largest V scale among its 128 tokens (each
 * the largest by itself: they may be different tokens'); f32: q to 2^-24 of itself and 2^-37 of
 * its row's largest entry, p to 2^-23 and 2^-38.  (A row's largest counts as 2^-92 at least.)
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_attend(const shadowkv_cache* c, int dtype, int h_q, const shadowkv_rows* q,
                                 float scale, int gather, float decay, const shadowkv_rows* out,
                                 float* lse, void* work, size_t work_bytes, void* stream);

/* Bytes of workspace shadowkv_cache_attend_tokens needs for h_q query heads and s tokens on
 * the current device (0 if the arguments are not valid). */
size_t shadowkv_cache_attend_tokens_workspace(const shadowkv_cache* c, int h_q, int s);

/*
 * Attention of several tokens per sequence over the cache: a piece of a prompt or
 * drafted tokens, whose own keys and values have been appended (causal = 1), or
 * queries over the states of an encoder (causal = 0):
 *   out_j = sum_t p_t V_t,  p = softmax_t(scale q_j . K_t)  over the tokens t that query j sees:
 *   causal = 1: t <= n_tok - lens[i] + j (the sequence's last token is query lens[i] - 1);
 *   causal = 0: all n_tok of the pair.
 * Query head g reads KV head g / (h_q / h_kv); h_q / h_kv <= 128.
 *   dtype : SKV_DTYPE_F32 or SKV_DTYPE_BF16, of q and out.
 *   q, out: device rows b x h_q x s x d, aligned to their elements (the loads are widest where
 *           pointers and strides are multiples of 16 bytes); out may be q itself (same pointer and
 *           strides), else it does not overlap q.
 *   lens  : device int32, b: queries of each sequence, 0..s (others are clamped and recorded); NULL: s
 *           each.  q is not read past them, and out and lse stay as they were there.
 *   lse   : device f32, b x h_q x s: log sum_t exp(scale q_j . K_t), or NULL.
 *   work  : device, 256-byte aligned, at least shadowkv_cache_attend_tokens_workspace bytes; its
 *           contents before and after mean nothing.  Calls that may run at the same time need
 *           workspaces of their own.
 * No block weights are gathered.  A query that sees no token gives zeros and an lse of -inf.  A key or value that is NaN reaches the
 * queries that see it and no others; a query with an entry that is not finite gives NaN.
 * The products run on fp16 operands, accumulated in fp32: codes exactly; a bf16 query exactly from 2^-31 of its row's
 * largest entry on and to 2^-39 of that below, p times its V scale to 2^-20 of itself (beside its logit's own rounding to 24
 * bits) and 2^-36 of the largest p times the largest V scale among the tokens that the query sees (each the largest by itself);
 * f32: q and p to 2^-22 of themselves, with the same floors.
 * Results do not depend on timing.
 * s h_q / h_kv <= 2^24 (SKV_ERR_UNSUPPORTED).  s = 0 does nothing.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_attend_tokens(const shadowkv_cache* c, int dtype, int h_q, int s, const shadowkv_rows* q,
                                        const int32_t* lens, int causal, float scale, const shadowkv_rows* out, float* lse,
                                        void* work, size_t work_bytes, void* stream);

/*
 * Evicts whole blocks by gathered weight.  A pair with more than `keep`
 * blocks (its last, partly filled one counts) keeps its first `sink`, its
 * last `recent`, and of the others those of largest weight (ties to the lower index, NaN
 * below everything), `keep` in all, in their order; n_tok falls accordingly.
 * The freed blocks' ids follow the kept ones in the table, so that
 * later appends reuse them; weights past the kept blocks become 0.
 * Other pairs stay as they are (their weights past the blocks held become 0).
 *   dst  : gets table, n_tok and weight; NULL or the same memory: in place.
 *          Its sizes must be src's; its pool is not used.
 *   kept : device int32, b x h_kv x keep: the old index of every block that is still held, -1 behind
 *          the last; or NULL.
 * Needs 1 <= keep <= max_blocks, sink, recent >= 0, sink + recent <= keep, and weights.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_evict(const shadowkv_cache* src, const shadowkv_cache* dst, int keep, int sink,
                                int recent, int32_t* kept, void* stream);

/* ------------------------------------------------ a pool that sequences share
 * The calls above take a table as it is.  Those below keep one over a pool that may be
 * smaller than all tables together, whose blocks several sequences may name:
 *   refs : device int32, n_pool: the table entries that name each block.  A block with
 *          refs 0 is free.
 * A table entry of -1 names no block.  An empty cache of this kind has tables of
 * -1, refs of 0 and n_tok of 0.  Every call leaves refs as the entries say; eviction in
 * place does too (an evicted block stays in its pair's table, and with it its reference, until
 * shadowkv_cache_truncate), one into another cache's tables does not.
 * Before an append, shadowkv_cache_reserve gives every pair the blocks it writes to;
 * without it an append through -1 is dropped and recorded, and one into a block that
 * others name changes theirs. */

/*
 * Forks: sequence dst[k] becomes a copy of sequence src[k] (tokens, weights) that names
 * the same blocks, k < n; no codes are moved.  What dst[k] named before is given back.
 *   src, dst : device int32, n each; n <= b.
 * All sources are read as they were before the call: a dst[k] that is any source, that an earlier
 * dst names too, or a number outside 0..b-1 leaves fork k out and is recorded in *status.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_share(const shadowkv_cache* c, int32_t* refs, int n, const int32_t* src, const int32_t* dst,
                                void* stream);

/* Bytes of workspace shadowkv_cache_reserve needs for s tokens (0 if the arguments are not valid). */
size_t shadowkv_cache_reserve_workspace(const shadowkv_cache* c, int s);

/*
 * Room for an append of s tokens per sequence (lens as there): the blocks from the one the next
 * token goes to, as far as the tokens reach, become the pair's own, a partly filled one
 * also where lens is 0.  An entry of -1, and one whose block others name too,
 * gets a free block: the lowest ones, in order of sequence, head and entry; a
 * partly filled block is copied first (codes and scales).  Blocks this call gives
 * back are free for later calls.
 *   granted : device int32, b: lens[i] (s without lens) where sequence i has its blocks, else 0:
 *          the lens to append with.  A sequence gets all its blocks or none: those of the sequences
 *          up to it, granted or not, have to be free (one that needs none is always granted).  One whose
 *          tokens would pass max_blocks block, or whose partly filled block is missing (recorded), needs
 *          none and is not granted.
 *   work  : device, 256-byte aligned, at least shadowkv_cache_reserve_workspace bytes; its contents
 *          before and after mean nothing.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_reserve(const shadowkv_cache* c, int32_t* refs, int s, const int32_t* lens, int32_t* granted,
                                  void* work, size_t work_bytes, void* stream);

/*
 * Takes tokens off the end of every sequence: n_tok = max(n_tok - drop[i], 0) for each of
 * its pairs.  Table entries past the tokens are given back and become -1, their weights 0.
 *   refs  : NULL for a cache whose pool is not shared: its tables stay as they are.
 *   drop  : device int32, b (a negative one counts as 0 and is recorded); NULL: none, which
 *           gives back what eviction and unused reservations hold.
 * A block that keeps some of its tokens stays as the others left it: with the scales that a large one of them has
 * raised (its tokens' entries are then off by up to 2^-10 of the new scale, and later tokens are held by it), and with the weight that it
 * gathered.  Drafts come off without a trace where the sequence was forked before their append: shadowkv_cache_share to a spare
 * sequence, whose partly filled block shadowkv_cache_reserve then copies, and back.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_truncate(const shadowkv_cache* c, int32_t* refs, const int32_t* drop, void* stream);

/* Bytes of workspace shadowkv_cache_compact needs (0 if the arguments are not valid). */
size_t shadowkv_cache_compact_workspace(const shadowkv_cache* src);

/*
 * Moves a cache to a pool of another size: the blocks in use (refs > 0), in order,
 * become blocks 0, 1, ... of dst's pool, and dst gets the tables (with the new numbers), counts,
 * weights (0 where src keeps none) and references.  dst's blocks behind them stay as they were; their references are 0.
 * Where dst's pool has too few blocks, dst becomes an empty cache, recorded in its status.
 * dst has src's b, h_kv, d, block and max_blocks, and memory of its own.
 *   work  : as above, of shadowkv_cache_compact_workspace bytes.
 * Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_cache_compact(const shadowkv_cache* src, const int32_t* refs, const shadowkv_cache* dst,
                                  int32_t* dst_refs, void* work, size_t work_bytes, void* stream);

/* Synchronizes the current device and reads the cache's status word;
 * SKV_ERR_DEVICE_CHECK if a kernel recorded an id, a length, a token count or a sequence out of range, or too small a pool. */
skv_status shadowkv_cache_check(const shadowkv_cache* c);

/* ------------------------------------------------ verification of drafted tokens */
typedef struct shadowkv_verify_params {
  int b, s;            /* sequences, drafted tokens of each at most */
  int vocab;           /* tokens of the vocabulary: 1..2^19 */
  int dtype;           /* SKV_DTYPE_F32 or SKV_DTYPE_BF16, of the logits */
  double temperature;  /* of every sequence, where no temperatures are given; 0: greedy */
  long long logits_sb, logits_ss;   /* strides of sequences and positions, in elements */
  long long probs_sb, probs_ss;
} shadowkv_verify_params;

/* Bytes of workspace shadowkv_verify_drafts needs (0 if the arguments are not valid). */
size_t shadowkv_verify_workspace(const shadowkv_verify_params* p);

/*
 * How many of a sequence's drafted tokens stand, and the token that follows them, such
 * that the tokens are distributed as if sampled one by one from the target (speculative sampling):
 *   p_j = softmax(logits_j / T); T = 0: 1 at the first largest logit, else 0;
 *   draft x_j stands if those before it do and accept_j q_j(x_j) < p_j(x_j);
 *   the next token is drawn from p_n if all n stand, else from max(p_a - q_a, 0), a being the
 *   first that does not (p_a, if that is 0 everywhere): the lowest v with sum_{w <= v} > sample times the total.
 *   logits : device, b x (s + 1) x vocab, the vocab elements of a row adjacent; row j follows j drafts.
 *            NaN counts as -inf, +inf as the largest float.
 *   drafts : device int32, b x s; one outside the vocabulary does not stand.
 *   probs  : device f32, b x s x vocab: q_j, the distributions the drafts were sampled from; or
 *            NULL: drafts that were not sampled (looked up): q_j is 1 at x_j.  A negative or NaN entry
 *            counts as 0 in what is left of p_a.
 *   accept, sample : device f32, b x s and b: random numbers in [0, 1).  An accept that is NaN
 *            does not stand; a sample below 0 or NaN counts as 0, one of 1 or more as the largest below 1.
 *   lens   : device int32, b: drafts of each sequence (clamped to 0..s; nothing is read past them); NULL: s each.
 *   temperatures : device f32, b, or NULL.  One below 1e-30 or NaN counts as 0, one above 1e30 as that.
 *   tokens : device int32, b x (s + 1): the drafts that stand, the next token, then -1.  A row without a
 *            logit above -inf accepts nothing and gives -1.
 *   accepted : device int32, b: drafts that stand.
 *   work   : device, 256-byte aligned, at least shadowkv_verify_workspace bytes; its contents before
 *            and after mean nothing.
 * The sampled row's weights exp((l - max) / T) are whole numbers of 2^-43, each within 2^-37 of
 * itself and 2^-44 (half a unit: a token less likely than 2^-44 times the likeliest has no weight), and their sums exact.
 * Acceptance is decided to 2^-36 + vocab 2^-44 of its border, the sampled token to as much of the total.  Results do not depend on
 * timing.  b (s + 1) <= 65535 (SKV_ERR_UNSUPPORTED).
 * b = 0 does nothing.  Asynchronous on `stream`; runs on the current device.
 */
skv_status shadowkv_verify_drafts(const shadowkv_verify_params* p, const void* logits, const int32_t* drafts,
                                  const float* probs, const float* accept, const float* sample, const int32_t* lens,
                                  const float* temperatures, int32_t* tokens, int32_t* accepted, void* work,
                                  size_t work_bytes, void* stream);

/* ------------------------------------------------------ timing / counting */
/* Kernels are numbered 0..shadowkv_num_kernels()-1 with stable names. */
int shadowkv_num_kernels(void);
const char* shadowkv_kernel_name(int id);
/* With SKV_OPT_TIMING on: total milliseconds and launch count per kernel id
 * since the last reset (arrays of n entries), of the context's own kernels.  Synchronizes.  With K/V
 * records (bf16, d = 128) the value fetch runs inside the "attention" launch
 * (or, with SKV_OPT_SPLIT_TOKENS set, inside the "rebuild" launch), and
 * "fetch" counts no launches.  The events recorded between launches
 * remove the overlap between consecutive kernels, so the per-kernel times sum
 * to more than a step takes with timing off. */
skv_status shadowkv_kernel_times(shadowkv_ctx* ctx, double* ms, long long* launches, int n);
skv_status shadowkv_reset_timers(shadowkv_ctx* ctx);

/* ---------------------------------------------------------- introspection */
enum {
  SKV_FIELD_A = 0,            /* dtype b x s x r */
  SKV_FIELD_BT = 1,           /* dtype b x h_kv x d x r  (B transposed per head) */
  SKV_FIELD_L = 2,            /* dtype b x h_kv x n x d */
  SKV_FIELD_MIN_COS = 3,      /* f32 b x h_kv x n  (prefill only) */
  SKV_FIELD_OUTLIER_IDS = 4,  /* i32 b x h_kv x o */
  SKV_FIELD_K_OUT = 5,        /* dtype b x h_kv x (o c) x d */
  SKV_FIELD_V_OUT = 6,        /* dtype b x h_kv x (o c) x d */
  SKV_FIELD_K_LOC = 7,        /* dtype b x h_kv x (w + max_new) x d */
  SKV_FIELD_V_LOC = 8,        /* dtype b x h_kv x (w + max_new) x d */
  SKV_FIELD_SEL = 9,          /* i32 b x h_kv x k: last step's chunks, ascending */
  SKV_FIELD_SEL_SLOT = 10,    /* i32 b x h_kv x k: cache slot holding each selected chunk */
  SKV_FIELD_HITS = 11,        /* i32 b x h_kv: last step's cache hits */
  SKV_FIELD_LOGITS = 12,      /* f32 b x h_q x n: last step's q.L/sqrt(d) (outliers included) */
  SKV_FIELD_K_SPARSE = 13,    /* dtype b x h_kv x (k c) x d: last step's RoPE(Gather(A,I) B) */
  SKV_FIELD_SLOT_CHUNK = 14,  /* i32 b x h_kv x k: chunk in each cache slot (-1 empty) */
  SKV_FIELD_SLOT_V = 15,      /* dtype b x h_kv x k x c x d: cached values */
  SKV_FIELD_V_CPU = 16,       /* dtype b x h_kv x s x d: the pinned host copy of V */
  SKV_FIELD_SVD_BASIS = 17,   /* f32 b x r x (h_kv d): orthonormal rows spanning the rank-r
                                 right singular subspace (prefill only) */
  SKV_FIELD_COUNT = 18
};
/* Size in bytes of a field. Host-only. */
skv_status shadowkv_field_bytes(const shadowkv_ctx* ctx, int field, size_t* bytes);
/* Copies a field to host memory dst (bytes must equal the field size).
 * Synchronizes the context's streams. */
skv_status shadowkv_export(shadowkv_ctx* ctx, int field, void* dst, size_t bytes);

#ifdef __cplusplus
}
#endif
#endif /* SHADOWKV_H */
