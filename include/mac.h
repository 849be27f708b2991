/*
 * mac.h -- C ABI of the GB300 (sm_103a) MAC-Attention decode-step library.
 *
 * MAC-Attention ("Match-Amend-Complete", arXiv 2604.00235) accelerates one
 * decode step of attention by reusing the attention summary of a recent,
 * similar query.  Per request and per query head, at decode position m:
 *
 *   Match    (paper, Figure 2(a); abstract "pre-RoPE L2 matching over a short
 *            local window"): compare the pre-RoPE query q~_m with a small
 *            ring of recent pre-RoPE queries; if the nearest one, at position
 *            p, passes an L2 threshold, fetch its attention summary
 *            AS_{1:p-r}; otherwise run full attention.
 *   Complete (Figure 2(b)): attention of the post-RoPE query q_m over the
 *            band+tail [p-r+1, m] only, merged in the log domain with the
 *            fetched AS_{1:p-r}; KV [1, p-r] is not read.
 *   Amend    (Figure 2(c), asynchronous): recompute the rectification term
 *            AS_{m-r+1:m}, obtain AS_{1:m-r} by log-domain removal from the
 *            step's AS_{1:m}, and insert <q~_m, AS_{1:m-r}> into the rings.
 *
 * An attention summary AS = (o, lse): o is the softmax-normalised attention
 * output over a token set, lse the log-sum-exp of its scaled scores.
 *
 * Conventions
 *  - Every pointer argument named dev_* is CUDA device memory on the current
 *    device; host_* pointers are host memory.
 *  - Tensors are dense, row-major, with no padding: queries and outputs
 *    [batch][heads][head_dim]; new/appended K, V [n][kv_heads][head_dim].
 *    bf16 values are IEEE bfloat16 bit patterns (uint16).  Device tensors
 *    must be 16-byte aligned (fp32 lse: 4-byte aligned).
 *  - A `stream` argument is a cudaStream_t passed as void* (NULL = the legacy
 *    default stream).  Calls marked "async" only enqueue work on it.
 *  - Request i of a batched call is request slot i of the handle.
 *  - Ownership: the caller owns every buffer it passes, including the three
 *    backing buffers handed to mac_create, which must outlive the handle.
 *    The library owns one side stream, its events and nothing else.
 *  - Errors: every call returns a mac_status; no exception or abort crosses
 *    the ABI.  A CUDA error is sticky: the handle returns MAC_ERR_CUDA from
 *    then on.  A handle is not thread-safe.
 *  - Stream capture: the step calls enqueue only kernels (and, with
 *    amend_band 1, event records and waits), so a decode loop can be
 *    captured into a CUDA graph.  Call mac_sync before beginning a capture
 *    and, with amend_band 1, mac_join on the capturing stream before ending
 *    it.  Host-side length checks run at capture time: a replayed graph
 *    advances the device state, not the checks.  Calls made after a replay
 *    must be ordered after it (same stream, or after synchronising).
 */
#ifndef MAC_H
#define MAC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mac_ctx *mac_handle;

typedef enum {
    MAC_OK = 0,
    MAC_ERR_INVALID_ARG = -1,  /* bad pointer, size, index or configuration   */
    MAC_ERR_OOM = -2,          /* a backing buffer is too small or misaligned  */
    MAC_ERR_CUDA = -3,         /* a CUDA call failed (sticky)                  */
    MAC_ERR_CAPACITY = -4,     /* KV store or page table of a request is full  */
    MAC_ERR_TIMEOUT = -5,      /* mac_sync gave up waiting                     */
    MAC_ERR_STATE = -6         /* a device-side bounds check fired (sticky)    */
} mac_status;

/* Configuration of one attention layer (one handle per layer). */
typedef struct {
    int heads;          /* query heads H                                        */
    int kv_heads;       /* KV heads H_kv; heads % kv_heads == 0 and the group   */
                        /* G = heads / kv_heads is one of 1, 2, 4, 8, 16, 32     */
    int head_dim;       /* d; must be 128                                        */
    int ring_len;       /* L: ring entries per (request, head), 1..4096; rings   */
                        /* over 32 entries are scanned by a separate grid-wide  */
                        /* kernel before Match decides                          */
    int band_r;         /* r: rectification band width in tokens, >= 1           */
    double tau;         /* L2 threshold, relative: hit iff                       */
                        /* ||q~_m - q~_e|| < tau * ||q~_m||; tau >= 0           */
    int max_batch;      /* request slots, >= 1; max_batch * kv_heads <= 1024    */
    int64_t max_ctx;    /* tokens per request, 1 .. 2^30                         */
    int page_size;      /* 0: contiguous KV per request; 16: paged KV            */
    int num_pages;      /* paged: pages in the pool (0: max_batch*ceil(max_ctx/16)) */
    float sm_scale;     /* score scale; 0 selects 1/sqrt(head_dim)               */
    int plan_mode;      /* 0: span-proportional work split (the paper's          */
                        /* load-balanced planning, Figure 3(b)); 1: equal split  */
                        /* per KV group regardless of span (unbalanced baseline) */
    int amend_band;     /* where Amend's rectification term AS_{m-r+1:m} comes   */
                        /* from: 0 = the band segment Complete already streams   */
                        /* (the band lies inside band+tail and inside [1, m]);   */
                        /* 1 = recomputed by the Amend kernel from the KV store  */
                        /* (Figure 2(c) as drawn).  Same value either way.       */
} mac_config;

/* Cumulative device counters (mac_get_stats). */
typedef struct {
    uint64_t steps;           /* mac_decode_step + mac_full_step calls          */
    uint64_t head_decisions;  /* (request, head) Match decisions               */
    uint64_t hits;            /* of which reuse the ring (hits)                 */
    uint64_t kv_tokens_read;  /* sum over (request, KV head) of tokens streamed */
    uint64_t kv_tokens_full;  /* same for full attention over [1, m]            */
    uint64_t removal_direct;  /* Amend removals too ill-conditioned for fp32    */
                              /* (1 - e^delta < 1/32), formed directly instead  */
    uint64_t work_items;      /* attention work items planned                   */
    uint32_t device_error;    /* bounds-check bits (0 = none; any set makes     */
                              /* mac_sync return MAC_ERR_STATE and the handle   */
                              /* sticky): 1 a page-table entry outside          */
                              /* the pool or a page past the table (its tokens  */
                              /* are not read; the request's output is then     */
                              /* wrong, other requests' are not touched); 2 a   */
                              /* forced slot that holds no entry (taken as a    */
                              /* miss); 4 more work                             */
                              /* items than the scratch holds; 8 a wait in the  */
                              /* tcgen05 kernel gave up (its CTA stopped early) */
    uint32_t reserved;
    uint64_t tcgen05_steps;   /* of the steps, those whose attention ran on the */
                              /* tcgen05 kernel (groups of 32 heads, steps of   */
                              /* at least 16384 KV tokens); the others ran on   */
                              /* the mma.sync kernel                            */
} mac_stats;

/* Accumulated GPU time per phase since profiling was enabled (ms). */
typedef struct {
    double match_plan_ms;     /* KV append + Match (+ the ring scan of long     */
                              /* rings)                                         */
    double attention_ms;      /* work plan + split-KV band+tail / full          */
                              /* attention kernel                               */
    double combine_ms;        /* log-domain merge kernel (with Amend's removal  */
                              /* and ring insert when amend_band is 0)          */
    double amend_ms;          /* Amend kernel (side stream, amend_band 1); 0    */
                              /* when Amend runs inside the merge kernel        */
    uint64_t steps;           /* steps timed                                    */
} mac_profile;

/* Bytes of the three backing buffers a configuration needs.  Pure host
 * arithmetic (no GPU needed).  kv: the K and V store; ring: the rings of
 * pre-RoPE queries and summaries (per request and head, L slots of bf16 q~,
 * fp32 o and fp32 lse -- 772 B per slot per query head at d = 128 -- plus
 * one int32 position per request and slot); scratch: decisions, work list,
 * partial summaries and counters.  MAC_ERR_INVALID_ARG for a bad config. */
mac_status mac_query_sizes(const mac_config *cfg, size_t *kv_bytes, size_t *ring_bytes,
                           size_t *scratch_bytes);

/* Create a handle over caller-allocated device buffers (each 256-byte
 * aligned and at least the size mac_query_sizes gives; MAC_ERR_OOM if not).
 * Zeroes the KV store; clears rings, lengths and counters; creates the side
 * stream and events.
 * Synchronous. */
mac_status mac_create(const mac_config *cfg, void *dev_kv, size_t kv_bytes, void *dev_ring,
                      size_t ring_bytes, void *dev_scratch, size_t scratch_bytes, mac_handle *out);

/* Wait for outstanding work, then release the stream and events.  The
 * backing buffers stay the caller's. */
mac_status mac_destroy(mac_handle h);

/* Paged mode: install request req's page table, n_pages int32 page indices
 * into the pool (each < num_pages), copied device-to-device.  Logical page i
 * holds tokens [16 i, 16 i + 16).  The caller's KV manager chooses the pages
 * (paper abstract: composes with paged-KV managers).  Async on stream. */
mac_status mac_set_page_table(mac_handle h, int req, const int32_t *dev_pages, int n_pages,
                              void *stream);

/* Append n_tokens tokens of post-RoPE K and of V (device bf16
 * [n_tokens][kv_heads][head_dim]) after request req's current length, e.g.
 * the prefill.  The rings are not touched.  MAC_ERR_CAPACITY if the request
 * would exceed max_ctx or its page table.  Async on stream. */
mac_status mac_append_kv(mac_handle h, int req, const void *dev_k, const void *dev_v, int64_t n_tokens,
                         void *stream);

/* One MAC decode step for requests 0..batch-1 (Figure 2 (a)->(b)->(c)):
 * appends k_new/v_new (device bf16 [batch][kv_heads][head_dim], post-RoPE)
 * at position m = length + 1, runs Match on q_pre (pre-RoPE, device bf16
 * [batch][heads][head_dim]), Complete with q_post (post-RoPE, same shape),
 * and writes out (device bf16 [batch][heads][head_dim]) and, if lse_out is
 * not NULL, the natural-log LSE of AS_{1:m} (device fp32 [batch][heads]).
 * Amend runs on the library's side stream after Complete; the next call on
 * this handle waits for it.  The inputs may be reused by later work on
 * `stream` (Amend keeps its own copies).  Async on stream. */
mac_status mac_decode_step(mac_handle h, int batch, const void *dev_q_pre, const void *dev_q_post,
                           const void *dev_k_new, const void *dev_v_new, void *dev_out, float *dev_lse_out,
                           void *stream);

/* mac_decode_step with its inputs and results in page-locked host memory
 * (cudaHostAlloc / cudaMallocHost / cudaHostRegister; same layouts and
 * alignment as above): the step's kernels read q_pre, q_post, k_new and v_new and write
 * out and lse_out in place over the host link (NVLink-C2C on Grace
 * systems), so the transfers ride inside the step's three launches instead
 * of separate copies.  The host buffers must stay untouched until the work
 * on `stream` is complete; results are valid after a stream/event sync.
 * MAC_ERR_INVALID_ARG if a buffer is not page-locked host memory the device
 * can address (pageable memory is refused, not staged).  Async on stream. */
mac_status mac_decode_step_host(mac_handle h, int batch, const void *host_q_pre, const void *host_q_post,
                                const void *host_k_new, const void *host_v_new, void *host_out,
                                float *host_lse_out, void *stream);

/* Full split-KV decode attention (the miss path for every head; no Match,
 * no ring update): append, then out = AS_{1:m}(q_post).  The in-library
 * baseline the MAC path is compared against.  Async on stream. */
mac_status mac_full_step(mac_handle h, int batch, const void *dev_q_post, const void *dev_k_new,
                         const void *dev_v_new, void *dev_out, float *dev_lse_out, void *stream);

/* Make `stream` wait (device-side) for the handle's outstanding Amend. */
mac_status mac_join(mac_handle h, void *stream);

/* Block until the outstanding Amend has finished, polling; MAC_ERR_TIMEOUT
 * after timeout_ms (< 0: wait forever).  Then checks the device bounds-check
 * word (MAC_ERR_STATE if set). */
mac_status mac_sync(mac_handle h, int timeout_ms);

/* Copy the device counters out (waits for the device first). */
mac_status mac_get_stats(mac_handle h, mac_stats *out);
mac_status mac_reset_stats(mac_handle h);

/* Seed request req's rings with n entries <q~, AS_{1:pos-r}> -- for example
 * the last prefill queries and the summaries the caller's prefill attention
 * produced -- so the first decode steps can already reuse them (the paper's
 * 512-2048-entry match windows, Figure 6 and Tables 5 and 7, reach back into
 * the prompt; the pages do not say how those entries are formed, so the
 * caller supplies them).  dev_q_pre bf16 [n][heads][head_dim] (pre-RoPE),
 * dev_o fp32 [n][heads][head_dim] (normalised output of AS_{1:pos-r}),
 * dev_lse fp32 [n][heads] (its natural-log LSE; -inf for the empty set),
 * host_pos int64 [n]: 1-based positions, strictly increasing, each <= the
 * request's length.  Entries are inserted in order exactly as decode steps
 * insert theirs (slot = step mod L, step + 1), so only the last L survive.
 * Seed before decoding (positions must grow with insertion order).
 * Synchronous (waits for stream). */
mac_status mac_seed_ring(mac_handle h, int req, int n, const void *dev_q_pre, const float *dev_o,
                         const float *dev_lse, const int64_t *host_pos, void *stream);

/* Forget request req: length 0, empty rings, step counter 0.  Async on
 * stream (after outstanding Amend). */
mac_status mac_reset_request(mac_handle h, int req, void *stream);

/* Per-phase GPU timing with CUDA events around each launch (adds event
 * records to every step; off by default).  mac_get_profile synchronises and
 * reports the totals since profiling was (re-)enabled. */
mac_status mac_set_profiling(mac_handle h, int enable);
mac_status mac_get_profile(mac_handle h, mac_profile *out);

/* ---- test hooks --------------------------------------------------------- */

/* Override the next decode step's decisions: dev_slot [batch][heads] int32,
 * -1 = miss, otherwise the ring slot to reuse (it must hold an entry, else
 * the step treats it as a miss and sets a bounds-check bit).  The Match
 * kernel still computes and records its own decision.  One-shot.  Async. */
mac_status mac_debug_force_decisions(mac_handle h, const int32_t *dev_slot, int batch, void *stream);

/* The last decode step's own Match results for requests 0..batch-1 (host
 * [batch][heads] each; NULL skips): nearest valid slot (-1 if the ring was
 * empty), its hit flag, its squared distance D and ||q~||^2 in fp32.
 * Synchronous. */
mac_status mac_debug_get_decisions(mac_handle h, int batch, int32_t *host_slot, int32_t *host_hit,
                                   float *host_D, float *host_qn2);

/* Copy request req's rings to the host (NULL skips): positions [L] (1-based,
 * 0 = empty), q~ [heads][L][head_dim] bf16 bits, o [heads][L][head_dim]
 * fp32, lse [heads][L] fp32; and its length and step counter.  Synchronous. */
mac_status mac_debug_read_ring(mac_handle h, int req, int32_t *host_pos, uint16_t *host_q, float *host_o,
                               float *host_lse, int64_t *kv_len, int64_t *steps);

/* ---- decode attention without any device allocation --------------------- */

/* No counterpart in the paper: this entry point exists for callers that may
 * not allocate device memory at the point where they run attention -- a
 * runtime that plans every byte of device memory in one arena at start-up
 * and forbids later allocations, a latency-critical loop that must not call
 * cudaMalloc (it can synchronise the device), or a plug-in host that hands
 * the library nothing but its input and output buffers.  Every handle-based
 * call above needs a scratch buffer allocated for mac_create; this one
 * needs none.
 *
 * It computes what mac_full_step computes (full split-KV decode attention,
 * out = AS_{1:len}(q) per request and query head) over a KV cache the caller
 * holds, without appending to it:
 *   dev_k, dev_v  bf16 [batch][kv_heads][ctx_stride][head_dim]; token j of
 *                 request b, KV head g starts at element
 *                 ((b * kv_heads + g) * ctx_stride + j) * head_dim
 *                 (the contiguous layout of a mac_create handle with
 *                 page_size 0, ctx_stride = max_ctx rounded up to 16)
 *   host_lens     host int32 [batch], tokens of each request, 1..ctx_stride;
 *                 slots past a request's length are never used, whatever
 *                 they hold (NaN included)
 *   dev_q         bf16 [batch][heads][head_dim], post-RoPE query
 *   dev_out       bf16 [batch][heads][head_dim]; dev_lse fp32 [batch][heads]
 *                 natural-log LSE, or NULL
 *   sm_scale      score scale, 0 selects 1/sqrt(head_dim)
 * Limits: head_dim 128, heads / kv_heads in {1, 2, 4, 8, 16, 32}, batch
 * 1..64, batch * kv_heads <= 1024, ctx_stride a multiple of 16.  Its work list and partial summaries
 * live in a fixed 16 MiB device array inside the library, which every GPU
 * that loads the library holds until the process exits; a call whose
 * scratch would exceed it returns MAC_ERR_CAPACITY and launches nothing.
 * The first call on each device looks up that array's device address and
 * the kernels' launch shapes (with that device current); make that first
 * call before any stream capture.  All calls on a device share the array
 * and overwrite it: calls whose GPU work can overlap (other streams, other
 * host threads) race and must be serialised by the caller.  Async on
 * stream; returns MAC_ERR_INVALID_ARG for bad arguments, MAC_ERR_CUDA if a
 * launch fails.  Every block index the kernels form is checked on the host
 * first (lengths within ctx_stride), so this call has no device-side error
 * to report and none is read back: MAC_OK means the work was launched. */
mac_status mac_attention_noalloc(int batch, int heads, int kv_heads, int head_dim, int64_t ctx_stride,
                                 const void *dev_k, const void *dev_v, const int32_t *host_lens,
                                 const void *dev_q, void *dev_out, float *dev_lse, float sm_scale,
                                 void *stream);

/* ---- operators around the decode step ----------------------------------- */

/* What a serving loop runs around a layer's decode attention: the QKV
 * projection's norms and rotation, the page bookkeeping of a step, and a KV
 * store of 4 bits per value with the attention over it.  None of them
 * allocates, synchronises with the host or reads anything back; all may be
 * captured into a CUDA graph, and every size that changes from step to step
 * (lengths, positions, slots, pages) is read from device memory when the work
 * runs.  Tensors they read and write must not overlap unless stated. */

/* Per-head RMS norm, rotary embedding and split of a QKV projection. */
typedef struct {
    int heads, kv_heads;   /* heads % kv_heads == 0, heads <= 1024              */
    int head_dim;          /* must be 128                                        */
    int rotary_dim;        /* r: the first r elements of a head are rotated;     */
                           /* a multiple of 8, 0..128                            */
    int interleaved;       /* pairs (i, i + r/2) (0) or (2 i, 2 i + 1) (1)       */
    float eps;             /* added to the mean of squares; >= 0                 */
    double rope_base;      /* pair i turns by pos * rope_base^(-2 i / r); >= 1   */
} mac_rope_config;

/* Made once by mac_rope_init from a configuration and kept by the caller;
 * plain host data, shared freely between calls, streams and devices. */
typedef struct {
    mac_rope_config cfg;
    uint64_t turns[64];    /* whole turns per position, as a fraction of 2^64    */
} mac_rope;

mac_status mac_rope_init(const mac_rope_config *cfg, mac_rope *out);

/* For n_tokens tokens (0: nothing is done): y = x / sqrt(mean(x^2) + eps) * w
 * for every query and key head (y = x where w is NULL), then
 *   q_pre = y, q_post = rotated y   (queries),  k_out = rotated y   (keys),
 *   v_out = the values unchanged,
 * computed in fp32 (angles in 64-bit fixed point, good to 2^-22 rad at any
 * int32 position) and rounded to bf16 once.  These are the q_pre, q_post, k_new and
 * v_new of mac_decode_step.
 *   dev_q, dev_k, dev_v  bf16, token t's heads at element t * stride (strides
 *                        in elements, multiples of 8, at least the heads'
 *                        size), so slices of one projection are read in
 *                        place; dev_v and dev_v_out may both be NULL
 *   dev_w_q, dev_w_k     bf16 [head_dim] norm weights, or NULL for no norm
 *   dev_pos              int32 [n_tokens] 0-based positions
 *   dev_q_pre, dev_q_post  bf16 [n_tokens][heads][head_dim]; q_pre may be NULL
 *   dev_k_out, dev_v_out bf16 [n_tokens][kv_heads][head_dim]
 * All bf16 pointers 16-byte aligned.  Async on stream. */
mac_status mac_qkv_norm_rope(const mac_rope *rope, int n_tokens, const void *dev_q, int64_t q_stride,
                             const void *dev_k, int64_t k_stride, const void *dev_v, int64_t v_stride,
                             const void *dev_w_q, const void *dev_w_k, const int32_t *dev_pos,
                             void *dev_q_pre, void *dev_q_post, void *dev_k_out, void *dev_v_out,
                             void *stream);

/* One serving step's page bookkeeping for `batch` requests (1..1024) over a
 * pool of num_pages 16-token pages (below 2^27): page-table entries for the
 * new tokens, the positions and slots of the packed new tokens, the new
 * lengths, and the pages of finished requests back on the free list.
 *   dev_len_in   int32 [batch] tokens a request holds
 *   dev_new      int32 [batch] its new tokens; a negative number: it is
 *                finished, its pages are freed and its length becomes 0
 *   dev_table    int32 [batch] rows of table_cols entries, table_stride apart;
 *                the entries of new pages are written, all others are left
 *   dev_ring     int32 [num_pages] ring of free page ids; entry
 *                (head + i) % num_pages, i < count, is free; freed ids are
 *                written behind the last
 *   dev_state_in int32 [2] {head, count}
 *   dev_len_out, dev_state_out   the new lengths and state (may be the same
 *                memory as the inputs)
 *   dev_starts   int32 [batch + 1]: request b's new tokens are the packed
 *                tokens starts[b] .. starts[b + 1] - 1 (at most max_tokens)
 *   dev_pos      int32 [max_tokens] 0-based position of each packed token
 *   dev_slot     int32 [max_tokens] page * 16 + offset where it is stored, or
 *                -1: it has none.  Past the last packed token: position 0,
 *                slot -1
 *   dev_status   int32 [1], written by every call: 0, or bits
 *                1  the pool has too few pages: in request order, the first
 *                   request that does not fit and every later one that needs
 *                   a page is denied
 *                2  a request would outgrow its table row: denied
 *                4  a length or the state out of range, or a page id outside
 *                   the pool met in the table or ring (its tokens get slot
 *                   -1; of a finished request that holds one, no page is
 *                   freed, so that it cannot get into the ring)
 *                8  a request's tokens would end past max_tokens: denied
 *                16 more pages released than the ring has room for: none is.
 *                   A state out of range leaves no room, either
 * A denied request keeps its length and gets no page; its packed tokens have
 * slot -1.  A length says which entries of its row a request holds, so a caller
 * must not set one back by itself (rejected drafts: mac_page_step_ex), or the
 * pages past it are lost.  max_tokens 1..2^30.  Async on stream. */
mac_status mac_page_step(int batch, int max_tokens, int num_pages, const int32_t *dev_len_in, const int32_t *dev_new,
                         int32_t *dev_len_out, int32_t *dev_table, int64_t table_stride, int table_cols,
                         int32_t *dev_ring, const int32_t *dev_state_in, int32_t *dev_state_out,
                         int32_t *dev_starts, int32_t *dev_pos, int32_t *dev_slot, int32_t *dev_status, void *stream);

/* mac_page_step with rejected drafts, and one more output.
 *   dev_rejected int32 [batch], or NULL: tokens taken back from the end of each
 *                request before its new ones, 0 .. its length (else status 4,
 *                and the request stays as it is); a finished request's does
 *                not count.  The pages that it then does not need go to the
 *                ring, those that it does need stay where they are.  A denied
 *                request keeps its length less what was taken back.  Where
 *                its pages cannot be given back (bits 4, 16) it is denied and
 *                keeps its whole length
 *   dev_unreleased  int32 [batch], or NULL: the tokens of a finished request
 *                whose pages were not freed (bits 4, 16), which are still those of
 *                its table row; 0 for every other request.  The length of a
 *                finished request becomes 0 all the same, so in a step in
 *                place nothing else says which pages it holds */
mac_status mac_page_step_ex(int batch, int max_tokens, int num_pages, const int32_t *dev_len_in, const int32_t *dev_new,
                            int32_t *dev_len_out, int32_t *dev_table, int64_t table_stride, int table_cols,
                            int32_t *dev_ring, const int32_t *dev_state_in, int32_t *dev_state_out, int32_t *dev_starts,
                            int32_t *dev_pos, int32_t *dev_slot, int32_t *dev_status, const int32_t *dev_rejected,
                            int32_t *dev_unreleased, void *stream);

/* A paged KV store of 4 bits per value, one layer per handle.  16 consecutive
 * elements x of a head share a scale s = e4m3(max|x| / 6) and are held as
 * e2m1(x / s) (both to nearest even, saturating; a block with a NaN or an
 * infinity reads back as NaN).  x is the bf16 element divided by k_scale or
 * v_scale.  144 bytes per token and KV head for K and V, against 512 in bf16. */
typedef struct mac_quant_ctx *mac_quant_handle;

typedef struct {
    int heads, kv_heads;   /* heads % kv_heads == 0, heads <= 4096               */
    int head_dim;          /* must be 128                                        */
    int page_size;         /* must be 16                                         */
    int num_pages;         /* pages in the store, 1 .. 2^27 - 1                  */
    int max_batch;         /* requests per attention call, 1..1024               */
    int max_query;         /* query tokens per request and call, >= 1;           */
                           /* heads / kv_heads * max_query <= 32                 */
    float sm_scale;        /* score scale; 0 selects 1/sqrt(head_dim)            */
    float k_scale, v_scale;/* global scales, powers of two in 2^-60 .. 2^59: the */
                           /* block scale covers max|x| from 0.006 to 2688       */
} mac_quant_config;

/* Bytes of the two backing buffers (host arithmetic).  store: the pages;
 * scratch: partial summaries of one attention call and the error word. */
mac_status mac_quant_query_sizes(const mac_quant_config *cfg, size_t *store_bytes, size_t *scratch_bytes);

/* A handle over caller-allocated device buffers (256-byte aligned, at least
 * the sizes above; MAC_ERR_OOM if not) on the current device.  Zeroes both
 * (an unwritten slot reads as zeros), but for a scratch that a live handle uses.  Synchronous.  Every call below needs
 * that device to be current (MAC_ERR_INVALID_ARG otherwise).  Calls on one
 * handle, replays of graphs captured from it among them, must be ordered
 * with one another (one stream, or events): they share the scratch.  Handles
 * (the layers of a model) whose calls are ordered may share one scratch
 * buffer, each at its start; they then share its error word too: what the
 * calls of any met is reported once, by the first to be asked. */
mac_status mac_quant_create(const mac_quant_config *cfg, void *dev_store, size_t store_bytes, void *dev_scratch,
                            size_t scratch_bytes, mac_quant_handle *out);

/* Waits for the device, then frees the handle; the buffers stay the caller's. */
mac_status mac_quant_destroy(mac_quant_handle h);

/* Store n_tokens tokens of K (post-RoPE) and V, bf16, token t's kv_heads x 128
 * elements at t * stride (elements, multiples of 8; 16-byte aligned), at
 * dev_slots[t] = page * 16 + offset; a negative slot skips its token, one past
 * the store is refused (nothing is written, mac_quant_sync reports it).  Slots
 * of one call must differ: where two tokens share one, what it holds
 * afterwards is a mix of both.  Async on stream. */
mac_status mac_quant_append(mac_quant_handle h, int n_tokens, const void *dev_k, int64_t k_stride, const void *dev_v,
                            int64_t v_stride, const int32_t *dev_slots, void *stream);

/* Read tokens back: dev_k, dev_v bf16 [n_tokens][kv_heads][128], the stored
 * values (exact in bf16; zeros for a negative or refused slot).  For a
 * prefill's own attention, or to hand a request to a bf16 store.  Async. */
mac_status mac_quant_gather(mac_quant_handle h, int n_tokens, const int32_t *dev_slots, void *dev_k, void *dev_v,
                            void *stream);

/* Decode attention of n_query query tokens for each of `batch` requests over
 * the stored tokens; query i of a request of len tokens sees the first
 * len - (n_query - 1) + i of them (its own among them: append first).
 *   dev_q      bf16 [batch][n_query][heads][128], post-RoPE
 *   dev_table  int32, request b's pages at b * table_stride, table_cols of them
 *   dev_lens   int32 [batch] tokens of each request, 0 .. 16 table_cols; a
 *              request without tokens (an idle slot) gives out 0, lse -inf
 *   dev_out    bf16 [batch][n_query][heads][128]; dev_lse fp32
 *              [batch][n_query][heads] natural-log LSE, or NULL
 * What slots past a request's length hold, NaN included, has no effect, nor
 * has what the tokens hold that a query does not see.  A query row with a NaN
 * or an infinity gives NaN (out and lse) where it sees a token.
 * Results do not depend on other requests' values, nor a row's on other heads'
 * or query tokens' queries, whatever their size; but the split of the work,
 * and with it the order of sums, depends on all lengths of the call.  A page
 * outside the store or a length outside the table is not read; the request's
 * output is then wrong and mac_quant_sync reports it.  Async on stream. */
mac_status mac_quant_attention(mac_quant_handle h, int batch, int n_query, const void *dev_q, const int32_t *dev_table,
                               int64_t table_stride, int table_cols, const int32_t *dev_lens, void *dev_out,
                               float *dev_lse, void *stream);

/* A decode step's new tokens, packed as mac_page_step leaves them, as n_query
 * rows for each of `batch` requests: row b * n_query + i is request b's i-th
 * new token.  The packed arrays hold only tokens that exist, so behind a request
 * without any (idle, finished) they and the rows of a padded batch differ.
 *   n_packed     entries of dev_pos and dev_slots
 *   dev_starts   int32 [batch + 1], mac_page_step's, or NULL: every request has
 *                n_query packed tokens (n_packed >= batch * n_query)
 *   dev_table, dev_lens  as the attention takes them, lengths after the step
 *   dev_pos_out, dev_slots_out  int32 [batch * n_query], for mac_qkv_norm_rope
 *                and mac_quant_append;  dev_lens_out  int32 [batch], for the attention
 * A request's rows count if it has exactly n_query packed tokens and their slots
 * are those that its table gives the last n_query tokens of its length.
 * Otherwise its rows get position 0 and slot -1 and its length becomes 0 (not
 * stored; out 0, lse -inf), which mac_quant_sync reports, unless it has no packed
 * token or none of them has a slot (idle, finished, denied).  Outputs must not
 * overlap the inputs.  Async on stream. */
mac_status mac_quant_step_rows(mac_quant_handle h, int batch, int n_query, int n_packed, const int32_t *dev_starts,
                               const int32_t *dev_pos, const int32_t *dev_slots, const int32_t *dev_table,
                               int64_t table_stride, int table_cols, const int32_t *dev_lens, int32_t *dev_pos_out,
                               int32_t *dev_slots_out, int32_t *dev_lens_out, void *stream);

/* Wait for the device and report what its checks met since the last call:
 * MAC_ERR_STATE (text in mac_quant_last_error), which is then cleared. */
mac_status mac_quant_sync(mac_quant_handle h);

/* Text of the handle's last error, or "" (owned by the handle). */
const char *mac_quant_last_error(mac_quant_handle h);

/* Human-readable text for a status code (static storage). */
const char *mac_status_string(mac_status s);

/* Text of the handle's sticky error, or "" (owned by the handle). */
const char *mac_last_error(mac_handle h);

#ifdef __cplusplus
}
#endif

#endif /* MAC_H */
