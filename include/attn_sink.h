/*
 * attn_sink.h -- C ABI of a GB300 (sm_103a) library for attention with an
 * attention sink.
 *
 * Two forms of the sink are implemented:
 *
 *  1. A learnable per-head sink logit (flash-attention PR "feat: Implement Sink
 *     Attention", Description; sglang PR "openai oss attention sink support
 *     with trtllm-gen backend", Summary of Changes).  For query head h the
 *     value sink[h] is one extra logit that enters the softmax denominator and
 *     carries no value vector:
 *         m_i   = max(sink[h], max_j s_ij)
 *         Z_i   = exp(sink[h] - m_i) + sum_j exp(s_ij - m_i)
 *         O_i   = sum_j exp(s_ij - m_i) v_j / Z_i
 *         LSE_i = m_i + ln Z_i
 *     with s_ij = scale * q_i . k_j over the keys j that row i sees.  sink is
 *     in the units of the scaled logits.  sink == NULL means "no sink"
 *     (sink = -inf, i.e. plain softmax attention).
 *
 *  2. First-window + last-window KV selection over a paged KV cache (sglang PR
 *     "To implement attention-sink", Motivation and the review's suggested
 *     code: keep the first 1024 and the last 7168 tokens of every sequence).
 *     A query at absolute position p sees the keys
 *         [0, min(F, p+1))  U  [max(p+1-W, min(F, p+1)), p+1)
 *     where F = win_first and W = win_last.  win_last <= 0 turns selection
 *     off (plain causal).  The window is applied per sequence, token-exactly;
 *     partial pages are masked per token.  Selection needs causal attention.
 *
 * Conventions shared by every entry point:
 *  - Tensors are device pointers owned by the caller; the library keeps no
 *    pointer after it returns.  Layouts are dense row-major as documented.
 *  - bf16 tensors hold raw IEEE bfloat16 bits (attn_bf16).
 *  - Work is queued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and is asynchronous: a zero return means "validated and
 *    launched", not "finished".
 *  - Query row t of a request with Lq queries and Lk keys sits at absolute
 *    position Lk - Lq + t (bottom-right alignment: a cached prefix precedes
 *    the new chunk).  A row that sees no key has O = 0 and LSE = sink (or
 *    -inf without a sink); its gradients are 0.
 *  - scale <= 0 selects 1/sqrt(head_dim).
 *  - Scratch memory (split-KV partials, the fp32 dQ accumulator) is taken
 *    from a library-owned stream-ordered pool on `stream` and returned on
 *    the same stream; no call synchronises the host.
 *  - Return values: ATTN_SINK_OK, or a negative status.  The text of the
 *    last failure of the calling thread is available from
 *    attn_sink_last_error().
 *  - Out-of-range page ids and sequence lengths longer than the page table
 *    are caught on the device: the offending load is skipped and a sticky
 *    device status is set, which attn_sink_device_status() reports.
 *  - One call takes at most 65535 requests (batch) in the forward, paged
 *    forward, decode, append, tree, compaction, eviction, verification and page entry points,
 *    and at most 65535 * 128 query
 *    rows per request in the forward ones (each is one grid dimension of the
 *    launch); larger calls return ATTN_SINK_ERR_UNSUPPORTED.
 */
#ifndef ATTN_SINK_H
#define ATTN_SINK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t attn_bf16;

enum {
    ATTN_SINK_OK = 0,
    ATTN_SINK_ERR_INVALID = -1,      /* NULL pointer, negative size, bad flag combination */
    ATTN_SINK_ERR_UNSUPPORTED = -2,  /* head_dim, group size, page_size or a size limit   */
    ATTN_SINK_ERR_CUDA = -3,         /* a CUDA call failed (allocation, launch)            */
    ATTN_SINK_ERR_DEVICE = -4        /* a device-side check failed (see device_status)     */
};

/* Device-side status bits reported by attn_sink_device_status(). */
enum {
    ATTN_SINK_DEV_PAGE_OOB = 1,      /* a page-table entry was outside [0, num_pages)       */
    ATTN_SINK_DEV_SEQLEN_OOB = 2,    /* a sequence length exceeded max_pages * page_size    */
    ATTN_SINK_DEV_TIMEOUT = 4,       /* a pipeline wait ran out of time; the kernel gave up */
    ATTN_SINK_DEV_LAYOUT = 8,        /* the dynamic shared-memory base was not 1024-byte
                                        aligned; the forward kernel did nothing            */
    ATTN_SINK_DEV_ORDER = 16,        /* attn_sink_kv_compact: a source token that is not after
                                        the one before it, or lies before its destination  */
    ATTN_SINK_DEV_TREE = 32,         /* attn_sink_tree_paged: a parent outside [-1, own index);
                                        attn_sink_verify_draft: outside [0, own index)     */
    ATTN_SINK_DEV_VALUE = 64,        /* attn_sink_kv_append_q8: an infinity or NaN was replaced */
    ATTN_SINK_DEV_PROB = 128,        /* attn_sink_verify_draft: a drafted token outside the
                                        vocabulary, or a row without any probability       */
    ATTN_SINK_DEV_POOL = 256         /* attn_sink_pages_*: too few free pages, or a table,
                                        lengths and counts that contradict each other      */
};

/*
 * Forward attention with a sink over varlen requests (prefill, chunked
 * extend, training forward).  Pages: flash-attention PR "feat: Implement Sink
 * Attention" (Key Changes: forward functions and their variable-length
 * counterparts take the sink); sglang PR "openai oss attention sink support with trtllm-gen backend" (Highlights: the extend path
 * passes sink=).
 *
 *   q            (total_q, hq, head_dim) bf16, total_q = cu_seqlens_q[batch]
 *   k, v         (total_k, hkv, head_dim) bf16; request b owns key rows
 *                [cu_seqlens_k[b], cu_seqlens_k[b+1]) (cached prefix then chunk)
 *   sink         (hq,) fp32 or NULL
 *   cu_seqlens_q, cu_seqlens_k   (batch+1,) int32 device, non-decreasing, [0]=0
 *   total_q, total_k             host row counts of q and k/v (the tensors'
 *                first extents); cu_seqlens_*[batch] must not exceed them --
 *                rows past them are never read or written and set
 *                ATTN_SINK_DEV_SEQLEN_OOB
 *   max_seqlen_q, max_seqlen_k   host upper bounds of the per-request lengths
 *                (size the grid; no device-to-host read)
 *   win_first, win_last          window selection (needs causal = 1)
 *   out          (total_q, hq, head_dim) bf16
 *   lse          (hq, total_q) fp32, natural log, includes the sink; may be NULL
 * Supported: head_dim 64 or 128; hq % hkv == 0.  A request's results depend on its
 * own rows only: the value rows that its last key tile covers past its last
 * key (another request's, or beyond cu_seqlens_k[batch]) are replaced by zeros
 * in shared memory, so they may hold anything, NaN included.
 * Input range: the online softmax exponentiates each tile against a running
 * reference that may lag the true row maximum by up to a factor 2^64, so the
 * un-normalised weights reach 2^64 and the fp32 accumulator of P V stays
 * finite while max|v| * Lk < 1.8e19 (|v| < 1.7e13 at a million keys); an
 * exact softmax would stay finite for any finite value.
 */
int attn_sink_fwd(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v,
                  const float* sink, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                  int batch, int total_q, int total_k, int hq, int hkv, int head_dim,
                  int max_seqlen_q, int max_seqlen_k,
                  int win_first, int win_last, int causal, float scale,
                  attn_bf16* out, float* lse, void* stream);

/*
 * attn_sink_fwd with explicit row strides, for packed layouts (the varlen
 * forward functions of flash-attention PR "feat: Implement Sink Attention",
 * Key Changes, come in packed-QKV and packed-KV forms).  q_row_stride,
 * k_row_stride, v_row_stride are the distances in elements between
 * consecutive token rows of q, k and v (0: contiguous, heads * head_dim).
 * Within a row the heads stay contiguous, head_dim elements apart.  A packed
 * (total, hq + 2*hkv, head_dim) QKV buffer is q = base, k = base + hq*head_dim,
 * v = base + (hq+hkv)*head_dim, all with row stride (hq + 2*hkv)*head_dim.
 * Strides must be 0 or >= heads*head_dim and multiples of 8; out stays
 * contiguous.  Everything else as in attn_sink_fwd.
 */
int attn_sink_fwd_strided(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v,
                          long long q_row_stride, long long k_row_stride, long long v_row_stride,
                          const float* sink, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                          int batch, int total_q, int total_k, int hq, int hkv, int head_dim,
                          int max_seqlen_q, int max_seqlen_k,
                          int win_first, int win_last, int causal, float scale,
                          attn_bf16* out, float* lse, void* stream);

/*
 * Paged single-token decode with a sink and optional first/last-window
 * selection.  Pages: sglang PR "openai oss attention sink support with trtllm-gen backend" (Highlights: the decode path passes
 * sink=); sglang PR "To implement attention-sink" (page table rows built from the first and last
 * windows, per sequence); flash-attention PR "feat: Implement Sink Attention" (a user reports the sink
 * giving wrong decode results through the KV-cache API -- here the sink is
 * folded exactly once, after the split-KV partials are merged).
 *
 *   q            (batch, hq, head_dim) bf16, one new token per request
 *   k_cache, v_cache  (num_pages, page_size, hkv, head_dim) bf16
 *   page_table   (batch, max_pages) int32 physical page ids; logical token t
 *                of request b lives in page page_table[b][t / page_size],
 *                row t % page_size.  Entries past a request's last page are
 *                never read.
 *   seqlens      (batch,) int32: cache length including the new token
 *   sink         (hq,) fp32 or NULL
 *   out          (batch, hq, head_dim) bf16
 *   lse          (batch, hq) fp32 or NULL
 * Supported: head_dim 64 or 128; hq % hkv == 0; page_size >= 1.
 */
int attn_sink_decode_paged(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                           const int32_t* page_table, int max_pages, const int32_t* seqlens,
                           int batch, int hq, int hkv, int head_dim, int page_size, int num_pages,
                           const float* sink, int win_first, int win_last, float scale,
                           attn_bf16* out, float* lse, void* stream);

/*
 * Allocation-free paged decode.  The paper has no counterpart: this entry
 * point exists for callers that cannot allocate device memory at call time
 * (an engine that reserved the whole GPU up front, a latency-critical path
 * that must not take the allocator's locks or its implicit synchronisation,
 * a host that only hands the library existing buffers).
 *
 * Same arguments, semantics and results as attn_sink_decode_paged (up to
 * rounding when it has to use longer splits), but its split-KV scratch lives
 * in one static 32 MiB device array inside the library instead of coming
 * from a memory pool.  It calls no cudaMalloc, cudaFree or other allocating
 * routine.
 *  - The array is shared by every call on a device and keeps the previous
 *    call's contents; every scratch entry a call reads is written earlier in
 *    the same call, so nothing needs clearing.  Calls whose work overlaps on
 *    the GPU (e.g. on two streams without ordering between them) race on the
 *    array: order them on one stream or with events.
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress) and caches it; make that first call before any
 *    stream capture.
 *  - A GPU holds the 32 MiB from the moment the library's module is loaded
 *    on it until the process exits.
 *  - Requests whose partials cannot fit in 32 MiB even with one split per
 *    (request, head) -- batch * hq * (head_dim * 4 + 8) bytes -- are
 *    rejected with ATTN_SINK_ERR_UNSUPPORTED and a message naming the size.
 */
int attn_sink_decode_paged_noalloc(const attn_bf16* q, const attn_bf16* k_cache,
                                   const attn_bf16* v_cache, const int32_t* page_table,
                                   int max_pages, const int32_t* seqlens, int batch, int hq,
                                   int hkv, int head_dim, int page_size, int num_pages,
                                   const float* sink, int win_first, int win_last, float scale,
                                   attn_bf16* out, float* lse, void* stream);

/*
 * Writes new tokens' K/V rows into a paged cache (the cache update that
 * precedes attention in KV-cache decode: flash-attention PR "feat: Implement
 * Sink Attention", Description; a request's tokens are reached through its
 * page-table row: sglang PR "To implement attention-sink", suggested code).
 *
 *   k_new, v_new   (rows, hkv, head_dim) bf16; request b's new rows are
 *                  [cu_new[b], cu_new[b+1]), or row b alone when cu_new is NULL
 *   cu_new         (batch+1,) int32 device or NULL (then max_new must be 1)
 *   seqlens        (batch,) int32 device: cache length INCLUDING the new rows,
 *                  so request b's n_b new rows become its logical tokens
 *                  seqlens[b] - n_b .. seqlens[b] - 1
 *   page_table     (batch, max_pages) int32 device, as in attn_sink_decode_paged
 *   max_new        host upper bound of n_b (sizes the grid); a request with more
 *                  new rows than max_new has its extra rows left unwritten and
 *                  sets ATTN_SINK_DEV_SEQLEN_OOB
 *   k_cache, v_cache   (num_pages, page_size, hkv, head_dim) bf16, written in place
 * A row whose slot would fall outside the cache (page id outside
 * [0, num_pages), or more new rows than cached tokens) is skipped and sets
 * ATTN_SINK_DEV_PAGE_OOB / ATTN_SINK_DEV_SEQLEN_OOB.  Rows of different
 * requests must not share a slot (the write order between them is undefined).
 * Supported: head_dim 64 or 128.
 */
int attn_sink_kv_append(const attn_bf16* k_new, const attn_bf16* v_new, const int32_t* cu_new,
                        const int32_t* seqlens, const int32_t* page_table, int max_pages, int batch,
                        int hkv, int head_dim, int page_size, int num_pages, int max_new,
                        attn_bf16* k_cache, attn_bf16* v_cache, void* stream);

/*
 * Paged decode with the new token's K/V appended in the same call: writes
 * k_new[b], v_new[b] ((batch, hkv, head_dim) bf16) at logical token
 * seqlens[b] - 1 of each request, then runs attn_sink_decode_paged on the
 * updated caches (KV-cache decode with a sink: flash-attention PR "feat:
 * Implement Sink Attention", Description).  Every other argument as in
 * attn_sink_decode_paged; k_cache / v_cache are written.  The call makes no
 * host synchronisation and depends only on its arguments, so it can be
 * captured in a CUDA graph (its scratch comes from a stream-ordered pool).
 */
int attn_sink_decode_paged_append(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new,
                                  attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table,
                                  int max_pages, const int32_t* seqlens, int batch, int hq, int hkv,
                                  int head_dim, int page_size, int num_pages, const float* sink,
                                  int win_first, int win_last, float scale, attn_bf16* out,
                                  float* lse, void* stream);

/*
 * attn_sink_fwd on HOST-resident tensors: the library copies each request's
 * q / k / v rows to the device, runs the forward for that request and copies
 * its out / lse rows back, pipelined on library-owned streams so that the copies
 * of neighbouring requests overlap the kernel (same arithmetic and results as
 * attn_sink_fwd).  All tensor arguments, cu_seqlens_q and cu_seqlens_k
 * included, are host pointers; the layouts are those of attn_sink_fwd and the
 * row counts come from cu_seqlens_*[batch].  Host buffers should be
 * page-locked (cudaHostAlloc / cudaHostRegister) for the copies to overlap;
 * pageable buffers still give correct results, without overlap.  Returns once
 * the work is queued; `stream` waits for all of it (synchronise `stream`
 * before reading out / lse).  Device scratch for the whole batch comes from the
 * library's stream-ordered pool.  Supported: head_dim 64 or 128; hq % hkv == 0.
 */
int attn_sink_fwd_host(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v,
                       const float* sink, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                       int batch, int hq, int hkv, int head_dim, int win_first, int win_last,
                       int causal, float scale, attn_bf16* out, float* lse, void* stream);

/*
 * Varlen extend / prefill whose keys and values live in a paged cache (the
 * serving extend path: sglang PR "openai oss attention sink support with
 * trtllm-gen backend", Highlights: the extend path passes sink=; the prefix is
 * reached through the page table: sglang PR "To implement attention-sink",
 * suggested code).  Request b's query rows [cu_seqlens_q[b], cu_seqlens_q[b+1])
 * are the LAST Lq_b of its seqlens_k[b] cached tokens (bottom-right causal
 * alignment, as in attn_sink_fwd).
 *
 *   q            (total_q, hq, 64) bf16
 *   k_new, v_new (total_q, hkv, 64) bf16, the chunk's own K/V, or both NULL.
 *                When given they are first appended into the cache at the
 *                chunk's positions (attn_sink_kv_append with cu_new =
 *                cu_seqlens_q); when NULL the cache must already hold them.
 *   k_cache, v_cache  (num_pages, page_size, hkv, 64) bf16
 *   page_table   (batch, max_pages) int32 device
 *   seqlens_k    (batch,) int32 device, prefix + chunk
 *   max_seqlen_q, max_seqlen_k   host upper bounds (grid sizing, append grid)
 *   sink, win_first, win_last, causal, scale, out, lse: as in attn_sink_fwd
 * Supported: head_dim 64 or 128; hq % hkv == 0; page_size a power of two >= 8
 * (a 128-key tile is then one TMA copy per page segment).  Cache slots that a
 * request does not own (the rest of its last page, any other page) never
 * reach its results and may hold anything, NaN included.
 */
int attn_sink_fwd_paged(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new,
                        attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table,
                        int max_pages, const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                        int batch, int total_q, int hq, int hkv, int head_dim, int page_size,
                        int num_pages, int max_seqlen_q, int max_seqlen_k, const float* sink,
                        int win_first, int win_last, int causal, float scale, attn_bf16* out,
                        float* lse, void* stream);

/*
 * Backward of attn_sink_fwd: gradients of sum(dout * out) with respect to q,
 * k, v and the sink.  Page: flash-attention PR "feat: Implement Sink Attention" (Key Changes: the
 * backward pass computes and returns the gradient of the learnable sink).
 * dsink[h] = -sum_i exp(sink[h] - LSE_i) * rowsum(dout_i * out_i).
 *
 *   q, k, v, sink, cu_seqlens_*, sizes, windows, causal, scale: as in attn_sink_fwd
 *   out, lse     the forward's outputs (lse is required here)
 *   dout         (total_q, hq, head_dim) bf16
 *   dq           (total_q, hq, head_dim) bf16
 *   dk, dv       (total_k, hkv, head_dim) bf16 (summed over the query heads
 *                of each KV head)
 *   dsink        (hq,) fp32; must be non-NULL iff sink is non-NULL; written
 *                (not accumulated)
 * Supported: head_dim 64 or 128 (one pass each: 128-row query steps at 64,
 * 64-row steps at 128); hq % hkv == 0.  A request's gradients depend on
 * its own rows only: the rows that its last query or key tile covers past its
 * own (another request's, or past total_q / total_k) are replaced by zeros in
 * shared memory, so they may hold anything, NaN included.
 */
int attn_sink_bwd(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, const float* sink,
                  const attn_bf16* out, const float* lse, const attn_bf16* dout,
                  const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                  int batch, int total_q, int total_k, int hq, int hkv, int head_dim,
                  int max_seqlen_q, int max_seqlen_k,
                  int win_first, int win_last, int causal, float scale,
                  attn_bf16* dq, attn_bf16* dk, attn_bf16* dv, float* dsink, void* stream);

/*
 * attn_sink_bwd with explicit row strides for q, k, v (inputs) and dq, dk, dv
 * (outputs), for packed QKV / KV layouts (as in attn_sink_fwd_strided; a packed
 * dQKV output uses the same offsets and stride as the packed QKV input).  out,
 * lse and dout stay contiguous.  With any of the dk / dv strides non-zero, dk/dv
 * rows past cu_seqlens_k[batch] are left untouched (instead of zeroed).
 */
int attn_sink_bwd_strided(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v,
                          long long q_row_stride, long long k_row_stride, long long v_row_stride,
                          const float* sink, const attn_bf16* out, const float* lse,
                          const attn_bf16* dout, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int batch, int total_q, int total_k, int hq,
                          int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
                          int win_first, int win_last, int causal, float scale,
                          attn_bf16* dq, attn_bf16* dk, attn_bf16* dv,
                          long long dq_row_stride, long long dk_row_stride, long long dv_row_stride,
                          float* dsink, void* stream);

/*
 * Rotary positions.  Pair i of a head's first rotary_dim dimensions -- elements
 * i and i + rotary_dim/2, or 2i and 2i + 1 when interleaved != 0 -- becomes
 *     (x cos a - y sin a, y cos a + x sin a) * attn_scale,
 *     a = positions[row] * inv_freq[i]   (-a when inverse != 0),
 * and dimensions rotary_dim .. head_dim - 1 are copied bit for bit.  The gradient
 * of the rotation is the same call with inverse = 1.  The angle of any int32 position
 * (negative ones included) is off by at most 1e-7 + |position| inv_freq 2^-52 radians.
 *
 *   q, q_out     (rows, hq, head_dim) bf16; q_out may be q
 *   k, k_out     (rows, hkv, head_dim) bf16, or both NULL (then hkv is ignored);
 *                k_out may be k
 *   *_row_stride distances in elements between consecutive rows (0: contiguous);
 *                0 or >= heads * head_dim, multiples of 8
 *   positions    (rows,) int32 device
 *   inv_freq     (rotary_dim / 2,) fp64 device, radians per position
 * An output may be its own input (same pointer and stride); any other overlap
 * of outputs with inputs or each other gives undefined values.
 * Supported: head_dim 64 or 128; rotary_dim even, 2 .. head_dim; at most 16384
 * heads (hq + hkv).
 */
int attn_sink_rope(const attn_bf16* q, attn_bf16* q_out, const attn_bf16* k, attn_bf16* k_out,
                   long long q_row_stride, long long q_out_row_stride, long long k_row_stride,
                   long long k_out_row_stride, const int32_t* positions, const double* inv_freq, int rows,
                   int hq, int hkv, int head_dim, int rotary_dim, int interleaved, int inverse,
                   float attn_scale, void* stream);

/*
 * attn_sink_rope on new tokens' queries and keys, with the rotated keys and the
 * values written into a paged cache in the same launch (attn_sink_kv_append's
 * slots, checks and status bits).
 *
 *   q, q_out        (total_new, hq, head_dim) bf16; q_out may be q
 *   k_new, v_new    (total_new, hkv, head_dim) bf16
 *   cu_new          (batch+1,) int32 device, or NULL: request b's one new row is row b
 *   positions       (total_new,) int32 device, or NULL: the row's logical token.
 *                   (Drafted trees pass prefix + depth.)
 *   total_new       host row count of q, k_new and v_new; cu_new[batch] must not
 *                   exceed it (rows past it are left alone, ATTN_SINK_DEV_SEQLEN_OOB)
 * Rows of q_out behind the last request's are left as they were.  Everything
 * else as in attn_sink_rope (forward rotation) and attn_sink_kv_append.
 * Supported: head_dim 64 or 128; at most 16384 heads (hq + 2 hkv), 65535 requests.
 */
int attn_sink_rope_kv_append(const attn_bf16* q, attn_bf16* q_out, const attn_bf16* k_new,
                             const attn_bf16* v_new, long long q_row_stride, long long q_out_row_stride,
                             long long k_row_stride, long long v_row_stride, const int32_t* cu_new,
                             const int32_t* positions, const double* inv_freq, const int32_t* seqlens,
                             const int32_t* page_table, int max_pages, int batch, int total_new, int hq,
                             int hkv, int head_dim, int rotary_dim, int page_size, int num_pages,
                             int max_new, int interleaved, float attn_scale, attn_bf16* k_cache,
                             attn_bf16* v_cache, void* stream);

/*
 * Attention of a tree of drafted tokens over a paged cache (the check of a
 * speculative draft).  Request b's rows [cu_seqlens_q[b], cu_seqlens_q[b+1]) are
 * its n nodes, in the order of the last n of its seqlens_k[b] cached tokens
 * (their K/V are in the cache already: attn_sink_kv_append or
 * attn_sink_rope_kv_append).  Node i hangs on node parents[row i] of the same
 * request, an earlier one, or on the prefix (the other P = seqlens_k[b] - n
 * tokens) when that is -1.  Nodes on the prefix have depth 0, others one more
 * than their parent; node i stands at position P + depth and sees the prefix,
 * its ancestors and itself, each by the first/last-window rule on positions.
 *
 *   q            (total_q, hq, head_dim) bf16
 *   parents      (total_q,) int32 device, each in [-1, own index in the request);
 *                any other value is read as -1 and sets ATTN_SINK_DEV_TREE
 *   max_seqlen_q host upper bound of n, at most 256.  Rows of a request past it
 *                are left alone and set ATTN_SINK_DEV_SEQLEN_OOB.
 *   max_seqlen_k host bound of seqlens_k, as attn_sink_fwd_paged takes it; at present
 *                only checked (>= 0): the keys are split by the lengths on the device
 *   out          (total_q, hq, head_dim) bf16
 *   lse          (hq, total_q) fp32, as in attn_sink_fwd; may be NULL
 * A request with fewer cached tokens than nodes sees no key (out 0, lse the
 * sink) and sets ATTN_SINK_DEV_SEQLEN_OOB.  Keys read through an out-of-range
 * page id take no weight.  Rows of out and lse behind the last request's are
 * left as they were.  Cache slots that a request does not own never reach its results,
 * and a cached token's infinities and NaNs only the nodes that see it.
 * As in every attention call here, scores, sums and lse are fp32, and the weights are
 * rounded to bf16 where they meet V (out is off by at most 2^-8 of sum p |v| for it).
 * Supported: head_dim 64 or 128; hq % hkv == 0, hq / hkv <= 128; page_size a
 * power of two >= 8.  No gradient.
 */
int attn_sink_tree_paged(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                         const int32_t* page_table, int max_pages, const int32_t* cu_seqlens_q,
                         const int32_t* seqlens_k, const int32_t* parents, int batch, int total_q, int hq,
                         int hkv, int head_dim, int page_size, int num_pages, int max_seqlen_q,
                         int max_seqlen_k, const float* sink, int win_first, int win_last, float scale,
                         attn_bf16* out, float* lse, void* stream);

/*
 * Moves cached rows of each request down in its token order: for j < counts[b],
 * token src[b][h][j] of request b becomes its token base[b] + j, in K and V, for
 * KV head h (src_heads == hkv) or for all heads (src_heads == 1).  With base the
 * prefix's length and src an accepted path's tokens, the drafted rows that were
 * accepted follow the prefix.
 *
 *   src      (batch, src_heads, max_rows) int32 device: increasing tokens,
 *            src[j] >= base + j; a row that breaks this sets ATTN_SINK_DEV_ORDER and
 *            is skipped, and the rows after it of its list may hold either value
 *   counts   (batch,) int32 device, at most max_rows
 *   base     (batch,) int32 device, or NULL: 0
 * In place and safe for any such src: a row is read before it is overwritten.
 * Pages that two requests share must not be written by either.  k_cache and
 * v_cache must be different tensors.  Supported: head_dim 64 or 128.
 */
int attn_sink_kv_compact(attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                         const int32_t* src, const int32_t* counts, const int32_t* base, int batch,
                         int src_heads, int max_rows, int hkv, int head_dim, int page_size, int num_pages,
                         void* stream);

/*
 * attn_sink_decode_paged that also accumulates the attention weight of every
 * cached token:
 *     weights[b][h][t] += sum_{g in h} exp(s_gt - LSE_g)
 * over the query heads g of KV head h (weight_heads == hkv) or over all query
 * heads (weight_heads == 1), for the visible tokens t of request b, from fp32 scores
 * and sums (only where they meet V are the weights rounded to bf16).  A token's
 * weights of one call and query head sum to 1 less the sink's share.
 *
 *   weights  (batch, weight_heads, weight_cap) fp32 device, updated in place; the
 *            caller sets new tokens' entries to 0 before their first call.  Tokens
 *            t >= weight_cap are left out and set ATTN_SINK_DEV_SEQLEN_OOB.
 * The sums have a fixed order (no atomics).  Scratch for scores: 4 bytes per query head
 * (those of a KV head rounded up to 1, 2, 4, 8 or a multiple of 16), request and token
 * that has an accumulator and that the page table can hold (or the window can show); at
 * most 2 GiB at a time, or one request's: batches that need more are taken in rounds of
 * requests.  (The lengths are on the device: a table much wider than they are costs
 * scratch and time, unless attn_sink_decode_paged_weights_bounded is told the longest.)
 * Everything else as in attn_sink_decode_paged; hq at most 4096, and with
 * weight_heads == 1 at most 6144 query heads, those of a KV head rounded up to 8 or a
 * multiple of 16.
 */
int attn_sink_decode_paged_weights(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                                   const int32_t* page_table, int max_pages, const int32_t* seqlens,
                                   int batch, int hq, int hkv, int head_dim, int page_size, int num_pages,
                                   const float* sink, int win_first, int win_last, float scale,
                                   float* weights, int weight_heads, int weight_cap, attn_bf16* out,
                                   float* lse, void* stream);

/*
 * attn_sink_decode_paged_weights with a host bound of seqlens, max_seqlen >= 0.  Launches
 * and scratch are sized by it instead of by the page table, which may be much wider
 * than the requests are long; lengths past it are cut there (ATTN_SINK_DEV_SEQLEN_OOB).
 */
int attn_sink_decode_paged_weights_bounded(const attn_bf16* q, const attn_bf16* k_cache,
                                           const attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                                           const int32_t* seqlens, int batch, int hq, int hkv, int head_dim,
                                           int page_size, int num_pages, int max_seqlen, const float* sink,
                                           int win_first, int win_last, float scale, float* weights,
                                           int weight_heads, int weight_cap, attn_bf16* out, float* lse,
                                           void* stream);

/*
 * Eviction by accumulated weight.  A request with more than `budget` cached
 * tokens keeps its first keep_first, its last keep_last and, of the others, the
 * budget - keep_first - keep_last of largest weight (equal weights, +0 and -0
 * among them: the earlier token; NaN below every number); the kept tokens become
 * its tokens 0 .. budget - 1, in their order.  Each KV head keeps tokens of its
 * own (weight_heads == hkv) or all heads the same ones (weight_heads == 1).
 * Requests of at most `budget` tokens keep everything.
 *
 *   k_cache, v_cache  moved in place (different tensors; a page that two requests
 *                share must not be written by either)
 *   weights      (batch, weight_heads, weight_cap) fp32; lengths past weight_cap are
 *                cut there (ATTN_SINK_DEV_SEQLEN_OOB)
 *   weights_out  the same shape, or weights itself: the kept tokens' weights,
 *                then 0 up to weight_cap
 *   kept         (batch, weight_heads, budget) int32: the kept tokens, increasing,
 *                then -1
 *   new_seqlens  (batch,) int32: min(length, budget); must not be seqlens
 * Supported: head_dim 64 or 128; 1 <= budget, 0 <= keep_first, keep_last,
 * keep_first + keep_last <= budget; at most 21845 weight heads, 65535 requests.
 */
int attn_sink_evict_paged(attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                          const int32_t* seqlens, const float* weights, int batch, int weight_heads,
                          int weight_cap, int hkv, int head_dim, int page_size, int num_pages, int budget,
                          int keep_first, int keep_last, float* weights_out, int32_t* kept,
                          int32_t* new_seqlens, void* stream);

/* Formats of an 8-bit cache and types of probabilities. */
enum { ATTN_SINK_E4M3 = 0, ATTN_SINK_INT8 = 1 };
enum { ATTN_SINK_F32 = 0, ATTN_SINK_BF16 = 1, ATTN_SINK_F16 = 2 };

/*
 * The 8-bit paged cache.  k_cache and v_cache are (num_pages, page_size, hkv, head_dim)
 * codes, e4m3 or int8; k_scale and v_scale are (num_pages, page_size / block, hkv) fp32,
 * one scale for `block` tokens of a KV head.  block divides page_size.  A code c stands for
 * c * scale.
 *
 * attn_sink_kv_append_q8 writes new K/V rows into it (attn_sink_kv_append's slots, checks
 * and status bits).  For every block of tokens that receives rows, and each KV head of K
 * and of V, with qmax = 448 (e4m3) or 127 (int8):
 *   - needed = the least power of two s >= 2^-64 with max|x| <= qmax s over the new rows;
 *   - scale = needed where the block's first token is new, else max(old scale, needed);
 *   - codes = x / scale, rounded to nearest, ties to even.  If the scale grew, the codes of
 *     the tokens that the block has are scaled down by the quotient and rounded again.
 * Infinities become the largest code of their sign, NaN 0; both set
 * ATTN_SINK_DEV_VALUE and do not count for the scale.  Codes behind the last token of a
 * block are left as they were, and are rewritten with the block's scale when they are appended.
 * Pages that two requests share must not be written by either (attn_sink_pages_reserve copies
 * them).
 *
 *   k_new, v_new    (total_new, hkv, head_dim) bf16; *_row_stride as in attn_sink_rope
 *   cu_new          (batch+1,) int32 device, or NULL: request b's one new row is row b
 *   seqlens         (batch,) int32 device, the new rows included
 *   total_new       host row count of k_new and v_new; rows past it are left out
 *   max_new         host upper bound of the new rows of a request; rows past it are left out
 * Supported: head_dim 64 or 128; any page size.
 */
int attn_sink_kv_append_q8(const attn_bf16* k_new, const attn_bf16* v_new, long long k_row_stride,
                           long long v_row_stride, const int32_t* cu_new, const int32_t* seqlens,
                           const int32_t* page_table, int max_pages, int batch, int total_new, int hkv,
                           int head_dim, int page_size, int num_pages, int max_new, int block, int format,
                           void* k_cache, void* v_cache, float* k_scale, float* v_scale, void* stream);

/*
 * attn_sink_decode_paged over the 8-bit cache.  Scales may be any positive numbers up to 2^122
 * (those of V count as at least 2^-64), not only the powers of two that the append writes; the codes
 * of a request's tokens have to be numbers (the append writes no NaN).  The products are
 * fp16 with fp32 accumulation, in which both formats are exact: q enters them off by at
 * most 2^-25 of its row's largest magnitude, a weight times its V scale by at most 2^-11 of
 * itself or 2^-32 of the row's largest such product, whichever is more; scores, sums and lse are
 * fp32.  Where V's scales of the tokens that a row sees are more than 2^100 apart, tokens
 * of the small ones may be missing from the denominator and lse too.
 *
 *   max_seqlen  host bound of seqlens (INT_MAX: none); sizes launches and scratch.  Lengths
 *               past it are cut there (ATTN_SINK_DEV_SEQLEN_OOB)
 *   lse         (batch, hq) fp32; may be NULL
 * Supported: head_dim 64 or 128; hq % hkv == 0; any page size.
 */
int attn_sink_decode_paged_q8(const attn_bf16* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, int block, int format,
                              const int32_t* page_table, int max_pages, const int32_t* seqlens, int batch,
                              int hq, int hkv, int head_dim, int page_size, int num_pages, int max_seqlen,
                              const float* sink, int win_first, int win_last, float scale, attn_bf16* out,
                              float* lse, void* stream);

/*
 * attn_sink_fwd_paged over the 8-bit cache (which has the chunk's tokens already:
 * attn_sink_kv_append_q8).  Few rows (max_seqlen_q * hq / hkv small: drafts in a row) are
 * computed from the codes as in attn_sink_decode_paged_q8.  For more, the visible tokens
 * are expanded to bf16 (exactly, where the scales are powers of two, as the append writes them;
 * else rounded to it) in scratch of 4 hkv head_dim bytes per request and token
 * of max_seqlen_k, at most 2 GiB at a time (or one request's; larger batches in rounds of
 * requests), and read by the kernel of attn_sink_tree_paged (as a chain) or of
 * attn_sink_fwd_paged, with their rounding of the weights to bf16 (2^-8).  Position i of a
 * request's n rows is seqlens_k - n + i; rows before position 0 see nothing.  What rows that see
 * a token behind an out-of-range page id get is not defined; nothing outside the cache is read.
 *   max_seqlen_q  host upper bound of a request's rows.  A request with more sets
 *                 ATTN_SINK_DEV_SEQLEN_OOB; its rows up to the bound keep their positions, those past
 *                 it are left as they were or computed
 *   max_seqlen_k  host upper bound of seqlens_k, which must hold (it sizes scratch and launches;
 *                 no memory behind the page table or the scratch is read where it does not)
 *   lse           (hq, total_q) fp32; may be NULL
 * Supported: head_dim 64 or 128; hq % hkv == 0; any page size.
 */
int attn_sink_fwd_paged_q8(const attn_bf16* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale, int block, int format,
                           const int32_t* page_table, int max_pages, const int32_t* cu_seqlens_q,
                           const int32_t* seqlens_k, int batch, int total_q, int hq, int hkv, int head_dim,
                           int page_size, int num_pages, int max_seqlen_q, int max_seqlen_k, const float* sink,
                           int win_first, int win_last, int causal, float scale, attn_bf16* out, float* lse,
                           void* stream);

/*
 * Verification of drafted tokens by given random numbers.  Request b's rows [cu[b], cu[b+1])
 * are its nodes: node 0 is its last token, which stands; the others are drafted, each hangs
 * on an earlier one, its parent.  p_i and q_i are the target's and the draft model's
 * probabilities of the token that follows node i.  From node 0 on, the children of the node
 * reached are tested in their order; child number r, with token x and random number u, is
 * taken if
 *     u q_i(x) Z_r < max(p_i(x) - S_r q_i(x), 0),      S_0 = 0, Z_0 = 1,
 * and refused otherwise, with
 *     S_{r+1} = S_r + Z_r,   Z_{r+1} = sum_y max(p_i(y) - S_{r+1} q_i(y), 0).
 * With draft == NULL it is taken if u Z_r < p_i(x) with Z_r = 1 less p_i of the refused
 * siblings' tokens (each token once; a token that was refused is refused again).  Where no
 * child is taken (or there is none), the next token is the least x with
 *     sum_{y <= x} w(y) > u_next sum_y w(y),
 * w(y) = max(p_i(y) - S q_i(y), 0), or p_i without the refused tokens; p_i itself where that
 * leaves nothing.  The tokens are distributed as the target's where siblings are drawn
 * independently from q_i (draft given) or are chosen without regard to the random numbers.
 * Probabilities count as clamped to [0, 1] (NaN: 0) and enter sums as multiples of 2^-44;
 * u_next is clamped to [0, 1) (NaN: 0); a negative u counts as 0 (NaN: refused).
 *
 *   target, draft  (total, vocab) of type dtype (ATTN_SINK_F32, BF16 or F16); row i of a
 *                  request: after its node i.  *_row_stride in elements (0: vocab)
 *   tokens         (total,) int32; node 0's is not read.  One outside the vocabulary is refused
 *                  and sets ATTN_SINK_DEV_PROB
 *   parents        (total,) int32, or NULL: each node hangs on the one before it.  Node 0's is
 *                  not looked at; another's must be in [0, own index), else the node is left out
 *                  and sets ATTN_SINK_DEV_TREE
 *   u, u_next      (total,) and (batch,) fp32; node 0's u is not used
 *   base           (batch,) int32, or NULL: 0
 *   max_nodes      host upper bound of a request's nodes, at most 256; further ones are left out
 *                  and set ATTN_SINK_DEV_SEQLEN_OOB
 *   src            (batch, max_nodes) int32: base[b] + index of the nodes that stand, node 0
 *                  first, then -1 (attn_sink_kv_compact's src, with base the prefix's length)
 *   counts         (batch,) int32: how many stand (0 for a request without nodes)
 *   next_tokens    (batch,) int32: the next token; -1 for a request without nodes, and where
 *                  the row has no probability at all (ATTN_SINK_DEV_PROB)
 * Deterministic.  Supported: vocab below 2^20.
 */
int attn_sink_verify_draft(const void* target, const void* draft, long long target_row_stride,
                           long long draft_row_stride, int dtype, const int32_t* tokens,
                           const int32_t* parents, const int32_t* cu_seqlens, const float* u,
                           const float* u_next, const int32_t* base, int batch, int total, int max_nodes,
                           int vocab, int32_t* src, int32_t* counts, int32_t* next_tokens, void* stream);

/*
 * Bookkeeping of a paged cache's pages.  refs (num_pages,) int32 device counts, for every
 * page, the page-table entries that hold it (0: the page is free).  A request of L tokens holds
 * the first ceil(L / page_size) entries of its row.  `pools` is a host array of num_pools (at
 * most 8) device tensors whose pages move together (K, V, their scales), tensor i with
 * page_bytes[i] bytes a page; any alignment, fastest where both are multiples of 16.  All
 * results are the same in every run.  Entries outside [0, num_pages) set
 * ATTN_SINK_DEV_PAGE_OOB, lengths below 0 or above max_pages * page_size
 * ATTN_SINK_DEV_SEQLEN_OOB; what contradicts the counts sets ATTN_SINK_DEV_POOL.
 *
 * attn_sink_pages_copy: page src[i] of every tensor to page dst[i], i < n (device arrays;
 * -1 for both: no copy).  No page may be written twice, or be written and read.
 */
int attn_sink_pages_copy(void* const* pools, const long long* page_bytes, int num_pools, int num_pages,
                         const int32_t* src, const int32_t* dst, int n, void* stream);

/*
 * Row b of the new table (out_batch rows) is row src[b] of the old one (-1: a row without
 * tokens), with its length; refs follow: the old rows' entries are given up, the new ones'
 * are held.  Nothing else is copied: a row that then grows into a page that it shares calls
 * attn_sink_pages_reserve first.  Entries behind a row's pages are -1.  out_table and
 * out_seqlens must not be the inputs.  An old length below 0 counts as 0 (the row gives a new
 * one without tokens, and its own pages stay counted), one above the row as the whole row; a
 * src outside [-1, batch) counts as -1.
 */
int attn_sink_pages_fork(const int32_t* page_table, int32_t* refs, const int32_t* seqlens,
                         const int32_t* src, int batch, int out_batch, int max_pages, int page_size,
                         int num_pages, int32_t* out_table, int32_t* out_seqlens, void* stream);

/*
 * Gives back the pages of requests that shrink from seqlens[b] to new_seqlens[b] tokens (0: all
 * of them): their entries become -1.  A new length above the old one (ATTN_SINK_DEV_POOL), and a
 * new or old one out of range, change nothing.
 */
int attn_sink_pages_release(int32_t* page_table, int32_t* refs, const int32_t* seqlens,
                            const int32_t* new_seqlens, int batch, int max_pages, int page_size, int num_pages,
                            void* stream);

/*
 * Gives requests that grow from seqlens[b] to new_seqlens[b] tokens their pages, so that tokens
 * seqlens[b] .. new_seqlens[b] - 1 can be written: free pages, lowest first, to the requests in
 * order.  A request whose first new token goes into a page that others hold too gets a copy of
 * it (in all tensors) instead, before its new pages; of several such requests of one page the
 * last keeps the page, where they are all its holders.
 *   missing  (1,) int32: 0, or the pages that are too few; then nothing is changed
 *            (ATTN_SINK_DEV_POOL)
 * A request whose lengths are out of range or fall is left alone.
 */
int attn_sink_pages_reserve(void* const* pools, const long long* page_bytes, int num_pools,
                            int32_t* page_table, int32_t* refs, const int32_t* seqlens,
                            const int32_t* new_seqlens, int batch, int max_pages, int page_size, int num_pages,
                            int32_t* missing, void* stream);

/*
 * Brings the n held pages to the front: the i-th held page behind the first n goes to the i-th
 * free page among them, in all tensors, in the rows' entries and in refs.  The pages from n on are
 * free then.  Every entry that holds a page has to be in the given table: a page that is only
 * counted moves too, and who else remembers its number loses it.  In a row whose length is out of
 * range every entry that names a page follows it.
 *   held     (1,) int32: n
 */
int attn_sink_pages_compact(void* const* pools, const long long* page_bytes, int num_pools,
                            int32_t* page_table, int32_t* refs, const int32_t* seqlens, int batch,
                            int max_pages, int page_size, int num_pages, int32_t* held, void* stream);

/*
 * The visible token ranges of each decode request, as the decode kernels
 * compute them on the device (sglang PR "To implement attention-sink", suggested code: first window
 * [:F] and last window [L-W:L], per sequence).
 *   seqlens  (batch,) int32 device
 *   ranges   (batch, 4) int32 device: a0, b0, a1, b1 with visible =
 *            [a0,b0) U [a1,b1), disjoint and increasing.
 */
int attn_sink_visible_ranges(const int32_t* seqlens, int batch, int win_first, int win_last,
                             int32_t* ranges, void* stream);

/*
 * The physical KV slot of every visible token, in the order the decode
 * kernels read them: slot = page_table[b][t / page_size] * page_size
 * + t % page_size for the visible logical tokens t of request b.
 *   slots    (batch, max_visible) int32 device; row b holds the request's
 *            visible slots followed by -1 padding (and -1 where a page id
 *            is outside [0, num_pages), which also sets
 *            ATTN_SINK_DEV_PAGE_OOB).  max_visible must be at least the
 *            largest visible count.
 */
int attn_sink_visible_slots(const int32_t* seqlens, const int32_t* page_table, int max_pages,
                            int batch, int page_size, int num_pages, int win_first, int win_last,
                            int32_t* slots, int max_visible, void* stream);

/*
 * Reads and clears the sticky device status (a bitwise OR of the
 * ATTN_SINK_DEV_* bits set by kernels since the last call) for the current
 * device.  Synchronises `stream`.  Returns the bits, or ATTN_SINK_ERR_CUDA.
 */
int attn_sink_device_status(void* stream);

/*
 * Self-test of the bounded wait behind every pipeline barrier of the kernels
 * (no counterpart on the pages: it is how a stalled pipeline is detected).
 * Launches one single-thread kernel on `stream` that waits on an mbarrier of
 * its own.  complete != 0: the barrier's phase is completed first and the wait
 * returns at once (no status).  complete == 0: nothing arrives, the wait gives
 * up after its time limit (1 s), sets ATTN_SINK_DEV_TIMEOUT and the kernel
 * returns; the context stays usable.  Asynchronous; returns ATTN_SINK_OK or
 * ATTN_SINK_ERR_CUDA (launch failure).
 */
int attn_sink_selftest_wait(int complete, void* stream);

/* Text of the calling thread's last failure ("" if none).  Never NULL. */
const char* attn_sink_last_error(void);

/* Library version string. */
const char* attn_sink_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_SINK_H */
