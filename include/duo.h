/*
 * duo.h — C ABI of libduo: mixed-head (DuoAttention) attention on B200 (sm_100a).
 *
 * The method (DuoAttention abstract, pith.science review page, "read the
 * original abstract"; sourcepulse project card, "How It Works"): each KV head
 * of each layer is either a retrieval head, which keeps a full KV cache and
 * attends causally over every previous token, or a streaming head, which keeps
 * a constant-length KV cache of the first `sink` tokens (attention sinks) plus
 * the `recent` most recent tokens, and attends only to those. In GQA models
 * every query head inherits the type of its KV head. The library covers the two
 * phases the pages speed up (pre-filling, in chunks, and decoding) and the
 * per-head cache append/eviction behind them.
 *
 * Conventions (all calls):
 *  - Tensors are bf16, row-major, contiguous, in device memory owned by the
 *    caller, 16-byte aligned (DUO_ERR_ALIGNMENT otherwise).
 *      prefill q / out   [batch][n_tok][num_q_heads][head_dim]
 *      prefill k / v     [batch][n_tok][num_kv_heads][head_dim]
 *      decode  q / out   [batch][num_q_heads][head_dim]
 *      decode  k / v     [batch][num_kv_heads][head_dim]
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Every call is stream-ordered and asynchronous; host-side cache lengths are
 *    updated when the call is enqueued. Calls on one cache must be issued on
 *    one stream (or ordered by the caller): they share the cache's device state.
 *  - Argument errors are reported before any launch and leave the cache
 *    unchanged. DUO_ERR_CUDA reports a failed launch or CUDA call.
 *  - Positions are absolute token indices within a sequence, starting at 0.
 *    Each sequence of a batch has its own cache length (duo_cache_seq_lens).
 *  - Positional encodings are the caller's: q and k arrive already encoded and
 *    cached tokens keep their original positions (no re-indexing).
 *  - Softmax scale: layout.softmax_scale, or 1/sqrt(head_dim) when it is 0.
 */
#ifndef DUO_H_
#define DUO_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DUO_API __attribute__((visibility("default")))
#else
#define DUO_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum duo_status {
    DUO_OK = 0,
    DUO_ERR_INVALID_ARG = 1, /* bad layout, mask, layer, size or null pointer */
    DUO_ERR_CAPACITY = 2,    /* a retrieval cache would exceed max_len tokens */
    DUO_ERR_ALIGNMENT = 3,   /* a pointer is not 16-byte aligned */
    DUO_ERR_CUDA = 4,        /* a CUDA call or kernel launch failed */
    DUO_ERR_STATE = 5,       /* call not valid in the cache's current state */
    DUO_ERR_DEVICE = 6,      /* a kernel reported a device-side error (see duo_cache_error) */
    DUO_ERR_SCRATCH_LIMIT = 7, /* the request needs more than DUO_STATIC_SCRATCH_BYTES */
    DUO_ERR_HOST_MEMORY = 8    /* host memory ran out */
} duo_status;

/* Storage format of the retrieval heads' caches (streaming caches are always
 * bf16). The pages reach their longest contexts only with a quantized KV cache
 * (DuoAttention abstract: 3.3 million tokens on one GPU "combined with
 * quantization"); this library offers FP8 E4M3 with one scale per (layer, KV
 * head) for K and one for V:
 *   DUO_KV_BF16  bf16 rows (default)
 *   DUO_KV_E4M3  each element is stored as the E4M3 code of x * inv_scale (the
 *                product in fp32, inv_scale the fp32 reciprocal of the head's
 *                scale), rounded to nearest with ties to even and saturated to
 *                +-448, and read back as value(code) * scale. Halves the bytes a
 *                decode step reads from retrieval caches. */
#define DUO_KV_BF16 0
#define DUO_KV_E4M3 1

/* Largest head counts the kernels accept. */
#define DUO_MAX_Q_HEADS 256
#define DUO_MAX_KV_HEADS 128

/* Largest batch whose sequences may have different lengths (a ragged batch):
 * the per-sequence lengths travel with each launch. Larger batches keep one
 * length for all sequences. */
#define DUO_MAX_RAGGED_BATCH 64

/* Shape of the model's attention and of the caches.
 *   num_layers    >= 1
 *   batch         >= 1 sequences (each with its own cache length; see
 *                 duo_cache_seq_lens)
 *   num_q_heads   query heads, a multiple of num_kv_heads (GQA group size G)
 *   num_kv_heads  KV heads; the retrieval/streaming type is per (layer, KV head)
 *   head_dim      64 or 128
 *   sink          attention-sink tokens kept by streaming heads (>= 0)
 *   recent        recent tokens kept by streaming heads (>= 1); includes the
 *                 query's own token, so a streaming query at position p attends
 *                 to { j <= p : j < sink or p - j < recent }
 *   kv_format     DUO_KV_BF16 or DUO_KV_E4M3 (retrieval caches; see above)
 *   max_len       capacity of every retrieval cache in tokens
 *   softmax_scale 0 selects 1/sqrt(head_dim) */
typedef struct duo_layout {
    int32_t num_layers;
    int32_t batch;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t sink;
    int32_t recent;
    int32_t kv_format; /* DUO_KV_BF16 or DUO_KV_E4M3: storage of the retrieval caches */
    int64_t max_len;
    float softmax_scale;
    int32_t reserved1;
} duo_layout;

/* Opaque host object: the layout, the per-layer head maps and lengths, and
 * pointers into the caller's device buffer. */
typedef struct duo_cache duo_cache;

/* duo_cache_alloc — set up the two cache kinds of DuoAttention (a full cache per
 * retrieval head, a constant-length sink + recent cache per streaming head;
 * DuoAttention abstract) inside one caller-owned device buffer.
 *   layout        shape (see duo_layout); copied
 *   is_retrieval  host array [num_layers][num_kv_heads]: 1 = retrieval, 0 = streaming
 *   dev_buf       device buffer of at least *required_bytes bytes, 256-byte
 *                 aligned; NULL to only compute *required_bytes
 *   buf_bytes     size of dev_buf
 *   required_bytes out: bytes the cache needs (always written when non-NULL)
 *   stream        stream on which the buffer is zero-filled
 *   out           out: the new cache object (when dev_buf != NULL)
 * Device layout inside dev_buf (offsets in required_bytes order):
 *   retrieval K, V pools  [n_retrieval_heads_all_layers][batch][max_len][head_dim]
 *                         (bf16, or one-byte E4M3 codes for DUO_KV_E4M3)
 *   streaming K, V pools  [n_streaming_heads_all_layers][batch][sink+recent][head_dim]
 *   streaming slot rule   position p < sink -> slot p; otherwise slot
 *                         sink + (p - sink) mod recent (fixed sinks + a ring)
 *   decode scratch        split-KV partial results: batch x R x 256 splits x
 *                         (num_q_heads / num_kv_heads) x (head_dim + 1) fp32,
 *                         R = the most retrieval KV heads of any one layer
 *                         (streaming heads write none); per-(sequence, KV head)
 *                         split counters; an error word and the prefill's
 *                         work-item counters (one 256-byte block)
 *   E4M3 scales           DUO_KV_E4M3 only: [num_layers][num_kv_heads] x 4 fp32
 *                         (k_scale, v_scale and their fp32 reciprocals), 1 until
 *                         duo_cache_set_kv_scales
 * The caller keeps ownership of dev_buf and frees it after duo_cache_free. */
DUO_API duo_status duo_cache_alloc(const duo_layout* layout, const uint8_t* is_retrieval, void* dev_buf,
                           size_t buf_bytes, size_t* required_bytes, void* stream, duo_cache** out);

/* duo_cache_free — release the host object (not the device buffer). NULL is allowed. */
DUO_API duo_status duo_cache_free(duo_cache* cache);

/* duo_cache_append — append n_tok tokens per sequence to every KV head of `layer`
 * (the per-head cache update of DuoAttention: retrieval heads keep everything,
 * streaming heads keep sinks and evict the oldest recent token).
 *   k, v   device [batch][n_tok][num_kv_heads][head_dim] bf16, the tokens at
 *          positions [len_b, len_b + n_tok) of each sequence b (its own length)
 *   n_tok  >= 0 (0 is a no-op)
 * Retrieval heads write position p to slot p. Streaming heads write sink
 * positions to their slots and only the last min(n_tok, recent) non-sink
 * positions to their ring slots (earlier ones would be evicted within the call).
 * DUO_ERR_CAPACITY if some len_b + n_tok > max_len. Then every len_b += n_tok. */
DUO_API duo_status duo_cache_append(duo_cache* cache, int32_t layer, const void* k, const void* v, int64_t n_tok,
                            void* stream);

/* duo_cache_append_ragged — append a different number of tokens to each
 * sequence of `layer` (a ragged batch: sequences of different lengths).
 *   k, v     device [batch][max_tok][num_kv_heads][head_dim]; sequence b's rows
 *            [0, n_tok[b]) are its tokens at positions [len_b, len_b + n_tok[b]),
 *            the remaining rows are not read
 *   n_tok    host [batch], 0 <= n_tok[b] <= max_tok
 * Same slot rules as duo_cache_append, per sequence. Needs batch <=
 * DUO_MAX_RAGGED_BATCH unless every sequence has the same length and
 * n_tok[b] == max_tok for all b. DUO_ERR_CAPACITY if some len_b + n_tok[b] >
 * max_len (nothing is appended). Then len_b += n_tok[b]. */
DUO_API duo_status duo_cache_append_ragged(duo_cache* cache, int32_t layer, const void* k, const void* v,
                                   const int64_t* n_tok, int64_t max_tok, void* stream);

/* duo_prefill — attention of one prefill chunk of `layer` (DuoAttention
 * pre-filling; chunked as in the chunked-prefill work the pages cite).
 *   q      device [batch][n_tok][num_q_heads][head_dim], queries at positions
 *          [len, len + n_tok) with len = duo_cache_len(layer)
 *   k, v   device [batch][n_tok][num_kv_heads][head_dim], the chunk's own tokens
 *   out    device [batch][n_tok][num_q_heads][head_dim], written
 * Retrieval heads attend causally over the cache [0, len) and the chunk;
 * streaming heads over the sinks and the recent window, read from the
 * streaming cache for positions < len and from k/v for the chunk.
 * Does NOT modify the cache: call duo_cache_append(layer, k, v, n_tok) after it.
 * DUO_KV_E4M3 caches: the tensor-core prefill reads bf16 tiles only, so a chunk
 * is refused (DUO_ERR_STATE) once a retrieval head of the layer holds tokens;
 * prefill the prompt in one chunk, then decode.
 * Each sequence's chunk starts at its own length len_b (a ragged batch needs
 * batch <= DUO_MAX_RAGGED_BATCH, else DUO_ERR_STATE).
 * DUO_ERR_CAPACITY if a retrieval head could not hold len_b + n_tok tokens. */
DUO_API duo_status duo_prefill(duo_cache* cache, int32_t layer, const void* q, const void* k, const void* v, void* out,
                       int64_t n_tok, void* stream);

/* duo_prefill_ragged — duo_prefill with a different chunk length per sequence.
 *   q, k, v, out  as duo_prefill with max_tok rows per sequence; sequence b's
 *                 rows [0, n_tok[b]) are its chunk at positions
 *                 [len_b, len_b + n_tok[b]); its other rows are not read and its
 *                 other output rows are not written
 *   n_tok         host [batch], 0 <= n_tok[b] <= max_tok
 * Follow it with duo_cache_append_ragged(layer, k, v, n_tok, max_tok). Needs
 * batch <= DUO_MAX_RAGGED_BATCH unless all lengths and counts are equal. */
DUO_API duo_status duo_prefill_ragged(duo_cache* cache, int32_t layer, const void* q, const void* k, const void* v,
                              void* out, const int64_t* n_tok, int64_t max_tok, void* stream);

/* duo_decode — one decoding step of `layer` (DuoAttention decoding).
 *   q            device [batch][num_q_heads][head_dim], sequence b's query at
 *                position len_b (its cache length)
 *   k_new, v_new device [batch][num_kv_heads][head_dim], the new tokens
 *   out          device [batch][num_q_heads][head_dim], written
 * Appends each sequence's new token to every head's cache at that sequence's
 * own length (as duo_cache_append with one token), then attends: retrieval
 * heads over positions [0, len_b], streaming heads over the sinks and the last
 * `recent` positions. Then every len_b += 1. Sequences of different lengths
 * (a ragged batch) need batch <= DUO_MAX_RAGGED_BATCH, else DUO_ERR_STATE.
 * Uses the cache's decode scratch: decode calls on one cache must not overlap
 * on the device. DUO_ERR_CAPACITY if some len_b + 1 > max_len. */
DUO_API duo_status duo_decode(duo_cache* cache, int32_t layer, const void* q, const void* k_new, const void* v_new,
                      void* out, void* stream);

/* duo_cache_len — tokens appended so far to `layer` (host value; no sync).
 * DUO_ERR_STATE if its sequences have different lengths (see
 * duo_cache_seq_lens). */
DUO_API duo_status duo_cache_len(const duo_cache* cache, int32_t layer, int64_t* len);

/* duo_cache_set_len — set the host-side length of every sequence of `layer`,
 * e.g. to restore a snapshot taken with duo_cache_len (the device contents are
 * the caller's to restore). 0 <= len <= max_len. */
DUO_API duo_status duo_cache_set_len(duo_cache* cache, int32_t layer, int64_t len);

/* duo_cache_set_kv_scales — per-KV-head scales of a DUO_KV_E4M3 cache.
 *   k_scale, v_scale  host [num_kv_heads], finite and > 0 (the entries of
 *                     streaming heads are checked but not used)
 * The scales apply to tokens appended (and decoded) afterwards: set them before
 * the layer's first append. Copies them to the device on `stream`.
 * DUO_ERR_STATE for a bf16 cache; DUO_ERR_INVALID_ARG for a bad scale (nothing
 * changes). */
DUO_API duo_status duo_cache_set_kv_scales(duo_cache* cache, int32_t layer, const float* k_scale,
                                           const float* v_scale, void* stream);

/* duo_cache_seq_lens — per-sequence lengths of `layer`.
 *   lens  host [batch], written (host values; no sync) */
DUO_API duo_status duo_cache_seq_lens(const duo_cache* cache, int32_t layer, int64_t* lens);

/* duo_cache_set_seq_lens — set the per-sequence lengths of `layer`.
 *   lens  host [batch], 0 <= lens[b] <= max_len (nothing changes otherwise) */
DUO_API duo_status duo_cache_set_seq_lens(duo_cache* cache, int32_t layer, const int64_t* lens);

/* duo_cache_views — where one KV head's cache lives, for inspection.
 *   k, v          out: device pointers to [batch][slots][head_dim] bf16
 *                 (uint8 E4M3 codes for a retrieval head of a DUO_KV_E4M3 cache)
 *   slots         out: max_len (retrieval) or sink + recent (streaming)
 *   is_retrieval  out: 1 or 0
 * Any out pointer may be NULL. */
DUO_API duo_status duo_cache_views(const duo_cache* cache, int32_t layer, int32_t kv_head, void** k, void** v,
                           int64_t* slots, int32_t* is_retrieval);

/* duo_cache_error — read and clear the device-side error word of the cache
 * (bit flags set by kernels whose bounded waits ran out: DUO_ERR_BIT_PREFILL_WAIT,
 * DUO_ERR_BIT_DECODE_COPY). Synchronizes `stream`. *flags = 0 when no kernel
 * reported an error. */
DUO_API duo_status duo_cache_error(duo_cache* cache, void* stream, uint32_t* flags);

/* duo_decode_static_scratch — duo_decode for callers that cannot allocate device
 * memory when they call in. The pages have no counterpart to this call: it is a
 * deployment variant of the decode step.
 *
 * Some callers cannot call cudaMalloc at decode time: an inference-engine
 * plugin that only gets a memory arena planned before the run, a serving loop
 * that must not let cudaMalloc/cudaFree synchronize the device, or a process
 * whose device-memory budget belongs to another allocator. This call computes
 * exactly what duo_decode computes (same arguments, same cache update, same
 * result within rounding), but keeps the split-KV partial results in one
 * file-scope device array of DUO_STATIC_SCRATCH_BYTES instead of the cache's
 * scratch region. It allocates nothing and calls no allocating routine.
 *   - Every GPU that loads libduo holds the array until the process exits.
 *   - All calls on a device share the array; it keeps the previous call's
 *     contents (the call clears what must start at zero on `stream`). Calls
 *     whose kernels overlap on the GPU race on it: issue them on one stream.
 *   - The first call on a device looks up the array's address
 *     (cudaGetSymbolAddress, device current): make it before any stream capture.
 *     The address is kept per device and context; after a device reset the
 *     first call in the new context looks it up again (also before any capture).
 *   - DUO_ERR_SCRATCH_LIMIT when even one split per (sequence, retrieval head)
 *     does not fit: batch * retrieval KV heads * G * (head_dim + 1) * 4 bytes
 *     plus batch * num_kv_heads * 4 bytes of counters must stay below the limit.
 *     Long contexts are served with fewer, longer splits when the full split
 *     plan does not fit. */
#define DUO_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)
DUO_API duo_status duo_decode_static_scratch(duo_cache* cache, int32_t layer, const void* q, const void* k_new,
                                             const void* v_new, void* out, void* stream);

/* duo_cache_test_wait_timeout — a test of the kernels' failure detection; not
 * for production use. Every wait of a kernel on an asynchronous copy is bounded
 * (1 s); when one runs out the kernel sets a bit in the cache's error word
 * (duo_cache_error), finishes without the missing data and returns, and the
 * call that launched it has already returned DUO_OK. This call arms the next
 * launch of the kinds in `launches` on this cache to exercise that path without
 * any fault: one of its CTAs does not issue one of its copies, and the wait for
 * that copy gives up after `timeout_ns` (1 us .. 1 s) instead of 1 s. Every
 * other copy is issued and waited for as usual, so nothing is left in flight.
 *   DUO_TEST_WAIT_DECODE  the next duo_decode launch: warp 0 of its first CTA
 *                         withholds its first K/V block; error bit
 *                         DUO_ERR_BIT_DECODE_COPY; that step's output is wrong,
 *                         the cache update and every later call are not affected
 *   DUO_TEST_WAIT_PREFILL the next duo_prefill launch: its first CTA withholds
 *                         its first K tile; the CTA's MMA issuer gives up, the
 *                         CTA's other roles stop at their next wait and drain
 *                         what they issued; error bit DUO_ERR_BIT_PREFILL_WAIT;
 *                         the output rows of that CTA's work items are not
 *                         written, every other item's rows are
 * 0 disarms. DUO_ERR_INVALID_ARG for an unknown kind or a limit out of range. */
#define DUO_TEST_WAIT_DECODE 1
#define DUO_TEST_WAIT_PREFILL 2
#define DUO_ERR_BIT_PREFILL_WAIT 1u  /* duo_cache_error bits */
#define DUO_ERR_BIT_DECODE_COPY 2u
DUO_API duo_status duo_cache_test_wait_timeout(duo_cache* cache, int32_t launches, uint64_t timeout_ns);

/* ------------------------------------------------------------------------
 * Paged caches: many sequences of any length over one pool of pages.
 *
 * A duo_cache holds a fixed batch of sequences, each in a contiguous region of
 * max_len tokens. A duo_paged cache holds up to max_seqs sequences that come,
 * grow, branch and go: retrieval heads keep their tokens in pages of page_size
 * rows from one pool, listed per sequence in a page table that all layers
 * share; streaming heads keep the sink + ring window of duo_cache (same slot
 * rule), one window per sequence. Which rows a query attends to is as in
 * duo_prefill and duo_decode.
 *
 * All bookkeeping (page table, lengths, reference counts) lives in device
 * memory and is updated by kernels: no call waits for the device or reads from
 * it, and duo_paged_extend, _append, _prefill and _decode, captured into a CUDA
 * graph, serve as many steps as it is replayed for.
 *
 * Conventions beyond those at the top of this file:
 *  - `seqs`, `n_tok`, `row_start`, `src` and `dst` are device arrays of int32
 *    with n entries, 0 <= n <= DUO_PAGED_MAX_BATCH (n == 0 is a no-op; row_start
 *    has n + 1). An entry of seqs outside [0, max_seqs) is padding: it is
 *    skipped, and its rows of the call's tensors are neither read nor written.
 *  - One sequence may stand only once in a call's `seqs` (or `dst`); entries
 *    that name it twice are all skipped and DUO_ERR_BIT_PAGED_ARGUMENT is set.
 *  - What only the device can see (lengths, page numbers, duplicate entries, a
 *    pool without enough free pages) is checked there: the call does not do
 *    what it cannot do, as each call says, and sets bits in the cache's error
 *    word (duo_paged_error). No page number is used before it is checked.
 *  - Tensors are packed rows: token (or batch entry) r of q starts at
 *    q + r * q_stride elements, its heads are contiguous; k and v share
 *    kv_stride. A stride of 0 means dense (heads * head_dim); others are
 *    multiples of 8 elements, at least dense and at most 2^31 - 1. */
#define DUO_PAGED_MAX_SEQS 4096   /* sequences of one cache */
#define DUO_PAGED_MAX_BATCH 512   /* entries of one call */
#define DUO_PAGED_MAX_GROUP 8     /* query heads per KV head: 1 .. 8, any number */
#define DUO_PAGED_MAX_PAGES (1 << 20)  /* pages of one pool */

/* Shape of a paged cache. As duo_layout, except
 *   max_seqs    sequences the cache can hold
 *   page_size   tokens per page: 16, 32, 64 or 128
 *   num_pages   pages in the pool (>= 1)
 *   max_pages   pages of one sequence at most (the row length of the page table);
 *               max_pages x page_size <= 2^27
 *   num_q_heads num_kv_heads x (1 .. DUO_PAGED_MAX_GROUP) */
typedef struct duo_paged_layout {
    int32_t num_layers;
    int32_t max_seqs;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t sink;
    int32_t recent;
    int32_t kv_format; /* DUO_KV_BF16 or DUO_KV_E4M3: storage of the pages */
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages;
    float softmax_scale;
} duo_paged_layout;

/* Bytes of the device buffers of a paged cache (duo_paged_size). */
typedef struct duo_paged_sizes {
    size_t pages;      /* each of k_pages, v_pages */
    size_t windows;    /* each of k_window, v_window */
    size_t page_table;
    size_t seq_len;
    size_t page_ref;
    size_t workspace;
} duo_paged_sizes;

/* The device buffers, owned by the caller, 256-byte aligned; a buffer of size 0
 * may be NULL. An empty cache has seq_len and page_ref all zero; the contents of
 * the others do not matter until they are written.
 *   k_pages, v_pages    [num_pages][R][page_size][head_dim], R = retrieval heads
 *                       of all layers, layer by layer in head order
 *                       (bf16, or one-byte E4M3 codes)
 *   k_window, v_window  [max_seqs][S][sink + recent][head_dim] bf16, S =
 *                       streaming heads of all layers, layer by layer
 *   page_table          int32 [max_seqs][max_pages]; the first
 *                       ceil(seq_len / page_size) entries of a row count
 *   seq_len             int32 [max_seqs], tokens of each sequence
 *   page_ref            int32 [num_pages], table entries that name the page
 *                       (0: the page is free)
 *   workspace           scratch of the calls, the error word and the E4M3 scales */
typedef struct duo_paged_buffers {
    void* k_pages;
    void* v_pages;
    void* k_window;
    void* v_window;
    int32_t* page_table;
    int32_t* seq_len;
    int32_t* page_ref;
    void* workspace;
} duo_paged_buffers;

/* Opaque host object: the layout, the head maps and the buffers' addresses. */
typedef struct duo_paged duo_paged;

/* duo_paged_size — bytes of each buffer (no device work). */
DUO_API duo_status duo_paged_size(const duo_paged_layout* layout, const uint8_t* is_retrieval, duo_paged_sizes* sizes);

/* duo_paged_alloc — a paged cache over the caller's buffers, on the current
 * device. Clears the workspace on `stream` (E4M3 scales become 1) and leaves the
 * other buffers as they are: they may already hold sequences. The caller frees
 * the buffers after duo_paged_free. */
DUO_API duo_status duo_paged_alloc(const duo_paged_layout* layout, const uint8_t* is_retrieval,
                                   const duo_paged_buffers* buffers, void* stream, duo_paged** out);

/* duo_paged_free — release the host object (not the buffers). NULL is allowed. */
DUO_API duo_status duo_paged_free(duo_paged* cache);

/* duo_paged_set_kv_scales — as duo_cache_set_kv_scales, for a paged cache. */
DUO_API duo_status duo_paged_set_kv_scales(duo_paged* cache, int32_t layer, const float* k_scale,
                                           const float* v_scale, void* stream);

/* duo_paged_extend — give sequence seqs[i] n_tok[i] more tokens (1 each when
 * n_tok is NULL): once per step, before the layers' calls. The new tokens are
 * the last n_tok[i] positions of the sequence; their rows are written by
 * duo_paged_append or duo_paged_decode, layer by layer.
 * Pages are taken lowest number first, entry by entry; a last page that is only
 * partly full and shared with other sequences (duo_paged_fork) is first replaced
 * by a copy (all layers; when all its sharers are extended in one call, the last
 * of them keeps the page). All or nothing: nothing changes and
 * DUO_ERR_BIT_PAGED_CAPACITY is set when a sequence would need more than
 * max_pages pages or the pool has too few free ones, DUO_ERR_BIT_PAGED_ARGUMENT
 * for a negative n_tok, a sequence named twice or a length or page number out of
 * range. */
DUO_API duo_status duo_paged_extend(duo_paged* cache, int32_t n, const int32_t* seqs, const int32_t* n_tok,
                                    void* stream);

/* duo_paged_append — write `layer`'s rows of the newest tokens of n sequences:
 * packed rows [row_start[i], row_start[i+1]) of k and v are the last tokens of
 * sequence seqs[i], in order (duo_paged_extend comes first). n_rows: rows of the
 * k and v tensors; rows outside every range are not read. Slots as in
 * duo_cache_append. An entry whose range is not within [0, n_rows], is longer
 * than the sequence or runs backwards is skipped (DUO_ERR_BIT_PAGED_ARGUMENT;
 * ranges behind it may then overlap others, and a call whose ranges hold more than
 * 2^30 tokens in all appends nothing); a row that would go into a page shared with another sequence is not written
 * (DUO_ERR_BIT_PAGED_SHARED: it would change that sequence too). */
DUO_API duo_status duo_paged_append(duo_paged* cache, int32_t layer, int32_t n, const int32_t* seqs,
                                    const int32_t* row_start, const void* k, const void* v, int64_t n_rows,
                                    int64_t kv_stride, void* stream);

/* duo_paged_prefill — attention of n whole prompts of `layer`, packed one behind
 * the other: rows [row_start[i], row_start[i+1]) of q, k, v and out are prompt
 * i, positions 0 .. ; each query attends within its own prompt (all of it up to
 * itself in retrieval heads, sinks and window in streaming heads). Rows of
 * another prompt or outside every range have no effect on it, whatever they
 * hold, and out rows outside every range are not written. An empty prompt is
 * allowed. Neither reads nor changes the cache (duo_paged_append stores the
 * rows). n_rows: rows of the tensors, below 2^30;
 * an entry whose range is not within [0, n_rows] or runs backwards is skipped
 * (DUO_ERR_BIT_PAGED_ARGUMENT). */
DUO_API duo_status duo_paged_prefill(duo_paged* cache, int32_t layer, int32_t n, const int32_t* row_start,
                                     const void* q, const void* k, const void* v, void* out, int64_t n_rows,
                                     int64_t q_stride, int64_t kv_stride, int64_t out_stride, void* stream);

/* duo_paged_decode — one decoding step of `layer` for n sequences: row i of
 * k_new and v_new is the last token of sequence seqs[i] (duo_paged_extend comes
 * first), at position len - 1; it is written into the sequence's page and
 * windows, and row i of q attends to the cache with it, as in duo_decode. Row i
 * of `out` is zero for an empty sequence. A last page that is shared is not
 * written (DUO_ERR_BIT_PAGED_SHARED); the row's own attention still sees the new
 * token. */
DUO_API duo_status duo_paged_decode(duo_paged* cache, int32_t layer, int32_t n, const int32_t* seqs, const void* q,
                                    const void* k_new, const void* v_new, void* out, int64_t q_stride,
                                    int64_t kv_stride, int64_t out_stride, void* stream);

/* duo_paged_fork — sequence dst[i], which must be empty, becomes sequence src[i]:
 * it shares all its pages and gets a copy of its windows (all layers). One
 * source may be forked many times in a call; a dst that stands among the src
 * entries, is not empty or is named twice is skipped
 * (DUO_ERR_BIT_PAGED_ARGUMENT). Fork between steps: not between duo_paged_extend
 * and the layers' calls that write the new rows. */
DUO_API duo_status duo_paged_fork(duo_paged* cache, int32_t n, const int32_t* src, const int32_t* dst, void* stream);

/* duo_paged_copy — as duo_paged_fork, but dst[i] gets pages of its own (lowest
 * free numbers first, entry by entry) with copies of the rows. Nothing is copied
 * for any entry when the pool has too few free pages
 * (DUO_ERR_BIT_PAGED_CAPACITY). */
DUO_API duo_status duo_paged_copy(duo_paged* cache, int32_t n, const int32_t* src, const int32_t* dst, void* stream);

/* duo_paged_release — sequences seqs[i] become empty; pages no other sequence
 * names are free again. */
DUO_API duo_status duo_paged_release(duo_paged* cache, int32_t n, const int32_t* seqs, void* stream);

/* duo_paged_compact — move pages so that the ones in use are the lowest numbers:
 * with u pages in use, those at number u and above go, in ascending order, to
 * the free numbers below u in ascending order; the page table follows. */
DUO_API duo_status duo_paged_compact(duo_paged* cache, void* stream);

/* duo_paged_error — read and clear the cache's error word. Synchronizes `stream`
 * (not during a capture). */
#define DUO_ERR_BIT_PAGED_ARGUMENT 4u  /* duo_paged_error bits: an entry, length or page number out of range */
#define DUO_ERR_BIT_PAGED_CAPACITY 8u  /* too few free pages, or more than max_pages for a sequence */
#define DUO_ERR_BIT_PAGED_SHARED 16u   /* a write to a shared page was left out */
#define DUO_ERR_BIT_PAGED_WAIT 32u     /* a bounded wait of a kernel ran out: the outputs since then are not
                                        * valid, and a new duo_paged over the same buffers is needed, with
                                        * which the step's prefill and decode calls can be made again */
DUO_API duo_status duo_paged_error(duo_paged* cache, void* stream, uint32_t* flags);

/* duo_paged_test_wait_timeout — as duo_cache_test_wait_timeout, for the next
 * duo_paged_decode (DUO_TEST_WAIT_DECODE) or duo_paged_prefill
 * (DUO_TEST_WAIT_PREFILL) launch that has work: its first CTA issues no K and V
 * tile, and the waits for them run out after the usual second. Error bit
 * DUO_ERR_BIT_PAGED_WAIT; the outputs of that CTA's share (decode), or of its
 * first work item (prefill), are wrong or not written, all others are right.
 * 0 disarms. DUO_ERR_INVALID_ARG for an unknown kind. */
DUO_API duo_status duo_paged_test_wait_timeout(duo_paged* cache, int32_t launches);

/* duo_status_str — static description of a status code. */
DUO_API const char* duo_status_str(duo_status status);

#ifdef __cplusplus
}
#endif

#endif /* DUO_H_ */
