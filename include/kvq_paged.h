/*
 * kvq_paged.h — C ABI of the paged KV cache (GB300, sm_103a): rows written to pages at given
 * slots (16-bit, or quantised as they are written), read back, and read by the attention of one
 * new token or of a chunk of new tokens per sequence; and the norm and rotation that queries and
 * keys go through before. It stands beside kvq.h: kvq_cache keeps one slot of fixed regions per
 * sequence and its lengths on the host; here sequences share a pool of pages through a page
 * table, and table, lengths and slots are device arrays, so a captured step can be replayed with
 * other sequences and lengths.
 *
 * Conventions are those of kvq.h (status codes, plain device pointers, caller-owned memory, work
 * enqueued on the given stream, no allocation), and:
 *  - Alignment: pools 256 bytes; value rows, cos_sin and workspaces 16 bytes; int32 arrays, slopes and
 *    lse 4 bytes.
 *  - `dtype` is KVQ_F16 or KVQ_BF16: the type of the call's q, k, v and out (kv_paged_read also
 *    takes KVQ_PAGED_F32).
 *  - Strides count elements between tokens; a token's heads are contiguous ([heads][head_dim]).
 *    Strides are multiples of 8 and at least one token's elements; q may be a slice of a wider
 *    projection output.
 *  - What only the device knows is checked there and reported by kv_paged_get_status (bits below):
 *    an index out of range is skipped, never followed.
 *  - Calls on one handle may run on several streams at once as long as they do not write pages that
 *    another one reads, and do not share a workspace.
 *  - A call refused on the host (any status but KVQ_OK) has enqueued nothing.
 */
#ifndef KVQ_PAGED_H
#define KVQ_PAGED_H

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { KVQ_PAGED_F32 = 100 };   /* dtype of kv_paged_read: fp32 rows */

/* Bits of the status word (kv_paged_get_status). */
enum {
    KVQ_PAGED_NONFINITE = 1,    /* a quantised block had a non-finite scale (the page holds it) */
    KVQ_PAGED_TIMEOUT = 2,      /* a bounded device wait ran out; that launch's outputs are invalid */
    KVQ_PAGED_BAD_INDEX = 4,    /* a slot or a page number was out of range: a write was skipped, a page read as zeros */
    KVQ_PAGED_BAD_LENGTH = 8,   /* a length, row offset or max_q was out of range: lengths are cut to what the page
                                   table holds, rows beyond the call's buffers or max_q are skipped */
    KVQ_PAGED_RANGE = 16        /* a quantised block reaches beyond fp16's 65,504: the page holds it and kv_paged_read
                                   gives it, the attentions cut its scale (kv_paged_decode_attn) */
};

typedef struct {
    int32_t n_layers;
    int32_t n_kv_heads;
    int32_t head_dim;       /* 64, 128 or 256 */
    int32_t n_q_heads;      /* a multiple of n_kv_heads, with n_q_heads / n_kv_heads <= 16 */
    int32_t page_size;      /* positions per page: 16, 32, 64, 128 or 256 */
    int32_t n_pages;        /* pages per layer (one page table serves all layers); n_pages x page_size < 2^31 */
    int32_t k_fmt;          /* KVQ_F16, KVQ_BF16, KVQ_Q8_0 or KVQ_Q4_0 */
    int32_t v_fmt;          /* equal to k_fmt, or KVQ_Q4_0 beside KVQ_Q8_0 keys */
    float softmax_scale;    /* 0 selects 1/sqrt(head_dim) */
    int32_t reserved;
} kvq_paged_config;

typedef struct kvq_paged kvq_paged;   /* opaque host-side handle */

/* Options of the two attention calls; a null pointer in their place means none. Applied in this
 * order to the score s = scale <q, k_j> of the query at position i and position j:
 *   softcap > 0:  s = softcap * tanh(s / softcap)          (1e-30 to 2e38)
 *   slopes:       s = s - slopes[query head] * |i - j|        (device fp32 [n_q_heads])
 *   visibility:   j <= i, and j > i - window when window > 0; positions j < prefix[sequence] are
 *                 visible to every query, behind the window and after it too (device int32 [n_seq])
 * A query that sees no position gives zeros and lse = -inf; a NaN among the scores it sees gives NaN in both.
 *   lse:          device fp32 [query rows][n_q_heads], the log of the sum of exp(s) (may be null) */
typedef struct {
    float softcap;
    int32_t window;
    const float* slopes;
    const int32_t* prefix;
    float* lse;
} kvq_attn_opts;

/* kv_paged_required_bytes — pool bytes of a config, and workspace bytes of attention calls with up
 * to max_seqs sequences and (kv_paged_prefill_attn) max_tokens query rows in all. Host pointers
 * out; either may be null. KVQ_EINVAL on a bad config. */
kvq_status kv_paged_required_bytes(const kvq_paged_config* cfg, int32_t max_seqs, int64_t max_tokens,
                                   size_t* pool_bytes, size_t* workspace_bytes);

/* kv_paged_create — bind a config to a caller-owned pool (256-byte aligned, >= pool_bytes) on the
 * current device `device`. Zeroes the status word (synchronously); the pages keep their contents.
 * The layout (byte offsets) is fixed: [256 B status area], then per layer the K area and the V area,
 * each padded to 256 bytes; an area holds one unit per (page, KV head), page-major: page_size code
 * rows of head_dim values, then for Q8_0 / Q4_0 the scales [page_size][head_dim / 32] fp16. */
kvq_status kv_paged_create(const kvq_paged_config* cfg, void* pool, size_t pool_bytes, int device, kvq_paged** out);
kvq_status kv_paged_destroy(kvq_paged* h);

/* kv_paged_get_status — wait for all work on the device, then read the status word and clear the bits
 * read. KVQ_EDEVICE if any bit was set. */
kvq_status kv_paged_get_status(kvq_paged* h, uint32_t* word);

/* kv_paged_write — k, v [n_tok][n_kv_heads][head_dim] (strides k_stride, v_stride) to the pages of
 * `layer`: token t goes to page slots[t] / page_size, row slots[t] % page_size (device int32
 * [n_tok]). A negative slot skips the token (padding). Values are rounded to the nearest even (16-bit
 * pages) or quantised by the block codec's definition. Slots of one call must be distinct: of two
 * tokens with one slot either may be stored, or parts of both. Nothing else of the pool changes. */
kvq_status kv_paged_write(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_tok, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* slots, void* stream);

/* kv_paged_read — positions start[b] .. start[b] + cu_rows[b+1] - cu_rows[b] - 1 of each sequence b
 * into rows cu_rows[b].. of k_out and v_out ([n_rows][n_kv_heads][head_dim], contiguous; either may
 * be null): code x scale in fp32, rounded once to dtype. cu_rows: device int32 [n_seq + 1],
 * non-decreasing; start: device int32 [n_seq] or null (zeros). page_table: device int32, row b at
 * page_table + b * table_stride, max_pages entries. Rows outside [cu_rows[0], cu_rows[n_seq]) stay as they are. */
kvq_status kv_paged_read(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, const int32_t* page_table,
                         int32_t max_pages, int64_t table_stride, const int32_t* cu_rows, const int32_t* start,
                         int32_t n_rows, void* k_out, void* v_out, void* stream);

/* kv_paged_decode_attn — attention of one query per sequence, the newest position's: sequence b
 * holds lens[b] positions (device int32, the new one included and already written), its query
 * sits at position lens[b] - 1. q [n_seq][n_q_heads][head_dim] (stride q_stride), out contiguous.
 * 16-bit pages take queries of their own type; rows of Q8_0 / Q4_0 pages enter as code x scale
 * rounded to fp16, with queries of either type. Scales above 515.5 (Q8_0) or 9352 (Q4_0) are taken as
 * these, as code x scale would be no fp16 number (their write has set KVQ_PAGED_RANGE). lens[b] = 0 gives
 * zeros. max_pages x page_size is at most 2^31 - 256. workspace: device, 16-byte aligned,
 * >= kv_paged_required_bytes for n_seq; written before it is read. */
kvq_status kv_paged_decode_attn(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, const void* q,
                                int64_t q_stride, const int32_t* page_table, int32_t max_pages, int64_t table_stride,
                                const int32_t* lens, void* out, const kvq_attn_opts* opts, void* workspace,
                                size_t ws_bytes, void* stream);

/* kv_paged_prefill_attn — attention of a chunk of new tokens per sequence: the rows
 * cu_q[b] .. cu_q[b+1] - 1 of q ([n_rows][n_q_heads][head_dim], stride q_stride) are the last
 * positions of sequence b, which holds lens[b] positions with the chunk (its rows already in the
 * pages). cu_q: device int32 [n_seq + 1], non-decreasing; max_q (host): at least the longest chunk; of a longer
 * one the first max_q rows are computed, the others stay as they are, and the status word says so. n_seq up to 65,535,
 * n_rows below 2^27, max_q up to 524,280. Rows at a negative position (a chunk longer than lens[b]) see nothing:
 * zeros. Rows of out and lse outside [cu_q[0], cu_q[n_seq]) stay as they are. Types, table and workspace as above. */
kvq_status kv_paged_prefill_attn(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, int32_t n_rows,
                                 int32_t max_q, const void* q, int64_t q_stride, const int32_t* cu_q,
                                 const int32_t* page_table, int32_t max_pages, int64_t table_stride,
                                 const int32_t* lens, void* out, const kvq_attn_opts* opts, void* workspace,
                                 size_t ws_bytes, void* stream);

/* Arguments of kv_qk_norm_rope. Outputs may be the inputs (in place, equal strides); otherwise they
 * must not overlap them. The rows of q and k are different rows (slices of one buffer, not the same slice). */
typedef struct {
    int32_t dtype;             /* KVQ_F16 or KVQ_BF16: q, k, weights, outputs */
    int32_t n_tok;
    int32_t n_q_heads;         /* >= 0 */
    int32_t n_k_heads;         /* >= 0, not both 0 */
    int32_t head_dim;          /* 64, 128, 256 or 512 */
    int32_t rot_dim;           /* rotated channels, 0 .. head_dim: a multiple of 16 (of 32 at head_dim 512) */
    int32_t interleaved;       /* pairs (2i, 2i+1) if nonzero, else (i, i + rot_dim/2) */
    int32_t max_pos;           /* rows of cos_sin */
    float eps;
    int32_t reserved;
    const void* q;             /* device [n_tok][n_q_heads][head_dim], stride q_stride */
    const void* k;
    const void* q_weight;      /* device [head_dim]; null: no norm of the queries */
    const void* k_weight;      /* null: no norm of the keys */
    const float* cos_sin;      /* device fp32 [max_pos][rot_dim]: rot_dim/2 cosines, then the sines (null if rot_dim is 0) */
    const int32_t* positions;  /* device int32 [n_tok] (null if rot_dim is 0) */
    void* q_out;
    void* k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
} kvq_norm_rope_args;

/* kv_qk_norm_rope — every query and key head: y = x * rsqrt(mean(x^2) + eps) * weight, then the
 * rotation of its first rot_dim channels by the token's position, (a, b) -> (a cos - b sin,
 * b cos + a sin); fp32 arithmetic, one rounding at the end. The rows of a token whose position is
 * outside [0, max_pos) are set to NaN. Needs no cache handle; the current device's pointers. */
kvq_status kv_qk_norm_rope(const kvq_norm_rope_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_PAGED_H */
