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
/* A page format of its own: e4m3 codes with one scale for 16 positions of a head (a block: positions 16 i .. 16 i + 15 of a
 * sequence), a power of two: the smallest with the block's largest magnitude within 448 times it, 2^-126 at least. It grows
 * as rows come (kv_paged_append); the rows that are there are then rounded to it. */
enum { KVQ_PAGED_E4M3 = 101 };

/* Bits of the status word (kv_paged_get_status). */
enum {
    KVQ_PAGED_NONFINITE = 1,    /* a quantised block had a non-finite scale (the page holds it); KVQ_PAGED_E4M3: a value was no
                                   finite number (it is stored as NaN, the block's others by their own scale) */
    KVQ_PAGED_TIMEOUT = 2,      /* a bounded device wait ran out; that launch's outputs are invalid */
    KVQ_PAGED_BAD_INDEX = 4,    /* a slot or a page number was out of range: a write was skipped, a page read as zeros */
    KVQ_PAGED_BAD_LENGTH = 8,   /* a length, row offset or max_q was out of range: lengths are cut to what the page
                                   table holds, rows beyond the call's buffers or max_q are skipped */
    KVQ_PAGED_RANGE = 16,       /* a quantised block reaches beyond fp16's 65,504: the page holds it and kv_paged_read
                                   gives it, the attentions cut its scale (kv_paged_decode_attn) */
    KVQ_PAGED_NO_PAGES = 32     /* kv_pages_extend: fewer free pages than the call needs; it changed nothing */
};

typedef struct {
    int32_t n_layers;
    int32_t n_kv_heads;
    int32_t head_dim;       /* 64, 128 or 256 */
    int32_t n_q_heads;      /* a multiple of n_kv_heads, with n_q_heads / n_kv_heads <= 16 */
    int32_t page_size;      /* positions per page: 16, 32, 64, 128 or 256 */
    int32_t n_pages;        /* pages per layer (one page table serves all layers); n_pages x page_size < 2^31 */
    int32_t k_fmt;          /* KVQ_F16, KVQ_BF16, KVQ_Q8_0, KVQ_Q4_0 or KVQ_PAGED_E4M3 */
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
 * rows of head_dim values, then for Q8_0 / Q4_0 the scales [page_size][head_dim / 32] fp16, for KVQ_PAGED_E4M3 the
 * scales [page_size / 16] fp32, padded to 32 bytes. */
kvq_status kv_paged_create(const kvq_paged_config* cfg, void* pool, size_t pool_bytes, int device, kvq_paged** out);
kvq_status kv_paged_destroy(kvq_paged* h);

/* kv_paged_get_status — wait for all work on the device, then read the status word and clear the bits
 * read. KVQ_EDEVICE if any bit was set. */
kvq_status kv_paged_get_status(kvq_paged* h, uint32_t* word);

/* kv_paged_write — k, v [n_tok][n_kv_heads][head_dim] (strides k_stride, v_stride) to the pages of
 * `layer`: token t goes to page slots[t] / page_size, row slots[t] % page_size (device int32
 * [n_tok]). A negative slot skips the token (padding). Values are rounded to the nearest even (16-bit
 * pages) or quantised by the block codec's definition. Slots of one call must be distinct: of two
 * tokens with one slot either may be stored, or parts of both. Nothing else of the pool changes.
 * KVQ_EUNSUPPORTED for KVQ_PAGED_E4M3 pages, whose scales serve 16 positions: kv_paged_append. */
kvq_status kv_paged_write(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_tok, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* slots, void* stream);

/* kv_paged_append — rows cu_rows[b] .. cu_rows[b+1] - 1 of k, v ([n_rows][n_kv_heads][head_dim], strides k_stride,
 * v_stride) become the positions start[b].. of each sequence b, in KVQ_PAGED_E4M3 pages of `layer` (KVQ_EUNSUPPORTED for other
 * formats: kv_paged_write). cu_rows, start and the page table as for kv_paged_read. A block whose first position is among the rows
 * begins anew; otherwise its positions up to start[b] - 1 are there and count: its scale grows to what the rows need, never
 * shrinks, and where it grows those positions' codes are rounded to the new one. What the blocks hold behind the rows is not
 * looked at and stays as it is. A row of positions that the table does not hold is skipped (KVQ_PAGED_BAD_LENGTH).
 * Sequences that share a page must not write in it (kv_pages_extend sees to it). */
kvq_status kv_paged_append(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, const int32_t* page_table,
                           int32_t max_pages, int64_t table_stride, const int32_t* cu_rows, const int32_t* start,
                           int32_t n_rows, const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* stream);

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
 * these, as code x scale would be no fp16 number (their write has set KVQ_PAGED_RANGE). KVQ_PAGED_E4M3 rows likewise, with
 * scales up to 2^7 (a chunk may take code x scale as an fp16 number, which it is from scales of 2^-15 on; decode does not round
 * it). lens[b] = 0 gives
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

/* Page tables that the device keeps. A row is a sequence: lens[r] positions in the pages table[r][0] .. (device int32
 * [rows][max_pages], rows table_stride apart); what stands behind them is not looked at. refs[p] says how many rows hold page p
 * (device int32 [n_pages]; 0: free), and whoever else keeps a page counts in it too. A new cache's refs and lens are zeros. */
typedef struct {
    int32_t rows;
    int32_t max_pages;
    int64_t table_stride;
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
} kvq_page_tables;

/* Sequences forked, made longer, cut and freed, pages copied and moved, in all layers at once. Nothing is read back, so that the
 * calls can be captured; the same call on the same tables gives the same pages. Calls on the same tables, and calls that read or
 * write the pages concerned, go on one stream or wait for one another. Workspaces: device, 16-byte aligned,
 * >= kv_pages_required_bytes, written before they are read, one each for calls that may overlap. */
kvq_status kv_pages_required_bytes(const kvq_paged_config* cfg, size_t* workspace_bytes);

/* kv_pages_copy — page src[i] to page dst[i], i < n (device int32 [n]), K and V of every layer. A pair with a negative number is
 * skipped; no page may be a destination twice, nor both a source and a destination. */
kvq_status kv_pages_copy(kvq_paged* h, int32_t n, const int32_t* src, const int32_t* dst, void* stream);

/* kv_pages_fork — row children[i] becomes what row parents[i] is, i < n <= 65,535 (device int32 [n]): all pages are shared. A negative
 * child is skipped. A child that holds positions, has come before in the call or is a parent in it is left out
 * (KVQ_PAGED_BAD_INDEX); several children of one parent are fine. */
kvq_status kv_pages_fork(kvq_paged* h, const kvq_page_tables* t, int32_t n, const int32_t* parents, const int32_t* children, void* stream);

/* kv_pages_extend — row r will hold add[r] more positions (device int32 [rows], >= 0; 0 leaves a row as it is): lens grows, and
 * pages for them come from the free ones, lowest first, row after row. A row that would go on in a part-filled page that is held
 * by others too gets a copy of it instead (of several rows that go on in one page all of whose holders go on, the lowest
 * keeps it), so that what is then written at the new positions is the row's own. If the free pages do not suffice for the
 * whole call it changes nothing and sets KVQ_PAGED_NO_PAGES (lens stays; rows must not be written behind it then); a row that would outgrow its table, or whose last page is no
 * page, is left out (KVQ_PAGED_BAD_LENGTH, KVQ_PAGED_BAD_INDEX). */
kvq_status kv_pages_extend(kvq_paged* h, const kvq_page_tables* t, const int32_t* add, void* workspace, size_t ws_bytes, void* stream);

/* kv_pages_free — row rows[i] is cut to keep[i] positions (keep null: to none), i < n (device int32 [n]): the pages behind them
 * are given back (held once less), their entries become -1. A negative row is skipped, a row that is shorter stays as it is, one
 * that comes twice is cut to the lower number. */
kvq_status kv_pages_free(kvq_paged* h, const kvq_page_tables* t, int32_t n, const int32_t* rows, const int32_t* keep, void* stream);

/* kv_pages_compact — the L pages in use become pages 0 .. L - 1: those behind are moved to the free ones before, both in order, with
 * their counts, and the rows' entries are renumbered. remap (device int32 [n_pages], written): the new number of each page, -1 for
 * a free one. */
kvq_status kv_pages_compact(kvq_paged* h, const kvq_page_tables* t, int32_t* remap, void* workspace, size_t ws_bytes, void* stream);

/* Arguments of kv_prompt_attn: packed prompts, sequence b's tokens in rows cu[b] .. cu[b+1] - 1 of q, k, v and out. */
typedef struct {
    int32_t dtype;             /* KVQ_F16 or KVQ_BF16: q, k, v, out */
    int32_t n_seq;             /* up to 65,535 */
    int32_t n_rows;
    int32_t max_q;             /* at least the longest prompt; of a longer one only the first max_q tokens are computed */
    int32_t n_q_heads;         /* a multiple of n_kv_heads, with n_q_heads / n_kv_heads <= 16 */
    int32_t n_kv_heads;
    int32_t head_dim;          /* 64, 128 or 256 */
    float softmax_scale;       /* 0 selects 1/sqrt(head_dim) */
    const void* q;             /* device [n_rows][n_q_heads][head_dim], stride q_stride */
    const void* k;             /* device [n_rows][n_kv_heads][head_dim], stride k_stride */
    const void* v;
    const int32_t* cu;         /* device [n_seq + 1], non-decreasing */
    void* out;                 /* device [n_rows][n_q_heads][head_dim], contiguous */
    int64_t q_stride, k_stride, v_stride;
} kvq_prompt_args;

/* kv_prompt_attn — causal attention of whole prompts over their own rows: the token at position i of a sequence sees its positions
 * 0 .. i (options as for the paged calls). No cache is read or needed: before or beside the calls that store k and v, of either
 * cache. out overlaps none of q, k and v. Rows of out and lse outside [cu[0], cu[n_seq]) stay as they are, and so do those of a sequence whose bounds are
 * no rows of the call. workspace: device, 16-byte aligned, >= kv_prompt_required_bytes for the call; its first 256 bytes
 * hold a status word (the bits above), which its owner zeroes once and kv_prompt_get_status reads; the rest is written before
 * it is read. Calls that may overlap need workspaces of their own. The current device's pointers. */
kvq_status kv_prompt_required_bytes(int64_t n_rows, int32_t n_q_heads, int32_t head_dim, size_t* workspace_bytes);
kvq_status kv_prompt_attn(const kvq_prompt_args* args, const kvq_attn_opts* opts, void* workspace, size_t ws_bytes, void* stream);
/* kv_prompt_get_status — as kv_paged_get_status, of the calls with this workspace. */
kvq_status kv_prompt_get_status(void* workspace, uint32_t* word);

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

/* kv_qk_norm_rope_axes — kv_qk_norm_rope with positions on 1 to 4 axes (time, height and width of a patch, say): positions
 * is device int32 [n_axes][n_tok], and frequency i of the rot_dim / 2 turns its pair by the token's position on one of the axes,
 * sections[a] (host, >= 0, rot_dim / 2 in all) of them by axis a: in runs, axis after axis, or (cyclic != 0) dealt to the axes in
 * turn until each has its number. One table serves all axes. The rows of a token that has a position outside [0, max_pos) on an
 * axis with frequencies are set to NaN. rot_dim is above 0. */
kvq_status kv_qk_norm_rope_axes(const kvq_norm_rope_args* args, int32_t n_axes, const int32_t* sections, int32_t cyclic,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_PAGED_H */
