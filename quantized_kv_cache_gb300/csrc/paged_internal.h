// Internal definitions of the paged cache shared by its host side and its kernels: the pool's
// geometry, row encodings and the launch parameter blocks. Not part of the public C ABI.
#pragma once
#include "kvq_internal.h"
#include "../../include/kvq_paged.h"

namespace kvq {

constexpr int kTile = 16;            // positions per attention tile: every page size is a multiple
constexpr int kMaxSms = 192;         // bound of the SMs that a chunk's splits are spread over (sizes the workspace)
constexpr int kMaxDecodeCtas = 1024; // bound of a decode launch's CTAs (sizes the workspace)
// Largest scales that the attention takes as they are (fp16 bits of 515.5 and 9352): 127 and 7 times the next ones round to
// fp16's infinity.
constexpr uint32_t kMaxScaleQ8 = 0x6007, kMaxScaleQ4 = 0x7091;

// Exponents of an e4m3 block's power of two: 448 2^120 is above bf16's largest number. The attentions take powers up to 2^7
// (448 2^7 is an fp16 number, 448 2^8 is none).
constexpr int kMinPower = -126, kMaxPower = 120, kMaxPowerAttn = 7;

// Bytes of one code row (D values), and of the scales of a unit: a row's by 32 values, or one for a tile of an e4m3 unit (padded to
// 32 bytes, so that rows and units stay on sectors).
KVQ_HD int paged_row_bytes(int fmt, int D) { return fmt == KVQ_Q8_0 || fmt == KVQ_PAGED_E4M3 ? D : (fmt == KVQ_Q4_0 ? D / 2 : 2 * D); }
KVQ_HD int paged_scale_bytes(int fmt, int D, int ps) {
    if (fmt == KVQ_PAGED_E4M3) return ps / kTile * 4 < 32 ? 32 : ps / kTile * 4;
    return (fmt == KVQ_Q8_0 || fmt == KVQ_Q4_0) ? ps * (D / 16) : 0;
}
KVQ_HD int64_t paged_unit_bytes(int fmt, int D, int ps) {
    return (int64_t)ps * paged_row_bytes(fmt, D) + paged_scale_bytes(fmt, D, ps);
}

// One layer of the pool as the kernels see it.
struct PagedView {
    uint8_t* base[2];        // first unit of the K, V area
    int64_t unit[2];         // bytes of a unit
    uint32_t* status;
    int32_t fmt[2];
    int32_t H, D, ps, ps_shift, n_pages;
};

struct WriteParams {
    PagedView v;
    const void* src[2];
    int64_t stride[2];       // elements
    const int32_t* slots;
    int32_t n_tok, dtype;
};

struct PagedAppendParams {
    PagedView v;
    const void* src[2];
    int64_t stride[2];       // elements
    const int32_t* table;
    const int32_t* cu;
    const int32_t* start;
    int64_t table_stride;
    int32_t n_seq, max_pages, n_rows, dtype;
};

struct ReadParams {
    PagedView v;
    const int32_t* table;
    const int32_t* cu;
    const int32_t* start;
    void* out[2];
    int64_t table_stride;
    int32_t n_seq, max_pages, n_rows, dtype;
};

struct PagedAttnParams {
    PagedView v;
    const void* q;
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;       // prefill only
    const int32_t* prefix;
    const float* slopes;
    float* ws;
    int64_t q_stride, table_stride;
    int32_t n_seq, max_pages, Hq, G, dtype;
    int32_t n_rows, max_q;   // prefill only
    int32_t window;
    int32_t n_cta;           // decode only: CTAs of the split launch
    float scale, softcap;
};

// Page tables on the device, and the whole pool: v is layer 0, layers are layer_bytes apart.
struct PagesParams {
    PagedView v;
    int64_t layer_bytes, table_stride;
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int32_t n_layers, rows, max_pages, sm_count;
};
// int32 of workspace: a header, then up to five numbers per page
KVQ_HD int64_t pages_ws_ints(int64_t n_pages) { return 16 + 5 * n_pages; }

// Resident CTAs per SM of a kernel on the current device; lets it use `smem` bytes of dynamic shared memory.
// Asked once per kernel and device. Returns a cudaError_t as int.
int resident_ctas(const void* kernel, int threads, int smem, int* ctas);

int launch_paged_clear_status(uint32_t* status, uint32_t bits);   // on the legacy stream
// The axis of each frequency of a rotation, two bits each, eight to a word; and the axes that have any, by bit.
struct RopeAxes {
    uint32_t n, used;
    uint16_t of8[32];
};
// Frequencies in runs of sections[a], or dealt to the axes in turn until each has its number.
inline void rope_axes(int n_axes, const int32_t* sections, bool cyclic, RopeAxes* x) {
    *x = RopeAxes{};
    x->n = (uint32_t)n_axes;
    int left[4] = {}, total = 0, f = 0;
    for (int a = 0; a < n_axes; ++a) {
        left[a] = sections[a];
        total += sections[a];
        if (sections[a] > 0) x->used |= 1u << a;
    }
    const auto put = [&](int a) { x->of8[f / 8] = (uint16_t)(x->of8[f / 8] | a << 2 * (f % 8)); ++f; --left[a]; };
    while (f < total)
        for (int a = 0; a < n_axes; ++a)
            if (cyclic) {
                if (left[a] > 0) put(a);
            } else {
                while (left[a] > 0) put(a);
            }
}

int launch_norm_rope(const kvq_norm_rope_args& a, int sm_count, void* stream);
int launch_norm_rope_axes(const kvq_norm_rope_args& a, const RopeAxes& x, int sm_count, void* stream);
int launch_paged_write(const WriteParams& p, void* stream);
int launch_paged_append(const PagedAppendParams& p, void* stream);
int launch_paged_read(const ReadParams& p, void* stream);
int launch_pages_copy(const PagesParams& p, int n, const int32_t* src, const int32_t* dst, void* stream);
int launch_pages_fork(const PagesParams& p, int n, const int32_t* parents, const int32_t* children, void* stream);
int launch_pages_free(const PagesParams& p, int n, const int32_t* rows, const int32_t* keep, void* stream);
int launch_pages_extend(const PagesParams& p, const int32_t* add, int32_t* ws, void* stream);
int launch_pages_compact(const PagesParams& p, int32_t* remap, int32_t* ws, void* stream);
int launch_paged_decode_64(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_decode_128(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_decode_256(const PagedAttnParams& p, int sm_count, void* stream);
// maps: two CUtensorMap, the layer's K and V area as [units][page_size][head_dim] of 16-bit values in boxes of
// prefill_box_rows rows x 64 (16-bit pages; read for no other format)
int launch_paged_draft_64(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_draft_128(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_draft_256(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_prefill_64(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
int launch_paged_prefill_128(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
int launch_paged_prefill_256(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
// maps: two CUtensorMap, K and V rows as [rows][heads][head_dim] in boxes of prefill_tile rows x 1 x 64
int launch_prompt_attn_64(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
int launch_prompt_attn_128(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
int launch_prompt_attn_256(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
KVQ_HD constexpr int prefill_tile(int D) { return D == 256 ? 64 : 128; }    // positions of a KV tile
KVQ_HD int prefill_box_rows(int D, int ps) { return ps < prefill_tile(D) ? ps : prefill_tile(D); }
// A run's partial result of a head: 16 maxima, 16 sums, the outputs.
KVQ_HD int64_t partial_floats(int G, int D) { return 32 + (int64_t)G * D; }
// Before the partials: n_seq + 1 int64, the tiles before each sequence.
KVQ_HD int64_t line_floats(int64_t n_seq) { return (2 * (n_seq + 1) + 3) & ~(int64_t)3; }

// Chunks of a few tokens over e4m3 pages (kernels_paged_draft.cu): CTAs per SM (nq: blocks of eight rows of a warp), the floats of the
// partial results (maxima, sums, outputs) that the CTAs of an SM leave, each once: 64 rows of two CTAs, at D = 256 32 of two; and of all
// runs, two partials each.
KVQ_HD constexpr int draft_ctas(int D, int nq) { return nq == 4 || D == 256 ? 2 : (D == 128 ? 3 : 4); }
KVQ_HD constexpr int draft_part_floats(int D) { return D == 256 ? 2 * (64 + 32 * D) : 2 * (128 + 64 * D); }
KVQ_HD int64_t paged_draft_ws_floats(int D, int64_t n_seq) { return line_floats(n_seq) + (int64_t)kMaxSms * 2 * draft_part_floats(D); }
// Whether a chunk goes there: up to 64 rows a KV head, over as many positions of heads as make its even split worth more than the
// chunk kernel's tensor cores and split positions (their lengths are on the device: as many as the table holds). Of 40 heads on 8 x 128, us,
// chunk kernel / few-row kernel, 15 rows: 2 sequences up to 8,000 24 / 26, 4 36 / 30, 8 up to 2,000 23 / 23, 16 34 / 28 and up to 32,000
// 472 / 167; 30 rows: 4 up to 8,000 37 / 39, 8 70 / 54, 16 up to 2,000 34 / 37; one up to 32,000 39 / 36 and 41 / 44. D = 64 and 256
// cross at the same products. 60 rows (two warps of 32 on a tile): 16 up to 8,000 126 / 125, 20 up to 16,001 293 / 242.
KVQ_HD bool draft_better(int64_t rows, int64_t n_seq, int64_t H, int64_t positions) {
    return rows <= 64 && n_seq * H * positions >= (rows <= 16 ? 160000 : rows <= 32 ? 270000 : 1100000);
}

// A chunk's positions are split when its row tiles alone leave SMs without work: as many splits as leave one CTA per SM.
constexpr int kMaxSplits = 16;
KVQ_HD int prefill_splits(int64_t rows, int n_seq, int H, int tile_rows, int sm_count) {
    const int64_t ctas = (rows / tile_rows + n_seq) * H;       // at most one part-filled tile per sequence
    const int64_t s = (sm_count < kMaxSms ? sm_count : kMaxSms) / (ctas > 0 ? ctas : 1);
    return (int)(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}
// Whole prompts: the row tiles of all of them, at most one part-filled per sequence; and splits that leave each some four of the
// position tiles of the longest one's last rows (333 tokens, 4 heads on 2 x 128: unsplit 20 us, two 25; 1,024 tokens of one head unsplit 31,
// four 27, eight 25; 8,191 unsplit 113, four 49, more 49).
KVQ_HD int64_t prompt_tiles(int64_t n_rows, int64_t n_seq, int G, int D) { return n_rows * G / (D == 256 ? 128 : 256) + n_seq; }
KVQ_HD int prompt_splits(int max_q, int D) { return 1 + max_q / prefill_tile(D) / 4; }
// The splits' partials in the workspace: (maximum, sum) of all `pairs` (split, query row, head), then from float
// split_out_at on their outputs. Those go by 16-byte accesses, and pairs may be odd: rounded up to four floats.
KVQ_HD int64_t split_out_at(int64_t pairs) { return (2 * pairs + 3) & ~(int64_t)3; }
// The splits times the rows stay below one CTA per SM's worth of row tiles, and below kMaxSplits times the rows.
KVQ_HD int64_t paged_prefill_ws_floats(int D, int64_t head_rows) {   // query rows x query heads
    const int64_t most = head_rows * kMaxSplits, full = (int64_t)kMaxSms * 256, pairs = most < full ? most : full;
    return split_out_at(pairs) + pairs * D;
}

}  // namespace kvq
