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

// Bytes of one code row (D values) and of a row's scales.
KVQ_HD int paged_row_bytes(int fmt, int D) { return fmt == KVQ_Q8_0 ? D : (fmt == KVQ_Q4_0 ? D / 2 : 2 * D); }
KVQ_HD int paged_scale_bytes(int fmt, int D) { return (fmt == KVQ_Q8_0 || fmt == KVQ_Q4_0) ? D / 16 : 0; }
KVQ_HD int64_t paged_unit_bytes(int fmt, int D, int ps) {
    return (int64_t)ps * (paged_row_bytes(fmt, D) + paged_scale_bytes(fmt, D));
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

// Resident CTAs per SM of a kernel on the current device; lets it use `smem` bytes of dynamic shared memory.
// Asked once per kernel and device. Returns a cudaError_t as int.
int resident_ctas(const void* kernel, int threads, int smem, int* ctas);

int launch_paged_clear_status(uint32_t* status, uint32_t bits);   // on the legacy stream
int launch_norm_rope(const kvq_norm_rope_args& a, int sm_count, void* stream);
int launch_paged_write(const WriteParams& p, void* stream);
int launch_paged_read(const ReadParams& p, void* stream);
int launch_paged_decode_64(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_decode_128(const PagedAttnParams& p, int sm_count, void* stream);
int launch_paged_decode_256(const PagedAttnParams& p, int sm_count, void* stream);
// maps: two CUtensorMap, the layer's K and V area as [units][page_size][head_dim] of 16-bit values in boxes of
// prefill_box_rows rows x 64 (16-bit pages; read for no other format)
int launch_paged_prefill(const PagedAttnParams& p, const void* maps, int sm_count, void* stream);
int prefill_box_rows(int D, int ps);
// A run's partial result of a head: 16 maxima, 16 sums, the outputs.
KVQ_HD int64_t partial_floats(int G, int D) { return 32 + (int64_t)G * D; }
// Before the partials: n_seq + 1 int64, the tiles before each sequence.
KVQ_HD int64_t line_floats(int64_t n_seq) { return (2 * (n_seq + 1) + 3) & ~(int64_t)3; }

// A chunk's positions are split when its row tiles alone leave SMs without work: as many splits as leave one CTA per SM.
constexpr int kMaxSplits = 16;
KVQ_HD int prefill_splits(int64_t rows, int n_seq, int H, int tile_rows, int sm_count) {
    const int64_t ctas = (rows / tile_rows + n_seq) * H;       // at most one part-filled tile per sequence
    const int64_t s = (sm_count < kMaxSms ? sm_count : kMaxSms) / (ctas > 0 ? ctas : 1);
    return (int)(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}
// The splits' partials in the workspace: (maximum, sum) of all `pairs` (split, query row, head), then from float
// split_out_at on their outputs. Those go by 16-byte accesses, and pairs may be odd: rounded up to four floats.
KVQ_HD int64_t split_out_at(int64_t pairs) { return (2 * pairs + 3) & ~(int64_t)3; }
// The splits times the rows stay below one CTA per SM's worth of row tiles, and below kMaxSplits times the rows.
KVQ_HD int64_t paged_prefill_ws_floats(int D, int64_t head_rows) {   // query rows x query heads
    const int64_t most = head_rows * kMaxSplits, full = (int64_t)kMaxSms * 256, pairs = most < full ? most : full;
    return split_out_at(pairs) + pairs * D;
}

}  // namespace kvq
