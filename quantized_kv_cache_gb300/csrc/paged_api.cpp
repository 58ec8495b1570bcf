// Host side of the paged cache's C ABI (include/kvq_paged.h): configuration and argument checks, the
// pool's layout and the launches. Everything that is refused is refused here, before anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstring>
#include <exception>
#include <map>
#include <mutex>
#include <new>
#include <utility>
#include <vector>
#include "paged_internal.h"

using namespace kvq;

struct kvq_paged {
    kvq_paged_config cfg;
    uint8_t* pool;
    int device, sm_count;
    std::vector<CUtensorMap> maps;   // 16-bit pages: K and V area of every layer
};

namespace {

struct Geometry {
    int64_t area[2], layer, total;   // bytes of a layer's K, V areas; of a layer; of the pool
};

bool geometry(const kvq_paged_config& c, Geometry* g) {
    if (c.n_layers <= 0 || c.n_kv_heads <= 0 || c.n_q_heads <= 0 || c.n_pages <= 0) return false;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return false;
    if (c.n_q_heads % c.n_kv_heads || c.n_q_heads / c.n_kv_heads > kMaxG) return false;
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return false;
    if ((int64_t)c.n_pages * c.page_size >= (int64_t)1 << 31) return false;
    const bool k16 = c.k_fmt == KVQ_F16 || c.k_fmt == KVQ_BF16, kq = c.k_fmt == KVQ_Q8_0 || c.k_fmt == KVQ_Q4_0;
    if (!k16 && !kq) return false;
    if (c.v_fmt != c.k_fmt && !(c.k_fmt == KVQ_Q8_0 && c.v_fmt == KVQ_Q4_0)) return false;
    if (!(c.softmax_scale >= 0.f) || !std::isfinite(c.softmax_scale)) return false;
    const int fmt[2] = {c.k_fmt, c.v_fmt};
    const int64_t limit = (int64_t)1 << 44;      // 16 TB: keeps every product below far from overflow
    const int64_t units = (int64_t)c.n_pages * c.n_kv_heads;
    for (int w = 0; w < 2; ++w) {
        const int64_t u = paged_unit_bytes(fmt[w], c.head_dim, c.page_size);
        if (units >= (int64_t)1 << 31 || units > limit / u) return false;
        g->area[w] = align256(units * u);
    }
    g->layer = g->area[0] + g->area[1];
    if (g->layer > limit / c.n_layers) return false;
    g->total = 256 + g->layer * c.n_layers;
    return true;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

kvq_status check(const kvq_paged* h, int layer) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers) return KVQ_EINVAL;
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess || d != h->device) return KVQ_EINVAL;
    return KVQ_OK;
}

bool dtype16(int d) { return d == KVQ_F16 || d == KVQ_BF16; }
bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0; }

PagedView view(const kvq_paged* h, int layer) {
    Geometry g;
    geometry(h->cfg, &g);
    const kvq_paged_config& c = h->cfg;
    PagedView v{};
    v.base[0] = h->pool + 256 + g.layer * layer;
    v.base[1] = v.base[0] + g.area[0];
    v.fmt[0] = c.k_fmt;
    v.fmt[1] = c.v_fmt;
    for (int w = 0; w < 2; ++w) v.unit[w] = paged_unit_bytes(v.fmt[w], c.head_dim, c.page_size);
    v.status = (uint32_t*)h->pool;
    v.H = c.n_kv_heads;
    v.D = c.head_dim;
    v.ps = c.page_size;
    v.ps_shift = log2_of(c.page_size);
    v.n_pages = c.n_pages;
    return v;
}

size_t workspace_floats(const kvq_paged_config& c, int64_t seqs, int64_t rows) {
    const int G = c.n_q_heads / c.n_kv_heads;
    const size_t a = (size_t)(line_floats(seqs) + (kMaxDecodeCtas + seqs * c.n_kv_heads) * partial_floats(G, c.head_dim));
    const size_t b = (size_t)paged_prefill_ws_floats(c.head_dim, rows * c.n_q_heads);
    return a > b ? a : b;
}

// The tensor maps of a 16-bit pool: per layer K, then V, as [units][page_size][head_dim].
bool make_maps(kvq_paged* h) {
    const kvq_paged_config& c = h->cfg;
    h->maps.resize(2 * (size_t)c.n_layers);
    if (c.k_fmt != KVQ_F16 && c.k_fmt != KVQ_BF16) return true;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return false;
    const auto encode = (decltype(&cuTensorMapEncodeTiled))fn;
    for (int l = 0; l < c.n_layers; ++l) {
        const PagedView v = view(h, l);
        for (int w = 0; w < 2; ++w) {
            const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages * c.n_kv_heads};
            const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)v.unit[w]};
            const cuuint32_t box[3] = {64, (cuuint32_t)prefill_box_rows(c.head_dim, c.page_size), 1}, one[3] = {1, 1, 1};
            if (encode(&h->maps[2 * l + w], c.k_fmt == KVQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       3, v.base[w], dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return false;
        }
    }
    return true;
}

kvq_status launched(int e) { return e == 0 ? KVQ_OK : KVQ_ECUDA; }

// What the two attention calls share. rows: query rows (decode: n_seq).
kvq_status attn_params(kvq_paged* h, int layer, int dtype, int n_seq, int64_t rows, const void* q, int64_t q_stride,
                       const int32_t* table, int max_pages, int64_t table_stride, const int32_t* lens, void* out,
                       const kvq_attn_opts* opts, void* ws, size_t ws_bytes, PagedAttnParams* p) {
    const kvq_paged_config& c = h->cfg;
    if (!q || !table || !lens || !out || !ws) return KVQ_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(ws) || !aligned4(table) || !aligned4(lens)) return KVQ_EINVAL;
    if (!stride_ok(q_stride, (int64_t)c.n_q_heads * c.head_dim)) return KVQ_EINVAL;
    if (max_pages <= 0 || table_stride < max_pages) return KVQ_EINVAL;
    if ((int64_t)max_pages * c.page_size > ((int64_t)1 << 31) - 256) return KVQ_EINVAL;   // the end of a tile behind the last position too is below 2^31
    if (dtype16(c.k_fmt) && dtype != c.k_fmt) return KVQ_EUNSUPPORTED;
    *p = PagedAttnParams{};
    if (opts) {
        if (!(opts->softcap >= 0.f) || !std::isfinite(opts->softcap) || opts->window < 0) return KVQ_EINVAL;
        if (opts->softcap > 0.f && opts->softcap < 1e-30f) return KVQ_EINVAL;    // its reciprocal has to be finite
        if (opts->softcap > 2e38f) return KVQ_EINVAL;                            // and its multiple by log2(e)
        if (!aligned4(opts->slopes) || !aligned4(opts->prefix) || !aligned4(opts->lse)) return KVQ_EINVAL;
        p->softcap = opts->softcap;
        // a window of all that the table holds hides nothing
        p->window = opts->window >= (int64_t)max_pages * c.page_size ? 0 : opts->window;
        p->slopes = opts->slopes;
        p->prefix = opts->prefix;
        p->lse = opts->lse;
    }
    if (ws_bytes < workspace_floats(c, n_seq, rows) * 4) return KVQ_EINVAL;
    p->v = view(h, layer);
    p->q = q;
    p->out = out;
    p->table = table;
    p->lens = lens;
    p->ws = (float*)ws;
    p->q_stride = q_stride;
    p->table_stride = table_stride;
    p->n_seq = n_seq;
    p->max_pages = max_pages;
    p->Hq = c.n_q_heads;
    p->G = c.n_q_heads / c.n_kv_heads;
    p->dtype = dtype;
    p->scale = c.softmax_scale > 0.f ? c.softmax_scale : 1.0f / std::sqrt((float)c.head_dim);
    return KVQ_OK;
}

}  // namespace

namespace kvq {

int resident_ctas(const void* kernel, int threads, int smem, int* ctas) try {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, int> known;
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return (int)e;
    std::lock_guard<std::mutex> lk(mu);
    const auto it = known.find({kernel, d});
    if (it != known.end()) {
        *ctas = it->second;
        return 0;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, threads, smem);
    if (e != cudaSuccess) return (int)e;
    if (*ctas < 1) return (int)cudaErrorInvalidConfiguration;
    known[{kernel, d}] = *ctas;
    return 0;
} catch (const std::exception&) {     // of the map or the mutex: none leaves the C ABI
    return (int)cudaErrorMemoryAllocation;
}

}  // namespace kvq

extern "C" {

kvq_status kv_paged_required_bytes(const kvq_paged_config* cfg, int32_t max_seqs, int64_t max_tokens,
                                   size_t* pool_bytes, size_t* workspace_bytes) {
    Geometry g;
    if (!cfg || max_seqs < 0 || max_tokens < 0 || max_tokens >= (int64_t)1 << 31 || !geometry(*cfg, &g)) return KVQ_EINVAL;
    if (pool_bytes) *pool_bytes = (size_t)g.total;
    if (workspace_bytes) *workspace_bytes = workspace_floats(*cfg, max_seqs, max_tokens) * 4;
    return KVQ_OK;
}

kvq_status kv_paged_create(const kvq_paged_config* cfg, void* pool, size_t pool_bytes, int device, kvq_paged** out) {
    Geometry g;
    if (!cfg || !pool || !out || !geometry(*cfg, &g)) return KVQ_EINVAL;
    if (pool_bytes < (size_t)g.total || ((uintptr_t)pool & 255)) return KVQ_EINVAL;
    int d = -1, sms = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d != device) return KVQ_EINVAL;
    if (cudaMemset(pool, 0, 256) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) return KVQ_ECUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return KVQ_ECUDA;
    kvq_paged* h = new (std::nothrow) kvq_paged;
    if (!h) return KVQ_EINVAL;
    h->cfg = *cfg;
    h->pool = (uint8_t*)pool;
    h->device = device;
    h->sm_count = sms;
    try {
        if (!make_maps(h)) {
            delete h;
            return KVQ_ECUDA;
        }
    } catch (const std::bad_alloc&) {
        delete h;
        return KVQ_EINVAL;
    }
    *out = h;
    return KVQ_OK;
}

kvq_status kv_paged_destroy(kvq_paged* h) {
    if (!h) return KVQ_EINVAL;
    delete h;
    return KVQ_OK;
}

kvq_status kv_paged_get_status(kvq_paged* h, uint32_t* word) {
    const kvq_status st = check(h, 0);
    if (st != KVQ_OK) return st;
    // the word of all that was enqueued before, on any stream; then exactly the bits that are reported are taken out, so
    // that one that a later call sets meanwhile stays for the next reading
    uint32_t w = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return KVQ_ECUDA;
    if (cudaMemcpy(&w, h->pool, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return KVQ_ECUDA;
    if (w && (launch_paged_clear_status((uint32_t*)h->pool, w) || cudaStreamSynchronize(nullptr) != cudaSuccess)) return KVQ_ECUDA;
    if (word) *word = w;
    return w ? KVQ_EDEVICE : KVQ_OK;
}

kvq_status kv_paged_write(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_tok, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* slots, void* stream) {
    const kvq_status st = check(h, layer);
    if (st != KVQ_OK) return st;
    if (!dtype16(dtype) || n_tok < 0) return KVQ_EINVAL;
    if (n_tok == 0) return KVQ_OK;
    const int64_t row = (int64_t)h->cfg.n_kv_heads * h->cfg.head_dim;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || !aligned4(slots)) return KVQ_EINVAL;
    if (!stride_ok(k_stride, row) || !stride_ok(v_stride, row)) return KVQ_EINVAL;
    WriteParams p{};
    p.v = view(h, layer);
    p.src[0] = k;
    p.src[1] = v;
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.slots = slots;
    p.n_tok = n_tok;
    p.dtype = dtype;
    return launched(launch_paged_write(p, stream));
}

kvq_status kv_paged_read(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, const int32_t* page_table,
                         int32_t max_pages, int64_t table_stride, const int32_t* cu_rows, const int32_t* start,
                         int32_t n_rows, void* k_out, void* v_out, void* stream) {
    const kvq_status st = check(h, layer);
    if (st != KVQ_OK) return st;
    if ((!dtype16(dtype) && dtype != KVQ_PAGED_F32) || n_seq < 0 || n_rows < 0) return KVQ_EINVAL;
    if (n_seq == 0 || n_rows == 0) return KVQ_OK;
    if (!page_table || !cu_rows || (!k_out && !v_out) || max_pages <= 0 || table_stride < max_pages) return KVQ_EINVAL;
    if (!aligned4(page_table) || !aligned4(cu_rows) || !aligned4(start) || !aligned16(k_out) || !aligned16(v_out))
        return KVQ_EINVAL;
    ReadParams p{};
    p.v = view(h, layer);
    p.table = page_table;
    p.cu = cu_rows;
    p.start = start;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.table_stride = table_stride;
    p.n_seq = n_seq;
    p.max_pages = max_pages;
    p.n_rows = n_rows;
    p.dtype = dtype;
    return launched(launch_paged_read(p, stream));
}

kvq_status kv_paged_decode_attn(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, const void* q,
                                int64_t q_stride, const int32_t* page_table, int32_t max_pages, int64_t table_stride,
                                const int32_t* lens, void* out, const kvq_attn_opts* opts, void* workspace,
                                size_t ws_bytes, void* stream) {
    kvq_status st = check(h, layer);
    if (st != KVQ_OK) return st;
    if (!dtype16(dtype) || n_seq < 0) return KVQ_EINVAL;
    if (n_seq == 0) return KVQ_OK;
    PagedAttnParams p;
    st = attn_params(h, layer, dtype, n_seq, 0, q, q_stride, page_table, max_pages, table_stride, lens, out, opts,
                     workspace, ws_bytes, &p);
    if (st != KVQ_OK) return st;
    const auto launch = p.v.D == 64 ? launch_paged_decode_64 : (p.v.D == 128 ? launch_paged_decode_128 : launch_paged_decode_256);
    return launched(launch(p, h->sm_count, stream));
}

kvq_status kv_paged_prefill_attn(kvq_paged* h, int32_t layer, int32_t dtype, int32_t n_seq, int32_t n_rows,
                                 int32_t max_q, const void* q, int64_t q_stride, const int32_t* cu_q,
                                 const int32_t* page_table, int32_t max_pages, int64_t table_stride,
                                 const int32_t* lens, void* out, const kvq_attn_opts* opts, void* workspace,
                                 size_t ws_bytes, void* stream) {
    kvq_status st = check(h, layer);
    if (st != KVQ_OK) return st;
    if (!dtype16(dtype) || n_seq < 0 || n_rows < 0 || max_q < 0) return KVQ_EINVAL;
    if (n_seq == 0 || n_rows == 0 || max_q == 0) return KVQ_OK;
    if (!cu_q || !aligned4(cu_q)) return KVQ_EINVAL;
    // grid rows: one per sequence, one per 128 rows of the longest chunk; a head's row numbers stay below 2^31
    if (n_seq > 65535 || (int64_t)n_rows * kMaxG >= (int64_t)1 << 31 || (int64_t)(max_q < n_rows ? max_q : n_rows) * kMaxG > 65535 * (int64_t)128) return KVQ_EUNSUPPORTED;
    PagedAttnParams p;
    st = attn_params(h, layer, dtype, n_seq, n_rows, q, q_stride, page_table, max_pages, table_stride, lens, out, opts,
                     workspace, ws_bytes, &p);
    if (st != KVQ_OK) return st;
    p.cu = cu_q;
    p.n_rows = n_rows;
    p.max_q = max_q < n_rows ? max_q : n_rows;
    return launched(launch_paged_prefill(p, &h->maps[2 * (size_t)layer], h->sm_count, stream));
}

kvq_status kv_qk_norm_rope(const kvq_norm_rope_args* a, void* stream) {
    if (!a || !dtype16(a->dtype) || a->n_tok < 0 || a->n_q_heads < 0 || a->n_k_heads < 0) return KVQ_EINVAL;
    if (a->n_q_heads + (int64_t)a->n_k_heads == 0 || (int64_t)a->n_q_heads + a->n_k_heads > 1 << 20) return KVQ_EINVAL;
    const int D = a->head_dim, align = D == 512 ? 32 : 16;
    if (D != 64 && D != 128 && D != 256 && D != 512) return KVQ_EINVAL;
    if (a->rot_dim < 0 || a->rot_dim > D || a->rot_dim % align) return KVQ_EINVAL;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return KVQ_EINVAL;
    if (a->n_tok == 0) return KVQ_OK;
    if (a->rot_dim && (!a->cos_sin || !a->positions || a->max_pos <= 0)) return KVQ_EINVAL;
    if (!aligned16(a->cos_sin) || !aligned4(a->positions)) return KVQ_EINVAL;
    struct Side { int heads; const void* in; const void* w; const void* out; int64_t si, so; };
    const Side sides[2] = {{a->n_q_heads, a->q, a->q_weight, a->q_out, a->q_stride, a->q_out_stride},
                           {a->n_k_heads, a->k, a->k_weight, a->k_out, a->k_stride, a->k_out_stride}};
    for (const Side& s : sides) {
        if (!s.heads) continue;
        const int64_t row = (int64_t)s.heads * D;
        if (!s.in || !s.out || !aligned16(s.in) || !aligned16(s.out) || !aligned16(s.w)) return KVQ_EINVAL;
        if (!stride_ok(s.si, row) || !stride_ok(s.so, row)) return KVQ_EINVAL;
        if (s.in == s.out && s.si != s.so) return KVQ_EINVAL;
    }
    int d = 0, sms = 0;
    if (cudaGetDevice(&d) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d) != cudaSuccess)
        return KVQ_ECUDA;
    return launched(launch_norm_rope(*a, sms, stream));
}

}  // extern "C"
