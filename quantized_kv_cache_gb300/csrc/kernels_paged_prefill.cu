// Attention of chunks of new tokens over pages.
//
// The rows of a KV head are the chunk's tokens times the G query heads that read it, row r = token r / G,
// head r % G, so the KV rows are read once for all of them. A CTA takes 64 rows of one (sequence, KV
// head), 16 per warp, and walks the 16-position tiles that any of its rows sees.
#include "paged_frag.cuh"

namespace kvq {
namespace {

constexpr int kPW = 4;
constexpr int kPT = kPW * 32;
constexpr int kRowsCta = kPW * 16;

// One sequence's chunk: rows of q, and the positions they sit at.
struct Chunk {
    int row0, n, len, pos0, pre;     // first row of q, tokens, positions held, position of the first token, prefix
};
__device__ __forceinline__ Chunk chunk_of(const PagedAttnParams& p, int b, bool report) {
    Chunk c;
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    const int len = p.lens[b], c0 = p.cu[b], c1 = p.cu[b + 1];
    c.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
    c.row0 = c0;
    c.n = c0 < 0 || c1 > p.n_rows || c1 < c0 ? 0 : c1 - c0;
    if (report && (len < 0 || len > cap || c0 < 0 || c1 > p.n_rows || c1 < c0 || c.n > p.max_q))
        raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
    c.pos0 = c.len - c.n;
    c.pre = p.prefix ? min(max(p.prefix[b], 0), c.len) : 0;
    return c;
}

// o += p V over the positions of the tile that each row sees (a score of -inf is one it does not see).
template <int D, int VF, typename T, typename SRC>
__device__ __noinline__ void add_seen(const SRC& src, int g, int t, const float (&s)[2][4], const float (&base)[2],
                                      float (&o)[D / 8][4]) {
    using V = VGeo<D, VF>;
    for (int j = 0; j < 16; ++j) {
        float x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float a = j < 8 ? s[0][2 * k] : s[1][2 * k], b = j < 8 ? s[0][2 * k + 1] : s[1][2 * k + 1];
            x[k] = __shfl_sync(kAll, (j & 1) ? b : a, 4 * g + (j & 7) / 2);
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int k = c >> 1;
                const float v = tile_value<D, VF, T>(src, j, ochan<D, VF>(d / V::CH, 2 * t + (c & 1)) + d % V::CH);
                if (x[k] != -INFINITY) o[d][c] = fmaf(ex2(x[k] - base[k]), v, o[d][c]);
            }
    }
}

template <int D, int KF, int VF, typename T, typename TQ>
__global__ void __launch_bounds__(kPT) prefill_kernel(PagedAttnParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.z, h = blockIdx.y, G = p.G;
    const Chunk c = chunk_of(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int rows = c.n * G, base_row = blockIdx.x * kRowsCta + warp * 16;
    if (base_row >= rows) return;
    const ScoreRule rule = score_rule(p);
    auto qrow = [&](int r) -> const TQ* {
        const int i = base_row + r;
        if (i >= rows) return nullptr;
        return (const TQ*)p.q + (int64_t)(c.row0 + i / G) * p.q_stride + ((int64_t)h * G + i % G) * D;
    };
    uint32_t qf[D / 16][4];
    float back[2], slope[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4] = {};
    load_queries<D, KF, T, TQ>(qrow, g, t, qf, back);
    int pos[2], lo[2], pre[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = base_row + g + 8 * k;
        pos[k] = i < rows ? c.pos0 + i / G : -1;
        lo[k] = p.window > 0 ? pos[k] - p.window + 1 : 0;
        pre[k] = pos[k] >= 0 ? c.pre : 0;
        slope[k] = p.slopes && i < rows ? p.slopes[h * G + i % G] * kL2e : 0.f;
    }
    // the warp's tiles: [0, n0) of the prefix, [t1, end) from its first row's window to its last row
    const int last = c.pos0 + (min(base_row + 16, rows) - 1) / G, first = c.pos0 + base_row / G;
    const int end = last < 0 ? 0 : (max(last + 1, c.pre) + kTile - 1) / kTile;
    const int t1 = min(end, p.window > 0 ? max(0, first - p.window + 1) / kTile : 0);
    const int n0 = min((last < 0 ? 0 : c.pre + kTile - 1) / kTile, t1);

    for (int i = 0; i < n0 + end - t1; ++i) {
        const int p0 = (i < n0 ? i : t1 + i - n0) * kTile, off = p0 & (p.v.ps - 1);
        int page = p.table[b * p.table_stride + (p0 >> p.v.ps_shift)];
        unsigned live = c.len - p0 >= kTile ? 0xffffu : (1u << max(0, c.len - p0)) - 1;
        if (page < 0 || page >= p.v.n_pages) {
            if (lane == 0) raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
            page = 0;
            live = 0;
        }
        float s[2][4] = {};
        tile_scores<D, KF, T>(global_tile<KGeo<D, KF>::RB>(p.v, 0, page, h, off, live), g, t, qf, s);
        float mx[2] = {-INFINITY, -INFINITY};
        bool hidden = false;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = e >> 1, j = p0 + 8 * n + 2 * t + (e & 1);
                const bool see = j < c.len && ((j <= pos[k] && j >= lo[k]) || j < pre[k]);
                const float x = rule(s[n][e] * rule.factor(back[k]), abs(pos[k] - j), slope[k]);
                s[n][e] = see ? x : -INFINITY;
                hidden |= !see && base_row + g + 8 * k < rows;
                mx[k] = fmaxf(mx[k], s[n][e]);
            }
        float base[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            mx[k] = fmaxf(mx[k], __shfl_xor_sync(kAll, mx[k], 1));
            mx[k] = fmaxf(mx[k], __shfl_xor_sync(kAll, mx[k], 2));
            const float mn = fmaxf(m[k], mx[k]);
            base[k] = mn == -INFINITY ? 0.f : mn;
            const float a = ex2(m[k] - base[k]);
            m[k] = mn;
            l[k] *= a;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][2 * k] *= a;
                o[d][2 * k + 1] *= a;
            }
        }
        uint32_t pa[4], pl[4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float x = ex2(s[n][2 * k] - base[k]), y = ex2(s[n][2 * k + 1] - base[k]);
                l[k] += x + y;
                pa[2 * n + k] = Two<T>::pack(x, y);
            }
        const GlobalTile<VGeo<D, VF>::RB> vt = global_tile<VGeo<D, VF>::RB>(p.v, 1, page, h, off, live);
        // a weight of 0 does not keep an infinity or NaN out of the product: where some row does not see the
        // whole tile and the tile holds one, every row adds what it sees by itself
        const bool part = __any_sync(kAll, hidden);
        if (part && tile_nonfinite<D, VF, T>(vt, lane)) {
            add_seen<D, VF, T>(vt, g, t, s, base, o);
            continue;
        }
        tile_values<D, VF, T, false>(vt, g, t, pa, pl, o);
    }
    using V = VGeo<D, VF>;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(kAll, l[k], 1);
        l[k] += __shfl_xor_sync(kAll, l[k], 2);
        const int i = base_row + g + 8 * k;
        if (i >= rows) continue;
        const int64_t at = (int64_t)(c.row0 + i / G) * p.Hq + h * G + i % G;
        const float inv = l[k] > 0.f ? 1.f / l[k] : 0.f;
        TQ* out = (TQ*)p.out + at * D;
#pragma unroll
        for (int j = 0; j < V::NJ; ++j)
#pragma unroll
            for (int e = 0; e < V::CH; e += 2)
#pragma unroll
                for (int col = 0; col < 2; ++col)
                    *reinterpret_cast<uint32_t*>(out + ochan<D, VF>(j, 2 * t + col) + e) =
                        Two<TQ>::pack(o[V::CH * j + e][2 * k + col] * inv, o[V::CH * j + e + 1][2 * k + col] * inv);
        if (p.lse && t == 0) p.lse[at] = l[k] > 0.f ? (m[k] + log2f(l[k])) * kLn2 : -INFINITY;
    }
}

template <int D, int KF, int VF, typename T, typename TQ> int prefill_run(const PagedAttnParams& p, cudaStream_t s) {
    const dim3 grid((unsigned)(((int64_t)p.max_q * p.G + kRowsCta - 1) / kRowsCta), p.v.H, p.n_seq);
    prefill_kernel<D, KF, VF, T, TQ><<<grid, kPT, 0, s>>>(p);
    return (int)cudaGetLastError();
}

template <int D> int prefill_d(const PagedAttnParams& p, cudaStream_t s) {
    const int kf = p.v.fmt[0], vf = p.v.fmt[1];
    if (kf == KVQ_F16) return prefill_run<D, PF_16, PF_16, __half, __half>(p, s);
    if (kf == KVQ_BF16) return prefill_run<D, PF_16, PF_16, __nv_bfloat16, __nv_bfloat16>(p, s);
    if (p.dtype == KVQ_F16) {
        if (kf == KVQ_Q4_0) return prefill_run<D, PF_Q4, PF_Q4, __half, __half>(p, s);
        if (vf == KVQ_Q4_0) return prefill_run<D, PF_Q8, PF_Q4, __half, __half>(p, s);
        return prefill_run<D, PF_Q8, PF_Q8, __half, __half>(p, s);
    }
    if (kf == KVQ_Q4_0) return prefill_run<D, PF_Q4, PF_Q4, __half, __nv_bfloat16>(p, s);
    if (vf == KVQ_Q4_0) return prefill_run<D, PF_Q8, PF_Q4, __half, __nv_bfloat16>(p, s);
    return prefill_run<D, PF_Q8, PF_Q8, __half, __nv_bfloat16>(p, s);
}

}  // namespace

size_t paged_prefill_ws_floats(int, int, int, int64_t) { return 0; }

int launch_paged_prefill(PagedAttnParams p, int, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    if (p.v.D == 64) return prefill_d<64>(p, s);
    if (p.v.D == 128) return prefill_d<128>(p, s);
    return prefill_d<256>(p, s);
}

}  // namespace kvq
