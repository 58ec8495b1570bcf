// Chunks of a few tokens over e4m3 pages (drafted tokens looked at by the target): attention with few rows for each KV head, split over
// positions and joined.
//
// A head has tokens x G query rows here, up to 16, 32 or 64 of which are a group. As in decode, the 16-position tiles of all
// (sequence, KV head, group) are one line that is cut into equal runs, one per CTA, on the device; a CTA's four warps take the tiles
// of a run in turn, positions or channels on M of mma.sync, the group's rows on N in blocks of eight, two or four blocks a warp, and
// where those are not enough two warps on one tile. The rows' fragments wait in shared memory, one copy for the four warps; the outputs
// stay in registers.
// A run writes a group that it holds whole and leaves (m, l, o) of the at most two that its ends cut, which the merge kernel
// joins. Rows see different positions: where a tile is not seen whole by all of them the scores are hidden row by row, and rows
// of V that hold a NaN are added to the rows that see them and taken out before the product.
//
// On the tensor cores of the chunk kernel a tile of 128 rows would be a fifth full, and its softmax a chain of one
// tile after the other: 20 sequences of 12 tokens up to 16,001 positions, 40 heads on 8 x 128 (60 rows a KV head): 293 us there,
// 242 here, and of five tokens (25 rows) 139 (HBM's floor 64). Where little is held that kernel is the faster one (draft_better). Bound by latency: a tile of 16 positions takes a warp 590 instructions, the matrix pipe 540 of
// a scheduler's 1,550 cycles, and two warps a scheduler do not fill the waits between them. Other forms of the same batch: up to 16
// rows 113 us (two blocks of rows, three CTAs an SM; with four blocks 147); 25 rows as two warps on a tile 151; 4 x 256, 30
// rows 152 (as two groups 172). The scores of the next tile formed beside the values of this one: 143-149, the registers spill.
#include "device_common.cuh"
#include "paged_frag.cuh"

namespace kvq {
namespace {

constexpr int kDW = 4;                    // warps of a CTA
constexpr int kDT = kDW * 32;
constexpr int kMinTiles = 4;              // smallest run: one tile per warp
constexpr float kUp = 15.f, kFirst = 8.f; // as in decode: a maximum moves when a weight would be above 2^15, to the largest score less 8

// A sequence's rows and the tiles that any of them sees: [0, n0) and [t1, t1 + n - n0).
struct Rows {
    int row0, n, first, last, len, pre;   // first row of q; tokens; positions of the first and last one; positions held; prefix
    int n0, t1, tiles, groups;            // groups of the sequence's rows (none where no tile is seen)
    __device__ __forceinline__ int tile(int i) const { return i < n0 ? i : t1 + i - n0; }
};
template <int RP> __device__ __forceinline__ Rows rows_of(const PagedAttnParams& p, int b, bool report) {
    Rows s;
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    const int len = p.lens[b], c0 = p.cu[b], c1 = p.cu[b + 1];
    const bool bad = c0 < 0 || c1 > p.n_rows || c1 < c0;
    s.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
    s.row0 = c0;
    s.n = bad ? 0 : c1 - c0;
    if (report && (len < 0 || len > cap || bad || s.n > p.max_q)) raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
    s.first = s.len - s.n;
    s.n = min(s.n, p.max_q);
    s.last = s.first + s.n - 1;
    s.pre = p.prefix ? min(max(p.prefix[b], 0), s.len) : 0;
    const bool none = s.n == 0 || s.last < 0;
    const int end = none ? 0 : (max(s.last + 1, s.pre) + kTile - 1) / kTile;
    s.t1 = min(end, p.window > 0 && s.first >= p.window ? (s.first - p.window + 1) / kTile : 0);
    s.n0 = none ? 0 : min((s.pre + kTile - 1) / kTile, s.t1);
    s.tiles = s.n0 + end - s.t1;
    s.groups = s.tiles ? (s.n * p.G + RP - 1) / RP : 0;
    return s;
}

__device__ __forceinline__ int64_t run_tiles(int64_t total, int n_cta) {
    const int64_t u = (total + n_cta - 1) / n_cta;
    return u < kMinTiles ? kMinTiles : u;
}

template <int D, int NQ, int SPLIT> struct DGeo {                 // blocks of eight rows of a warp; warps on one tile
    static constexpr int RP = 8 * NQ * SPLIT, W = kDW / SPLIT;    // rows of a group; tiles in hand at a time
    static constexpr int ctas = draft_ctas(D, NQ);                // per SM
    static constexpr int tile = tile_bytes<D, PF_E4>(), slot = 2 * tile, q_bytes = RP * D * 2;
    static constexpr int fit = ((226 / ctas - 3) * 1024 - q_bytes) / W / slot, NS = fit > 8 ? 8 : fit;
    static constexpr int join = W * RP * D * 4;                   // the outputs at a group's end
    static constexpr int rings = NS * slot * W > join ? NS * slot * W : join;
    static constexpr int smem = q_bytes + rings, part = 2 * RP + RP * D;
    static_assert(NS >= 3, "tiles in flight beside the one in use");
};
// The warps on one tile wait for one another.
template <int SPLIT> __device__ __forceinline__ void sync_tile(int stream) {
    if constexpr (SPLIT == 1) __syncwarp();
    else asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(1 + stream), "n"(32 * SPLIT) : "memory");
}

// s[q] += K Q^T: a piece of K decoded, then all blocks of rows from their fragments at `q`.
template <int D, int NQ, typename PLACE>
__device__ __forceinline__ void draft_scores(uint32_t base, const PLACE& at, uint32_t q, float (&s)[NQ][4]) {
    using K = KGeo<D, PF_E4>;
    constexpr int KS = K::CH / 16;                                // pairs of k-steps of a piece
#pragma unroll
    for (int j = 0; j < K::NJ; ++j) {
        const uint32_t a = base + (j & 1 ? at.k[1] : at.k[0]) + j / 2 * 128;
        const Words<K::NW> x = ld_words<K::NW>(a), y = ld_words<K::NW>(a + 8 * K::RB);     // rows g, g + 8
        uint32_t f[K::NW][4];
#pragma unroll
        for (int i = 0; i < K::NW; ++i) {
            e4m3_four(x.w[i], f[i][0], f[i][2]);
            e4m3_four(y.w[i], f[i][1], f[i][3]);
        }
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {                        // a block's products wait for one another: the blocks in turn
            Words<4> z[NQ];
#pragma unroll
            for (int k = 0; k < NQ; ++k) z[k] = ld_words<4>(q + ((k * (D / 32) + 2 * KS * j + i) * 32) * 16);
#pragma unroll
            for (int k = 0; k < NQ; ++k) mma_t(s[k], f[2 * i], z[k].w[0], z[k].w[1], __half());
#pragma unroll
            for (int k = 0; k < NQ; ++k) mma_t(s[k], f[2 * i + 1], z[k].w[2], z[k].w[3], __half());
        }
    }
}

template <int D, int NQ, int SPLIT, typename TQ>
__global__ void __launch_bounds__(kDT, draft_ctas(D, NQ)) draft_kernel(PagedAttnParams p) {
    using GE = DGeo<D, NQ, SPLIT>;
    constexpr int RP = GE::RP, W = GE::W;
    extern __shared__ __align__(128) float smem[];                // fragments of the rows; the rings, or [W][RP][D] outputs
    __shared__ float s_m[W][RP], s_l[W][RP], s_f[RP];
    __shared__ int64_t red[kDW];
    __shared__ int s_b, s_h, s_i;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int H = p.v.H, G = p.G;
    const int stream = warp / SPLIT, half = warp % SPLIT, block0 = half * NQ;     // the warp's tiles; its rows' first block
    const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(smem), ring = q_at + GE::q_bytes + stream * GE::NS * GE::slot;
    float* s_out = smem + GE::q_bytes / 4;
    grid_dep_wait();

    // this CTA's run of the line, and the (sequence, head and group, tile) where it starts
    int64_t mine = 0;
    const int per = (p.n_seq + kDT - 1) / kDT;
    for (int b = threadIdx.x * per; b < min(p.n_seq, (int)(threadIdx.x + 1) * per); ++b) {
        const Rows r = rows_of<RP>(p, b, blockIdx.x == 0);
        mine += (int64_t)r.tiles * r.groups * H;
    }
    int64_t before = mine;                                        // inclusive scan over the warp
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int64_t y = __shfl_up_sync(kAll, before, s);
        if (lane >= s) before += y;
    }
    if (lane == 31) red[warp] = before;
    __syncthreads();
    int64_t total = 0;
    for (int i = 0; i < kDW; ++i) {
        if (i < warp) before += red[i];
        total += red[i];
    }
    before -= mine;
    const int64_t U = run_tiles(total, p.n_cta), first = blockIdx.x * U;
    if (blockIdx.x == 0) {                                        // tiles before each sequence, for the merge
        int64_t* line = (int64_t*)p.ws;
        int64_t at = before;
        for (int b = threadIdx.x * per; b < min(p.n_seq, (int)(threadIdx.x + 1) * per); ++b) {
            line[b] = at;
            const Rows r = rows_of<RP>(p, b, false);
            at += (int64_t)r.tiles * r.groups * H;
        }
        if (threadIdx.x == 0) line[p.n_seq] = total;
    }
    for (int b = blockIdx.x; b < p.n_seq; b += gridDim.x) {       // rows that see nothing give zeros
        const Rows r = rows_of<RP>(p, b, false);
        if (r.tiles) continue;
        uint4* out = reinterpret_cast<uint4*>((TQ*)p.out + (int64_t)r.row0 * p.Hq * D);
        for (int64_t e = threadIdx.x; e < (int64_t)r.n * p.Hq * D / 8; e += kDT) out[e] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int e = threadIdx.x; e < r.n * p.Hq; e += kDT) p.lse[(int64_t)r.row0 * p.Hq + e] = -INFINITY;
    }
    int64_t left = min(U, total - first);
    if (left <= 0) return;
    if (first >= before && first < before + mine) {
        int64_t at = first - before;
        for (int b = threadIdx.x * per;; ++b) {
            const Rows r = rows_of<RP>(p, b, false);
            const int64_t n = (int64_t)r.tiles * r.groups * H;
            if (at < n) {
                s_b = b;
                s_h = (int)(at / r.tiles);
                s_i = (int)(at % r.tiles);
                break;
            }
            at -= n;
        }
    }
    __syncthreads();
    int b = s_b, hg = s_h, i0 = s_i;                              // hg: KV head x groups + group
    const ScoreRule rule = score_rule(p);
    const bool plain = rule.plain();
    const LanePlace<D, PF_E4, PF_E4> place(g, t);
    const uint32_t k_at = copy_lane<D, PF_E4, false>(lane), v_at = copy_lane<D, PF_E4, true>(lane);

    for (; left > 0; ++hg, i0 = 0) {
        Rows st = rows_of<RP>(p, b, false);
        if (hg >= H * st.groups) {
            ++b;
            hg = -1;
            continue;
        }
        const int h = hg / st.groups, base_row = hg % st.groups * RP, rows = min(RP, st.n * G - base_row);
        const int i1 = (int)min((int64_t)st.tiles, i0 + left);
        left -= i1 - i0;
        const int nt = (i1 - i0 - stream + W - 1) / W;            // this warp's tiles
        // the copies run ahead, K and V of a tile in one slot (of two warps one brings K, the other V)
        int pages = 0, unit_page = 0, unit_off = 0, put = 0, item = 0;
        auto copy_next = [&]() {
            if (item < nt) {
                const uint32_t dst = ring + put * GE::slot;
                if ((item & 31) == 0) {                           // the next 32 tiles' page numbers, one per lane
                    const int k = min(item + lane, nt - 1) * W + i0 + stream;
                    pages = p.table[b * p.table_stride + ((st.tile(k) * kTile) >> p.v.ps_shift)];
                    if (pages < 0 || pages >= p.v.n_pages) {
                        raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
                        pages = -1;
                    } else {
                        pages = pages * H + h;                    // the unit's number
                    }
                }
                unit_page = __shfl_sync(kAll, pages, item & 31);
                unit_off = (st.tile(item * W + i0 + stream) * kTile) & (p.v.ps - 1);
                const auto unit = [&](int w) -> const uint8_t* {
                    return unit_page < 0 ? nullptr : p.v.base[w] + (uint64_t)(uint32_t)unit_page * (uint32_t)p.v.unit[w];
                };
                if (half == 0) copy_tile<D, PF_E4, false>(dst, k_at, unit(0), p.v.ps, unit_off, lane);
                if (half == SPLIT - 1) copy_tile<D, PF_E4, true>(dst + GE::tile, v_at, unit(1), p.v.ps, unit_off, lane);
            }
            cp_commit();
            ++item;
            put = put + 1 == GE::NS ? 0 : put + 1;
        };
#pragma unroll 1
        for (int i = 0; i < GE::NS - 1; ++i) copy_next();

        // the rows' fragments, a block of eight rows a warp
        for (int k = warp; k < RP / 8; k += kDW) {
            uint32_t qf[D / 16][1][2];
            float back[1];
            load_queries<D, PF_E4, 1, __half, TQ>(
                [&](int r) {
                    r += 8 * k;
                    if (r >= rows) return (const TQ*)nullptr;
                    const int x = base_row + r, tok = x / G;
                    return (const TQ*)p.q + (int64_t)(st.row0 + tok) * p.q_stride + (int64_t)(h * G + x - tok * G) * D;
                },
                g, t, qf, back);
            if (t == 0) s_f[8 * k + g] = fminf(rule.factor(back[0]), kMaxFactor);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(q_at + ((k * (D / 32) + i) * 32 + lane) * 16), "r"(qf[2 * i][0][0]),
                             "r"(qf[2 * i][0][1]), "r"(qf[2 * i + 1][0][0]), "r"(qf[2 * i + 1][0][1])
                             : "memory");
        }
        __syncthreads();
        float f[NQ][2], m[NQ][2], l[NQ][2] = {}, o[D / 16][NQ][4] = {};
#pragma unroll
        for (int k = 0; k < NQ; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[k][e] = s_f[8 * (block0 + k) + 2 * t + e];
                m[k][e] = -INFINITY;
            }
        // position of a row of the group (rows behind the last one: the last token's)
        const auto row_at = [&](int k, int e) { return 8 * (block0 + k) + 2 * t + e; };
        const auto pos_of = [&](int r) { return st.first + min(base_row + r, st.n * G - 1) / G; };
        const int lo_last = p.window > 0 && st.last >= p.window ? st.last - p.window + 1 : 0;
        ValueScale values;
        int get = 0;
        for (int i = 0; i < nt; ++i) {
            const int p0 = st.tile(i * W + i0 + stream) * kTile;
            cp_wait<GE::NS - 2>();
            sync_tile<SPLIT>(stream);                             // the tile has landed, and the one before it is done with
            const uint32_t k_tile = ring + get * GE::slot, v_tile = k_tile + GE::tile;
            get = get + 1 == GE::NS ? 0 : get + 1;
            copy_next();
            float s[NQ][4] = {};                                  // (position g, g + 8) x (row 2t, 2t + 1)
            draft_scores<D, NQ>(k_tile, place, q_at + (block0 * D + lane) * 16, s);
            const bool all = st.first >= 0 && (p0 + kTile <= st.pre || (p0 + kTile - 1 <= st.first && p0 >= lo_last));
            const float d = tile_scale<D>(k_tile);
#pragma unroll
            for (int k = 0; k < NQ; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[k][c] *= f[k][c & 1] * d;
            // does the row at position x see position j?
            const auto sees = [&](int x, int j) {
                return x >= 0 && ((j <= x && (p.window <= 0 || j > x - p.window)) || j < st.pre);
            };
            if (!plain) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = row_at(k, e), x = pos_of(r);
                        const float slope = p.slopes && r < rows ? p.slopes[h * G + (base_row + r) % G] * kL2e : 0.f;
                        s[k][e] = rule(s[k][e], abs(x - p0 - g), slope);
                        s[k][2 + e] = rule(s[k][2 + e], abs(x - p0 - g - 8), slope);
                    }
            }
            if (!all) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int x = pos_of(row_at(k, e));
                        if (!sees(x, p0 + g)) s[k][e] = -INFINITY;
                        if (!sees(x, p0 + g + 8)) s[k][2 + e] = -INFINITY;
                    }
            }
            bool moved = false;                                   // one vote says whether a maximum has to move
#pragma unroll
            for (int k = 0; k < NQ; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) moved |= fmaxf(s[k][e], s[k][2 + e]) > m[k][e] + kUp;
            if (__any_sync(kAll, moved)) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[k][e], s[k][2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
                        if (mx > m[k][e] + kUp) {
                            const float a = ex2(m[k][e] - (mx - kFirst));
                            m[k][e] = mx - kFirst;
                            l[k][e] *= a;
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                o[c][k][e] *= a;
                                o[c][k][2 + e] *= a;
                            }
                        }
                    }
            }
            const float by = values.take(tile_scale<D>(v_tile), [&](float x) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
#pragma unroll
                    for (int k = 0; k < NQ; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[c][k][e] *= x;
            });
            uint32_t pb[NQ][2], lo[NQ][2];
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
                const float b0 = m[k][0] == -INFINITY ? 0.f : m[k][0], b1 = m[k][1] == -INFINITY ? 0.f : m[k][1];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x = ex2(s[k][2 * n] - b0), y = ex2(s[k][2 * n + 1] - b1);
                    l[k][0] += x;
                    l[k][1] += y;
                    s[k][2 * n] = x * by;
                    s[k][2 * n + 1] = y * by;
                    pb[k][n] = transpose8(Two<__half>::pack(x * by, y * by));
                }
            }
            if (!all) {
                // rows of V with a NaN: lane r looks at row r
                using V = VGeo<D, PF_E4>;
                bool odd = false;
                if (lane < kTile)
                    for (int c = 0; c < D; c += 16) {
                        const Words<4> x = ld_words<4>(v_tile + tile_swizzle<D, true>(lane * D + c));
#pragma unroll
                        for (int i = 0; i < 4; ++i) odd |= __vcmpeq4(x.w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                    }
                const unsigned bad = __ballot_sync(kAll, odd);
                for (unsigned rest = bad; rest; rest &= rest - 1) {
                    const int j = __ffs(rest) - 1;
                    float w[NQ][2];
#pragma unroll
                    for (int k = 0; k < NQ; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float u = __shfl_sync(kAll, s[k][e], 4 * (j & 7) + t), v = __shfl_sync(kAll, s[k][2 + e], 4 * (j & 7) + t);
                            w[k][e] = j < 8 ? u : v;
                        }
#pragma unroll
                    for (int jj = 0; jj < V::NJ; ++jj) {
                        const Words<V::NW> x = ld_words<V::NW>(v_tile + tile_swizzle<D, true>(j * D + V::CB * (g + 8 * jj)));
#pragma unroll
                        for (int c = 0; c < V::CH; c += 2) {
                            const float2 y = __half22float2(h2(e4m3_pair(x.w[c / 4] >> (8 * (c & 2)) & 0xffffu)));
#pragma unroll
                            for (int k = 0; k < NQ; ++k)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (sees(pos_of(row_at(k, e)), p0 + j)) {
                                        float (&acc)[4] = o[(V::CH * jj + c) / 2][k];
                                        acc[e] = fmaf(w[k][e], y.x, acc[e]);
                                        acc[2 + e] = fmaf(w[k][e], y.y, acc[2 + e]);
                                    }
                        }
                    }
                }
                if (bad) {
                    sync_tile<SPLIT>(stream);
                    clear_rows<D, PF_E4>(v_tile, ~bad, lane);
                    sync_tile<SPLIT>(stream);
                }
            }
            tile_values<D, PF_E4, NQ, __half, false>(v_tile, place, pb, lo, o);
        }
        cp_wait<0>();
        __syncthreads();                                          // the rings become the join's space

        // join the warps: rows' maxima and sums, then the outputs rescaled to the common maximum
#pragma unroll
        for (int k = 0; k < NQ; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[k][e] += __shfl_xor_sync(kAll, l[k][e], 4);
                l[k][e] += __shfl_xor_sync(kAll, l[k][e], 8);
                l[k][e] += __shfl_xor_sync(kAll, l[k][e], 16);
                if (g == 0) {
                    s_m[stream][row_at(k, e)] = m[k][e];
                    s_l[stream][row_at(k, e)] = l[k][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NQ; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row_at(k, e);
                float mm = -INFINITY;
                for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][r]);
                const float a = (mm == -INFINITY ? 0.f : ex2(m[k][e] - mm)) * values.unit;
                float* dst = s_out + (stream * RP + r) * D;
                using V = VGeo<D, PF_E4>;
#pragma unroll
                for (int j = 0; j < V::NJ; ++j)
#pragma unroll
                    for (int c = 0; c < V::CH; ++c) dst[ochan<D, PF_E4>(j, g) + c] = o[(V::CH * j + c) / 2][k][2 * (c & 1) + e] * a;
            }
        __syncthreads();
        const bool whole = i0 == 0 && i1 == st.tiles;
        // a run leaves at most two partials: of a group that it goes on with, and of one that it begins
        float* part = p.ws + line_floats(p.n_seq) + ((int64_t)blockIdx.x * 2 + (i0 == 0)) * GE::part;
        for (int e = threadIdx.x; e < rows * D / 2; e += kDT) {
            const int r = 2 * e / D;
            float x = 0.f, y = 0.f;
            for (int w = 0; w < W; ++w) {
                const float2 z = *reinterpret_cast<const float2*>(s_out + w * RP * D + 2 * e);
                x += z.x;
                y += z.y;
            }
            if (whole) {
                float mm = -INFINITY, ll = 0.f;
                for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][r]);
                for (int w = 0; w < W; ++w) ll += s_l[w][r] * (mm == -INFINITY ? 0.f : ex2(s_m[w][r] - mm));
                const float inv = inverse_sum(ll);
                const int z = base_row + r, tok = z / G;
                const int64_t at = (int64_t)(st.row0 + tok) * p.Hq + h * G + z - tok * G;
                reinterpret_cast<uint32_t*>((TQ*)p.out + at * D)[e - r * (D / 2)] = Two<TQ>::pack(x * inv, y * inv);
            } else {
                *reinterpret_cast<float2*>(part + 2 * RP + 2 * e) = make_float2(x, y);
            }
        }
        if (threadIdx.x < rows) {
            const int r = threadIdx.x;
            float mm = -INFINITY, ll = 0.f;
            for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][r]);
            for (int w = 0; w < W; ++w) ll += s_l[w][r] * (mm == -INFINITY ? 0.f : ex2(s_m[w][r] - mm));
            if (!whole) {
                part[r] = mm;
                part[RP + r] = ll;
            } else if (p.lse) {
                const int z = base_row + r, tok = z / G;
                p.lse[(int64_t)(st.row0 + tok) * p.Hq + h * G + z - tok * G] = log_sum(mm, ll);
            }
        }
        __syncthreads();
    }
}

// Joins the partials of the groups that runs share: a block per run and eight rows of a group. At most one group is cut by the start of
// a run, and its first cut joins it: a warp a row.
constexpr int kMT = 256;
template <int D, int RP, typename TQ> __global__ void __launch_bounds__(kMT) draft_merge_kernel(PagedAttnParams p) {
    constexpr int PF = 2 * RP + RP * D, C = D / 32;      // floats of a partial, channels of a lane
    grid_dep_wait();
    const int64_t* line = (const int64_t*)p.ws;
    const int id = blockIdx.x, G = p.G, lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int64_t total = line[p.n_seq], U = run_tiles(total, p.n_cta), at = (int64_t)id * U;
    if (id == 0 || at >= total) return;
    int b = 0, hi = p.n_seq - 1;                         // the last sequence that starts at or before the run
    while (b < hi) {
        const int mid = (b + hi + 1) >> 1;
        if (line[mid] <= at) b = mid; else hi = mid - 1;
    }
    const Rows st = rows_of<RP>(p, b, false);
    const int hg = (int)((at - line[b]) / st.tiles);
    const int64_t s0 = line[b] + (int64_t)hg * st.tiles;
    const int c0 = (int)(s0 / U), nc = (int)((s0 + st.tiles - 1) / U) - c0 + 1;
    if (s0 == at || c0 != id - 1) return;                // not cut here, or cut before
    const int h = hg / st.groups, row = hg % st.groups * RP + r;
    if (row >= st.n * G) return;
    const float* base = p.ws + line_floats(p.n_seq);
    // the partial of run c0 + c: the group begins in the first one
    const auto part = [&](int c) { return base + ((int64_t)(c0 + c) * 2 + (c == 0)) * PF; };
    float m = -INFINITY, l = 0.f;
    for (int c = lane; c < nc; c += 32) m = fmaxf(m, part(c)[r]);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, s));
    float o[C] = {};
#pragma unroll 4
    for (int c = 0; c < nc; ++c) {
        const float* x = part(c);
        const float a = m == -INFINITY ? 0.f : ex2(x[r] - m);
        l += x[RP + r] * a;
#pragma unroll
        for (int e = 0; e < C; e += 2) {
            const float2 y = *reinterpret_cast<const float2*>(x + 2 * RP + r * D + lane * C + e);
            o[e] = fmaf(y.x, a, o[e]);
            o[e + 1] = fmaf(y.y, a, o[e + 1]);
        }
    }
    const float inv = inverse_sum(l);
    const int tok = row / G;
    const int64_t to = (int64_t)(st.row0 + tok) * p.Hq + h * G + row - tok * G;
    uint32_t* out = reinterpret_cast<uint32_t*>((TQ*)p.out + to * D + lane * C);
#pragma unroll
    for (int e = 0; e < C; e += 2) out[e / 2] = Two<TQ>::pack(o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[to] = log_sum(m, l);
}

template <int D, int NQ, int SPLIT, typename TQ> int draft_run(const PagedAttnParams& p, int sm_count, cudaStream_t s) {
    PagedAttnParams a = p;
    using GE = DGeo<D, NQ, SPLIT>;
    static_assert(GE::part * GE::ctas <= draft_part_floats(D), "the workspace's");
    const auto k = draft_kernel<D, NQ, SPLIT, TQ>;
    int res = 0;
    if (const int e = resident_ctas((const void*)k, kDT, GE::smem, &res)) return e;
    a.n_cta = min(kMaxSms * GE::ctas, sm_count * res);
    cudaError_t e = launch_k(k, dim3(a.n_cta), dim3(kDT), GE::smem, s, true, a);
    if (e == cudaSuccess) e = launch_k(draft_merge_kernel<D, GE::RP, TQ>, dim3((unsigned)a.n_cta, GE::RP / 8), dim3(kMT), 0, s, true, a);
    return (int)e;
}
template <int D, typename TQ> int draft_rows_run(const PagedAttnParams& p, int sm_count, cudaStream_t s) {
    const int rows = p.max_q * p.G;
    if (rows <= 16) return draft_run<D, 2, 1, TQ>(p, sm_count, s);
    if constexpr (D == 256) return draft_run<D, 2, 2, TQ>(p, sm_count, s);
    else return rows <= 32 ? draft_run<D, 4, 1, TQ>(p, sm_count, s) : draft_run<D, 4, 2, TQ>(p, sm_count, s);
}

}  // namespace

// One head dimension per compilation of this file (KVQ_D), so that they build side by side.
#define KVQ_NAME2(d) launch_paged_draft_##d
#define KVQ_NAME(d) KVQ_NAME2(d)
int KVQ_NAME(KVQ_D)(const PagedAttnParams& p, int sms, void* stream) {
    return p.dtype == KVQ_F16 ? draft_rows_run<KVQ_D, __half>(p, sms, (cudaStream_t)stream)
                              : draft_rows_run<KVQ_D, __nv_bfloat16>(p, sms, (cudaStream_t)stream);
}

}  // namespace kvq
