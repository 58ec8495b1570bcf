// Decode attention over pages: one query per sequence, split over positions and joined.
//
// The work is one line of 16-position tiles: sequences in order, in each its KV heads in order, in
// each head the tiles that hold a visible position. The line is cut into equal runs, one per CTA, on
// the device (lengths are device arrays), so ragged batches balance and a captured call follows new
// lengths. A CTA's four warps take the tiles of a run in turn, each with its own running maximum, sum
// and output (fp32, registers); at the end of a head they join through shared memory. A head that lies
// in one run is written out at once; others leave (m, l, o) per run, which the merge kernel joins.
//
// Bound by HBM over 16-bit pages (48 ragged sequences up to 24,001 positions, 8 x 128 bf16: 407 us, 99% of the measured
// rate; 4 up to 262,144, 4 x 256 fp16: 465 us, 104%), by the instructions that turn codes into operands over
// quantised ones (131,072 positions, 8 x 128, q8_0 / q4_0: 59 us, 54%; issue slots 65% busy, two thirds of the 566
// instructions of a tile in the two products' decoding). Groups of 16, two query tiles a warp: 16 sequences up to 32,768 on
// 2 x 128, fp16 94 us (65%), q8_0 / q4_0 68 us (37%).
//
// e4m3 pages (24 ragged sequences up to 50,001, 8 x 128: 236 us, 81%): a code becomes fp16 by one conversion for two, and the scales,
// one for a tile, go to the scores and to the weights, 320 instructions a tile. What is left is latency (four warps a scheduler,
// issue slots 39-42% busy) and SMs that end before others (a tenth of the time: with six times as many runs 235 us against 252 there,
// but one sequence of 131,072 106 us against 78). Three CTAs an SM 260 us, five 270.
#include "device_common.cuh"
#include "paged_frag.cuh"

namespace kvq {
namespace {

constexpr int kDW = 4;                    // warps of a CTA
constexpr int kDT = kDW * 32;
constexpr int kMinTiles = 4;              // smallest run: one tile per warp

// Visible tiles of a sequence: [0, n0) (the prefix) and [t1, t1 + n1) (the window, or everything).
struct SeqTiles {
    int len, lo, pre, n0, t1, n;          // n: tiles in all
    __device__ __forceinline__ int tile(int i) const { return i < n0 ? i : t1 + i - n0; }
    __device__ __forceinline__ bool sees(int pos) const { return pos < len && (pos >= lo || pos < pre); }
};
__device__ __forceinline__ SeqTiles seq_tiles(const PagedAttnParams& p, int b) {
    SeqTiles s;
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    const int n = p.lens[b];
    s.len = n < 0 ? 0 : (n > cap ? (int)cap : n);
    s.lo = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
    const int x = p.prefix ? p.prefix[b] : 0;
    s.pre = min(max(x, 0), s.len);
    const int end = (s.len + kTile - 1) / kTile;
    s.t1 = s.lo / kTile;
    s.n0 = min((s.pre + kTile - 1) / kTile, s.t1);
    s.n = s.n0 + end - s.t1;
    return s;
}

__device__ __forceinline__ int64_t run_tiles(int64_t total, int n_cta) {
    const int64_t u = (total + n_cta - 1) / n_cta;
    return u < kMinTiles ? kMinTiles : u;
}

// Each warp stages its tiles through a ring of its own in shared memory, K and V tiles in turn or together, NS slots
// with NS - 1 copies in flight (cp.async; no barrier but the warp's). Rows of codes keep the warps busy with decoding, so
// there a third (D = 256) or fourth CTA an SM is worth more than deeper rings; 16-bit rows want the bytes in flight.
template <int D, int KF, int VF, int NQ> struct Ring {
    static constexpr int ctas = (D == 256 ? 2 : 3) + (KF != PF_16 && NQ == 1 ? 1 : 0);   // per SM
    static constexpr int kb = tile_bytes<D, KF>(), vb = tile_bytes<D, VF>();
    static constexpr int budget = (226 / ctas - 2) * 1024 / kDW;
    // K and V of a tile in one slot, copied and awaited together (half of the bookkeeping), where three such slots fit
    static constexpr bool one = KF != PF_16 && budget / (kb + vb) >= 3;
    static constexpr int slot = one ? kb + vb : (kb > vb ? kb : vb);
    static constexpr int fit = budget / slot;
    static constexpr int NS = fit > 8 ? 8 : fit;
    static constexpr int join = 8 * NQ * D * 4 * kDW;      // the warps' outputs at a head's end
    static constexpr int bytes = NS * slot * kDW > join ? NS * slot * kDW : join;
    static_assert(NS >= 3, "a tile of each kind in flight beside the one in use");
};

template <int D, int KF, int VF, int NQ, typename T, typename TQ>
__global__ void __launch_bounds__(kDT, (Ring<D, KF, VF, NQ>::ctas)) decode_kernel(PagedAttnParams p) {
    constexpr bool LO = std::is_same<T, __nv_bfloat16>::value;   // P in two bf16 parts: 16 bits of it
    // fp16 weights are 2^(s - (max - 15)): the largest is 2^15, and those down to 2^-29 of it keep all bits, down to 2^-40 some
    // (at 2^(s - max) what lies 2^-25 below the largest would be lost to the outputs but not to the sums). m is max - kUp
    // everywhere, sums and outputs are in its units; bf16 has the exponents.
    // e4m3: m moves only when a weight would be above 2^15, and then to the largest score less kFirst.
    constexpr float kUp = LO ? 0.f : 15.f, kFirst = 8.f;
    using R = Ring<D, KF, VF, NQ>;
    extern __shared__ __align__(128) float smem[];               // the rings; [kDW][G][D] outputs at a head's end
    __shared__ float s_m[kDW][16], s_l[kDW][16];
    __shared__ int64_t red[kDW];
    __shared__ int s_b, s_h, s_i;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int H = p.v.H, G = p.G;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * R::NS * R::slot;
    grid_dep_wait();

    // this CTA's run of the line, and the head where it starts
    int64_t mine = 0;
    const int per = (p.n_seq + kDT - 1) / kDT;
    for (int b = threadIdx.x * per; b < min(p.n_seq, (int)(threadIdx.x + 1) * per); ++b) {
        mine += (int64_t)seq_tiles(p, b).n * H;
        const int n = p.lens[b];
        if (blockIdx.x == 0 && (n < 0 || n > ((int64_t)p.max_pages << p.v.ps_shift))) raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
    }
    int64_t before = mine;                                       // inclusive scan over the warp
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
    // a launch that leaves half of its CTAs without work lets the merge's start beside it (in a full one they would
    // take the place of its own)
    if (total <= p.n_cta / 2 * U) grid_dep_launch();
    if (blockIdx.x == 0) {                                       // tiles before each sequence, for the merge
        int64_t* line = (int64_t*)p.ws;
        int64_t at = before;
        for (int b = threadIdx.x * per; b < min(p.n_seq, (int)(threadIdx.x + 1) * per); ++b) {
            line[b] = at;
            at += (int64_t)seq_tiles(p, b).n * H;
        }
        if (threadIdx.x == 0) line[p.n_seq] = total;
    }
    for (int b = blockIdx.x; b < p.n_seq; b += gridDim.x) {      // sequences without a visible position give zeros
        if (seq_tiles(p, b).n) continue;
        uint32_t* out = reinterpret_cast<uint32_t*>((TQ*)p.out + (int64_t)b * p.Hq * D);
        for (int e = threadIdx.x; e < p.Hq * D / 2; e += kDT) out[e] = 0;
        if (p.lse)
            for (int e = threadIdx.x; e < p.Hq; e += kDT) p.lse[(int64_t)b * p.Hq + e] = -INFINITY;
    }
    int64_t left = min(U, total - first);
    if (left <= 0) return;
    if (first >= before && first < before + mine) {
        int64_t at = first - before;
        for (int b = threadIdx.x * per;; ++b) {
            const int64_t n = seq_tiles(p, b).n;
            if (at < n * H) {
                s_b = b;
                s_h = (int)(at / n);
                s_i = (int)(at % n);
                break;
            }
            at -= n * H;
        }
    }
    __syncthreads();
    int b = s_b, h = s_h, i0 = s_i;
    const ScoreRule rule = score_rule(p);
    const bool plain = rule.plain();
    const LanePlace<D, KF, VF> place(g, t);
    const uint32_t k_at = copy_lane<D, KF, false>(lane), v_at = copy_lane<D, VF, true>(lane);

    for (; left > 0; ++h, i0 = 0) {
        if (h == H) { h = 0; ++b; }
        const SeqTiles st = seq_tiles(p, b);
        if (st.n == 0) { h = H - 1; continue; }
        const int i1 = (int)min((int64_t)st.n, i0 + left);
        left -= i1 - i0;
        const int nt = (i1 - i0 - warp + kDW - 1) / kDW;          // this warp's tiles
        // the copies run ahead: item 2i is K of the warp's tile i, item 2i + 1 its V; with one slot for both, item i
        int pages = 0, unit_page = 0, unit_off = 0, put = 0, item = 0;
        auto copy_next = [&]() {
            const int i = R::one ? item : item >> 1;
            if (i < nt) {
                const uint32_t dst = ring + put * R::slot;
                if (R::one || !(item & 1)) {
                    if ((i & 31) == 0) {                         // the next 32 tiles' page numbers, one per lane
                        const int k = min(i + lane, nt - 1) * kDW + i0 + warp;
                        pages = p.table[b * p.table_stride + ((st.tile(k) * kTile) >> p.v.ps_shift)];
                        if (pages < 0 || pages >= p.v.n_pages) {
                            raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
                            pages = -1;
                        } else {
                            pages = pages * H + h;               // the unit's number
                        }
                    }
                    unit_page = __shfl_sync(kAll, pages, i & 31);
                    unit_off = (st.tile(i * kDW + i0 + warp) * kTile) & (p.v.ps - 1);
                }
                const auto unit = [&](int w) -> const uint8_t* {
                    return unit_page < 0 ? nullptr : p.v.base[w] + (uint64_t)(uint32_t)unit_page * (uint32_t)p.v.unit[w];
                };
                if (R::one || !(item & 1)) copy_tile<D, KF, false>(dst, k_at, unit(0), p.v.ps, unit_off, lane);
                if (R::one || (item & 1)) copy_tile<D, VF, true>(dst + (R::one ? R::kb : 0), v_at, unit(1), p.v.ps, unit_off, lane);
            }
            cp_commit();
            ++item;
            put = put + 1 == R::NS ? 0 : put + 1;
        };
#pragma unroll 1
        for (int i = 0; i < R::NS - 1; ++i) copy_next();
        int get = 0;
        // the next item has landed, and the slot of the item before it is free for a new copy
        auto take = [&]() -> uint32_t {
            cp_wait<R::NS - 2>();
            __syncwarp();
            const uint32_t a = ring + get * R::slot;
            get = get + 1 == R::NS ? 0 : get + 1;
            return a;
        };

        const TQ* q = (const TQ*)p.q + b * p.q_stride + (int64_t)h * G * D;
        // by query group and the lane's two queries in it (8 q + 2 t, 8 q + 2 t + 1)
        uint32_t qf[D / 16][NQ][2];
        float f[NQ][2], slope[NQ][2], m[NQ][2], l[NQ][2] = {}, o[D / 16][NQ][4] = {}, back[NQ];
        load_queries<D, KF, NQ, T, TQ>([&](int r) { return r < G ? q + r * D : (const TQ*)nullptr; }, g, t, qf, back);
#pragma unroll
        for (int k = 0; k < NQ; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * k + 2 * t + e;
                f[k][e] = rule.factor(__shfl_sync(kAll, back[k], 4 * (2 * t + e)));
                if constexpr (KF == PF_E4) f[k][e] = fminf(f[k][e], kMaxFactor);
                slope[k][e] = p.slopes && r < G ? p.slopes[h * G + r] * kL2e : 0.f;
                m[k][e] = -INFINITY;
            }

        ValueScale values;
        for (int i = 0; i < nt; ++i) {
            const int p0 = st.tile(i * kDW + i0 + warp) * kTile;
            const uint32_t k_tile = take();
            copy_next();
            float s[NQ][4] = {};                                  // (position g, g + 8) x (query 2t, 2t + 1)
            tile_scores<D, KF, NQ, T>(k_tile, place, qf, s);
            const bool all = p0 + kTile <= st.len && (p0 >= st.lo || p0 + kTile <= st.pre);
            unsigned see = 0xffffu;
            if (!all) see = __ballot_sync(kAll, lane < 16 && st.sees(p0 + lane));
            if constexpr (KF == PF_E4) {
                const float d = tile_scale<D>(k_tile);
#pragma unroll
                for (int k = 0; k < NQ; ++k) {
                    const float f0 = f[k][0] * d, f1 = f[k][1] * d;
                    s[k][0] *= f0;
                    s[k][1] *= f1;
                    s[k][2] *= f0;
                    s[k][3] *= f1;
                }
            } else {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[k][c] *= f[k][c & 1];
            }
            if (!plain) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[k][c] = rule(s[k][c], st.len - 1 - p0 - (g + 8 * (c >> 1)), slope[k][c & 1]);
            }
            if (!all) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!((see >> (g + 8 * (c >> 1))) & 1)) s[k][c] = -INFINITY;
            }
            float base[NQ][2], a[NQ][2], by = 1.f;
            bool moved = KF != PF_E4;
            if constexpr (KF == PF_E4) {                          // one vote says whether the maximum has to move
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) moved |= fmaxf(s[k][e], s[k][2 + e]) > m[k][e] + kUp;
                moved = __any_sync(kAll, moved);
            }
            if (moved) {
                moved = false;
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[k][e], s[k][2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
                        float mn = fmaxf(m[k][e], mx - kUp);
                        if constexpr (KF == PF_E4) mn = mx > m[k][e] + kUp ? mx - kFirst : m[k][e];
                        moved |= m[k][e] != mn;
                        a[k][e] = m[k][e];
                        m[k][e] = mn;
                    }
            }
#pragma unroll
            for (int k = 0; k < NQ; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) base[k][e] = m[k][e] == -INFINITY ? 0.f : m[k][e];
            if (KF == PF_E4 ? moved : __any_sync(kAll, moved)) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[k][e] = a[k][e] == m[k][e] ? 1.f : ex2(a[k][e] - base[k][e]);
                        l[k][e] *= a[k][e];
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            o[d][k][e] *= a[k][e];
                            o[d][k][2 + e] *= a[k][e];
                        }
                    }
            }
            uint32_t v_tile = k_tile + R::kb;
            if constexpr (KF == PF_E4) {
                if constexpr (!R::one) {
                    v_tile = take();
                    copy_next();
                }
                by = values.take(tile_scale<D>(v_tile), [&](float x) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
#pragma unroll
                        for (int k = 0; k < NQ; ++k)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[d][k][c] *= x;
                });
            }
            uint32_t pb[NQ][2], lo[NQ][2] = {};
#pragma unroll
            for (int k = 0; k < NQ; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x = ex2(s[k][2 * n] - base[k][0]), y = ex2(s[k][2 * n + 1] - base[k][1]);
                    l[k][0] += x;
                    l[k][1] += y;
                    const uint32_t w = KF == PF_E4 ? Two<T>::pack(x * by, y * by) : Two<T>::pack(x, y);
                    pb[k][n] = transpose8(w);
                    if constexpr (LO) {
                        const float2 hi = Two<T>::unpack(w);
                        lo[k][n] = transpose8(Two<T>::pack(x - hi.x, y - hi.y));
                    }
                }
            if constexpr (!R::one && KF != PF_E4) {
                v_tile = take();
                copy_next();
            }
            if (!all) {
                clear_rows<D, VF>(v_tile, see, lane);
                __syncwarp();
            }
            tile_values<D, VF, NQ, T, LO>(v_tile, place, pb, lo, o);
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
                    s_m[warp][8 * k + 2 * t + e] = m[k][e];
                    s_l[warp][8 * k + 2 * t + e] = l[k][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NQ; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * k + 2 * t + e;
                if (r >= G) continue;
                float mm = -INFINITY;
                for (int w = 0; w < kDW; ++w) mm = fmaxf(mm, s_m[w][r]);
                float a = mm == -INFINITY ? 0.f : ex2(m[k][e] - mm);
                if constexpr (KF == PF_E4) a *= values.unit;
                float* dst = smem + ((int64_t)warp * G + r) * D;
                using V = VGeo<D, VF>;
#pragma unroll
                for (int j = 0; j < V::NJ; ++j)
#pragma unroll
                    for (int c = 0; c < V::CH; ++c) dst[ochan<D, VF>(j, g) + c] = o[(V::CH * j + c) / 2][k][2 * (c & 1) + e] * a;
            }
        __syncthreads();
        const bool whole = i0 == 0 && i1 == st.n;
        float* part = p.ws + line_floats(p.n_seq) + ((int64_t)blockIdx.x + (int64_t)b * H + h) * partial_floats(G, D);
        for (int e = threadIdx.x; e < G * D / 2; e += kDT) {
            const int r = 2 * e / D;
            float x = 0.f, y = 0.f;
            for (int w = 0; w < kDW; ++w) {
                const float2 f = *reinterpret_cast<const float2*>(smem + (int64_t)w * G * D + 2 * e);
                x += f.x;
                y += f.y;
            }
            if (whole) {
                float mm = -INFINITY, ll = 0.f;
                for (int w = 0; w < kDW; ++w) mm = fmaxf(mm, s_m[w][r]);
                for (int w = 0; w < kDW; ++w) ll += s_l[w][r] * (mm == -INFINITY ? 0.f : ex2(s_m[w][r] - mm));
                const float inv = inverse_sum(ll);
                reinterpret_cast<uint32_t*>((TQ*)p.out + ((int64_t)b * p.Hq + h * G) * D)[e] = Two<TQ>::pack(x * inv, y * inv);
            } else {
                *reinterpret_cast<float2*>(part + 32 + 2 * e) = make_float2(x, y);
            }
        }
        if (threadIdx.x < G) {
            const int r = threadIdx.x;
            float mm = -INFINITY, ll = 0.f;
            for (int w = 0; w < kDW; ++w) mm = fmaxf(mm, s_m[w][r]);
            for (int w = 0; w < kDW; ++w) ll += s_l[w][r] * (mm == -INFINITY ? 0.f : ex2(s_m[w][r] - mm));
            if (!whole) {
                part[r] = mm;
                part[16 + r] = ll;
            } else if (p.lse) {
                p.lse[(int64_t)b * p.Hq + h * G + r] = log_sum(mm, ll);
            }
        }
        __syncthreads();
    }
}

// Joins the runs' partials of the heads that runs share: a CTA per (head, query of its group). Where there are more
// heads than runs, the CTAs go by runs instead: at most one head is cut by the start of a run, and its first cut joins
// it. The runs' maxima and sums give one weight per run; then the CTA's thread groups take the runs in turn.
constexpr int kMT = 256;
template <int D, typename TQ>
__global__ void __launch_bounds__(kMT) merge_kernel(PagedAttnParams p, bool by_runs) {
    constexpr int L = D / 4, N = kMT / L;                // threads of an output row (four channels each); groups
    __shared__ float s_w[kMaxDecodeCtas + 1], s_x[kMT / 32];
    __shared__ float4 s_o[N][L];
    const int H = p.v.H, G = p.G, r = blockIdx.x % G, id = blockIdx.x / G;
    // Up to 32 sequences: the line is known from their lengths, before the decode kernel has ended (its blocks wait for
    // what came before them first, so the lengths stand when this kernel starts). Else it is read as the kernel left it
    // (always read: 1,024 positions of 2 heads took 8.3 us in a graph, with the early line 7.1-7.2).
    const bool early = !by_runs && p.n_seq <= 32;
    const int64_t* line = (const int64_t*)p.ws;
    int b = id / H, h = id % H;
    int64_t total, start, n;                             // tiles in all, before sequence b, and of one head of b
    if (early) {
        const int lane = threadIdx.x & 31, mine = lane < p.n_seq ? seq_tiles(p, lane).n : 0;
        int64_t sum = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int64_t y = __shfl_up_sync(kAll, sum, s);
            if (lane >= s) sum += y;
        }
        total = __shfl_sync(kAll, sum, 31) * H;
        start = __shfl_sync(kAll, sum - mine, b) * H;
        n = __shfl_sync(kAll, mine, b);
    } else {
        grid_dep_wait();
        total = line[p.n_seq];
    }
    const int64_t U = run_tiles(total, p.n_cta);
    if (by_runs) {
        const int64_t at = (int64_t)id * U;
        if (id == 0 || at >= total) return;
        int lo = 0, hi = p.n_seq - 1;                    // the last sequence that starts at or before the run
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line[mid] <= at) lo = mid; else hi = mid - 1;
        }
        b = lo;
        h = (int)((at - line[b]) / ((line[b + 1] - line[b]) / H));
    }
    if (!early) {
        start = line[b];
        n = (line[b + 1] - start) / H;
    }
    const int64_t s0 = start + (int64_t)h * n;
    const int c0 = (int)(s0 / U), nc = (int)((s0 + n - 1) / U) - c0 + 1;
    if (early) grid_dep_wait();                          // before any return: what follows this kernel follows both
    if (n == 0 || nc == 1 || (by_runs && (s0 == (int64_t)id * U || c0 != id - 1))) return;
    const int64_t row = (int64_t)b * p.Hq + h * G + r;
    TQ* out = (TQ*)p.out + row * D;
    const int64_t pf = partial_floats(G, D);
    const float* part = p.ws + line_floats(p.n_seq) + ((int64_t)b * H + h + c0) * pf;
    float m = -INFINITY, l = 0.f;
    for (int c = threadIdx.x; c < nc; c += kMT) m = fmaxf(m, s_w[c] = part[c * pf + r]);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, s));
    if ((threadIdx.x & 31) == 0) s_x[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMT / 32; ++i) m = fmaxf(m, s_x[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < nc; c += kMT) {
        const float a = m == -INFINITY ? 0.f : ex2(s_w[c] - m);
        s_w[c] = a;
        l += part[c * pf + 16 + r] * a;
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) l += __shfl_xor_sync(kAll, l, s);
    if ((threadIdx.x & 31) == 0) s_x[threadIdx.x >> 5] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kMT / 32; ++i) l += s_x[i];
    const int col = threadIdx.x % L, grp = threadIdx.x / L;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = grp; c < nc; c += N) {
        const float4 f = *reinterpret_cast<const float4*>(part + c * pf + 32 + (int64_t)r * D + 4 * col);
        const float a = s_w[c];
        o.x = fmaf(f.x, a, o.x);
        o.y = fmaf(f.y, a, o.y);
        o.z = fmaf(f.z, a, o.z);
        o.w = fmaf(f.w, a, o.w);
    }
    s_o[grp][col] = o;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int i = 1; i < N; ++i) {
            const float4 f = s_o[i][col];
            o.x += f.x;
            o.y += f.y;
            o.z += f.z;
            o.w += f.w;
        }
        const float inv = inverse_sum(l);
        *reinterpret_cast<uint2*>(out + 4 * col) = make_uint2(Two<TQ>::pack(o.x * inv, o.y * inv), Two<TQ>::pack(o.z * inv, o.w * inv));
        if (p.lse && col == 0) p.lse[row] = log_sum(m, l);
    }
}

template <int KF, int VF, int NQ, typename T, typename TQ>
int decode_run(const PagedAttnParams& p, int sm_count, cudaStream_t s) {
    PagedAttnParams a = p;
    using R = Ring<KVQ_D, KF, VF, NQ>;
    const auto k = decode_kernel<KVQ_D, KF, VF, NQ, T, TQ>;
    int res = 0;
    if (const int e = resident_ctas((const void*)k, kDT, R::bytes, &res)) return e;
    a.n_cta = min(kMaxDecodeCtas, sm_count * res);
    cudaError_t e = launch_k(k, dim3(a.n_cta), dim3(kDT), R::bytes, s, true, a);
    const int64_t heads = (int64_t)p.n_seq * p.v.H;
    const bool by_runs = heads > a.n_cta;
    if (e == cudaSuccess)
        e = launch_k(merge_kernel<KVQ_D, TQ>, dim3((unsigned)(by_runs ? a.n_cta : heads) * p.G), dim3(kMT), 0, s, true, a, by_runs);
    return (int)e;
}
template <int KF, int VF, typename T, typename TQ> int decode_g(const PagedAttnParams& p, int sms, cudaStream_t s) {
    return p.G <= 8 ? decode_run<KF, VF, 1, T, TQ>(p, sms, s) : decode_run<KF, VF, 2, T, TQ>(p, sms, s);
}

}  // namespace

// One head dimension per compilation of this file (KVQ_D), so that they build side by side.
#define KVQ_NAME2(d) launch_paged_decode_##d
#define KVQ_NAME(d) KVQ_NAME2(d)
int KVQ_NAME(KVQ_D)(const PagedAttnParams& p, int sms, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    const int kf = p.v.fmt[0], vf = p.v.fmt[1];
    if (kf == KVQ_F16) return decode_g<PF_16, PF_16, __half, __half>(p, sms, s);
    if (kf == KVQ_BF16) return decode_g<PF_16, PF_16, __nv_bfloat16, __nv_bfloat16>(p, sms, s);
    if (kf == KVQ_PAGED_E4M3)
        return p.dtype == KVQ_F16 ? decode_g<PF_E4, PF_E4, __half, __half>(p, sms, s) : decode_g<PF_E4, PF_E4, __half, __nv_bfloat16>(p, sms, s);
    if (p.dtype == KVQ_F16) {
        if (kf == KVQ_Q4_0) return decode_g<PF_Q4, PF_Q4, __half, __half>(p, sms, s);
        if (vf == KVQ_Q4_0) return decode_g<PF_Q8, PF_Q4, __half, __half>(p, sms, s);
        return decode_g<PF_Q8, PF_Q8, __half, __half>(p, sms, s);
    }
    if (kf == KVQ_Q4_0) return decode_g<PF_Q4, PF_Q4, __half, __nv_bfloat16>(p, sms, s);
    if (vf == KVQ_Q4_0) return decode_g<PF_Q8, PF_Q4, __half, __nv_bfloat16>(p, sms, s);
    return decode_g<PF_Q8, PF_Q8, __half, __nv_bfloat16>(p, sms, s);
}

}  // namespace kvq
