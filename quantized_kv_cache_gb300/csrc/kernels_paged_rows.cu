// Row kernels of the paged cache: the norm and rotation of query and key heads, rows written to
// pages (copied, rounded or quantised), appended to blocks of e4m3 codes, and read back.
//
// All three move bytes: each input is read once and each output written once with 16-byte accesses, several vectors
// in flight per thread, fp32 arithmetic. On GB300 (measured HBM rate 6.79 TB/s): norm and rotation of 8,191 tokens x 48
// heads x 128 in 38.4 us, 78% of that rate (issue slots 67% busy, 72 registers); q8_0 rows of 65,536 + 57,855 + 60,559
// positions x 4 x 256 read as bf16 in 173 us, 98%; 16,383 tokens x 8 x 128 written as q8_0 / q4_0 in 22 us (bound by the
// quantiser's instructions, issue 83% busy).
#include <type_traits>
#include "device_common.cuh"
#include "paged_common.cuh"

namespace kvq {
namespace {

constexpr int kRowThreads = 256;

// ---------------------------------------------------------------------------- norm and rotation
// A head row of D values is held by D / V lanes, V values (V / 8 vectors) each: V = 8, and 16 at
// D = 512, so a row never spans two warps and a rotation pair (c, c + rot/2) sits in two lanes at
// the same place (rot/2 is a multiple of V) or, interleaved, in one lane. A warp works on one
// token: its cosines, sines and the weights stay in registers over the `heads` head rows it takes.
template <typename T, int D, bool ROT, bool INTER>
__global__ void __launch_bounds__(kRowThreads, D == 512 ? 2 : 3) norm_rope_kernel(kvq_norm_rope_args a, int heads, int parts) {
    constexpr int V = D == 512 ? 16 : 8, LPR = D / V, RPW = 32 / LPR, NV = V / 8;
    const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
    grid_dep_wait();
    const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(task / parts);
    if (t >= a.n_tok) return;
    const int nh = a.n_q_heads + a.n_k_heads;
    const int h0 = (int)(task % parts) * heads, h1 = min(nh, h0 + heads);
    const int c0 = V * li;                                    // this lane's first channel

    // the first rows are on their way before the position, and with it the table's row, is known; the next ones
    // while these are worked on
    constexpr int U = V == 8 ? 4 : 2;
    uint4 ahead[U][NV] = {};
    const auto load_rows = [&](int hb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub;
            if (h >= h1) continue;
            const T* src = h < a.n_q_heads ? (const T*)a.q + t * a.q_stride + (int64_t)h * D
                                           : (const T*)a.k + t * a.k_stride + (int64_t)(h - a.n_q_heads) * D;
#pragma unroll
            for (int i = 0; i < NV; ++i) ahead[u][i] = *reinterpret_cast<const uint4*>(src + c0 + 8 * i);
        }
    };
    load_rows(h0);

    // pairs (c, c + rot/2): lanes below rot/2 hold the first of a pair, the next rot/2 channels the
    // second; lanes past rot only norm
    const int half = a.rot_dim / 2;
    const bool rotated = ROT && c0 < a.rot_dim;
    const bool second = c0 >= half;
    const int partner = rotated && !INTER ? (second ? lane - half / V : lane + half / V) : lane;
    float cs[V], sn[V];
    bool bad = false;
    if constexpr (ROT) {
        const int pos = a.positions[t];
        bad = pos < 0 || pos >= a.max_pos;
        if (rotated && !bad) {
            const float* row = a.cos_sin + (int64_t)pos * a.rot_dim;
            constexpr int N = INTER ? V / 2 : V;
            const float* p = row + (INTER ? c0 / 2 : (second ? c0 - half : c0));
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 c = *reinterpret_cast<const float4*>(p + i);
                const float4 s = *reinterpret_cast<const float4*>(p + half + i);
                cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
                sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
            }
        }
    }
    for (int hb = h0; hb < h1; hb += U * RPW) {
        uint4 x[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NV; ++i) x[u][i] = ahead[u][i];
        load_rows(hb + U * RPW);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub;
            const bool live = h < h1;
            const bool isq = h < a.n_q_heads;
            float y[V], z[V];                                 // own values, the partner's
            float r = 1.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8];
                unpack8<T>(x[u][i], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[8 * i + e] = f[e];
                if constexpr (ROT && !INTER) {
                    const uint4 o = make_uint4(__shfl_sync(kAll, x[u][i].x, partner), __shfl_sync(kAll, x[u][i].y, partner),
                                               __shfl_sync(kAll, x[u][i].z, partner), __shfl_sync(kAll, x[u][i].w, partner));
                    unpack8<T>(o, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[8 * i + e] = f[e];
                }
            }
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
            for (int s = 1; s < LPR; s <<= 1) ss += __shfl_xor_sync(kAll, ss, s);
            if (!live) continue;
            const T* wt = (const T*)(isq ? a.q_weight : a.k_weight);
            if (wt) {
                r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float f[8];
                    unpack8<T>(*reinterpret_cast<const uint4*>(wt + c0 + 8 * i), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[8 * i + e] *= r * f[e];
                    if constexpr (ROT && !INTER) {
                        const int pc = rotated ? (second ? c0 - half : c0 + half) : c0;
                        unpack8<T>(*reinterpret_cast<const uint4*>(wt + pc + 8 * i), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[8 * i + e] *= r * f[e];
                    }
                }
            }
            if constexpr (ROT) {
                if (rotated) {
                    if constexpr (INTER) {
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) {
                            const float p = y[2 * e], q = y[2 * e + 1];
                            y[2 * e] = p * cs[e] - q * sn[e];
                            y[2 * e + 1] = q * cs[e] + p * sn[e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) y[e] = y[e] * cs[e] + (second ? z[e] * sn[e] : -(z[e] * sn[e]));
                    }
                }
                if (bad) {
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = __int_as_float(0x7fffffff);
                }
            }
            T* dst = isq ? (T*)a.q_out + t * a.q_out_stride + (int64_t)h * D
                         : (T*)a.k_out + t * a.k_out_stride + (int64_t)(h - a.n_q_heads) * D;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = y[8 * i + e];
                *reinterpret_cast<uint4*>(dst + c0 + 8 * i) = pack8<T>(f);
            }
        }
    }
}

template <typename T, int D>
int norm_rope_d(const kvq_norm_rope_args& a, int sm_count, cudaStream_t s) {
    constexpr int RPW = D >= 256 ? 1 : 256 / D;
    const int nh = a.n_q_heads + a.n_k_heads;
    // head rows per warp: all of a token's while that gives every SM 32 warps, fewer below (8,191 tokens of 48 heads of
    // 128: 38.6 us; with a target of 128 warps 47 us, the table's rows being read by four times as many)
    int heads = (nh + RPW - 1) / RPW * RPW;
    const int64_t want = (int64_t)sm_count * 32;
    while (heads > RPW && (int64_t)a.n_tok * ((nh + heads - 1) / heads) < want) heads = (heads / 2 + RPW - 1) / RPW * RPW;
    const int parts = (nh + heads - 1) / heads;
    const int64_t warps = (int64_t)a.n_tok * parts;
    const unsigned grid = (unsigned)((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
    const auto k = !a.rot_dim ? norm_rope_kernel<T, D, false, false>
                              : (a.interleaved ? norm_rope_kernel<T, D, true, true> : norm_rope_kernel<T, D, true, false>);
    return (int)launch_k(k, dim3(grid), dim3(kRowThreads), 0, s, true, a, heads, parts);
}

template <typename T>
int norm_rope_t(const kvq_norm_rope_args& a, int sm_count, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return norm_rope_d<T, 64>(a, sm_count, s);
        case 128: return norm_rope_d<T, 128>(a, sm_count, s);
        case 256: return norm_rope_d<T, 256>(a, sm_count, s);
        default: return norm_rope_d<T, 512>(a, sm_count, s);
    }
}

// ---------------------------------------------------------------------------- norm and rotation, positions on several axes
// A lane holds both values of each of its eight pairs, 16 channels: two pieces of eight, half of the rotated channels apart (or, with
// pairs (2i, 2i + 1), next to one another), so that no value is fetched from another lane or weighed twice. Its eight
// cosines and sines come once per token, each from the table's row of its frequency's axis; arithmetic goes two values at a time.
// 12,001 tokens x 28 heads x 256 (three axes dealt in turn): 61.6 us, 84% of the measured HBM rate, the rest latency at 16 warps an SM
// (three CTAs an SM: the registers spill, 113 us; one row of a lane in flight instead of two 79 us).
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads, 2) norm_rope_axes_kernel(const __grid_constant__ kvq_norm_rope_args a,
                                                                        const __grid_constant__ RopeAxes ax, int heads, int parts) {
    constexpr int LPR = D / 16, RPW = 32 / LPR, U = 2;           // lanes of a row, rows of a warp, in flight
    const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
    grid_dep_wait();
    const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(task / parts);
    if (t >= a.n_tok) return;
    const int nh = a.n_q_heads + a.n_k_heads;
    const int h0 = (int)(task % parts) * heads, h1 = min(nh, h0 + heads);
    const int half = a.rot_dim / 2, np = half / 8;
    const bool rotated = li < np;
    // first channels of the lane's two pieces; lanes behind the rotated ones take two pieces side by side
    const int c0 = INTER || !rotated ? 16 * li : 8 * li, c1 = INTER || !rotated ? c0 + 8 : c0 + half;
    const auto row_of = [&](int h) {
        return h < a.n_q_heads ? (const T*)a.q + t * a.q_stride + (int64_t)h * D
                               : (const T*)a.k + t * a.k_stride + (int64_t)(h - a.n_q_heads) * D;
    };
    uint4 ahead[U][2] = {};
    const auto load_rows = [&](int hb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub;
            if (h >= h1) continue;
            const T* src = row_of(h);
            ahead[u][0] = *reinterpret_cast<const uint4*>(src + c0);
            ahead[u][1] = *reinterpret_cast<const uint4*>(src + c1);
        }
    };
    load_rows(h0);
    int pos[4] = {};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((ax.used >> i) & 1) {
            pos[i] = a.positions[(int64_t)i * a.n_tok + t];
            bad |= pos[i] < 0 || pos[i] >= a.max_pos;
        }
    float2 cs[4] = {}, sn[4] = {};                               // of pairs 2 i, 2 i + 1 of the lane's
    if (rotated && !bad) {
        const uint32_t of = ax.of8[li];
        const auto at = [&](int e) {
            const int x = (of >> (2 * e)) & 3;
            return a.cos_sin + (int64_t)(x & 2 ? (x & 1 ? pos[3] : pos[2]) : (x & 1 ? pos[1] : pos[0])) * a.rot_dim + 8 * li + e;
        };
        if (of == (of & 3) * 0x5555u) {                          // one axis: its row by vectors
            const float* p = at(0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 c = *reinterpret_cast<const float4*>(p + 4 * i), s = *reinterpret_cast<const float4*>(p + half + 4 * i);
                cs[2 * i] = make_float2(c.x, c.y);
                cs[2 * i + 1] = make_float2(c.z, c.w);
                sn[2 * i] = make_float2(s.x, s.y);
                sn[2 * i + 1] = make_float2(s.z, s.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *p = at(2 * i), *q = at(2 * i + 1);
                cs[i] = make_float2(*p, *q);
                sn[i] = make_float2(p[half], q[half]);
            }
        }
    }
    float2 w[8];                                                  // the side's weights, channel by channel as the values
    bool weighed = false;
    int side = -1;
    for (int hb = h0; hb < h1; hb += U * RPW) {
        uint4 x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u][0] = ahead[u][0];
            x[u][1] = ahead[u][1];
        }
        load_rows(hb + U * RPW);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub, now = h < a.n_q_heads ? 0 : 1;
            float2 y[8];                                          // piece 0: y[0..3], piece 1: y[4..7]
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                y[4 * i] = Two<T>::unpack(x[u][i].x);
                y[4 * i + 1] = Two<T>::unpack(x[u][i].y);
                y[4 * i + 2] = Two<T>::unpack(x[u][i].z);
                y[4 * i + 3] = Two<T>::unpack(x[u][i].w);
            }
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s2 = __ffma2_rn(y[i], y[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int s = 1; s < LPR; s <<= 1) ss += __shfl_xor_sync(kAll, ss, s);
            if (h >= h1) continue;
            if (now != side) {
                side = now;
                const T* wt = (const T*)(now ? a.k_weight : a.q_weight);
                weighed = wt != nullptr;
                if (weighed) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 z = *reinterpret_cast<const uint4*>(wt + (i ? c1 : c0));
                        w[4 * i] = Two<T>::unpack(z.x);
                        w[4 * i + 1] = Two<T>::unpack(z.y);
                        w[4 * i + 2] = Two<T>::unpack(z.z);
                        w[4 * i + 3] = Two<T>::unpack(z.w);
                    }
                }
            }
            if (weighed) {
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(y[i], __fmul2_rn(w[i], make_float2(r, r)));
            }
            if (rotated) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // first and second values of pairs 2 i, 2 i + 1
                    const float2 p = INTER ? make_float2(y[2 * i].x, y[2 * i + 1].x) : y[i];
                    const float2 q = INTER ? make_float2(y[2 * i].y, y[2 * i + 1].y) : y[4 + i];
                    const float2 f = __ffma2_rn(p, cs[i], neg2(__fmul2_rn(q, sn[i]))), g = __ffma2_rn(q, cs[i], __fmul2_rn(p, sn[i]));
                    if constexpr (INTER) {
                        y[2 * i] = make_float2(f.x, g.x);
                        y[2 * i + 1] = make_float2(f.y, g.y);
                    } else {
                        y[i] = f;
                        y[4 + i] = g;
                    }
                }
            }
            if (bad) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i].x = y[i].y = __int_as_float(0x7fffffff);
            }
            T* dst = now ? (T*)a.k_out + t * a.k_out_stride + (int64_t)(h - a.n_q_heads) * D
                         : (T*)a.q_out + t * a.q_out_stride + (int64_t)h * D;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint4*>(dst + (i ? c1 : c0)) =
                    make_uint4(Two<T>::pack(y[4 * i].x, y[4 * i].y), Two<T>::pack(y[4 * i + 1].x, y[4 * i + 1].y),
                               Two<T>::pack(y[4 * i + 2].x, y[4 * i + 2].y), Two<T>::pack(y[4 * i + 3].x, y[4 * i + 3].y));
        }
    }
}

template <typename T, int D>
int norm_rope_axes_d(const kvq_norm_rope_args& a, const RopeAxes& x, int sm_count, cudaStream_t s) {
    constexpr int RPW = 512 / D;
    const int nh = a.n_q_heads + a.n_k_heads;
    // head rows per warp: all of a token's while that gives every SM 32 warps, fewer below (as for one axis)
    int heads = (nh + RPW - 1) / RPW * RPW;
    const int64_t want = (int64_t)sm_count * 32;
    while (heads > RPW && (int64_t)a.n_tok * ((nh + heads - 1) / heads) < want) heads = (heads / 2 + RPW - 1) / RPW * RPW;
    const int parts = (nh + heads - 1) / heads;
    const unsigned grid = (unsigned)(((int64_t)a.n_tok * parts + kRowThreads / 32 - 1) / (kRowThreads / 32));
    const auto k = a.interleaved ? norm_rope_axes_kernel<T, D, true> : norm_rope_axes_kernel<T, D, false>;
    return (int)launch_k(k, dim3(grid), dim3(kRowThreads), 0, s, true, a, x, heads, parts);
}

template <typename T>
int norm_rope_axes_t(const kvq_norm_rope_args& a, const RopeAxes& x, int sm_count, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return norm_rope_axes_d<T, 64>(a, x, sm_count, s);
        case 128: return norm_rope_axes_d<T, 128>(a, x, sm_count, s);
        case 256: return norm_rope_axes_d<T, 256>(a, x, sm_count, s);
        default: return norm_rope_axes_d<T, 512>(a, x, sm_count, s);
    }
}

// ---------------------------------------------------------------------------- write
// Quantises 16 values; a 32-value block is two neighbouring lanes. The block's largest magnitude is taken on the
// bits (a NaN compares above infinity, so it reaches the scale). c: the codes as the low bits of 1.5 * 2^23 + q, which
// is rint(x * (1 / d)) clamped to +-top: one fp32 rounding per operation, as the codec is defined (clamping first
// gives the same integer).
template <typename T>
__device__ __forceinline__ __half quantise16(const uint4 (&x)[2], float top, uint32_t (&c)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                 __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(kAll, m, 1));
    const __half dh = __float2half_rn(__fdiv_rn(Two<T>::unpack(m).x, top));
    const float d = __half2float(dh);
    const float inv = d == 0.f ? 0.f : __fdiv_rn(1.0f, d);
    // A normal d is within 2^-11 of amax / top, so that no |x * inv| rounds above top: clamped only where some block's d
    // is subnormal (or 0, or not finite).
    const bool clamp = __any_sync(kAll, !(d >= 6.1035156e-5f && d <= 65504.f));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[8];
        unpack8<T>(x[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = __fmul_rn(f[e], inv);
            if (clamp) v = fminf(fmaxf(v, -top), top);
            c[8 * i + e] = __float_as_uint(__fadd_rn(v, 12582912.f));
        }
    }
    return dh;
}

// The lowest bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// grid.y: 0 = K, 1 = V; a thread per 16 channels of a token, kWriteTokens tokens a CTA. FMT is the pages' format.
constexpr int kWriteTokens = 4;
template <typename T, int FMT, int D> __device__ __forceinline__ void write_rows(const WriteParams& p, int w) {
    const PagedView& v = p.v;
    constexpr int P = D / 16;
    const int per = v.H * P, t0 = blockIdx.x * kWriteTokens;
    const int n = min(kWriteTokens, p.n_tok - t0) * per, round = (n + 31) & ~31;    // whole warps: a block is two lanes
    for (int i = threadIdx.x; i < round; i += kRowThreads) {
        const int t = i / per, in = i - t * per, head = in / P, ch = in % P * 16;
        int slot = -1;
        uint4 x[2] = {};
        if (i < n) {
            slot = p.slots[t0 + t];
            const uint4* src = reinterpret_cast<const uint4*>((const T*)p.src[w] + (int64_t)(t0 + t) * p.stride[w] + 16 * in);
            x[0] = src[0];
            x[1] = src[1];
        }
        const int page = slot >> v.ps_shift, row = slot & (v.ps - 1);
        const bool ok = slot >= 0 && page < v.n_pages;
        if (slot >= 0 && !ok && in == 0) raise_status(v.status, KVQ_PAGED_BAD_INDEX);
        uint8_t* unit = const_cast<uint8_t*>(unit_at(v, w, ok ? page : 0, head));
        const int at = row * D + ch;
        if constexpr (FMT == KVQ_F16 || FMT == KVQ_BF16) {
            if constexpr ((FMT == KVQ_F16) != std::is_same<T, __half>::value) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float f[8];
                    unpack8<T>(x[k], f);
                    x[k] = FMT == KVQ_F16 ? pack8<__half>(f) : pack8<__nv_bfloat16>(f);
                }
            }
            if (ok) {
                uint4* dst = reinterpret_cast<uint4*>(unit + 2 * at);
                dst[0] = x[0];
                dst[1] = x[1];
            }
        } else {
            uint32_t c[16];
            const __half dh = quantise16<T>(x, FMT == KVQ_Q8_0 ? 127.f : 7.f, c);
            if (!ok) continue;
            if constexpr (FMT == KVQ_Q8_0) {
                *reinterpret_cast<uint4*>(unit + at) =
                    make_uint4(low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7]),
                               low_bytes(c[8], c[9], c[10], c[11]), low_bytes(c[12], c[13], c[14], c[15]));
            } else {
                uint32_t o[2] = {};
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e >> 3] |= ((c[e] + 8u) & 15u) << (4 * (e & 7));
                *reinterpret_cast<uint2*>(unit + at / 2) = make_uint2(o[0], o[1]);
            }
            if ((ch & 31) == 0) {
                const uint32_t bits = __half_as_ushort(dh);
                if (bits > (FMT == KVQ_Q8_0 ? kMaxScaleQ8 : kMaxScaleQ4))
                    raise_status(v.status, bits < 0x7c00 ? KVQ_PAGED_RANGE : KVQ_PAGED_NONFINITE);
                constexpr int RB = FMT == KVQ_Q8_0 ? D : D / 2;
                reinterpret_cast<__half*>(unit + v.ps * RB)[row * (D / 32) + ch / 32] = dh;
            }
        }
    }
}

template <typename T, int KF, int VF, int D> __global__ void __launch_bounds__(kRowThreads) write_kernel(WriteParams p) {
    grid_dep_wait();
    if (blockIdx.y == 0) write_rows<T, KF, D>(p, 0);
    else write_rows<T, VF, D>(p, 1);
}

// ---------------------------------------------------------------------------- append
// e4m3 blocks: 16 positions of a head under one power of two. A warp takes a whole block (one head of K or V), all its new rows
// in registers: their largest magnitude on the bits, the power, the codes. Rows that were there are rounded to the new power
// where it grew; in a decode step (one such load after the other) their codes are loaded beside the new rows, before that is known.
// No two warps touch the same bytes, and no order of anything matters. Bound by HBM: three prompts of 41,331 rows in all, 4 x 256 fp16, in
// 41 us, 91% of the measured rate (with 16 rows a CTA and all old codes loaded 54 us).
//
// The warps find their blocks from the rows: a row that begins a block, or its sequence's rows, leads one. With R = 32 a CTA looks at
// 32 rows, of which two lead where sequences bring many; with R = 1 (a decode step) a CTA takes one row's block.
constexpr int kAppendWarps = 4;
template <typename T, int D, int R> __global__ void __launch_bounds__(32 * kAppendWarps) paged_append_kernel(PagedAppendParams p) {
    const PagedView& v = p.v;
    const int lane = threadIdx.x & 31, task = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
    grid_dep_wait();
    if (task >= 2 * v.H) return;
    const int w = task >= v.H, head = task - (w ? v.H : 0), r0 = blockIdx.x * R, r = r0 + (lane < R ? lane : 0);
    const bool tell = task == 0;
    // the last sequence whose rows begin at or before this lane's row
    int b = 0;
    if (p.n_seq <= (R == 1 ? 1024 : 64)) {
        for (int i = 0; i < p.n_seq; i += 32) {
            const int c = i + lane + 1 < p.n_seq ? p.cu[i + lane + 1] : 0x7fffffff;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int n = __popc(__ballot_sync(kAll, c <= r0 + k));
                if (R == 1 || lane == k) b += n;
            }
        }
    } else {
        int hi = p.n_seq - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (p.cu[mid] <= r) b = mid; else hi = mid - 1;
        }
    }
    const int c0 = p.cu[b], c1 = min(p.cu[b + 1], p.n_rows);
    if (tell && r0 == 0 && lane == 0 && (p.cu[0] < 0 || p.cu[p.n_seq] > p.n_rows)) raise_status(v.status, KVQ_PAGED_BAD_LENGTH);
    const int64_t pos = (int64_t)(p.start ? p.start[b] : 0) + r - c0;
    int off = (int)(pos & (kTile - 1)), n = min(kTile - off, c1 - r), unit = -1;
    if (lane < R && r >= c0 && r < c1 && c0 >= 0 && (off == 0 || r == c0)) {
        const int64_t e = pos >> v.ps_shift;
        if (pos < 0 || e >= p.max_pages) {
            if (tell) raise_status(v.status, KVQ_PAGED_BAD_LENGTH);
        } else {
            const int page = p.table[b * p.table_stride + e];
            if (page >= 0 && page < v.n_pages) unit = page * v.H + head;
            else if (tell) raise_status(v.status, KVQ_PAGED_BAD_INDEX);
        }
    }
    constexpr int VPR = D / 8, RPI = 32 / VPR, IT = kTile / RPI;    // vectors of a row, rows of an iteration, iterations
    const int sub = lane / VPR, col = lane % VPR * 8;
    for (unsigned lead = __ballot_sync(kAll, unit >= 0); lead; lead &= lead - 1) {
        const int from = __ffs(lead) - 1;
        const int un = __shfl_sync(kAll, unit, from), o = __shfl_sync(kAll, off, from), cnt = __shfl_sync(kAll, n, from);
        const int row0 = (int)__shfl_sync(kAll, pos, from) & (v.ps - 1) & ~(kTile - 1);
        uint8_t* base = v.base[w] + (int64_t)un * v.unit[w];
        uint8_t* code = base + row0 * D + col;
        float* scale = reinterpret_cast<float*>(base + v.ps * D) + row0 / kTile;
        const T* src = (const T*)p.src[w] + (r0 + from) * p.stride[w] + (int64_t)head * D + col;
        uint4 x[IT];
        uint2 old[R == 1 ? IT : 1] = {};
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int k = i * RPI + sub;
            x[i] = make_uint4(0, 0, 0, 0);
            if (k < cnt) x[i] = *reinterpret_cast<const uint4*>(src + k * p.stride[w]);
        }
        int held = kMinPower;
        if (o > 0) {
            held = min(max(exponent_of(*scale), kMinPower), kMaxPower);
            if constexpr (R == 1) {
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    if (i * RPI + sub < o) old[i] = *reinterpret_cast<const uint2*>(code + (i * RPI + sub) * D);
            }
        }
        constexpr uint32_t inf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < IT; ++i)
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        m = max(m & 0xffffu, m >> 16);
        const bool odd = __any_sync(kAll, m >= inf);                 // an infinity or NaN: the block goes by its other values
        if (odd) {
            m = 0;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t a = (y[k / 2] >> (16 * (k & 1))) & 0x7fffu;
                    m = max(m, a < inf ? a : 0u);
                }
            }
            if (lane == 0) raise_status(v.status, KVQ_PAGED_NONFINITE);
        }
        m = __reduce_max_sync(kAll, m);
        const uint32_t top = __float_as_uint(Two<T>::unpack(m).x);  // of 1.75 x 2^8 = 448: one more above a mantissa of 0.75
        int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u);
        e = max(max(e, kMinPower), held);
        if (lane == 0 && e > kMaxPowerAttn) raise_status(v.status, KVQ_PAGED_RANGE);
        const float inv = power_of(-e);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int k = i * RPI + sub;
            float f[8];
            unpack8<T>(x[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (odd && !isfinite(f[q])) f[q] = __int_as_float(0x7fffffff);
                f[q] *= inv;
            }
            const uint2 c = make_uint2(e4m3_codes(f[0], f[1]) | (e4m3_codes(f[2], f[3]) << 16),
                                       e4m3_codes(f[4], f[5]) | (e4m3_codes(f[6], f[7]) << 16));
            if (k < cnt) *reinterpret_cast<uint2*>(code + (o + k) * D) = c;
        }
        if (o > 0 && e > held) {
            const float by = power_of(max(held - e, kMinPower));
#pragma unroll(R == 1 ? IT : 1)
            for (int i = 0; i < IT; ++i) {
                if (R > 1 && i * RPI + sub < o) old[0] = *reinterpret_cast<const uint2*>(code + (i * RPI + sub) * D);
                const uint32_t y[2] = {old[R == 1 ? i : 0].x, old[R == 1 ? i : 0].y};
                uint32_t c[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 a = __half22float2(h2(e4m3_pair(y[k] & 0xffffu))), d = __half22float2(h2(e4m3_pair(y[k] >> 16)));
                    c[k] = e4m3_codes(a.x * by, a.y * by) | (e4m3_codes(d.x * by, d.y * by) << 16);
                }
                if (i * RPI + sub < o) *reinterpret_cast<uint2*>(code + (i * RPI + sub) * D) = make_uint2(c[0], c[1]);
            }
        }
        if (lane == 0) *scale = power_of(e);
    }
}

// ---------------------------------------------------------------------------- read
// A CTA takes kReadRows output rows: one thread per row finds the row's sequence (binary search over cu) and page, then
// all threads move the rows' pieces, head by head, so that neighbouring lanes read neighbouring rows of a unit.
// A piece is 16 bytes of output, so that a warp's store fills whole sectors; U of a thread's are loaded together.
// Codes x scale in fp32 (exact: at most 19 bits), rounded once to the output's type.
constexpr int kReadRows = 16;

template <typename TO, int FMT, int D> __device__ __forceinline__ void read_rows(const ReadParams& p, int w, const int* s_page, const int* s_row) {
    const PagedView& v = p.v;
    constexpr bool E4 = FMT == KVQ_PAGED_E4M3, BYTES = FMT == KVQ_Q8_0 || E4, CODES = BYTES || FMT == KVQ_Q4_0;
    constexpr bool WIDE = std::is_same<TO, float>::value;
    constexpr int CH = WIDE ? 4 : 8, P = D / CH, RB = BYTES ? D : (FMT == KVQ_Q4_0 ? D / 2 : 2 * D);
    using Scale = typename std::conditional<E4, uint32_t, uint16_t>::type;
    // 16-bit rows out: four pieces (q8_0 rows of 3 sequences: 173 us, with eight 205: fewer warps fit); fp32: eight (123 us, 125)
    constexpr int U = WIDE ? 8 : 4;
    const int row0 = blockIdx.x * kReadRows, n = v.H * kReadRows * P;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * kRowThreads) {
        uint32_t x[U][4];
        Scale d[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRowThreads, ch = i % P * CH, r = i / P % kReadRows, head = i / (P * kReadRows);
            live[u] = i < n && s_page[r] >= -1;
            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0;
            d[u] = 0;
            if (live[u] && s_page[r] >= 0) {
                const uint8_t* unit = unit_at(v, w, s_page[r], head);
                const uint8_t* a = unit + s_row[r] * RB + (CODES ? (BYTES ? ch : ch / 2) : 2 * ch);
                constexpr int B = CODES ? (BYTES ? CH : CH / 2) : 2 * CH;                // bytes of a piece
                if constexpr (B == 16) {
                    const uint4 y = *reinterpret_cast<const uint4*>(a);
                    x[u][0] = y.x;
                    x[u][1] = y.y;
                    x[u][2] = y.z;
                    x[u][3] = y.w;
                } else if constexpr (B == 8) {
                    const uint2 y = *reinterpret_cast<const uint2*>(a);
                    x[u][0] = y.x;
                    x[u][1] = y.y;
                } else if constexpr (B == 4) {
                    x[u][0] = *reinterpret_cast<const uint32_t*>(a);
                } else {
                    x[u][0] = *reinterpret_cast<const uint16_t*>(a);
                }
                if constexpr (E4) d[u] = reinterpret_cast<const uint32_t*>(unit + v.ps * RB)[s_row[r] / kTile];
                else if constexpr (CODES) d[u] = reinterpret_cast<const uint16_t*>(unit + v.ps * RB)[s_row[r] * (D / 32) + ch / 32];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!live[u]) continue;
            const int i = i0 + u * kRowThreads, ch = i % P * CH, r = i / P % kReadRows, head = i / (P * kReadRows);
            TO* out = (TO*)p.out[w] + ((int64_t)(row0 + r) * v.H + head) * D + ch;
            if constexpr (!CODES && ((FMT == KVQ_F16 && std::is_same<TO, __half>::value) ||
                                     (FMT == KVQ_BF16 && std::is_same<TO, __nv_bfloat16>::value))) {
                *reinterpret_cast<uint4*>(out) = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
                continue;
            }
            float f[8];
            float scale;
            if constexpr (E4) scale = __uint_as_float(d[u]);
            else scale = __half2float(__ushort_as_half(d[u]));
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                if constexpr (E4) {
                    const float2 y = __half22float2(h2(e4m3_pair(x[u][e >> 2] >> (16 * (e >> 1 & 1)) & 0xffffu)));
                    f[e] = scale * (e & 1 ? y.y : y.x);
                } else if constexpr (FMT == KVQ_Q8_0) {
                    f[e] = scale * (float)(int8_t)(x[u][e >> 2] >> (8 * (e & 3)));
                } else if constexpr (FMT == KVQ_Q4_0) {
                    f[e] = scale * (float)((int)((x[u][0] >> (4 * e)) & 15u) - 8);
                } else {
                    const float2 y = Two<typename std::conditional<FMT == KVQ_F16, __half, __nv_bfloat16>::type>::unpack(x[u][e >> 1]);
                    f[e] = e & 1 ? y.y : y.x;
                }
            }
            if constexpr (WIDE) *reinterpret_cast<float4*>(out) = make_float4(f[0], f[1], f[2], f[3]);
            else *reinterpret_cast<uint4*>(out) = pack8<TO>(f);
        }
    }
}

template <typename TO, int KF, int VF, int D> __global__ void __launch_bounds__(kRowThreads) read_kernel(ReadParams p) {
    const PagedView& v = p.v;
    __shared__ int s_page[kReadRows], s_row[kReadRows];   // page: -1 reads zeros, -2 leaves the row as it is
    grid_dep_wait();
    const int w = p.out[0] ? blockIdx.y : 1, row0 = blockIdx.x * kReadRows;
    if (threadIdx.x < kReadRows) {
        const int r = row0 + threadIdx.x;
        int page = -2, in = 0;
        if (r == 0 && blockIdx.y == 0 && (p.cu[0] < 0 || p.cu[p.n_seq] > p.n_rows)) raise_status(v.status, KVQ_PAGED_BAD_LENGTH);
        if (r < p.n_rows && r >= p.cu[0] && r < p.cu[p.n_seq]) {
            int lo = 0, hi = p.n_seq - 1;                 // the last b with cu[b] <= r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.cu[mid] <= r) lo = mid; else hi = mid - 1;
            }
            const int64_t pos = (int64_t)r - p.cu[lo] + (p.start ? p.start[lo] : 0);
            page = -1;
            const int64_t e = pos >> v.ps_shift;
            if (pos < 0 || e >= p.max_pages) {
                raise_status(v.status, KVQ_PAGED_BAD_LENGTH);
            } else {
                page = p.table[lo * p.table_stride + e];
                if (page < 0 || page >= v.n_pages) {
                    raise_status(v.status, KVQ_PAGED_BAD_INDEX);
                    page = -1;
                }
            }
            in = (int)(pos & (v.ps - 1));
        }
        s_page[threadIdx.x] = page;
        s_row[threadIdx.x] = in;
    }
    __syncthreads();
    if (w == 0) read_rows<TO, KF, D>(p, 0, s_page, s_row);
    else read_rows<TO, VF, D>(p, 1, s_page, s_row);
}

__global__ void clear_status_kernel(uint32_t* status, uint32_t bits) { atomicAnd(status, ~bits); }

// fn(key format, value format) as constants, of the pairs a config may have.
template <typename F> int by_formats(const PagedView& v, F fn) {
    if (v.fmt[0] == KVQ_F16) return fn(std::integral_constant<int, KVQ_F16>(), std::integral_constant<int, KVQ_F16>());
    if (v.fmt[0] == KVQ_BF16) return fn(std::integral_constant<int, KVQ_BF16>(), std::integral_constant<int, KVQ_BF16>());
    if (v.fmt[0] == KVQ_Q4_0) return fn(std::integral_constant<int, KVQ_Q4_0>(), std::integral_constant<int, KVQ_Q4_0>());
    if (v.fmt[1] == KVQ_Q4_0) return fn(std::integral_constant<int, KVQ_Q8_0>(), std::integral_constant<int, KVQ_Q4_0>());
    return fn(std::integral_constant<int, KVQ_Q8_0>(), std::integral_constant<int, KVQ_Q8_0>());
}

template <typename T, int D> int write_d(const WriteParams& p, cudaStream_t s) {
    return by_formats(p.v, [&](auto k, auto v) {
        const dim3 grid((unsigned)((p.n_tok + kWriteTokens - 1) / kWriteTokens), 2);
        return (int)launch_k(write_kernel<T, k.value, v.value, D>, grid, dim3(kRowThreads), 0, s, true, p);
    });
}
template <typename T> int write_t(const WriteParams& p, cudaStream_t s) {
    return p.v.D == 64 ? write_d<T, 64>(p, s) : (p.v.D == 128 ? write_d<T, 128>(p, s) : write_d<T, 256>(p, s));
}
template <typename T, int D> int append_d(const PagedAppendParams& p, cudaStream_t s) {
    // 32 rows a CTA where there are many and a sequence brings four or more, on the mean (a row a CTA against 32, in us: 32
    // sequences of 16 rows 10 / 12, of 64 14 / 12; 512 sequences of one 16 / 51, of four 25 / 23, of eight 35 / 18)
    const int rows = p.n_rows >= 2048 && p.n_rows / 4 >= p.n_seq ? 32 : 1;
    const dim3 grid((unsigned)((p.n_rows + (int64_t)rows - 1) / rows), (unsigned)((2 * p.v.H + kAppendWarps - 1) / kAppendWarps));
    const auto k = rows == 1 ? paged_append_kernel<T, D, 1> : paged_append_kernel<T, D, 32>;
    return (int)launch_k(k, grid, dim3(32 * kAppendWarps), 0, s, true, p);
}
template <typename T> int append_t(const PagedAppendParams& p, cudaStream_t s) {
    return p.v.D == 64 ? append_d<T, 64>(p, s) : (p.v.D == 128 ? append_d<T, 128>(p, s) : append_d<T, 256>(p, s));
}
template <typename TO, int D> int read_d(const ReadParams& p, cudaStream_t s) {
    const dim3 grid((unsigned)((p.n_rows + kReadRows - 1) / kReadRows), p.out[0] && p.out[1] ? 2 : 1);
    if (p.v.fmt[0] == KVQ_PAGED_E4M3)
        return (int)launch_k(read_kernel<TO, KVQ_PAGED_E4M3, KVQ_PAGED_E4M3, D>, grid, dim3(kRowThreads), 0, s, true, p);
    return by_formats(p.v, [&](auto k, auto v) {
        return (int)launch_k(read_kernel<TO, k.value, v.value, D>, grid, dim3(kRowThreads), 0, s, true, p);
    });
}
template <typename TO> int read_t(const ReadParams& p, cudaStream_t s) {
    return p.v.D == 64 ? read_d<TO, 64>(p, s) : (p.v.D == 128 ? read_d<TO, 128>(p, s) : read_d<TO, 256>(p, s));
}

}  // namespace

int launch_paged_clear_status(uint32_t* status, uint32_t bits) {
    return (int)launch_k(clear_status_kernel, dim3(1), dim3(1), 0, nullptr, false, status, bits);
}

int launch_norm_rope(const kvq_norm_rope_args& a, int sm_count, void* stream) {
    return a.dtype == KVQ_F16 ? norm_rope_t<__half>(a, sm_count, (cudaStream_t)stream)
                              : norm_rope_t<__nv_bfloat16>(a, sm_count, (cudaStream_t)stream);
}

int launch_norm_rope_axes(const kvq_norm_rope_args& a, const RopeAxes& x, int sm_count, void* stream) {
    return a.dtype == KVQ_F16 ? norm_rope_axes_t<__half>(a, x, sm_count, (cudaStream_t)stream)
                              : norm_rope_axes_t<__nv_bfloat16>(a, x, sm_count, (cudaStream_t)stream);
}

int launch_paged_write(const WriteParams& p, void* stream) {
    return p.dtype == KVQ_F16 ? write_t<__half>(p, (cudaStream_t)stream) : write_t<__nv_bfloat16>(p, (cudaStream_t)stream);
}

int launch_paged_append(const PagedAppendParams& p, void* stream) {
    return p.dtype == KVQ_F16 ? append_t<__half>(p, (cudaStream_t)stream) : append_t<__nv_bfloat16>(p, (cudaStream_t)stream);
}

int launch_paged_read(const ReadParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    if (p.dtype == KVQ_F16) return read_t<__half>(p, s);
    return p.dtype == KVQ_BF16 ? read_t<__nv_bfloat16>(p, s) : read_t<float>(p, s);
}

}  // namespace kvq
