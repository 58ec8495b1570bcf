// Row kernels of the paged cache: the norm and rotation of query and key heads, rows written to
// pages (copied, rounded or quantised) and read back.
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

// ---------------------------------------------------------------------------- read
// A CTA takes kReadRows output rows: one thread per row finds the row's sequence (binary search over cu) and page, then
// all threads move the rows' pieces, head by head, so that neighbouring lanes read neighbouring rows of a unit.
// A piece is 16 bytes of output, so that a warp's store fills whole sectors; U of a thread's are loaded together.
// Codes x scale in fp32 (exact: at most 19 bits), rounded once to the output's type.
constexpr int kReadRows = 16;

template <typename TO, int FMT, int D> __device__ __forceinline__ void read_rows(const ReadParams& p, int w, const int* s_page, const int* s_row) {
    const PagedView& v = p.v;
    constexpr bool CODES = FMT == KVQ_Q8_0 || FMT == KVQ_Q4_0, WIDE = std::is_same<TO, float>::value;
    constexpr int CH = WIDE ? 4 : 8, P = D / CH, RB = FMT == KVQ_Q8_0 ? D : (FMT == KVQ_Q4_0 ? D / 2 : 2 * D);
    // 16-bit rows out: four pieces (q8_0 rows of 3 sequences: 173 us, with eight 205: fewer warps fit); fp32: eight (123 us, 125)
    constexpr int U = WIDE ? 8 : 4;
    const int row0 = blockIdx.x * kReadRows, n = v.H * kReadRows * P;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * kRowThreads) {
        uint32_t x[U][4];
        uint16_t d[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRowThreads, ch = i % P * CH, r = i / P % kReadRows, head = i / (P * kReadRows);
            live[u] = i < n && s_page[r] >= -1;
            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0;
            d[u] = 0;
            if (live[u] && s_page[r] >= 0) {
                const uint8_t* unit = unit_at(v, w, s_page[r], head);
                const uint8_t* a = unit + s_row[r] * RB + (CODES ? (FMT == KVQ_Q8_0 ? ch : ch / 2) : 2 * ch);
                constexpr int B = CODES ? (FMT == KVQ_Q8_0 ? CH : CH / 2) : 2 * CH;      // bytes of a piece
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
                if constexpr (CODES) d[u] = reinterpret_cast<const uint16_t*>(unit + v.ps * RB)[s_row[r] * (D / 32) + ch / 32];
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
            const float scale = __half2float(__ushort_as_half(d[u]));
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                if constexpr (FMT == KVQ_Q8_0) {
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
template <typename TO, int D> int read_d(const ReadParams& p, cudaStream_t s) {
    return by_formats(p.v, [&](auto k, auto v) {
        const dim3 grid((unsigned)((p.n_rows + kReadRows - 1) / kReadRows), p.out[0] && p.out[1] ? 2 : 1);
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

int launch_paged_write(const WriteParams& p, void* stream) {
    return p.dtype == KVQ_F16 ? write_t<__half>(p, (cudaStream_t)stream) : write_t<__nv_bfloat16>(p, (cudaStream_t)stream);
}

int launch_paged_read(const ReadParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    if (p.dtype == KVQ_F16) return read_t<__half>(p, s);
    return p.dtype == KVQ_BF16 ? read_t<__nv_bfloat16>(p, s) : read_t<float>(p, s);
}

}  // namespace kvq
