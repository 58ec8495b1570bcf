// Row kernels of the paged cache: the norm and rotation of query and key heads, rows written to
// pages (copied, rounded or quantised) and read back.
//
// All three move bytes: each input is read once and each output written once with 16-byte accesses,
// several vectors in flight per thread, and the arithmetic (fp32 throughout) stays below the issue
// rate that the HBM rate leaves.
#include <type_traits>
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
__global__ void __launch_bounds__(kRowThreads) norm_rope_kernel(kvq_norm_rope_args a, int heads, int parts) {
    constexpr int V = D == 512 ? 16 : 8, LPR = D / V, RPW = 32 / LPR, NV = V / 8;
    const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
    const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(task / parts);
    if (t >= a.n_tok) return;
    const int nh = a.n_q_heads + a.n_k_heads;
    const int h0 = (int)(task % parts) * heads, h1 = min(nh, h0 + heads);
    const int c0 = V * li;                                    // this lane's first channel

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
    constexpr int U = V == 8 ? 4 : 2;                         // rows in flight
    for (int hb = h0; hb < h1; hb += U * RPW) {
        uint4 x[U][NV] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub;
            if (h >= h1) continue;
            const T* src = h < a.n_q_heads ? (const T*)a.q + t * a.q_stride + (int64_t)h * D
                                           : (const T*)a.k + t * a.k_stride + (int64_t)(h - a.n_q_heads) * D;
#pragma unroll
            for (int i = 0; i < NV; ++i) x[u][i] = *reinterpret_cast<const uint4*>(src + c0 + 8 * i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * RPW + sub;
            const bool live = h < h1;
            const bool isq = h < a.n_q_heads;
            const T* wt = (const T*)(isq ? a.q_weight : a.k_weight);
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
            if (wt) {
                r = rsqrtf(ss * (1.0f / D) + a.eps);
                float f[8];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    unpack8<T>(*reinterpret_cast<const uint4*>(wt + c0 + 8 * i), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[8 * i + e] *= r * f[e];
                    if constexpr (ROT && !INTER) {
                        if (rotated) {
                            const int pc = second ? c0 - half : c0 + half;
                            unpack8<T>(*reinterpret_cast<const uint4*>(wt + pc + 8 * i), f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) z[8 * i + e] *= r * f[e];
                        }
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
    // head rows per warp: all of a token's while that leaves every SM's 64 warps busy, fewer below
    int heads = (nh + RPW - 1) / RPW * RPW;
    const int64_t want = (int64_t)sm_count * 64;
    while (heads > RPW && (int64_t)a.n_tok * ((nh + heads - 1) / heads) < want) heads = (heads / 2 + RPW - 1) / RPW * RPW;
    const int parts = (nh + heads - 1) / heads;
    const int64_t warps = (int64_t)a.n_tok * parts;
    const unsigned grid = (unsigned)((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
    if (!a.rot_dim) norm_rope_kernel<T, D, false, false><<<grid, kRowThreads, 0, s>>>(a, heads, parts);
    else if (a.interleaved) norm_rope_kernel<T, D, true, true><<<grid, kRowThreads, 0, s>>>(a, heads, parts);
    else norm_rope_kernel<T, D, true, false><<<grid, kRowThreads, 0, s>>>(a, heads, parts);
    return (int)cudaGetLastError();
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
// Quantises one 8-value vector; a 32-value block is four neighbouring lanes. The block's largest
// magnitude is taken on the bits (a NaN compares above infinity, so it reaches the scale). c: the
// codes as the low bits of 1.5 * 2^23 + q, which is rint(x * (1 / d)) clamped to +-top: one fp32
// rounding per operation, as the codec is defined (clamping first gives the same integer).
template <typename T>
__device__ __forceinline__ __half quantise8(const uint4& x, float top, uint32_t (&c)[8]) {
    uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(kAll, m, 1));
    m = max(m, __shfl_xor_sync(kAll, m, 2));
    const __half dh = __float2half_rn(__fdiv_rn(Two<T>::unpack(m).x, top));
    const float d = __half2float(dh);
    const float inv = d == 0.f ? 0.f : __fdiv_rn(1.0f, d);
    float f[8];
    unpack8<T>(x, f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        c[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmul_rn(f[e], inv), -top), top), 12582912.f));
    return dh;
}

// grid.y: 0 = K, 1 = V. Every token's H * D / 8 vectors in order (a block's four lie in one warp),
// U per thread, loaded together.
template <typename T, int U>
__global__ void __launch_bounds__(kRowThreads) write_kernel(WriteParams p) {
    const PagedView& v = p.v;
    const int w = blockIdx.y, per = v.H * v.D / 8, fmt = v.fmt[w], ps = v.ps, D = v.D;
    const int64_t total = (int64_t)p.n_tok * per;
    const int64_t first = (int64_t)blockIdx.x * (kRowThreads * U) + threadIdx.x;
    uint4 x[U] = {};
    int slot[U], in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = first + u * kRowThreads;
        slot[u] = -1;
        in[u] = 0;
        if (e < total) {
            const int t = (int)(e / per);
            in[u] = (int)(e - (int64_t)t * per);
            slot[u] = p.slots[t];
            x[u] = *reinterpret_cast<const uint4*>((const T*)p.src[w] + t * p.stride[w] + 8 * in[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int page = slot[u] >> v.ps_shift, row = slot[u] & (ps - 1);
        const bool ok = slot[u] >= 0 && page < v.n_pages;
        if (slot[u] >= 0 && !ok && in[u] == 0) raise_status(v.status, KVQ_PAGED_BAD_INDEX);
        const int head = (in[u] * 8) / D, ch = (in[u] * 8) % D;
        uint8_t* unit = const_cast<uint8_t*>(unit_at(v, w, ok ? page : 0, head));
        const int64_t at = (int64_t)row * D + ch;
        if (fmt == KVQ_F16 || fmt == KVQ_BF16) {
            uint4 o = x[u];
            if ((fmt == KVQ_F16) != std::is_same<T, __half>::value) {
                float f[8];
                unpack8<T>(x[u], f);
                o = fmt == KVQ_F16 ? pack8<__half>(f) : pack8<__nv_bfloat16>(f);
            }
            if (ok) *reinterpret_cast<uint4*>(unit + at * 2) = o;
            continue;
        }
        uint32_t c[8];
        const __half dh = quantise8<T>(x[u], fmt == KVQ_Q8_0 ? 127.f : 7.f, c);
        if (!ok) continue;
        if (fmt == KVQ_Q8_0) {
            uint2 o;
            o.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
            o.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(unit + at) = o;
        } else {
            uint32_t o = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) o |= ((c[e] + 8u) & 15u) << (4 * e);
            *reinterpret_cast<uint32_t*>(unit + at / 2) = o;
        }
        if ((ch & 31) == 0) {
            if (!isfinite(__half2float(dh))) raise_status(v.status, KVQ_PAGED_NONFINITE);
            const int rb = fmt == KVQ_Q8_0 ? D : D / 2;
            reinterpret_cast<__half*>(unit + (int64_t)ps * rb)[row * (D / 32) + ch / 32] = dh;
        }
    }
}

// ---------------------------------------------------------------------------- read
// 8 values (ch .. ch + 7) of a row, code x scale in fp32 (exact: at most 19 bits).
__device__ __forceinline__ void load8(const uint8_t* unit, int fmt, int ps, int D, int row, int ch, float (&x)[8]) {
    const int64_t at = (int64_t)row * D + ch;
    if (fmt == KVQ_F16) {
        unpack8<__half>(*reinterpret_cast<const uint4*>(unit + at * 2), x);
        return;
    }
    if (fmt == KVQ_BF16) {
        unpack8<__nv_bfloat16>(*reinterpret_cast<const uint4*>(unit + at * 2), x);
        return;
    }
    const int rb = fmt == KVQ_Q8_0 ? D : D / 2;
    const float d = __half2float(reinterpret_cast<const __half*>(unit + (int64_t)ps * rb)[row * (D / 32) + ch / 32]);
    if (fmt == KVQ_Q8_0) {
        const uint2 c = *reinterpret_cast<const uint2*>(unit + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3))) * d;
    } else {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(unit + at / 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)((int)((c >> (4 * e)) & 15u) - 8) * d;
    }
}

__device__ __forceinline__ void store8(void* out, int dtype, int64_t e, const float (&x)[8]) {
    if (dtype == KVQ_PAGED_F32) {
        float4* o = reinterpret_cast<float4*>((float*)out + e);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>((uint16_t*)out + e) = dtype == KVQ_F16 ? pack8<__half>(x) : pack8<__nv_bfloat16>(x);
    }
}

// grid.y: 0 = K, 1 = V. A CTA takes kReadRows output rows: one thread per row finds the row's sequence
// (binary search over cu) and page, then all threads move the rows' vectors.
constexpr int kReadRows = 16;
__global__ void __launch_bounds__(kRowThreads) read_kernel(ReadParams p) {
    const PagedView& v = p.v;
    __shared__ int s_page[kReadRows], s_row[kReadRows];   // page: -1 reads zeros, -2 leaves the row as it is
    const int w = blockIdx.y, D = v.D, row0 = blockIdx.x * kReadRows;
    if (threadIdx.x < kReadRows) {
        const int r = row0 + threadIdx.x;
        int page = -2, in = 0;
        if (r == 0 && w == 0 && (p.cu[0] < 0 || p.cu[p.n_seq] > p.n_rows)) raise_status(v.status, KVQ_PAGED_BAD_LENGTH);
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
    const int per = v.H * D / 8;
    for (int e = threadIdx.x; e < kReadRows * per; e += kRowThreads) {
        const int r = e / per, c = (e - r * per) * 8, head = c / D, ch = c % D;
        const int page = s_page[r];
        if (page == -2) continue;
        float x[8] = {};
        if (page >= 0) load8(unit_at(v, w, page, head), v.fmt[w], v.ps, D, s_row[r], ch, x);
        store8(p.out[w], p.dtype, ((int64_t)(row0 + r) * v.H + head) * D + ch, x);
    }
}

}  // namespace

int launch_norm_rope(const kvq_norm_rope_args& a, int sm_count, void* stream) {
    return a.dtype == KVQ_F16 ? norm_rope_t<__half>(a, sm_count, (cudaStream_t)stream)
                              : norm_rope_t<__nv_bfloat16>(a, sm_count, (cudaStream_t)stream);
}

int launch_paged_write(const WriteParams& p, void* stream) {
    constexpr int U = 2;
    const int64_t total = (int64_t)p.n_tok * p.v.H * p.v.D / 8;
    const dim3 grid((unsigned)((total + kRowThreads * U - 1) / (kRowThreads * U)), 2);
    if (p.dtype == KVQ_F16) write_kernel<__half, U><<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(p);
    else write_kernel<__nv_bfloat16, U><<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(p);
    return (int)cudaGetLastError();
}

int launch_paged_read(const ReadParams& p, void* stream) {
    ReadParams r = p;
    int first = 0, n = 2;
    if (!p.out[0]) { first = 1; n = 1; }
    else if (!p.out[1]) n = 1;
    const dim3 grid((unsigned)((p.n_rows + kReadRows - 1) / kReadRows), (unsigned)n);
    if (first) {                       // V alone: the kernel's w = 0 takes the V area
        r.out[0] = p.out[1];
        r.v.base[0] = p.v.base[1];
        r.v.unit[0] = p.v.unit[1];
        r.v.fmt[0] = p.v.fmt[1];
    }
    read_kernel<<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(r);
    return (int)cudaGetLastError();
}

}  // namespace kvq
