// Device helpers shared by the paged cache's kernels: 16-bit conversions by type and page lookup.
#pragma once
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cstdint>
#include "paged_internal.h"

namespace kvq {
namespace {

constexpr unsigned kAll = 0xffffffffu;

template <typename T> struct Two;
template <> struct Two<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Two<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// 8 values of a 16-byte vector, widened.
template <typename T> __device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Two<T>::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T> __device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Two<T>::pack(x[0], x[1]), Two<T>::pack(x[2], x[3]), Two<T>::pack(x[4], x[5]),
                      Two<T>::pack(x[6], x[7]));
}

__device__ __forceinline__ void raise_status(uint32_t* status, uint32_t bits) { atomicOr(status, bits); }

// First byte of the unit of (page, head) in the K (w = 0) or V area.
__device__ __forceinline__ const uint8_t* unit_at(const PagedView& v, int w, int page, int head) {
    return v.base[w] + ((int64_t)page * v.H + head) * v.unit[w];
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kL2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A row's maximum m (units of log2) and sum l of 2^(s - m): the log of its sum of exp, and what its output is multiplied
// by. l is 0 only where nothing was seen. NaN scores leave m as it was (a maximum drops them) and make l NaN: so are both.
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// tanh to about 2^-23 of 1 and, below 1/4, of itself (the odd series' first five terms there; 1 - 2 / (1 +
// exp(2 |x|)) above).
__device__ __forceinline__ float tanh_small(float x) {
    const float q = x * x;
    return x * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 0.021869489f, -0.053968254f), 0.13333333f), -0.33333334f), 1.f);
}
__device__ __forceinline__ float tanh_any(float x) {
    const float a = fabsf(x), t = 1.f - __fdividef(2.f, 1.f + ex2(2.f * kL2e * a));
    return a < 0.25f ? tanh_small(x) : copysignf(t, x);
}

// The score options, in units of log2. A score x = q.k * f, f = (the row's power of two) * scale * log2(e);
// with a cap, f = .. * scale / softcap and x = softcap * log2(e) * tanh(q.k * f); then the bias.
struct ScoreRule {
    float scale, cap, cap_l2;      // softmax scale; softcap (0: none); softcap * log2(e)
    bool biased;
    __device__ __forceinline__ bool plain() const { return cap == 0.f && !biased; }
    // kept among fp32's normal numbers: 0 or an infinity times a score of infinity or 0 is no score
    __device__ __forceinline__ float factor(float back) const {
        return fminf(fmaxf(back * scale * (cap > 0.f ? 1.f / cap : kL2e), 1.17549435e-38f), 3.40282347e38f);
    }
    // dist: |distance| in positions; slope_l2: the head's slope * log2(e)
    __device__ __forceinline__ float operator()(float x, int dist, float slope_l2) const {
        if (cap > 0.f) x = cap_l2 * tanh_any(x);
        return biased ? x - slope_l2 * (float)dist : x;
    }
};
__device__ __forceinline__ ScoreRule score_rule(const PagedAttnParams& p) {
    ScoreRule r;
    r.scale = p.scale;
    r.cap = p.softcap;
    r.cap_l2 = p.softcap * kL2e;
    r.biased = p.slopes != nullptr;
    return r;
}

__device__ __forceinline__ __half2 h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// raw halves (1024 + u), u = code + off, times the scale pair d: fp16(code x scale), one rounding.
__device__ __forceinline__ uint32_t deq(uint32_t raw, float off1024, uint32_t d) {
    return u32(__hmul2(__hsub2(h2(raw), __float2half2_rn(off1024)), h2(d)));
}
// A pair of block scales (d <= 0x7c00 as they are written) cut to kMaxScale, so that code x scale stays below fp16's
// infinity; scales that are no number become NaN (0 x d), as the minimum alone would not keep them.
template <bool Q8> __device__ __forceinline__ uint32_t cut_scales(uint32_t d) {
    const uint32_t top = Q8 ? kMaxScaleQ8 * 0x10001u : kMaxScaleQ4 * 0x10001u;
    return u32(__hfma2(h2(d), h2(0u), __hmin2(h2(d), h2(top))));
}
}  // namespace
}  // namespace kvq
