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

}  // namespace
}  // namespace kvq
