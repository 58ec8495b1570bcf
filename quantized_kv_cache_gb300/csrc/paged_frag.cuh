// Warp-level pieces of the paged decode kernel: page rows turned into mma.sync operands.
//
// One warp holds 8 NQ query rows (N of m16n8k16) against a tile of 16 positions of one page. Both products take
// their operands from 16-byte pieces of the rows, in whatever order the lanes read them: the channel order of the
// score product is free (the query fragments follow it), and so is the channel order of the output. With
// g = lane / 4, t = lane % 4:
//  - scores, S^T[16 positions x 8] = K Q^T: lane (g, t) reads pieces t, t + 4, .. of rows g and g + 8; each piece
//    feeds k-steps whose channels qchan() names (eight consecutive ones for two steps);
//  - values, O^T[16 channels x 8] = V^T P^T: lane (g, t) reads pieces g, g + 8, .. of rows 2t, 2t+1, 2t+8, 2t+9 and
//    pairs the rows channel by channel (byte permutes); channels 2i and 2i + 1 of its piece are rows g and g + 8
//    of a product, so a lane ends with runs of consecutive output channels of queries 2t and 2t + 1.
// P^T comes from the accumulators of S^T by one 8 x 8 transposition per 8 positions. Codes become exact fp16
// integers (an exponent placed around the code bits, one subtract), then code x scale is rounded to fp16 once (scales cut to what keeps
// that finite: two operations a pair of blocks).
// Queries on N: a group of up to eight takes half of the products and of the registers that they would take on M.
#pragma once
#include <type_traits>
#include "paged_common.cuh"

namespace kvq {
namespace {

enum { PF_16 = 0, PF_Q8 = 1, PF_Q4 = 2 };   // row encodings: 16-bit values, int8 codes, nibbles

__device__ __forceinline__ void mma_t(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_t(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (r & 0x000f000f) | 0x64006400 and (r & 0x00ff00ff) ^ 0x64806480: one logic operation each.
__device__ __forceinline__ uint32_t nib_raw(uint32_t r) { return (r & 0x000f000fu) | 0x64006400u; }
// nibbles at bits 4-7 of each half: 1024 + 16 n
__device__ __forceinline__ uint32_t nib_raw_hi(uint32_t r) { return (r & 0x00f000f0u) | 0x64006400u; }
__device__ __forceinline__ uint32_t deq_hi(uint32_t raw, uint32_t d) {
    // (1024 + 16 n) / 16 - 72 = n - 8, exact
    return u32(__hmul2(__hfma2(h2(raw), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)), h2(d)));
}
__device__ __forceinline__ uint32_t byte_raw(uint32_t r) { return (r & 0x00ff00ffu) ^ 0x64806480u; }
// four nibbles of each half of r (two rows' halfwords): operand registers of nibble positions 0..3
__device__ __forceinline__ void nib_pairs(uint32_t r, uint32_t d, uint32_t (&o)[4]) {
    o[0] = deq(nib_raw(r), 1032.f, d);
    o[1] = deq_hi(nib_raw_hi(r), d);
    const uint32_t s = r >> 8;
    o[2] = deq(nib_raw(s), 1032.f, d);
    o[3] = deq_hi(nib_raw_hi(s), d);
}
// two signed bytes of each half of r
__device__ __forceinline__ void byte_pairs(uint32_t r, uint32_t d, uint32_t& o0, uint32_t& o1) {
    o0 = deq(byte_raw(r), 1152.f, d);
    o1 = deq(byte_raw(r >> 8), 1152.f, d);
}

template <int N> struct Words { uint32_t w[N]; };

template <int D, int PF> struct KGeo {
    static constexpr int RB = PF == PF_16 ? 2 * D : (PF == PF_Q8 ? D : D / 2);   // row bytes
    static constexpr int CB = RB / 4 < 16 ? RB / 4 : 16;                          // piece bytes
    static constexpr int NJ = RB / 4 / CB, NW = CB / 4;                           // pieces, words of one
    static constexpr int CH = PF == PF_16 ? CB / 2 : (PF == PF_Q8 ? CB : CB * 2); // channels of one
};
template <int D, int PF> struct VGeo {
    static constexpr int RB = KGeo<D, PF>::RB;
    static constexpr int CB = RB / 8 < 16 ? RB / 8 : 16;
    static constexpr int NJ = RB / 8 / CB, NW = CB / 4;
    static constexpr int CH = PF == PF_16 ? CB / 2 : (PF == PF_Q8 ? CB : CB * 2);
};

// First of the eight consecutive channels that k-steps 2 i and 2 i + 1 of lane t take. Their operand pairs are
// (0, 1), (2, 3) | (4, 5), (6, 7), or for nibbles (0, 4), (1, 5) | (2, 6), (3, 7), as the rows decode.
template <int D, int PF> __device__ __forceinline__ int qchan(int i, int t) {
    constexpr int CH = KGeo<D, PF>::CH, N = CH / 8;             // groups of eight in a piece
    return CH * (t + 4 * (i / N)) + 8 * (i % N);
}

// First of the CH consecutive output channels of lane group g in piece j.
template <int D, int PF> __device__ __forceinline__ int ochan(int j, int g) { return VGeo<D, PF>::CH * (g + 8 * j); }

// Where a lane finds its pieces and scales in a tile, fixed over the tiles: a tile in shared memory is 16 code rows of RB
// bytes, then (block formats) the rows' scales. The 16-byte pieces of a 128-byte line are permuted by row so
// that the eight lanes of a load phase (K: two rows, four neighbouring pieces; V: rows 0, 2, 4, 6, two
// neighbouring pieces) hit all banks.
template <int RB, bool VALUES> __device__ __forceinline__ uint32_t tile_swizzle(uint32_t byte) {
    const uint32_t row = byte / RB;
    if (VALUES) return byte ^ (RB >= 64 ? ((row >> 1) & 3) << 5 : ((row >> 2) & 1) << 5);
    return RB >= 128 ? byte ^ ((row & 1) << 6) : byte;
}
template <int D, int KF, int VF> struct LanePlace {
    using K = KGeo<D, KF>;
    using V = VGeo<D, VF>;
    uint32_t k[2], ks;        // K: pieces of even and odd j of row g; the row's first scale
    uint32_t v[2], vs;        // V: piece 0 of rows 2t, 2t + 1; the first scale of row 2t
    __device__ __forceinline__ LanePlace(int g, int t) {
        k[0] = tile_swizzle<K::RB, false>(g * K::RB + K::CB * t);
        k[1] = tile_swizzle<K::RB, false>(g * K::RB + (K::NJ > 1 ? K::CB * (t + 4) : K::CB * t));
        ks = 16 * K::RB + g * (D / 16) + K::CH * t / 32 * 2;
        v[0] = tile_swizzle<V::RB, true>(2 * t * V::RB + V::CB * g);
        v[1] = tile_swizzle<V::RB, true>((2 * t + 1) * V::RB + V::CB * g);
        vs = 16 * V::RB + 2 * t * (D / 16) + V::CH * g / 32 * 2;
    }
};
template <int N> __device__ __forceinline__ Words<N> ld_words(uint32_t a) {
    Words<N> w;
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(w.w[0]), "=r"(w.w[1]), "=r"(w.w[2]), "=r"(w.w[3]) : "r"(a));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(w.w[0]), "=r"(w.w[1]) : "r"(a));
    else
        asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w.w[0]) : "r"(a));
    return w;
}
__device__ __forceinline__ uint32_t ld_half(uint32_t a) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(x) : "r"(a));
    return x;
}

// s[q] += K Q^T of the tile at `base` and query group q.
template <int D, int PF, int NQ, typename T, typename PLACE>
__device__ __forceinline__ void tile_scores(uint32_t base, const PLACE& at, const uint32_t (&qf)[D / 16][NQ][2], float (&s)[NQ][4]) {
    using K = KGeo<D, PF>;
    static_assert(K::NJ == 1 || K::CB == 16, "pieces j and j + 2 are 128 bytes apart");
    const uint32_t even = base + at.k[0], odd = base + at.k[1], sc = base + at.ks;
    const auto step = [&](int ks, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        const uint32_t a[4] = {a0, a1, a2, a3};
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma_t(s[q], a, qf[ks][q][0], qf[ks][q][1], T());
    };
#pragma unroll
    for (int j = 0; j < K::NJ; ++j) {
        const uint32_t a = (j & 1 ? odd : even) + j / 2 * 128;
        const Words<K::NW> x = ld_words<K::NW>(a), y = ld_words<K::NW>(a + 8 * K::RB);     // rows g, g + 8
        constexpr int KS = K::CH / 4;
        if constexpr (PF == PF_16) {
            step(KS * j, x.w[0], y.w[0], x.w[1], y.w[1]);
            step(KS * j + 1, x.w[2], y.w[2], x.w[3], y.w[3]);
        } else {
            const uint32_t d1 = ld_half(sc + K::CH * j / 4), e1 = ld_half(sc + 8 * (D / 16) + K::CH * j / 4);
            const uint32_t d = cut_scales<PF == PF_Q8>(__byte_perm(d1, d1, 0x1010)), e = cut_scales<PF == PF_Q8>(__byte_perm(e1, e1, 0x1010));
#pragma unroll
            for (int i = 0; i < K::NW; ++i) {
                if constexpr (PF == PF_Q8) {
                    const uint32_t u = x.w[i] ^ 0x80808080u, v = y.w[i] ^ 0x80808080u;     // 1024 + 128 + b by an exponent byte
                    step(KS * j + i, deq(__byte_perm(u, 0x64646464u, 0x4140), 1152.f, d), deq(__byte_perm(v, 0x64646464u, 0x4140), 1152.f, e),
                         deq(__byte_perm(u, 0x64646464u, 0x4342), 1152.f, d), deq(__byte_perm(v, 0x64646464u, 0x4342), 1152.f, e));
                } else {
                    uint32_t o[4], r[4];                                   // (n0, n4), (n1, n5), (n2, n6), (n3, n7)
                    nib_pairs(x.w[i], d, o);
                    nib_pairs(y.w[i], e, r);
                    step(KS * j + 2 * i, o[0], r[0], o[1], r[1]);
                    step(KS * j + 2 * i + 1, o[2], r[2], o[3], r[3]);
                }
            }
        }
    }
}

// o += V^T P^T of the tile's 16 positions. With LO, P = p + lo (two bf16 parts).
template <int D, int PF, int NQ, typename T, bool LO, typename PLACE>
__device__ __forceinline__ void tile_values(uint32_t base, const PLACE& at, const uint32_t (&p)[NQ][2], const uint32_t (&lo)[NQ][2],
                                            float (&o)[D / 16][NQ][4]) {
    using V = VGeo<D, PF>;
    static_assert(V::NJ == 1 || V::CB == 16, "pieces j and j + 1 are 128 bytes apart");
    // rows 2t + 8 and 2t + 9: the same permutation (that of 32-byte rows too: two lines on)
    const uint32_t a0 = base + at.v[0], a1 = base + at.v[1], sc = base + at.vs;
#pragma unroll
    for (int j = 0; j < V::NJ; ++j) {
        const Words<V::NW> r0 = ld_words<V::NW>(a0 + 128 * j), r1 = ld_words<V::NW>(a1 + 128 * j);
        const Words<V::NW> r2 = ld_words<V::NW>(a0 + 128 * j + 8 * V::RB), r3 = ld_words<V::NW>(a1 + 128 * j + 8 * V::RB);
        uint32_t d01 = 0, d23 = 0;
        if constexpr (PF != PF_16) {
            const uint32_t x = sc + V::CH * j / 2;
            d01 = cut_scales<PF == PF_Q8>(__byte_perm(ld_half(x), ld_half(x + D / 16), 0x5410));
            d23 = cut_scales<PF == PF_Q8>(__byte_perm(ld_half(x + 8 * (D / 16)), ld_half(x + 9 * (D / 16)), 0x5410));
        }
#pragma unroll
        for (int i = 0; i < V::NW; ++i) {
            const uint32_t xl = __byte_perm(r0.w[i], r1.w[i], 0x5410), xh = __byte_perm(r0.w[i], r1.w[i], 0x7632);
            const uint32_t yl = __byte_perm(r2.w[i], r3.w[i], 0x5410), yh = __byte_perm(r2.w[i], r3.w[i], 0x7632);
            constexpr int N = V::CH / V::NW;      // channels of a word: 2, 4, 8
            uint32_t b0[N], b1[N];
            if constexpr (PF == PF_16) {
                b0[0] = xl; b0[1] = xh; b1[0] = yl; b1[1] = yh;
            } else if constexpr (PF == PF_Q8) {
                byte_pairs(xl, d01, b0[0], b0[1]);
                byte_pairs(xh, d01, b0[2], b0[3]);
                byte_pairs(yl, d23, b1[0], b1[1]);
                byte_pairs(yh, d23, b1[2], b1[3]);
            } else {
                nib_pairs(xl, d01, *(uint32_t(*)[4])&b0[0]);
                nib_pairs(xh, d01, *(uint32_t(*)[4])&b0[4]);
                nib_pairs(yl, d23, *(uint32_t(*)[4])&b1[0]);
                nib_pairs(yh, d23, *(uint32_t(*)[4])&b1[4]);
            }
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const uint32_t a[4] = {b0[c], b0[c + 1], b1[c], b1[c + 1]};
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    float (&acc)[4] = o[(V::CH * j + N * i + c) / 2][q];
                    mma_t(acc, a, p[q][0], p[q][1], T());
                    if constexpr (LO) mma_t(acc, a, lo[q][0], lo[q][1], T());
                }
            }
        }
    }
}

// Query fragments of a warp's 8 NQ rows; row r is at rows(r) (null: a row of zeros), of type TQ. fp16 operands of bf16
// queries are scaled by a power of two per row so that no exponent is out of range; back[] undoes it (of row g + 8q).
template <int D, int PF, int NQ, typename T, typename TQ, typename ROW>
__device__ __forceinline__ void load_queries(const ROW& rows, int g, int t, uint32_t (&qf)[D / 16][NQ][2], float (&back)[NQ]) {
    constexpr bool same = std::is_same<T, TQ>::value;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const TQ* p = rows(g + 8 * q);
        float up = 1.f;
        back[q] = 1.f;
        if constexpr (!same) {
            float a = 0.f;
            if (p) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float f[8];
                    unpack8<TQ>(*reinterpret_cast<const uint4*>(p + (D / 4) * t + 8 * i), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(f[e]));
                }
            }
            a = fmaxf(a, __shfl_xor_sync(kAll, a, 1));
            a = fmaxf(a, __shfl_xor_sync(kAll, a, 2));
            const int ex = (int)((__float_as_uint(a) >> 23) & 255) - 127;
            if (a > 0.f && ex < 128) {
                const int sh = min(14 - ex, 100);                    // the largest magnitude to [2^14, 2^15): from -113 on
                up = __uint_as_float((uint32_t)(127 + sh) << 23);
                back[q] = __uint_as_float((uint32_t)(127 - sh) << 23);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (p) {
                x = *reinterpret_cast<const uint4*>(p + qchan<D, PF>(i, t));
                if constexpr (!same) {
                    float y[8];
                    unpack8<TQ>(x, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= up;
                    x = pack8<T>(y);
                }
            }
            if constexpr (PF == PF_Q4)
                x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                               __byte_perm(x.y, x.w, 0x7632));
            qf[2 * i][q][0] = x.x;
            qf[2 * i][q][1] = x.y;
            qf[2 * i + 1][q][0] = x.z;
            qf[2 * i + 1][q][1] = x.w;
        }
    }
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
    return d;
}

template <int D, int PF> constexpr int tile_bytes() { return 16 * KGeo<D, PF>::RB + (PF == PF_16 ? 0 : D); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
__device__ __forceinline__ void st_zero16(uint32_t dst) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(dst), "r"(0) : "memory");
}

// A lane's place in a tile's copy: piece `lane` of every 512 bytes. The permutation is a xor by bits of the
// row, of which 512 * i and the lane set different ones: one offset per lane and a constant per i.
template <int D, int PF, bool VALUES> __device__ __forceinline__ uint32_t copy_lane(int lane) {
    return tile_swizzle<KGeo<D, PF>::RB, VALUES>(lane * 16);
}

// One warp starts the copy of a tile (16 rows from row `off` of a page's unit) to shared memory; a null
// unit (a page number out of range) gives zeros.
template <int D, int PF, bool VALUES>
__device__ __forceinline__ void copy_tile(uint32_t dst, uint32_t at, const uint8_t* unit, int ps, int off, int lane) {
    constexpr int RB = KGeo<D, PF>::RB, N = 16 * RB / 16;
    if (unit) {
        const uint8_t* src = unit + off * RB + lane * 16;
#pragma unroll
        for (int i = 0; i < (N + 31) / 32; ++i)
            if (N % 32 == 0 || lane < N) cp_async16(dst + 512 * i + (at ^ (tile_swizzle<RB, VALUES>(512 * i) - 512 * i)), src + 512 * i);
        if constexpr (PF != PF_16)
            if (lane < D / 16) cp_async16(dst + 16 * RB + lane * 16, unit + ps * RB + off * (D / 16) + lane * 16);
    } else {
        for (int i = lane; i < tile_bytes<D, PF>() / 16; i += 32) st_zero16(dst + i * 16);
    }
}

// Zeroes what the rows outside `live` would add (the values of 16-bit rows, the scales of the others): a
// weight of 0 does not keep an infinity or NaN of an unused row out of the product.
template <int D, int PF> __device__ __forceinline__ void clear_rows(uint32_t base, uint32_t live, int lane) {
    constexpr int RB = KGeo<D, PF>::RB;
    if constexpr (PF == PF_16) {
        for (int c = lane; c < RB; c += 32)            // 16 rows x RB / 16 pieces
            if (!((live >> (c / (RB / 16))) & 1)) st_zero16(base + tile_swizzle<RB, true>(c * 16));
    } else {
        for (int c = lane; c < 16 * (D / 32); c += 32)
            if (!((live >> (c / (D / 32))) & 1))
                asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(base + 16 * RB + 2 * c), "h"((uint16_t)0) : "memory");
    }
}

}  // namespace
}  // namespace kvq
