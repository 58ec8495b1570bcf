// Attention of chunks of new tokens over pages, and of whole prompts over their own rows, on the tensor cores (tcgen05).
//
// The rows of a KV head are the chunk's tokens times the G query heads that read it, row r = token r / G,
// head r % G, so K and V tiles serve all of them. A CTA holds NT tiles of 128 rows (two up to D = 128, one
// at D = 256, where the output takes half of the tensor memory) and walks the BN-position tiles that any of
// its rows sees. Its warps have fixed parts:
//  - producers bring K and V tiles into a ring of four shared-memory slots, page by page, as fp16 / bf16 in
//    the 128-byte-swizzled layout both products read: K with the summed axis contiguous, V with its other
//    axis contiguous. 16-bit pages come by tensor-map copies, one lane per page and 64 channels (16-byte
//    copies by the threads took 1,550 of the 2,400 cycles of a tile); a tile that ends behind the last position
//    is copied by the threads, zeros in place of the rows behind it. Quantised rows are decoded on the way. Prompts' own rows come
//    by tensor-map copies alone;
//  - one warp issues the products: S = Q K^T into tensor memory, and O += P V with P read from tensor memory;
//  - one thread per row does the softmax: S from tensor memory to registers, maximum, exponentials, P back
//    over S. The running maximum moves only when it grows by more than 2^4 (bf16 pages: 2^8), so that O is
//    rescaled rarely.
// With two row tiles, the products of one run while the other's softmax does; with one, S of the next
// tile is computed meanwhile (two S buffers).
//
// 4,096 tokens at 8,192 positions, 40 heads on 8 x 128, bf16: 412 us, 1,250 TFLOP/s (65% of the measured matrix rate); 9 packed
// prompts up to 8,191 tokens, their own rows: 2,614 us, 1,258 TFLOP/s. A row tile's turn is a chain: softmax 1,000 cycles, products
// 1,130 (1,024 at the peak), barriers and wake-ups 850; the other tile's turn fills most of the rest. 16-bit pages at D = 256
// (4,096 tokens at 8,192, 24 heads on 4): 620 us, 52%, the scores of 64 positions taking as long as those of 128 would; D = 64 (40
// heads on 8): 340 us, 39%. Over codes every row tile (two up to D = 128) decodes its positions anew: the 4,096 tokens take 483 us
// (q8_0) and 487 us (e4m3) at D = 128, 739 and 786 us at D = 256, where a tile of 64 positions is 2,600 cycles, its decoding 1,700 of
// them beside the chain. Capped scores cost the products of a polynomial (packed multiply-adds take two cycles): 5 chunks up to
// 1,501 tokens at 6,000, cap 30, 750 us over e4m3 pages of 4 x 256 (without the cap 655).
#include <cuda.h>
#include "stream_common.cuh"
#include "paged_common.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace {

template <int D, bool CODES> struct Geo {
    static constexpr int NT = D == 256 ? 1 : 2;              // row tiles of a CTA
    static constexpr int BN = prefill_tile(D);               // positions of a KV tile
    static constexpr int rows = 128 * NT;
    // warps: four softmax warps per row tile, one that issues the products, producers (decoding codes takes more)
    static constexpr int mma_warp = 4 * NT, first_prod = mma_warp + 1, prod = CODES ? 15 - mma_warp : 3;
    static constexpr int threads = 32 * (first_prod + prod);
    // registers (0: not moved): what the block is launched with, 384 x 168 or 512 x 128, is shared out between the softmax's
    // 128 NT threads and the others. Codes (5 chunks up to 1,501 tokens at 6,000 positions): at D = 256 152 and 120 (200 and 104, the decoding spilling: e4m3 700 us
    // against 655), at D = 128 168 and 88 (152 and 104: 473 against 434; 144 and 112: 442)
    static constexpr int soft_regs = NT == 2 ? (CODES ? 168 : 208) : (CODES ? 152 : 0);
    static constexpr int other_regs = NT == 2 ? 88 : (CODES ? 120 : 0);
    static constexpr int q_bytes = 128 * D * 2;              // of a row tile
    static constexpr int slot = BN * D * 2;
    static constexpr int smem = 1024 + NT * q_bytes + 4 * slot;
    // slots: K of tile i in place i & 1, V in place 2 + (i & 1)
    // tensor memory columns: S (and P over it), two buffers; O
    static constexpr int s_col(int i) { return i * BN; }
    static constexpr int o_col(int t) { return 256 + t * D; }
};

// One sequence's chunk: rows of q, and the positions they sit at.
struct Chunk {
    int row0, n, len, pos0, pre;     // first row of q, tokens worked on, positions held, position of the first token, prefix
};
__device__ __forceinline__ Chunk chunk_of(const PagedAttnParams& p, int b, bool report) {
    Chunk c;
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    const bool bad = c0 < 0 || c1 > p.n_rows || c1 < c0;
    const int len = p.lens ? p.lens[b] : (bad ? 0 : c1 - c0);       // a prompt holds its own rows
    c.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
    c.row0 = c0;
    c.n = bad ? 0 : c1 - c0;
    if (report && (len < 0 || len > cap || bad || c.n > p.max_q)) raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
    c.pos0 = c.len - c.n;
    c.n = min(c.n, p.max_q);                 // the grids hold max_q tokens of a chunk: its first ones
    c.pre = p.prefix ? min(max(p.prefix[b], 0), c.len) : 0;
    return c;
}

// The KV tiles of rows whose positions span [first, last]: [0, n0) of the prefix, then [t1, t1 + n - n0).
template <int BN> struct KvTiles {
    int n0, t1, n;
    __device__ __forceinline__ KvTiles(const Chunk& c, int first, int last, int window) {
        const int end = last < 0 ? 0 : (max(last + 1, c.pre) + BN - 1) / BN;
        t1 = min(end, window > 0 && first >= window ? (first - window + 1) / BN : 0);   // first may be far below 0
        n0 = last < 0 ? 0 : min((c.pre + BN - 1) / BN, t1);
        n = n0 + end - t1;
    }
    __device__ __forceinline__ int at(int i) const { return (i < n0 ? i : t1 + i - n0) * BN; }
};

// Byte of the 16-byte piece holding channels ch .. ch + 7 of row r in a tile of `rows` rows.
__device__ __forceinline__ uint32_t tile_byte(int rows, int r, int ch) {
    return (uint32_t)((ch >> 6) * rows * 128 + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// Eight channels of a quantised row as fp16: code x scale, rounded once (natural channel order).
__device__ __forceinline__ uint4 decode_q8(uint2 c, uint32_t d) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = (i ? c.y : c.x) ^ 0x80808080u;
        o[2 * i] = deq(__byte_perm(x, 0x64646464u, 0x4140), 1152.f, d);
        o[2 * i + 1] = deq(__byte_perm(x, 0x64646464u, 0x4342), 1152.f, d);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 decode_q4(uint32_t c, uint32_t d) {
    // a byte in both halves: its low nibble as 1024 + n, its high one as 1024 + 16 n; then n - 8 in one step
    const __half2 mul = __floats2half2_rn(1.f, 0.0625f), add = __floats2half2_rn(-1032.f, -72.f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = (__byte_perm(c, 0, 0x4040 + 0x101 * i) & 0x00f0000fu) | 0x64006400u;
        o[i] = u32(__hmul2(__hfma2(h2(r), mul, add), h2(d)));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight e4m3 codes as fp16: code x power, rounded once. The power comes as a factor of 2^-13 at least (with it a code is an fp16
// number) and, where `small`, what is left of it.
__device__ __forceinline__ uint4 decode_e4(uint2 c, uint32_t mul, uint32_t rest, bool small) {
    uint32_t o[4];
    e4m3_four(c.x, o[0], o[1]);
    e4m3_four(c.y, o[2], o[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = u32(__hmul2(h2(o[i]), h2(mul)));
        if (small) o[i] = u32(__hmul2(h2(o[i]), h2(rest)));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A wait on a barrier's phase, bounded as the streaming kernels' are (2 s, then the status bit and the CTA's
// abort flag), that looks at the clock and the flag only every 32nd time. False where it gave up.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* abort_flag) {
    uint64_t t0 = 0;
    for (int n = 1; !mbar_try(bar, parity); ++n) {
        if (n & 31) continue;
        if (*abort_flag) return false;
        const uint64_t t = gtime();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitNs) {
            raise_status(status, KVQ_PAGED_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// What one row's thread keeps.
struct RowState {
    int pos, lo;             // position (rows that see nothing: -1), first position of the window
    int hi, pre;             // last visible position; positions < pre are visible too
    float f, slope;          // factor of a raw score; slope * log2(e)
};

// o += p V over the positions of the tile that this row sees: used where some row does not see all of the
// tile and the tile holds an infinity or NaN, which a weight of 0 would not keep out of the product.
template <int D, int BN, typename T>
__device__ __noinline__ void add_seen(uint32_t v_tile, uint32_t o_addr, uint32_t p_addr, const RowState& r, int p0, bool first) {
    // the weights come back from tensor memory (rounded as the product would take them)
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t o[32];
        if (first) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
        } else {
            tmem_ld32(o_addr + d0, o);
            tmem_wait_ld(o);
        }
#pragma unroll 1
        for (int c = 0; c < BN / 64; ++c) {
            uint32_t w[32];
            tmem_ld32(p_addr + 32 * c, w);
            tmem_wait_ld(w);
#pragma unroll 1
            for (int e = 0; e < 64; ++e) {
                const int j = p0 + 64 * c + e;
                if (!((j <= r.hi && j >= r.lo) || j < r.pre)) continue;
                const float2 f = Two<T>::unpack(w[e / 2]);
                const float wt = e & 1 ? f.y : f.x;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
                    unpack8<T>(ld_shared16(v_tile + tile_byte(BN, 64 * c + e, d0 + 8 * q)), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[8 * q + k] = __float_as_uint(fmaf(wt, v[k], __uint_as_float(o[8 * q + k])));
                }
            }
        }
        tmem_st32(o_addr + d0, o);
        tmem_wait_st();
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
    return (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
}
__device__ __forceinline__ float2 unpair(uint64_t x) { return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32))); }

// Weights 2^(s f - m) of 32 scores, packed two by two into w; adds them to the sums and finds the largest score. A warp
// has its scheduler almost to itself here, and the exponential unit takes one instruction in four cycles: the
// instructions are written in the order in which they should issue, between two exponentials a multiply-add of
// the next pairs and the rounding, sum and maximum of the last (grouped by kind they took 240 cycles, not 128).
template <typename T>
__device__ __forceinline__ void weights32(const uint32_t (&x)[32], uint64_t f, uint64_t m, uint32_t* w, uint64_t (&sum)[4], float (&top)[4]) {
    uint64_t u[16];
    float v[32] = {};
    const auto first = [&](int e) {
        const uint64_t a = (uint64_t)x[2 * e] | ((uint64_t)x[2 * e + 1] << 32);
        asm volatile("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(u[e]) : "l"(a), "l"(f), "l"(m));
    };
    const auto last = [&](int e) {
        if constexpr (std::is_same<T, __half>::value)
            asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
        else
            asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
        asm volatile("add.rn.f32x2 %0, %0, %1;\n" : "+l"(sum[e & 3]) : "l"(pair(v[2 * e], v[2 * e + 1])));
    };
    constexpr int A = 2;                                      // pairs that the multiply-adds and the roundings are apart by
#pragma unroll
    for (int e = 0; e < A; ++e) first(e);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 y = unpair(u[e]);
        asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * e]) : "f"(y.x));
        if (e + A < 16) first(e + A);
        asm volatile("max.f32 %0, %0, %1, %2;\n" : "+f"(top[e & 3]) : "f"(__uint_as_float(x[2 * e])), "f"(__uint_as_float(x[2 * e + 1])));
        asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * e + 1]) : "f"(y.y));
        if (e >= A) last(e - A);
    }
#pragma unroll
    for (int e = 16 - A; e < 16; ++e) last(e);
}

// The exponentials of 16 pairs, packed, added to the sums; their largest arguments.
template <typename T>
__device__ __forceinline__ void exps32(const float2 (&x)[16], uint32_t* w, uint64_t (&sum)[4], float (&top)[4]) {
    float v[32] = {};
    const auto last = [&](int e) {                            // as in weights32
        if constexpr (std::is_same<T, __half>::value)
            asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
        else
            asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
        asm volatile("add.rn.f32x2 %0, %0, %1;\n" : "+l"(sum[e & 3]) : "l"(pair(v[2 * e], v[2 * e + 1])));
    };
    constexpr int A = 2;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * e]) : "f"(x[e].x));
        asm volatile("max.f32 %0, %0, %1, %2;\n" : "+f"(top[e & 3]) : "f"(x[e].x), "f"(x[e].y));
        asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * e + 1]) : "f"(x[e].y));
        if (e >= A) last(e - A);
    }
#pragma unroll
    for (int e = 16 - A; e < 16; ++e) last(e);
}

// weights32 with a cap alone, straight through: y = cap tanh(s f) = s (a0 + a1 s^2 + a2 s^4 + a3 s^6) for |s f| < 0.35 (a: of the
// polynomial below, with f and the cap in it). What is beyond that shows in `big`, the largest |s|. No branch parts the products from
// the exponentials, and they are written in the order in which they should issue, as in weights32: a pair's six products one step apart
// from the next pair's, so that none waits for the one before it. 5 chunks up to 1,501 tokens at 6,000 positions, 40 heads on 8 x 128,
// a cap of 30, 16-bit pages: 500 us, with rule_weights32 for every tile 684, without the cap 367. Over codes the registers bind (168 a
// softmax thread, where scores and weights of a tile are 128): 766 us, without the cap 434.
template <typename T>
__device__ __forceinline__ void cap_weights32(const uint32_t (&s)[32], const uint64_t (&a)[4], uint64_t m, uint32_t* w, uint64_t (&sum)[4],
                                              float (&top)[4], float& big) {
    uint64_t q[16], p[16];
    float v[32];
    const auto both = [&](int e) { return (uint64_t)s[2 * e] | ((uint64_t)s[2 * e + 1] << 32); };
#pragma unroll
    for (int n = -6; n < 18; ++n) {
        const auto at = [&](int e) { return e >= 0 && e < 16; };
        float2 y = make_float2(0.f, 0.f);
        if (at(n)) {
            y = unpair(p[n]);
            asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * n]) : "f"(y.x));
        }
        if (at(n + 6)) asm volatile("mul.rn.f32x2 %0, %1, %1;\n" : "=l"(q[n + 6]) : "l"(both(n + 6)));
        if (at(n + 5)) asm volatile("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(p[n + 5]) : "l"(q[n + 5]), "l"(a[3]), "l"(a[2]));
        if (at(n + 6))
            asm volatile("{ .reg .f32 x, y; abs.f32 x, %1; abs.f32 y, %2; max.f32 %0, %0, x, y; }\n"
                         : "+f"(big) : "f"(__uint_as_float(s[2 * (n + 6)])), "f"(__uint_as_float(s[2 * (n + 6) + 1])));
        if (at(n + 4)) asm volatile("fma.rn.f32x2 %0, %1, %0, %2;\n" : "+l"(p[n + 4]) : "l"(q[n + 4]), "l"(a[1]));
        if (at(n + 3)) asm volatile("fma.rn.f32x2 %0, %1, %0, %2;\n" : "+l"(p[n + 3]) : "l"(q[n + 3]), "l"(a[0]));
        if (at(n)) {
            asm volatile("max.f32 %0, %0, %1, %2;\n" : "+f"(top[n & 3]) : "f"(y.x), "f"(y.y));
            asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(v[2 * n + 1]) : "f"(y.y));
        }
        if (at(n + 2)) asm volatile("mul.rn.f32x2 %0, %0, %1;\n" : "+l"(p[n + 2]) : "l"(both(n + 2)));
        if (at(n + 1)) asm volatile("add.rn.f32x2 %0, %0, %1;\n" : "+l"(p[n + 1]) : "l"(m));       // by itself, as below
        if (at(n - 2)) {
            const int e = n - 2;
            if constexpr (std::is_same<T, __half>::value)
                asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
            else
                asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
            asm volatile("add.rn.f32x2 %0, %0, %1;\n" : "+l"(sum[e & 3]) : "l"(pair(v[2 * e], v[2 * e + 1])));
        }
    }
}

// weights32 with the cap and the bias on the way: scores of 32 positions from p0 on, in units of log2, less the row's maximum (m its
// negative) as it stands; `hide` takes out what the row does not see. Where all capped scores are below 0.35 of the cap no
// exponential is taken for them: tanh x = x (1 + q c(q)), q = x^2, with the polynomial of least relative error on that range
// (2^-24.5). top: the largest score less the maximum.
template <typename T, typename HIDE>
__device__ __forceinline__ void rule_weights32(uint32_t (&s)[32], const ScoreRule& rule, const RowState& r, int p0, float m, const HIDE& hide,
                                               uint32_t* w, uint64_t (&sum)[4], float (&top)[4]) {
    const float2 f = make_float2(r.f, r.f), back = make_float2(m, m);
    float2 x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
    if (rule.cap > 0.f) {
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = __fmul2_rn(x[e], f);
            big = max3(big, fabsf(x[e].x), fabsf(x[e].y));
        }
        const auto both = [&](float c) { return make_float2(c * rule.cap_l2, c * rule.cap_l2); };
        if (__all_sync(kAll, big < 0.35f)) {
            const float2 c0 = both(1.f), c1 = both(-0.33332664f), c2 = both(0.13299826f), c3 = both(-0.049148493f);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 q = __fmul2_rn(x[e], x[e]);
                x[e] = __fmul2_rn(x[e], __ffma2_rn(q, __ffma2_rn(q, __ffma2_rn(q, c3, c2), c1), c0));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = make_float2(rule.cap_l2 * tanh_any(x[e].x), rule.cap_l2 * tanh_any(x[e].y));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __fmul2_rn(x[e], f);
    }
    if (rule.biased) {
        const float d = (float)(r.pos - p0);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e].x = fmaf(-r.slope, fabsf(d - (float)(2 * e)), x[e].x);
            x[e].y = fmaf(-r.slope, fabsf(d - (float)(2 * e + 1)), x[e].y);
        }
    }
    // subtracted by itself: of large scores the rounding of the product would be left where it is fused
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __fadd2_rn(x[e], back);
    hide(x);
    exps32<T>(x, w, sum, top);
}

// Whole prompts: the row tiles of all sequences are one line, so that ragged ones leave no block without work. The sequence of
// tile `slot`, and the tile's number in it (-1: the line is shorter); called by whole warps.
__device__ __forceinline__ int find_tile(const PagedAttnParams& p, int slot, int tile_rows, bool report, int* tile) {
    const int lane = threadIdx.x & 31;
    int before = 0, found = -1;
    for (int i = 0; i < p.n_seq && (found < 0 || report); i += 32) {
        const int b = i + lane;
        int n = 0;
        if (b < p.n_seq) n = (chunk_of(p, b, report).n * p.G + tile_rows - 1) / tile_rows;
        int sum = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int y = __shfl_up_sync(kAll, sum, s);
            if (lane >= s) sum += y;
        }
        const unsigned m = __ballot_sync(kAll, found < 0 && before + sum > slot);
        if (m) {
            const int k = __ffs(m) - 1;
            found = i + k;
            *tile = slot - before - __shfl_sync(kAll, sum - n, k);
        }
        before += __shfl_sync(kAll, sum, 31);
    }
    return found;
}

// Where K and V rows come from: pages of 16-bit rows (0) or codes (1 int8, 2 nibbles, 3 e4m3), or the prompts' own rows (4).
constexpr int kRows = 4;
constexpr bool codes_of(int kf) { return kf > 0 && kf < kRows; }

template <int D, int KF, int VF, typename T, typename TQ, bool RULE>      // RULE: scores go through a cap or a bias
__global__ void __launch_bounds__(Geo<D, codes_of(KF)>::threads, 1) prefill_kernel(const __grid_constant__ PagedAttnParams p,
                                                                        const __grid_constant__ CUtensorMap k_map,
                                                                        const __grid_constant__ CUtensorMap v_map, int splits) {
    using GE = Geo<D, codes_of(KF)>;
    constexpr int NT = GE::NT, BN = GE::BN;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    // Weights are 2^(s - m), m = the largest score when m last moved, less kUp; it moves when a score is more than kLazy
    // above. fp16: up to 2^15, so that weights down to 2^-25 of the largest keep all bits and down to 2^-36 some (with
    // kUp = 0 what lies 2^-25 below the largest was lost to the outputs but not to the sums). bf16 has the exponents, so
    // that m moves more rarely; of a weight it keeps 8 bits (half a step is 2^-8 of it, which averages out over positions).
    constexpr float kUp = BF ? 0.f : 11.f, kLazy = BF ? 8.f : 4.f;
    extern __shared__ uint8_t raw[];
    // full / empty of the load stages; Q in place; S ready, P ready (by S buffer); O of a row tile up to date.
    // Stage u loads what the products take together: V of tile u - 1 and K of tile u.
    __shared__ uint64_t bars[2 + 2 + 1 + 2 + 2 + 2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_skip[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x, split = blockIdx.z % splits, G = p.G;
    const uint32_t full = su32(bars), empty = full + 16, q_full = full + 32, s_full = full + 40, p_full = full + 56,
                   o_done = full + 72;
    grid_dep_wait();
    int b = blockIdx.z / splits, tile = blockIdx.y;
    if constexpr (KF == kRows) {
        b = find_tile(p, blockIdx.y, GE::rows, h == 0 && blockIdx.y == 0 && split == 0 && warp == 0, &tile);
        if (b < 0) return;
    }
    const Chunk c = chunk_of(p, b, KF != kRows && h == 0 && blockIdx.y == 0 && split == 0 && threadIdx.x == 0);
    // tiles in descending order: the last rows see the most positions and start first
    const int rows = c.n * G, row_tiles = (rows + GE::rows - 1) / GE::rows;
    if (tile >= row_tiles) return;
    const int r0 = (row_tiles - 1 - tile) * GE::rows, r1 = min(rows, r0 + GE::rows);
    const KvTiles<BN> kv(c, c.pos0 + r0 / G, c.pos0 + (r1 - 1) / G, p.window);
    const int i0 = (int)((int64_t)kv.n * split / splits), nt = (int)((int64_t)kv.n * (split + 1) / splits) - i0;
    const int active = r1 - r0 > 128 ? 2 : 1;                  // row tiles that hold rows

    const uint32_t base = (su32(raw) + 1023) & ~1023u, ring = base + NT * GE::q_bytes;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 128 * active);
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + 8 * i, KF == kRows ? 32 : 32 * GE::prod);
            mbar_init(empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 128);
            mbar_init(o_done + 8 * i, 1);
        }
        s_abort = s_skip[0] = s_skip[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == GE::mma_warp) tmem_alloc512(su32(&s_tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint32_t bar, uint32_t parity) { return bounded_wait(bar, parity, p.v.status, &s_abort); };

    if (warp >= GE::mma_warp) {
        if constexpr (GE::other_regs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(GE::other_regs));
        if (warp == GE::mma_warp) {
            // ------------------------------------------------------------------ the products
            // One warp for both row tiles: it keeps them half a period apart, so that the softmax of one runs beside
            // the products of the other (with a warp each they fell into step: 594 us for what took 478 us this way).
            if (nt > 0) {
                const uint32_t tm = __shfl_sync(kAll, tmem, 0);
                const uint64_t q_desc = smem_desc(base, 0), k_desc = smem_desc(ring, 0), v_desc = smem_desc(ring + 2 * GE::slot, BN * 128);
                const auto scores = [&](int t, int i) {         // S of row tile t and KV tile i
                    const int buf = NT == 2 ? t : i & 1;
                    const uint64_t q = desc_at(q_desc, t * GE::q_bytes), k = desc_at(k_desc, (i & 1) * GE::slot);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        mma_ss(tm + GE::s_col(buf), desc_at(q, (s / 4) * 128 * 128 + (s % 4) * 32),
                               desc_at(k, (s / 4) * BN * 128 + (s % 4) * 32), mma_desc(BF, false, BN), s > 0);
                    tc_commit(s_full + 8 * buf);
                };
                const auto values = [&](int t, int i) {         // O of row tile t += P V of KV tile i
                    const int buf = NT == 2 ? t : i & 1;
                    const uint64_t v = desc_at(v_desc, (i & 1) * GE::slot);
#pragma unroll
                    for (int s = 0; s < BN / 16; ++s)
                        mma_ts(tm + GE::o_col(t), tm + GE::s_col(buf) + 8 * s, desc_at(v, s * 2048), mma_desc(BF, true, D), i > 0 || s > 0);
                };
                bool may = wait(q_full, 0);                     // after a wait that gave up nothing more is issued
                may &= wait(full, 0);
                tc_fence_after();
                if (elect_one() && may) {
                    for (int t = 0; t < active; ++t) scores(t, 0);
                    tc_commit(empty);
                }
                __syncwarp();
                for (int i = 0; i < nt; ++i) {
                    const int u = i + 1;
                    const bool more = u < nt;
                    may &= wait(full + 8 * (u & 1), (u >> 1) & 1);
                    if (NT == 1 && more) {
                        tc_fence_after();
                        if (elect_one() && may) scores(0, u);
                        __syncwarp();
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (t >= active) break;
                        const int buf = NT == 2 ? t : i & 1;
                        may &= wait(p_full + 8 * buf, NT == 2 ? i & 1 : (i >> 1) & 1);
                        tc_fence_after();
                        const int skip = *(volatile int*)&s_skip[buf];
                        if (elect_one() && may) {
                            if (!skip) values(t, i);
                            if (NT == 1 || !more) tc_commit(o_done + 8 * t);
                            if (NT == 2 && more) scores(t, u);
                            if (t == active - 1) tc_commit(empty + 8 * (u & 1));
                        }
                        __syncwarp();
                    }
                }
            }
        } else {
            // ------------------------------------------------------------------ K and V tiles
            const int pw = warp - GE::first_prod;               // 8-row blocks pw, pw + prod, ..
            const int32_t* table = p.table + (int64_t)b * p.table_stride;
            if constexpr (KF == kRows) {
                // Boxes of BN rows x 64 channels, one per lane of the first producer. A tile that ends behind the prompt
                // holds the next one's rows there (behind the last row zeros): no query here sees them.
                if (pw == 0) {
                    bool may = true;                                // as for the products
                    for (int n = 1; n <= 2 * nt; ++n) {             // items as for 16-bit pages below
                        const int u = n >> 1, w = n & 1 ? 0 : 1, i = w ? u - 1 : u;
                        const uint32_t bar = full + 8 * (u & 1);
                        if (w && u >= 2) may &= wait(empty + 8 * (u & 1), ((u >> 1) - 1) & 1);
                        if (lane == 0 && may) tc_expect(bar, GE::slot);
                        __syncwarp();
                        if (lane < D / 64 && may)
                            tma_load3(ring + (2 * w + (i & 1)) * GE::slot + tile_byte(BN, 0, 64 * lane), w ? &v_map : &k_map, 64 * lane, h,
                                      c.row0 + kv.at(i0 + i), bar);
                        if (w == 0 || u == nt) mbar_arrive(bar);    // the last item of the stage
                    }
                }
            } else if constexpr (KF == 0) {
                // page numbers of a tile's 16-row blocks, one per lane, loaded a tile ahead
                auto pages_of = [&](int i) {
                    int page = -1;
                    const int at = i < nt ? kv.at(i0 + i) + 16 * lane : c.len;
                    if (lane < BN / 16 && at < c.len) {
                        page = table[at >> p.v.ps_shift];
                        if (page < 0 || page >= p.v.n_pages) {
                            raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
                            page = -1;
                        }
                    }
                    return page;
                };
                int page = -1, next_page = pages_of(0);
                bool may = true;                                // as for the products
                // items: V of tile u - 1 and K of tile u, for u = 0 .. nt (no V in the first, no K in the last)
                for (int n = 1; n <= 2 * nt; ++n) {
                    const int u = n >> 1, w = n & 1 ? 0 : 1, i = w ? u - 1 : u, p0 = kv.at(i0 + i);
                    const uint32_t bar = full + 8 * (u & 1);
                    if (w == 0) {
                        page = next_page;
                        next_page = pages_of(i + 1);
                    }
                    if (w && u >= 2) may &= wait(empty + 8 * (u & 1), ((u >> 1) - 1) & 1);
                    const uint32_t dst = ring + (2 * w + (i & 1)) * GE::slot;
                    const bool arrive = w == 0 || u == nt;          // the last item of the stage
                    auto block_rows = [&](int blk, int& off) -> const uint8_t* {
                        const int pg = __shfl_sync(kAll, page, blk >> 1);
                        off = (p0 + 8 * blk) & (p.v.ps - 1);
                        return pg < 0 ? nullptr : unit_at(p.v, w, pg, h);
                    };
                    if (__all_sync(kAll, lane >= BN / 16 || page >= 0) && p0 + BN <= c.len) {
                        // boxes of min(page_size, BN) rows x 64 channels, one per lane of the first producer
                        const int rows = min(p.v.ps, BN), boxes = BN / rows * (D / 64);
                        const int k = lane / (D / 64), col = lane % (D / 64) * 64, at = p0 + k * rows;
                        const int pg = __shfl_sync(kAll, page, (k * rows >> 4) & (BN / 16 - 1));
                        if (pw == 0) {
                            if (lane == 0 && may) tc_expect(bar, GE::slot);
                            __syncwarp();
                            if (lane < boxes && may)
                                tma_load3(dst + tile_byte(BN, k * rows, col), w ? &v_map : &k_map, col, at & (p.v.ps - 1),
                                          pg * p.v.H + h, bar);
                        }
                    } else {
                        constexpr int per = D / 8;                  // 16-byte pieces of a row
                        for (int blk = pw; blk < BN / 8; blk += GE::prod) {
                            int off;
                            const uint8_t* u = block_rows(blk, off);
                            const int live = u ? c.len - p0 - 8 * blk : 0;         // rows of the block that hold positions
#pragma unroll
                            for (int e = 0; e < per / 4; ++e) {
                                const int x = e * 32 + lane, r = x / per, ch = x % per * 8;
                                uint4 y = make_uint4(0, 0, 0, 0);
                                if (r < live) y = *reinterpret_cast<const uint4*>(u + (off + r) * (2 * D) + 2 * ch);
                                st_shared16(dst + tile_byte(BN, 8 * blk + r, ch), y);
                            }
                        }
                    }
                    if (arrive) {
                        fence_async_smem();
                        mbar_arrive(bar);
                    }
                }
            } else {
                // Codes: a thread has the same pieces (16 channels of a row) of every tile; those of the next stage are on their
                // way while the products run. K and V have code of their own, with constant formats, and a tile's page
                // numbers are loaded a stage before they are looked at (item by item, with the number checked at once,
                // an item's loads took 1,500 cycles and the 6 prompts above 336 us, against 321 at that time).
                constexpr int per = D / 16, step = 32 * GE::prod / per, E = (BN + step - 1) / step;   // rows apart, of a thread
                // eight lanes take four pieces of two neighbouring rows: their stores hit all banks
                constexpr int nb = D / 64;
                const int row0 = pw * (32 / per) + ((lane >> 2) & 1) + 2 * (lane / 8 / nb), ch = 64 * (lane / 8 % nb) + 16 * (lane & 3);
                struct Codes {
                    uint4 c[E];
                    uint32_t d[E], held;                                // by bit: the row holds a position
                };
                const auto load = [&](auto fmt, int w, int tile, int units, Codes& x) {   // units: of the tile's 16-row blocks, by lane
                    constexpr bool E4 = decltype(fmt)::value == 3, Q8 = decltype(fmt)::value == 1 || E4;   // a byte a value
                    constexpr int RB = Q8 ? D : D / 2;
                    const uint8_t* base_w = w ? p.v.base[1] : p.v.base[0];
                    const uint32_t unit = (uint32_t)(w ? p.v.unit[1] : p.v.unit[0]);
                    const int p0 = kv.at(i0 + tile), live = c.len - p0;
                    // Loaded whether the row holds a position or not (of page 0 where there is no page): a load behind a branch
                    // goes to its place by a move, which waits for it.
                    x.held = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int r = min(row0 + e * step, BN - 1), un = __shfl_sync(kAll, units, r >> 4), row = (p0 + r) & (p.v.ps - 1);
                        if (un >= 0 && r < live) x.held |= 1u << e;
                        const uint8_t* a = base_w + (uint64_t)(uint32_t)max(un, 0) * unit;
                        if constexpr (E4) x.d[e] = *reinterpret_cast<const uint32_t*>(a + p.v.ps * RB + row / kTile * 4);
                        else x.d[e] = *reinterpret_cast<const uint16_t*>(a + (p.v.ps * RB + row * (D / 16) + ch / 32 * 2));
                        a += row * RB + (Q8 ? ch : ch / 2);
                        if constexpr (Q8) {
                            x.c[e] = *reinterpret_cast<const uint4*>(a);
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2*>(a);
                            x.c[e].x = y.x;
                            x.c[e].y = y.y;
                        }
                    }
                };
                const auto store = [&](auto fmt, uint32_t dst, const Codes& x) {
                    constexpr bool Q8 = decltype(fmt)::value == 1;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int r = row0 + e * step;
                        if (r >= BN) continue;
                        const bool held = (x.held >> e) & 1;
                        if constexpr (decltype(fmt)::value == 3) {
                            const float d = fminf(__uint_as_float(held ? x.d[e] : 0u), (float)(1 << kMaxPowerAttn)), mul = fmaxf(d, power_of(-13));
                            const bool small = mul > d;
                            const uint32_t dd = Two<__half>::pack(mul, mul), rest = Two<__half>::pack(d * 8192.f, d * 8192.f);
                            const uint4 y = held ? x.c[e] : make_uint4(0, 0, 0, 0);
                            st_shared16(dst + tile_byte(BN, r, ch), decode_e4(make_uint2(y.x, y.y), dd, rest, small));
                            st_shared16(dst + tile_byte(BN, r, ch + 8), decode_e4(make_uint2(y.z, y.w), dd, rest, small));
                            continue;
                        }
                        const uint32_t dd = held ? cut_scales<Q8>(x.d[e] | (x.d[e] << 16)) : 0u;
                        const uint4 y = x.c[e];
                        st_shared16(dst + tile_byte(BN, r, ch), Q8 ? decode_q8(make_uint2(y.x, y.y), dd) : decode_q4(y.x, dd));
                        st_shared16(dst + tile_byte(BN, r, ch + 8), Q8 ? decode_q8(make_uint2(y.z, y.w), dd) : decode_q4(y.y, dd));
                    }
                };
                const std::integral_constant<int, KF> kf;
                const std::integral_constant<int, VF> vf;
                // a tile's page numbers, one per lane: loaded a stage before they are looked at
                const auto table_of = [&](int tile) {
                    const int at = tile < nt ? kv.at(i0 + tile) + 16 * lane : c.len;
                    return lane < BN / 16 && at < c.len ? table[at >> p.v.ps_shift] : 0;
                };
                const auto units_of = [&](int page) {
                    if (page >= 0 && page < p.v.n_pages) return page * p.v.H + h;
                    raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
                    return -1;
                };
                const auto await_stage = [&](int u) { if (u >= 2) wait(empty + 8 * (u & 1), ((u >> 1) - 1) & 1); };
                const auto stage_full = [&](int u) {
                    fence_async_smem();
                    mbar_arrive(full + 8 * (u & 1));
                };
                // Stage u takes V of tile u - 1 and K of tile u; the next one's loads are issued behind it, without a branch (behind one
                // the loads' places are moved about, which waits for them), and the next page numbers are looked at before any of
                // them (a wait for these behind them would be one for those too).
                if (nt > 0) {
                    Codes kc, vc;
                    int units = units_of(table_of(0)), page = table_of(1);
                    load(kf, 0, 0, units, kc);
                    store(kf, ring, kc);
                    stage_full(0);
#pragma unroll 1
                    for (int u = 1; u < nt; ++u) {
                        const int old = units;
                        units = units_of(page);
                        page = table_of(u + 1);
                        load(vf, 1, u - 1, old, vc);
                        load(kf, 0, u, units, kc);
                        await_stage(u);
                        store(vf, ring + (2 + ((u - 1) & 1)) * GE::slot, vc);
                        store(kf, ring + (u & 1) * GE::slot, kc);
                        stage_full(u);
                    }
                    load(vf, 1, nt - 1, units, vc);
                    await_stage(nt);
                    store(vf, ring + (2 + ((nt - 1) & 1)) * GE::slot, vc);
                    stage_full(nt);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------------- the softmax
        if constexpr (GE::soft_regs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(GE::soft_regs));
        const int t = warp >> 2, in = threadIdx.x & 127, row = r0 + 128 * t + in;
        const bool alive = row < r1;
        const ScoreRule rule = score_rule(p);
        RowState rs;
        const int64_t at = (int64_t)(c.row0 + (alive ? row / G : 0)) * p.Hq + h * G + (alive ? row % G : 0);
        rs.pos = alive ? c.pos0 + row / G : -1;
        rs.lo = p.window > 0 && rs.pos >= p.window ? rs.pos - p.window + 1 : 0;
        rs.hi = min(rs.pos, c.len - 1);
        rs.pre = rs.pos >= 0 ? c.pre : 0;
        rs.slope = !RULE || !p.slopes || !alive ? 0.f : p.slopes[h * G + row % G] * kL2e;
        rs.f = rule.factor(1.f);
        float m = -INFINITY, l = 0.f;
        if (t < active) {
            // this row of Q to shared memory; bf16 queries over quantised pages become fp16, scaled by a power of two
            const uint32_t qs = base + t * GE::q_bytes;
            const TQ* src = alive ? (const TQ*)p.q + (int64_t)(c.row0 + row / G) * p.q_stride + ((int64_t)h * G + row % G) * D : nullptr;
            float up = 1.f;
            if constexpr (!std::is_same<T, TQ>::value) {
                float a = 0.f;
                if (src)
                    for (int d = 0; d < D; d += 8) {
                        float x[8];
                        unpack8<TQ>(*reinterpret_cast<const uint4*>(src + d), x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
                    }
                const int ex = (int)((__float_as_uint(a) >> 23) & 255) - 127;
                if (a > 0.f && ex < 128) {
                    // the largest magnitude to [2^14, 2^15): from -113 on; where scores are capped to [2^4, 2^5), for which the powers of
                    // their factor stay numbers (cap_weights32; what that costs is 2^-29 of the largest)
                    const int sh = min((RULE ? 4 : 14) - ex, 100);
                    up = __uint_as_float((uint32_t)(127 + sh) << 23);
                    rs.f = rule.factor(__uint_as_float((uint32_t)(127 - sh) << 23));
                }
            }
#pragma unroll 16
            for (int d = 0; d < D; d += 8) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (src) {
                    x = *reinterpret_cast<const uint4*>(src + d);
                    if constexpr (!std::is_same<T, TQ>::value) {
                        float y[8];
                        unpack8<TQ>(x, y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] *= up;
                        x = pack8<T>(y);
                    }
                }
                st_shared16(qs + tile_byte(128, in, d), x);
            }
            fence_async_smem();
            mbar_arrive(q_full);

            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), o_addr = lanes + GE::o_col(t);
            // the polynomial of cap_weights32, where f^7 and the cap leave its coefficients among the normal numbers
            const float f2 = rs.f * rs.f, a0 = rs.f * rule.cap_l2;
            const auto both = [](float c) { return pair(c, c); };
            const uint64_t cap[4] = {both(a0), both(-0.33332664f * f2 * a0), both(0.13299826f * f2 * f2 * a0), both(-0.049148493f * f2 * f2 * f2 * a0)};
            const bool cap_alone = RULE && __all_sync(kAll, rule.cap >= 1.f && rule.cap <= 1e6f && !rule.biased && rs.f >= 7.6e-6f && rs.f <= 16.f);
            int wide = 0;                                         // tiles for which scores beyond the polynomial are expected
            // positions of the row tile's first and last rows: what decides whether a KV tile is seen whole
            const int first = c.pos0 + (r0 + 128 * t) / G, last = c.pos0 + (min(r1, r0 + 128 * t + 128) - 1) / G;
            for (int i = 0; i < nt; ++i) {
                const int buf = NT == 2 ? t : i & 1, p0 = kv.at(i0 + i);
                const uint32_t s_addr = lanes + GE::s_col(buf);
                wait(s_full + 8 * buf, NT == 2 ? i & 1 : (i >> 1) & 1);
                tc_fence_after();
                const bool whole = p0 + BN <= c.pre ? first >= 0
                                                    : p0 + BN - 1 <= first && p0 + BN <= c.len &&
                                                          (p.window <= 0 || p0 >= last - p.window + 1);
                uint32_t sr[2][32], pr[BN / 64][32];
                float mx = -INFINITY, sum = 0.f;
                const auto hide = [&](int k, const auto& put) {           // put(e): position 32 k + e of the tile is not seen
                    const int hi = rs.hi - p0 - 32 * k, lo = rs.lo - p0 - 32 * k, pre = rs.pre - p0 - 32 * k;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((e <= hi && e >= lo) || e < pre)) put(e);
                };
                // scores that the visibility changes go back to S first (with options they are changed on their way to the weights)
                if (!RULE && !whole) {
                    tmem_ld32(s_addr, sr[0]);
#pragma unroll
                    for (int k = 0; k < BN / 32; ++k) {
                        uint32_t(&x)[32] = sr[k & 1];
                        tmem_wait_ld(x);
                        if (k + 1 < BN / 32) tmem_ld32(s_addr + 32 * (k + 1), sr[(k + 1) & 1]);
                        hide(k, [&](int e) { x[e] = 0xff800000u; });
                        tmem_st32(s_addr + 32 * k, x);
                    }
                    tmem_wait_st();
                }
                // With one row tile S runs ahead of the values: those of tile i - 1 are done before O is touched and before this
                // tile's weights go out (with two row tiles, S of tile i was issued after them).
                bool o_free = NT == 2 || i == 0;
                const auto await_o = [&]() {
                    if (o_free) return;
                    wait(o_done, (i - 1) & 1);
                    tc_fence_after();
                    o_free = true;
                };
                // The weights are formed with the maximum as it stands while the tile's own is found; only where that
                // is more than kLazy above (and for the first tile) the maximum moves and the weights are formed again.
                bool lean = RULE && cap_alone && whole && wide == 0;
                if (wide > 0) --wide;
                for (bool last_try = false;;) {
                    const float2 f2 = make_float2(rs.f, rs.f), mb = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(-m, -m);
                    uint64_t s2[4] = {};
                    float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, big = 0.f;
                    tmem_ld32(s_addr, sr[0]);
                    const auto each32 = [&](const auto& use) {            // use(scores, number) of every 32, the next on their way
#pragma unroll
                        for (int k = 0; k < BN / 32; ++k) {
                            uint32_t(&x)[32] = sr[k & 1];
                            tmem_wait_ld(x);
                            if (k + 1 < BN / 32) tmem_ld32(s_addr + 32 * (k + 1), sr[(k + 1) & 1]);
                            use(x, k);
                        }
                    };
                    if constexpr (!RULE)
                        each32([&](uint32_t (&x)[32], int k) { weights32<T>(x, pair(f2.x, f2.y), pair(mb.x, mb.y), &pr[k / 2][16 * (k & 1)], s2, y); });
                    else if (lean)
                        each32([&](uint32_t (&x)[32], int k) { cap_weights32<T>(x, cap, pair(mb.x, mb.y), &pr[k / 2][16 * (k & 1)], s2, y, big); });
                    else
                        each32([&](uint32_t (&x)[32], int k) {
                            rule_weights32<T>(x, rule, rs, p0 + 32 * k, mb.x, [&](float2 (&z)[16]) {
                                if (!whole) hide(k, [&](int e) { (e & 1 ? z[e / 2].y : z[e / 2].x) = -INFINITY; });
                            }, &pr[k / 2][16 * (k & 1)], s2, y);
                        });
                    {
                        const float2 a = unpair(s2[0]), b = unpair(s2[1]), c2 = unpair(s2[2]), d = unpair(s2[3]);
                        sum = ((a.x + a.y) + (b.x + b.y)) + ((c2.x + c2.y) + (d.x + d.y));
                    }
                    if (RULE && lean && __any_sync(kAll, !(big * rs.f < 0.35f))) {
                        lean = false;                             // some score is beyond the polynomial: this tile again, and the next
                        wide = 8;                                 // ones the other way
                        continue;
                    }
                    if (last_try) break;
                    mx = max3(fmaxf(y[0], y[1]), y[2], y[3]);
                    mx = (RULE ? mx - mb.x : mx * rs.f) - kUp;
                    const bool grow = mx > m + kLazy || (m == -INFINITY && mx > -INFINITY);
                    if (!__any_sync(kAll, grow)) break;
                    last_try = true;
                    const float a = grow ? ex2(m - mx) : 1.f;
                    if (grow) m = mx;
                    l *= a;
                    if (i > 0) {
                        await_o();
#pragma unroll 1
                        for (int d = 0; d < D; d += 32) {
                            tmem_ld32(o_addr + d, sr[0]);
                            tmem_wait_ld(sr[0]);
#pragma unroll
                            for (int e = 0; e < 32; ++e) sr[0][e] = __float_as_uint(__uint_as_float(sr[0][e]) * a);
                            tmem_st32(o_addr + d, sr[0]);
                        }
                    }
                }
                l += sum;
                await_o();
#pragma unroll
                for (int k = 0; k < BN / 64; ++k) tmem_st32(s_addr + 32 * k, pr[k]);
                tmem_wait_st();
                if (!whole) {
                    // does the V tile hold an infinity or NaN that some row must not see?
                    const uint32_t v_tile = ring + (2 + (i & 1)) * GE::slot;
                    wait(full + 8 * ((i + 1) & 1), ((i + 1) >> 1) & 1);
                    constexpr uint32_t top = BF ? 0x7f80u : 0x7c00u;
                    uint32_t bad = 0;
                    for (int e = in; e < BN * D / 8; e += 128) {
                        const uint4 y = ld_shared16(v_tile + 16 * e);
                        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) bad |= (w[q] & top) == top || ((w[q] >> 16) & top) == top;
                    }
                    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %0, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }\n"
                                 : "+r"(bad) : "r"(1 + t) : "memory");
                    if (bad) add_seen<D, BN, T>(v_tile, o_addr, s_addr, rs, p0, i == 0);
                    if (in == 0) s_skip[buf] = bad ? 1 : 0;
                } else if (in == 0) {
                    s_skip[buf] = 0;
                }
                tc_fence_before();
                mbar_arrive(p_full + 8 * buf);
            }
            if (nt > 0) {
                wait(o_done + 8 * t, NT == 2 ? 0 : (nt - 1) & 1);   // two row tiles: reported once, at the end
                tc_fence_after();
            }
            const float inv = inverse_sum(l);
            if (splits == 1) {
                TQ* out = (TQ*)p.out + at * D;
                if (p.lse && alive) p.lse[at] = log_sum(m, l);
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32] = {};
                    if (nt > 0) {
                        tmem_ld32(o_addr + d, o);
                        tmem_wait_ld(o);
                    }
                    if (!alive) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) y[q] = nt > 0 ? __uint_as_float(o[e + q]) * inv : 0.f;
                        *reinterpret_cast<uint4*>(out + d + e) = pack8<TQ>(y);
                    }
                }
            } else {
                const int64_t part = (int64_t)split * p.n_rows * p.Hq + at, all = (int64_t)splits * p.n_rows * p.Hq;
                float* o_part = p.ws + split_out_at(all) + part * D;
                if (alive) *reinterpret_cast<float2*>(p.ws + 2 * part) = make_float2(m, l);
#pragma unroll 1
                for (int d = 0; d < D && nt > 0; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_addr + d, o);
                    tmem_wait_ld(o);
                    if (!alive) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(o_part + d + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // A wait ran out: copies and products may still be on their way into this block's memory. They take microseconds; they
    // are given a millisecond before it is handed back.
    if (*(volatile int*)&s_abort) {
        const uint64_t t0 = gtime();
        for (int n = 0; n < 1 << 20 && gtime() - t0 < 1000000; ++n) {}
        __syncthreads();
    }
    if (warp == GE::mma_warp) tmem_free512(tmem);
}

// Joins the splits' partials: D / 8 threads a row, all rows of a chunk.
constexpr int kJT = 128;
template <int D, typename TQ> __global__ void __launch_bounds__(kJT) prefill_join_kernel(PagedAttnParams p, int splits) {
    grid_dep_wait();
    constexpr int L = D / 8;
    const int b = blockIdx.z, h = blockIdx.y, G = p.G;
    const Chunk c = chunk_of(p, b, false);
    const int row = blockIdx.x * (kJT / L) + threadIdx.x / L, ch = threadIdx.x % L * 8;
    if (row >= c.n * G) return;
    const int64_t at = (int64_t)(c.row0 + row / G) * p.Hq + h * G + row % G, n = (int64_t)p.n_rows * p.Hq;
    float m = -INFINITY;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, p.ws[2 * (s * n + at)]);
    float l = 0.f, o[8] = {};
    for (int s = 0; s < splits; ++s) {
        const float2 ml = *reinterpret_cast<const float2*>(p.ws + 2 * (s * n + at));
        if (ml.y == 0.f) continue;                       // nothing seen: no output was written (NaN scores: the sum is NaN)
        const float a = ex2(ml.x - m);
        l += ml.y * a;
        const float4* f = reinterpret_cast<const float4*>(p.ws + split_out_at(splits * n) + (s * n + at) * D + ch);
        const float4 x = f[0], y = f[1];
        const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(z[e], a, o[e]);
    }
    const float inv = inverse_sum(l);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    *reinterpret_cast<uint4*>((TQ*)p.out + at * D + ch) = pack8<TQ>(o);
    if (p.lse && ch == 0) p.lse[at] = log_sum(m, l);
}

template <int D, int KF, int VF, typename T, typename TQ>
int prefill_run(const PagedAttnParams& p, const CUtensorMap* maps, int sm_count, cudaStream_t s) {
    using GE = Geo<D, codes_of(KF)>;
    const auto k = p.softcap > 0.f || p.slopes ? prefill_kernel<D, KF, VF, T, TQ, true> : prefill_kernel<D, KF, VF, T, TQ, false>;
    int res = 0;
    if (const int e = resident_ctas((const void*)k, GE::threads, GE::smem, &res)) return e;
    const int64_t chunk = (int64_t)p.max_q * p.G;
    int splits = prefill_splits((int64_t)p.n_rows * p.G, p.n_seq, p.v.H, GE::rows, sm_count);
    dim3 grid(p.v.H, (unsigned)((chunk + GE::rows - 1) / GE::rows), (unsigned)(p.n_seq * splits));
    if constexpr (KF == kRows) {
        splits = min(splits, prompt_splits(p.max_q, D));
        grid.y = (unsigned)prompt_tiles(p.n_rows, p.n_seq, p.G, D);
        grid.z = splits;
    }
    cudaError_t e = launch_k(k, grid, dim3(GE::threads), GE::smem, s, true, p, maps[0], maps[1], splits);
    if (e == cudaSuccess && splits > 1) {
        constexpr int R = kJT / (D / 8);
        e = launch_k(prefill_join_kernel<D, TQ>, dim3((unsigned)((chunk + R - 1) / R), p.v.H, p.n_seq), dim3(kJT), 0, s, true, p, splits);
    }
    return (int)e;
}

template <int D> int prefill_d(const PagedAttnParams& p, const CUtensorMap* m, int n, cudaStream_t s) {
    const int kf = p.v.fmt[0], vf = p.v.fmt[1];
    if (kf == KVQ_F16) return prefill_run<D, 0, 0, __half, __half>(p, m, n, s);
    if (kf == KVQ_BF16) return prefill_run<D, 0, 0, __nv_bfloat16, __nv_bfloat16>(p, m, n, s);
    if (kf == KVQ_PAGED_E4M3)
        return p.dtype == KVQ_F16 ? prefill_run<D, 3, 3, __half, __half>(p, m, n, s) : prefill_run<D, 3, 3, __half, __nv_bfloat16>(p, m, n, s);
    if (p.dtype == KVQ_F16) {
        if (kf == KVQ_Q4_0) return prefill_run<D, 2, 2, __half, __half>(p, m, n, s);
        if (vf == KVQ_Q4_0) return prefill_run<D, 1, 2, __half, __half>(p, m, n, s);
        return prefill_run<D, 1, 1, __half, __half>(p, m, n, s);
    }
    if (kf == KVQ_Q4_0) return prefill_run<D, 2, 2, __half, __nv_bfloat16>(p, m, n, s);
    if (vf == KVQ_Q4_0) return prefill_run<D, 1, 2, __half, __nv_bfloat16>(p, m, n, s);
    return prefill_run<D, 1, 1, __half, __nv_bfloat16>(p, m, n, s);
}

}  // namespace

// One head dimension per compilation of this file (KVQ_D), so that they build side by side.
#define KVQ_NAME2(n, d) launch_##n##_##d
#define KVQ_NAME(n, d) KVQ_NAME2(n, d)
int KVQ_NAME(paged_prefill, KVQ_D)(const PagedAttnParams& p, const void* maps, int sms, void* stream) {
    return prefill_d<KVQ_D>(p, (const CUtensorMap*)maps, sms, (cudaStream_t)stream);
}
int KVQ_NAME(prompt_attn, KVQ_D)(const PagedAttnParams& p, const void* maps, int sms, void* stream) {
    const CUtensorMap* m = (const CUtensorMap*)maps;
    return p.dtype == KVQ_F16 ? prefill_run<KVQ_D, kRows, kRows, __half, __half>(p, m, sms, (cudaStream_t)stream)
                              : prefill_run<KVQ_D, kRows, kRows, __nv_bfloat16, __nv_bfloat16>(p, m, sms, (cudaStream_t)stream);
}

}  // namespace kvq
