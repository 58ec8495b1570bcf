// Pages shared, counted, copied, freed and moved: the page tables of a paged cache kept on the device.
//
// A page's count (refs) says how many table rows hold it. Decisions are taken by one block (prefix sums over the pages and rows,
// counts and minima whose order does not matter: the same call on the same tables gives the same pages), the bytes are
// moved by all of them: pages are copied in 16 KB pieces, a page's K or V of one layer being one run of bytes. 673 of 3,000 pages x 8
// layers x 64 KB move at 94% of the measured HBM rate (111 us; with the tables' part 126 us); the decisions take 3 to 10 us, one
// step after the other.
#include "device_common.cuh"
#include "paged_common.cuh"

namespace kvq {
namespace {

constexpr int kPT = 1024;            // threads of the deciding block

__device__ __forceinline__ int pages_of(int64_t len, int shift) { return (int)((len + (1 << shift) - 1) >> shift); }

// Exclusive prefix sum over the block's threads, in their order, and the total.
template <typename N> __device__ __forceinline__ N block_sums(N x, N* total) {
    __shared__ N s_sum[kPT / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    N sum = x;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const N y = __shfl_up_sync(kAll, sum, s);
        if (lane >= s) sum += y;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    const N w = s_sum[lane];
    N before = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const N y = __shfl_up_sync(kAll, before, s);
        if (lane >= s) before += y;
    }
    *total = __shfl_sync(kAll, before, 31);
    before = __shfl_sync(kAll, before - w, warp);
    __syncthreads();
    return before + sum - x;
}

// Four counts from page p on (pages behind the last one count as `none`).
__device__ __forceinline__ int4 refs_at(const int32_t* refs, int p, int n, int none) {
    if (p + 3 < n && ((uintptr_t)refs & 15) == 0) return *reinterpret_cast<const int4*>(refs + p);
    return make_int4(p < n ? refs[p] : none, p + 1 < n ? refs[p + 1] : none, p + 2 < n ? refs[p + 2] : none, p + 3 < n ? refs[p + 3] : none);
}

// ---------------------------------------------------------------------------- copies
// grid: any number of blocks; the pieces of all copies in turn. Pairs come as two arrays (a negative number skips one), or as the
// list that a deciding block left. With `remap` the rows' entries are renumbered too.
constexpr int kCT = 256, kCopyU = 4, kPiece = kCT * 16 * kCopyU;
__global__ void __launch_bounds__(kCT) copy_pages_kernel(PagesParams p, const int32_t* src, const int32_t* dst, const int32_t* count,
                                                         int n, const int32_t* remap) {
    grid_dep_wait();
    const PagedView& v = p.v;
    if (remap) {
        for (int b = blockIdx.x; b < p.rows; b += gridDim.x) {
            const int64_t cap = (int64_t)p.max_pages << v.ps_shift, len = p.lens[b];
            const int held = pages_of(len < 0 ? 0 : (len > cap ? cap : len), v.ps_shift);
            int32_t* row = p.table + b * p.table_stride;
            for (int e = threadIdx.x; e < held; e += kCT) {
                const int page = row[e], to = page >= 0 && page < v.n_pages ? remap[page] : -1;
                if (to < 0) raise_status(v.status, KVQ_PAGED_BAD_INDEX);
                else row[e] = to;
            }
        }
    }
    const int64_t k_bytes = v.H * v.unit[0], v_bytes = v.H * v.unit[1];
    const int k_parts = (int)((k_bytes + kPiece - 1) / kPiece), parts = k_parts + (int)((v_bytes + kPiece - 1) / kPiece);
    const int64_t per = (int64_t)p.n_layers * parts, all = (count ? *count : n) * per;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int c = (int)(i / per), in = (int)(i - c * per), layer = in / parts, k = in - layer * parts;
        const bool w = k >= k_parts;
        const int part = k - (w ? k_parts : 0);
        const int64_t bytes = w ? v_bytes : k_bytes;
        const int from = src[c], to = dst[c];
        if (from < 0 || to < 0 || from == to) continue;
        if (from >= v.n_pages || to >= v.n_pages) {
            if (in == 0 && threadIdx.x == 0) raise_status(v.status, KVQ_PAGED_BAD_INDEX);
            continue;
        }
        uint8_t* base = (w ? v.base[1] : v.base[0]) + layer * p.layer_bytes;
        const uint8_t* a = base + from * bytes;
        uint8_t* b = base + to * bytes;
        const int64_t at = (int64_t)part * kPiece + threadIdx.x * 16;
        uint4 x[kCopyU];
#pragma unroll
        for (int u = 0; u < kCopyU; ++u)
            if (at + u * (kCT * 16) < bytes) x[u] = *reinterpret_cast<const uint4*>(a + at + u * (kCT * 16));
#pragma unroll
        for (int u = 0; u < kCopyU; ++u)
            if (at + u * (kCT * 16) < bytes) *reinterpret_cast<uint4*>(b + at + u * (kCT * 16)) = x[u];
    }
}

// ---------------------------------------------------------------------------- fork
// A block per child: its row becomes its parent's, whose pages are held once more. A child that holds positions, comes twice or
// is a parent in the same call is left out (nothing that another block reads is written).
constexpr int kFT = 128;
__global__ void __launch_bounds__(kFT) fork_kernel(PagesParams p, int n, const int32_t* parents, const int32_t* children) {
    grid_dep_wait();
    const int i = blockIdx.x, c = children[i], from = parents[i];
    if (c < 0) return;
    bool bad = c >= p.rows || from < 0 || from >= p.rows;
    for (int j = threadIdx.x; j < n; j += kFT) {
        const int x = children[j];
        bad |= (x == c && j < i) || x == from;
    }
    int len = 0;
    if (!bad) {
        len = p.lens[from];
        bad = p.lens[c] != 0 || len < 0 || len > ((int64_t)p.max_pages << p.v.ps_shift);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
        return;
    }
    const int held = pages_of(len, p.v.ps_shift);
    const int32_t* a = p.table + from * p.table_stride;
    int32_t* b = p.table + c * p.table_stride;
    for (int e = threadIdx.x; e < held; e += kFT) {
        const int page = a[e];
        b[e] = page;
        if (page >= 0 && page < p.v.n_pages) atomicAdd(p.refs + page, 1);
        else raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
    }
    if (threadIdx.x == 0) p.lens[c] = len;
}

// ---------------------------------------------------------------------------- free
// A block per entry of `rows`: the row is cut to keep positions, and the pages behind them are given back. The old length is taken
// and the new one set by one atomic minimum and an entry by one exchange, so that a row that comes twice gives no page back twice.
__global__ void __launch_bounds__(kFT) free_kernel(PagesParams p, const int32_t* rows, const int32_t* keep) {
    __shared__ int s_old;
    grid_dep_wait();
    const int i = blockIdx.x, row = rows[i], to = keep ? keep[i] : 0;
    if (row < 0) return;
    if (row >= p.rows || to < 0) {
        if (threadIdx.x == 0) raise_status(p.v.status, row >= p.rows ? KVQ_PAGED_BAD_INDEX : KVQ_PAGED_BAD_LENGTH);
        return;
    }
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    if (threadIdx.x == 0) {
        const int old = atomicMin(p.lens + row, to);
        if (old < 0 || old > cap) raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
        s_old = old > cap ? (int)cap : old;
    }
    __syncthreads();
    if (s_old <= to) return;
    const int last = pages_of(s_old, p.v.ps_shift);
    for (int e = pages_of(to, p.v.ps_shift) + threadIdx.x; e < last; e += kFT) {
        const int page = atomicExch(p.table + row * p.table_stride + e, -1);
        if (page < 0 || page >= p.v.n_pages) {
            raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
        } else if (atomicSub(p.refs + page, 1) <= 0) {
            atomicAdd(p.refs + page, 1);                          // nobody held it: the count stays
            raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
        }
    }
}

// ---------------------------------------------------------------------------- extend
// What a row needs to go on by add[b] positions.
struct Growth {
    int have, want, last;      // pages it has and will have; the page that it goes on in (-1: none is part-filled)
    bool on;
};
__device__ __forceinline__ Growth growth(const PagesParams& p, const int32_t* add, int b, bool report) {
    Growth g = {0, 0, -1, false};
    const int64_t cap = (int64_t)p.max_pages << p.v.ps_shift;
    const int len = p.lens[b], more = add[b];
    if (more == 0) return g;
    if (more < 0 || len < 0 || (int64_t)len + more > cap) {
        if (report) raise_status(p.v.status, KVQ_PAGED_BAD_LENGTH);
        return g;
    }
    g.have = pages_of(len, p.v.ps_shift);
    g.want = pages_of((int64_t)len + more, p.v.ps_shift);
    if (len & (p.v.ps - 1)) {
        g.last = p.table[b * p.table_stride + g.have - 1];
        if (g.last < 0 || g.last >= p.v.n_pages) {
            if (report) raise_status(p.v.status, KVQ_PAGED_BAD_INDEX);
            return g;
        }
    }
    g.on = true;
    return g;
}

// One block. Workspace: [0] copies; from 16 on their sources and destinations [n_pages] each, the free pages in order
// [n_pages], and by page how many rows go on in it and the lowest of them [n_pages] each.
__global__ void __launch_bounds__(kPT, 1) extend_kernel(PagesParams p, const int32_t* add, int32_t* ws) {
    grid_dep_wait();
    const int n = p.v.n_pages;
    int32_t *src = ws + 16, *dst = src + n, *spare = dst + n, *going = spare + n, *lowest = going + n;
    for (int b = threadIdx.x; b < p.rows; b += kPT) {
        const Growth g = growth(p, add, b, true);
        if (g.on && g.last >= 0) {
            going[g.last] = 0;
            lowest[g.last] = 0x7fffffff;
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.rows; b += kPT) {
        const Growth g = growth(p, add, b, false);
        if (g.on && g.last >= 0) {
            atomicAdd(going + g.last, 1);
            atomicMin(lowest + g.last, b);
        }
    }
    __syncthreads();
    // a page stays with the lowest of its rows if all that hold it go on in it; all others go on in a copy
    for (int b = threadIdx.x; b < p.rows; b += kPT) {
        const Growth g = growth(p, add, b, false);
        if (g.on && g.last >= 0 && lowest[g.last] == b && going[g.last] < p.refs[g.last]) lowest[g.last] = -1;
    }
    __syncthreads();
    int64_t need = 0;
    for (int b = threadIdx.x; b < p.rows; b += kPT) {
        const Growth g = growth(p, add, b, false);
        if (g.on) need += g.want - g.have + (g.last >= 0 && lowest[g.last] != b);
    }
    int64_t total;
    block_sums(need, &total);
    if (threadIdx.x == 0) ws[0] = 0;
    if (total == 0) {
        for (int b = threadIdx.x; b < p.rows; b += kPT)
            if (growth(p, add, b, false).on) p.lens[b] += add[b];
        return;
    }
    int found = 0;                                                // free pages, lowest first, until there are enough
    for (int at = 0; at < n && found < total; at += 4 * kPT) {
        const int q = at + 4 * threadIdx.x;
        const int4 r = refs_at(p.refs, q, n, 1);
        int sum;
        int k = found + block_sums((r.x <= 0) + (r.y <= 0) + (r.z <= 0) + (r.w <= 0), &sum);
        if (r.x <= 0) spare[k++] = q;
        if (r.y <= 0) spare[k++] = q + 1;
        if (r.z <= 0) spare[k++] = q + 2;
        if (r.w <= 0) spare[k++] = q + 3;
        found += sum;
    }
    if (found < total) {                                          // too few: nothing changes
        if (threadIdx.x == 0) raise_status(p.v.status, KVQ_PAGED_NO_PAGES);
        return;
    }
    __syncthreads();
    int64_t before = 0;
    int copies = 0;
    __shared__ int s_first[kPT], s_from[kPT], s_n[kPT];
    for (int b0 = 0; b0 < p.rows; b0 += kPT) {
        const int b = b0 + threadIdx.x;
        Growth g = {0, 0, -1, false};
        if (b < p.rows) g = growth(p, add, b, false);
        const int copy = g.on && g.last >= 0 && lowest[g.last] != b, k = g.on ? g.want - g.have : 0;
        int64_t sum;
        int made;
        const int64_t first = before + block_sums((int64_t)(copy + k), &sum);
        const int at = copies + block_sums(copy, &made);
        before += sum;
        copies += made;
        if (copy) {
            const int page = spare[first];
            src[at] = g.last;
            dst[at] = page;
            p.table[b * p.table_stride + g.have - 1] = page;
            p.refs[page] = 1;
            atomicSub(p.refs + g.last, 1);
        }
        s_first[threadIdx.x] = (int)first + copy;
        s_from[threadIdx.x] = g.have;
        s_n[threadIdx.x] = k;
        if (g.on) p.lens[b] += add[b];
        __syncthreads();
        // new pages, a warp a row
        for (int r = threadIdx.x >> 5; r < kPT && b0 + r < p.rows; r += kPT / 32)
            for (int e = threadIdx.x & 31; e < s_n[r]; e += 32) {
                const int page = spare[s_first[r] + e];
                p.table[(b0 + r) * p.table_stride + s_from[r] + e] = page;
                p.refs[page] = 1;
            }
        __syncthreads();
    }
    if (threadIdx.x == 0) ws[0] = copies;
}

// ---------------------------------------------------------------------------- compact
// One block: of the L pages in use those behind page L - 1 move to the free ones before it, both in order. Workspace: [0] moves;
// from 16 on their sources and destinations [n_pages] each.
__global__ void __launch_bounds__(kPT, 1) compact_kernel(PagesParams p, int32_t* remap, int32_t* ws) {
    grid_dep_wait();
    const int n = p.v.n_pages;
    int32_t *src = ws + 16, *dst = src + n;
    int mine = 0, used;
    for (int q = 4 * threadIdx.x; q < n; q += 4 * kPT) {
        const int4 r = refs_at(p.refs, q, n, 0);
        mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
    block_sums(mine, &used);
    int moves = 0, holes = 0;
    for (int at = 0; at < n; at += 4 * kPT) {
        const int q = at + 4 * threadIdx.x;
        const int4 r4 = refs_at(p.refs, q, n, 0);
        const int r[4] = {r4.x, r4.y, r4.z, r4.w};
        int count = 0, sum;                                       // movers in the high half, free pages before L in the low one
#pragma unroll
        for (int i = 0; i < 4; ++i) count += q + i < used ? (r[i] <= 0) : (r[i] > 0) << 16;
        const int k = block_sums(count, &sum);
        int m = moves + (k >> 16), h = holes + (k & 0xffff);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (q + i >= n) break;
            const bool in_use = r[i] > 0;
            remap[q + i] = in_use ? q + i : -1;
            if (q + i < used) {
                if (!in_use) dst[h++] = q + i;
            } else if (in_use) {
                src[m++] = q + i;
            }
        }
        moves += sum >> 16;
        holes += sum & 0xffff;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += kPT) {
        const int a = src[i], b = dst[i];
        remap[a] = b;
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
    if (threadIdx.x == 0) ws[0] = moves;
}

int run_copies(const PagesParams& p, const int32_t* src, const int32_t* dst, const int32_t* count, int n, const int32_t* remap, cudaStream_t s) {
    int res = 0;
    if (const int e = resident_ctas((const void*)copy_pages_kernel, kCT, 0, &res)) return e;
    return (int)launch_k(copy_pages_kernel, dim3((unsigned)(p.sm_count * res)), dim3(kCT), 0, s, true, p, src, dst, count, n, remap);
}

}  // namespace

int launch_pages_copy(const PagesParams& p, int n, const int32_t* src, const int32_t* dst, void* stream) {
    return run_copies(p, src, dst, nullptr, n, nullptr, (cudaStream_t)stream);
}

int launch_pages_fork(const PagesParams& p, int n, const int32_t* parents, const int32_t* children, void* stream) {
    return (int)launch_k(fork_kernel, dim3((unsigned)n), dim3(kFT), 0, (cudaStream_t)stream, true, p, n, parents, children);
}

int launch_pages_free(const PagesParams& p, int n, const int32_t* rows, const int32_t* keep, void* stream) {
    return (int)launch_k(free_kernel, dim3((unsigned)n), dim3(kFT), 0, (cudaStream_t)stream, true, p, rows, keep);
}

int launch_pages_extend(const PagesParams& p, const int32_t* add, int32_t* ws, void* stream) {
    const cudaError_t e = launch_k(extend_kernel, dim3(1), dim3(kPT), 0, (cudaStream_t)stream, true, p, add, ws);
    return e != cudaSuccess ? (int)e : run_copies(p, ws + 16, ws + 16 + p.v.n_pages, ws, 0, nullptr, (cudaStream_t)stream);
}

int launch_pages_compact(const PagesParams& p, int32_t* remap, int32_t* ws, void* stream) {
    const cudaError_t e = launch_k(compact_kernel, dim3(1), dim3(kPT), 0, (cudaStream_t)stream, true, p, remap, ws);
    return e != cudaSuccess ? (int)e : run_copies(p, ws + 16, ws + 16 + p.v.n_pages, ws, 0, remap, (cudaStream_t)stream);
}

}  // namespace kvq
