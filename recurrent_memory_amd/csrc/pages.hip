// Pages of a pool of recurrent states: copies, forks and clears, and the moves
// that bring the live pages to the front.
//
// Both are copies, 8 bytes of HBM traffic per float moved, with a plan made from
// a list of page numbers in device memory.  Every workgroup makes the plan for
// itself from a bitmap of the pool's pages in LDS (one bit a page, 8 KiB at most),
// so that a call is one launch without workspace; a workgroup then takes 16 KiB
// pieces of pages in turn, four 16-byte loads a lane in flight (32 KiB pieces and 2048
// workgroups took 149 us for 250 MiB copied, this 104 us: 5.0 TB/s).  The plan is what
// bounds long lists of small pages: each workgroup reads the whole list (a copy within one
// pool twice) and marks its bitmap, 32768 copies of 64 floats 53 us for about 3 us of page
// traffic, 65536 slots compacted 33 us.
#include "common.h"
#include "kernels.h"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxGrid = 1024;             // workgroups of the copy loops: 4 per CU
constexpr int kWords = 65536 / 32;         // bitmap words of the largest pool

template <int V> struct Vec { typedef float T __attribute__((ext_vector_type(V))); };
template <> struct Vec<1> { typedef float T; };

// Piece c of a page of n vectors, by the whole workgroup; src == nullptr clears.
// Non-temporal stores leave the caches to the pages that are read (192 forks of 48 pages
// of 1 MiB: 59 us plain, 39 us so; loads non-temporal too: 64 us).
template <int V>
__device__ __forceinline__ void copy_piece(float* dst, const float* src, int64_t n, int64_t c) {
    typedef typename Vec<V>::T T;
    const int64_t i0 = c * (kThreads * kUnroll) + threadIdx.x;
    T v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        v[u] = T(0.f);
        if (src != nullptr && i < n) v[u] = reinterpret_cast<const T*>(src)[i];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i < n) __builtin_nontemporal_store(v[u], reinterpret_cast<T*>(dst) + i);
    }
}

// Pages of up to 128 vectors, `count` of them, as one run of vectors, so that every lane
// has work.  Calls of 16384 copies, us, a workgroup a page and so:  16 vectors 48 and 27,
// 64: 47 and 36, 128: 51 and 39, 256: 53 and 48, 512: 68 and 67; 32768 slots compacted, half of them
// live:  16: 35 and 21, 64: 35 and 22, 128: 35 and 25, 256: 37 and 38, 384: 40 and 45,
// 512: 41 and 54.  Short lists (48 entries) are the same up to 384 vectors; a page of 512 fills a
// workgroup, which then looks its numbers up once: 48 copies 4.4 us, 5.1 us so.
// find(k, &dst, &src) gives the k-th copy's pages (src == nullptr clears), or false if
// there is nothing to do.
constexpr int kSmallPage = kThreads / 2;
template <int V, typename Find>
__device__ __forceinline__ void copy_small_pages(int64_t count, uint32_t n, Find find) {
    typedef typename Vec<V>::T T;
    const uint32_t total = static_cast<uint32_t>(count) * n;      // at most 2^16 pages of 2^7 vectors
    for (uint32_t i0 = blockIdx.x * (kThreads * kUnroll) + threadIdx.x; i0 < total;
         i0 += gridDim.x * (kThreads * kUnroll)) {
        T v[kUnroll];
        T* to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t i = i0 + u * kThreads;
            float* dst;
            const float* src;
            v[u] = T(0.f);
            to[u] = nullptr;
            if (i < total && find(static_cast<int>(i / n), &dst, &src)) {
                to[u] = reinterpret_cast<T*>(dst) + i % n;
                if (src != nullptr) v[u] = reinterpret_cast<const T*>(src)[i % n];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] != nullptr) __builtin_nontemporal_store(v[u], to[u]);
    }
}

// Entries i, i + kThreads, ... of a list, all in flight at once; -1 beyond its end (for a
// destination or a slot: nothing to do).
constexpr int kList = 8;
__device__ __forceinline__ void load_list(const int* list, int i, int n, int* out) {
#pragma unroll
    for (int u = 0; u < kList; ++u) out[u] = i + u * kThreads < n ? list[i + u * kThreads] : -1;
}

// Entry i of a copy list does something: its numbers lie inside their pools, and
// it does not copy a page onto itself.
__device__ __forceinline__ bool acts(const PagesCopyArgs& p, int s, int d, bool same) {
    return d >= 0 && d < p.n_pages && s >= -1 && s < p.src_pages && !(same && s == d);
}

// The entries act in order.  If no destination is named twice or is also a
// source, the order does not matter and the pieces of all entries are copied at
// once, by position (piece 0 of every entry, then piece 1, ...), so that the
// forks of one page read it from cache.  Otherwise a lane owns a column of the
// pages and applies the whole list to it in order, one load and store after another:
// right for any list, and slow (4000 copies of 8 KiB pages 18 us, with one page named twice
// 1.95 ms; of 256-byte pages 10 us and 1.26 ms; 200 pages of 1 MiB copied 85 us, moved as
// copies each followed by a clear of its source 265 us).
template <int V>
__global__ __launch_bounds__(kThreads) void pages_copy_kernel(PagesCopyArgs p) {
    __shared__ uint32_t written[kWords];
    const bool same = p.src_pool == p.pool;
    for (int w = threadIdx.x; w < (p.n_pages + 31) / 32; w += kThreads) written[w] = 0;
    __syncthreads();
    bool clash = false;
    for (int i = threadIdx.x; i < p.n; i += kThreads * kList) {
        int s[kList], d[kList];
        load_list(p.src, i, p.n, s);
        load_list(p.dst, i, p.n, d);
#pragma unroll
        for (int u = 0; u < kList; ++u) {
            if (acts(p, s[u], d[u], same)) {
                const uint32_t bit = 1u << (d[u] & 31);
                clash |= (atomicOr(&written[d[u] >> 5], bit) & bit) != 0;
            }
        }
    }
    __syncthreads();
    if (same) {
        for (int i = threadIdx.x; i < p.n; i += kThreads * kList) {
            int s[kList], d[kList];
            load_list(p.src, i, p.n, s);
            load_list(p.dst, i, p.n, d);
#pragma unroll
            for (int u = 0; u < kList; ++u)
                if (acts(p, s[u], d[u], same) && s[u] >= 0) clash |= (written[s[u] >> 5] >> (s[u] & 31)) & 1u;
        }
    }
    const int64_t nv = p.page / V;
    if (!__syncthreads_or(clash)) {
        if (nv <= kSmallPage) {
            copy_small_pages<V>(p.n, static_cast<uint32_t>(nv), [&](int i, float** to, const float** from) {
                const int s = p.src[i], d = p.dst[i];
                *to = p.pool + d * p.page;
                *from = s < 0 ? nullptr : p.src_pool + s * p.page;
                return acts(p, s, d, same);
            });
            return;
        }
        const int64_t pieces = (nv + kThreads * kUnroll - 1) / (kThreads * kUnroll);
        for (int64_t u = blockIdx.x; u < pieces * p.n; u += gridDim.x) {
            const int i = static_cast<int>(u % p.n);
            const int s = p.src[i], d = p.dst[i];
            if (!acts(p, s, d, same)) continue;
            copy_piece<V>(p.pool + d * p.page, s < 0 ? nullptr : p.src_pool + s * p.page, nv, u / p.n);
        }
        return;
    }
    typedef typename Vec<V>::T T;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; c < nv; c += step) {
        for (int i = 0; i < p.n; ++i) {
            const int s = p.src[i], d = p.dst[i];
            if (!acts(p, s, d, same)) continue;
            T v = T(0.f);
            if (s >= 0) v = reinterpret_cast<const T*>(p.src_pool + s * p.page)[c];
            reinterpret_cast<T*>(p.pool + d * p.page)[c] = v;
        }
    }
}

// Live pages as a bitmap with the number of live pages before each word: the rank
// of a page and the page of a rank, for live and for free pages.
struct LiveMap {
    uint32_t bits[kWords + 1];
    int before[kWords + 1];

    __device__ int rank(int page) const {
        return before[page >> 5] + __popc(bits[page >> 5] & ((1u << (page & 31)) - 1u));
    }
    // The r-th (from 0) live (or, with FREE, free) page among `words` words.
    template <bool FREE>
    __device__ int select(int r, int words) const {
        int lo = 0, hi = words - 1;     // the last word with at most r such pages before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((FREE ? 32 * mid - before[mid] : before[mid]) <= r) lo = mid;
            else hi = mid - 1;
        }
        int k = r - (FREE ? 32 * lo - before[lo] : before[lo]);
        uint32_t w = FREE ? ~bits[lo] : bits[lo];
        int at = 0;
#pragma unroll
        for (int half = 16; half >= 1; half >>= 1) {
            const int c = __popc(w & ((1u << half) - 1u));
            if (k >= c) { k -= c; at += half; w >>= half; }
        }
        return 32 * lo + at;
    }
};

// With L live pages, the live pages at or above L (M of them) go to the free pages
// below L, k-th lowest to k-th lowest: sources and destinations are disjoint, so
// the moves need no order.
template <int V>
__global__ __launch_bounds__(kThreads) void pages_compact_kernel(PagesCompactArgs p) {
    __shared__ LiveMap map;
    __shared__ int wave_sum[kThreads / 64];
    const int words = (p.n_pages + 31) / 32;
    for (int w = threadIdx.x; w <= words; w += kThreads) map.bits[w] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kThreads * kList) {
        int s[kList];
        load_list(p.slots, i, p.n, s);
#pragma unroll
        for (int u = 0; u < kList; ++u)
            if (s[u] >= 0 && s[u] < p.n_pages) atomicOr(&map.bits[s[u] >> 5], 1u << (s[u] & 31));
    }
    __syncthreads();
    // live pages before each word: each thread sums a run of words, runs are scanned
    const int run = (words + kThreads - 1) / kThreads;
    const int w0 = min(static_cast<int>(threadIdx.x) * run, words), w1 = min(w0 + run, words);
    int sum = 0;
    for (int w = w0; w < w1; ++w) sum += __popc(map.bits[w]);
    int scan = sum;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(scan, d);
        if (lane >= d) scan += up;
    }
    if (lane == 63) wave_sum[threadIdx.x >> 6] = scan;
    __syncthreads();
    int base = scan - sum, L = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < static_cast<int>(threadIdx.x >> 6)) base += wave_sum[w];
        L += wave_sum[w];
    }
    for (int w = w0; w < w1; ++w) {
        map.before[w] = base;
        base += __popc(map.bits[w]);
    }
    if (threadIdx.x == 0) map.before[words] = L;
    __syncthreads();

    const int front = map.rank(L);   // live pages already below L
    const int M = L - front;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.n; i += gridDim.x * kThreads) {
        const int s = p.slots[i];
        int to = -1;
        if (s >= 0 && s < p.n_pages) to = s < L ? s : map.select<true>(map.rank(s) - front, words);
        p.slots_out[i] = to;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_live = L;

    const int64_t nv = p.page / V;
    if (nv <= kSmallPage) {
        copy_small_pages<V>(M, static_cast<uint32_t>(nv), [&](int k, float** to, const float** from) {
            *to = p.pool + map.select<true>(k, words) * p.page;
            *from = p.pool + map.select<false>(front + k, words) * p.page;
            return true;
        });
        return;
    }
    const int64_t pieces = (nv + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    for (int64_t u = blockIdx.x; u < pieces * M; u += gridDim.x) {
        const int k = static_cast<int>(u / pieces);
        const int64_t s = map.select<false>(front + k, words), d = map.select<true>(k, words);
        copy_piece<V>(p.pool + d * p.page, p.pool + s * p.page, nv, u % pieces);
    }
}

// Workgroups for `entries` pages: one per piece, up to kMaxGrid, at least one.
unsigned grid_for(int64_t page, int V, int64_t entries) {
    const int64_t piece = static_cast<int64_t>(kThreads) * kUnroll * V;
    const int64_t pieces = (page + piece - 1) / piece;
    int64_t all = entries > 0 && pieces > kMaxGrid ? kMaxGrid : pieces * entries;
    if (page <= kSmallPage * V) all = (page * entries + piece - 1) / piece;      // see copy_small_pages
    return static_cast<unsigned>(all < 1 ? 1 : all > kMaxGrid ? kMaxGrid : all);
}

}  // namespace

// 16-byte vectors where pages start on a multiple of 16 bytes, single floats otherwise.
hipError_t launch_pages_copy(const PagesCopyArgs& a, hipStream_t s) {
    const int V = a.page % 4 == 0 ? 4 : 1;
    const dim3 grid(grid_for(a.page, V, a.n)), block(kThreads);
    if (V == 4) hipLaunchKernelGGL((pages_copy_kernel<4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((pages_copy_kernel<1>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesCompactArgs& a, hipStream_t s) {
    const int V = a.page % 4 == 0 ? 4 : 1;
    // at most half of the pool, and one page per entry, can move
    const int64_t most = a.n < a.n_pages / 2 ? a.n : a.n_pages / 2;
    const dim3 grid(grid_for(a.page, V, most)), block(kThreads);
    if (V == 4) hipLaunchKernelGGL((pages_compact_kernel<4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((pages_compact_kernel<1>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace dr
