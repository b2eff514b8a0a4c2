// The pages of a state cache: explicit copies, forking a batch of beams and
// compacting. Fork and compaction are a plan (one workgroup: who keeps, who
// copies, what is free, written to the caller's workspace) followed by the
// copies, whose number only the device knows: a fixed grid walks the list.
#include "gdn_device.h"
#include "gdn_recurrent_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;        // threads of the copy kernel
constexpr int PIECE = 16384;   // bytes a workgroup copies at a time: 4 x 16 bytes a thread in flight
constexpr int COPY_WGS = 1024; // 4 workgroups per compute unit
constexpr int PT = 1024;       // threads of the plans

// NT_LOAD, NT_STORE: around the caches. Pools beyond the last-level cache
// (1.6 GB forked, 1.1 GB compacted): stores around it take 316 to 304 us and
// 203 to 196 us, loads as well 189 us where every page is read once, but 320
// where beams share parents, whose pages the caches serve.
template <bool NT_LOAD, bool NT_STORE>
__global__ __launch_bounds__(NT) void copy_kernel(PoolArgs a, const int32_t* dst_pages, const int32_t* src_pages,
                                                  int n, const int32_t* n_dev) {
    if (n_dev) {
        const int c = *n_dev;
        n = c < 0 ? 0 : (c < n ? c : n);
    }
    const int64_t pieces = (a.page_bytes + PIECE - 1) / PIECE;
    const int64_t per_pair = pieces * a.n_layers, items = per_pair * n;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t pair = it / per_pair, rest = it - pair * per_pair;
        const int64_t layer = rest / pieces, at = (rest - layer * pieces) * PIECE;
        const int sp = src_pages[pair], dp = dst_pages[pair];
        if (sp < 0 || sp >= a.src_pages || dp < 0 || dp >= a.dst_pages) continue;
        const char* src = a.src + (layer * a.src_pages + sp) * a.page_bytes + at;
        char* dst = a.dst + (layer * a.dst_pages + dp) * a.page_bytes + at;
        const int64_t left = a.page_bytes - at;
        u32x4 x[PIECE / NT / 16];
#pragma unroll
        for (int i = 0; i < PIECE / NT / 16; ++i) {
            const int64_t o = (int64_t)(threadIdx.x + i * NT) * 16;
            const u32x4* p = reinterpret_cast<const u32x4*>(src + o);
            if (o < left) x[i] = NT_LOAD ? __builtin_nontemporal_load(p) : *p;
        }
#pragma unroll
        for (int i = 0; i < PIECE / NT / 16; ++i) {
            const int64_t o = (int64_t)(threadIdx.x + i * NT) * 16;
            u32x4* p = reinterpret_cast<u32x4*>(dst + o);
            if (o < left) {
                if constexpr (NT_STORE) __builtin_nontemporal_store(x[i], p);
                else *p = x[i];
            }
        }
    }
}

// Exclusive sum of x over the workgroup's threads; total: the whole sum.
__device__ __forceinline__ int block_scan(int x, int* total, int* waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();   // waves[] of an earlier call has been read
    if (lane == 63) waves[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < PT / 64; ++w) {
        if (w < wave) before += waves[w];
        all += waves[w];
    }
    *total = all;
    return before + s - x;
}

__device__ __forceinline__ bool is_page(int p, int n_pages) { return p >= 0 && p < n_pages; }

// Every slot i: its source page is table[parent[i]]; the lowest child of a
// slot keeps it, the e-th other child copies into the e-th free page. A slot
// range of its own for each thread keeps the scans in slot order.
__global__ __launch_bounds__(PT) void fork_plan_kernel(int n_pages, const int32_t* table, const int32_t* parent, int n,
                                                       const int32_t* spare, int m, int32_t* new_table, int32_t* left,
                                                       int32_t* ws) {
    __shared__ int lowest[FORK_MAX];
    __shared__ int waves[PT / 64];
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += PT) lowest[i] = n;
    for (int i = tid; i < n + m; i += PT) left[i] = -1;
    __syncthreads();
    auto source = [&](int i) {   // the slot that i continues, or -1
        const int p = parent[i];
        return p >= 0 && p < n && is_page(table[p], n_pages) ? p : -1;
    };
    for (int i = tid; i < n; i += PT) {
        const int p = source(i);
        if (p >= 0) atomicMin(&lowest[p], i);
    }
    __syncthreads();
    const int per = (n + PT - 1) / PT, lo = min(tid * per, n), hi = min(lo + per, n);
    const int mper = (m + PT - 1) / PT, mlo = min(tid * mper, m), mhi = min(mlo + mper, m);
    int extra = 0, dead = 0, spares = 0;
    for (int i = lo; i < hi; ++i) {
        const int p = source(i);
        extra += p >= 0 && lowest[p] != i;
        dead += lowest[i] == n && is_page(table[i], n_pages);
    }
    for (int i = mlo; i < mhi; ++i) spares += is_page(spare[i], n_pages);
    int n_extra, n_dead, n_spare;
    int e = block_scan(extra, &n_extra, waves);
    int d = block_scan(dead, &n_dead, waves);
    int sp = n_dead + block_scan(spares, &n_spare, waves);
    const int copies = min(n_extra, n_dead + n_spare);
    int32_t* src = ws + 1;
    int32_t* dst = ws + 1 + n;
    // the free pages in order: the first `copies` are destinations, the rest is left
    auto free_page = [&](int rank, int page) {
        if (rank < copies) dst[rank] = page;
        else left[rank - copies] = page;
    };
    for (int i = lo; i < hi; ++i)
        if (lowest[i] == n && is_page(table[i], n_pages)) free_page(d++, table[i]);
    for (int i = mlo; i < mhi; ++i)
        if (is_page(spare[i], n_pages)) free_page(sp++, spare[i]);
    __syncthreads();
    for (int i = lo; i < hi; ++i) {
        const int p = source(i);
        int page = -1;
        if (p >= 0 && lowest[p] == i) {
            page = table[p];
        } else if (p >= 0) {
            if (e < copies) {
                src[e] = table[p];
                page = dst[e];
            }
            ++e;
        }
        new_table[i] = page;
    }
    if (tid == 0) ws[0] = copies;
}

// A bit for each used page; a page's rank among the pages that move, and a
// hole's rank among the holes, are counts of bits before it.
__global__ __launch_bounds__(PT) void compact_plan_kernel(int n_pages, const int32_t* table, int n, int32_t* new_table,
                                                          int32_t* count, int32_t* ws) {
    constexpr int WORDS = COMPACT_MAX / 32;
    __shared__ uint32_t used[WORDS];
    __shared__ int movers_before[WORDS];
    __shared__ int waves[PT / 64];
    const int tid = threadIdx.x, words = (n_pages + 31) / 32;
    for (int w = tid; w < words; w += PT) used[w] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += PT) {
        const int p = table[i];
        if (is_page(p, n_pages)) atomicOr(&used[p >> 5], 1u << (p & 31));
    }
    __syncthreads();
    const int per = (words + PT - 1) / PT, lo = min(tid * per, words), hi = min(lo + per, words);
    int mine = 0, total;
    for (int w = lo; w < hi; ++w) mine += __popc(used[w]);
    block_scan(mine, &total, waves);
    // bits of word w that are pages below the count
    auto below = [&](int w) -> uint32_t {
        const int b = total - 32 * w;
        return b <= 0 ? 0u : (b >= 32 ? ~0u : (1u << b) - 1u);
    };
    int movers = 0, holes = 0, n_movers, n_holes;
    for (int w = lo; w < hi; ++w) {
        movers += __popc(used[w] & ~below(w));
        holes += __popc(~used[w] & below(w));
    }
    int mv = block_scan(movers, &n_movers, waves);
    int ho = block_scan(holes, &n_holes, waves);
    int32_t* src = ws + 1;
    int32_t* dst = ws + 1 + n_pages;
    for (int w = lo; w < hi; ++w) {
        movers_before[w] = mv;
        for (uint32_t b = used[w] & ~below(w); b; b &= b - 1) src[mv++] = 32 * w + __ffs(b) - 1;
        for (uint32_t b = ~used[w] & below(w); b; b &= b - 1) dst[ho++] = 32 * w + __ffs(b) - 1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += PT) {
        int p = table[i];
        if (!is_page(p, n_pages)) {
            p = -1;
        } else if (p >= total) {
            const int w = p >> 5;
            p = dst[movers_before[w] + __popc(used[w] & ~below(w) & ((1u << (p & 31)) - 1u))];
        }
        new_table[i] = p;
    }
    if (tid == 0) {
        *count = total;
        ws[0] = n_movers;
    }
}

}  // namespace

hipError_t launch_pages_copy(const PoolArgs& pool, const int32_t* dst_pages, const int32_t* src_pages, int n,
                             const int32_t* n_dev, bool read_once, hipStream_t s) {
    const int64_t items = (pool.page_bytes + PIECE - 1) / PIECE * pool.n_layers * n;
    if (items == 0) return hipSuccess;
    const unsigned blocks = (unsigned)(items < COPY_WGS ? items : COPY_WGS);
    const bool large = (int64_t)pool.n_layers * pool.src_pages * pool.page_bytes > LAST_LEVEL_BYTES;
    if (large && read_once) copy_kernel<true, true><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    else if (large) copy_kernel<false, true><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    else copy_kernel<false, false><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    return hipGetLastError();
}

hipError_t launch_fork_plan(int n_pages, const int32_t* table, const int32_t* parent, int n, const int32_t* spare,
                            int m, int32_t* new_table, int32_t* left, int32_t* ws, hipStream_t s) {
    fork_plan_kernel<<<1, PT, 0, s>>>(n_pages, table, parent, n, spare, m, new_table, left, ws);
    return hipGetLastError();
}

hipError_t launch_compact_plan(int n_pages, const int32_t* table, int n, int32_t* new_table, int32_t* count,
                               int32_t* ws, hipStream_t s) {
    compact_plan_kernel<<<1, PT, 0, s>>>(n_pages, table, n, new_table, count, ws);
    return hipGetLastError();
}

}  // namespace gdn
