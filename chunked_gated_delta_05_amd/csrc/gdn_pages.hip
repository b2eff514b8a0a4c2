// The pages of a state cache: explicit copies, forking a batch of beams and
// compacting. Fork and compaction are a plan (who keeps, who copies, what is
// free) and the copies it lists, whose number only the device knows: a fixed
// grid walks the list. Few slots or pages: one kernel, in which every
// workgroup makes the plan for itself in LDS and the first writes the new
// table. Many: the plan is a kernel of one workgroup that leaves its list in
// the caller's workspace.
#include "gdn_device.h"
#include "gdn_recurrent_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;        // threads of the copy kernel
constexpr int PIECE = 16384;   // bytes a workgroup copies at a time: 4 x 16 bytes a thread in flight
constexpr int PT = 1024;       // threads of the plans

// The first n pairs of the lists, every layer, spread over the grid.
// NT_LOAD, NT_STORE: around the caches, where a call walks through more than
// they hold (beyond_caches). Stores around them: 128 slots of 16.8 MB forked
// 325 to 268 us. Loads as well only where no page is read twice: 1.1 GB
// compacted 196 to 189 us, but a page copied to 128 others 322 to 525 (128
// different ones 656 to 648).
template <bool NT_LOAD, bool NT_STORE>
__device__ __forceinline__ void copy_pairs(const PoolArgs& a, const int32_t* dst_pages, const int32_t* src_pages, int n) {
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

template <bool NT_LOAD, bool NT_STORE>
__global__ __launch_bounds__(NT) void copy_kernel(PoolArgs a, const int32_t* dst_pages, const int32_t* src_pages,
                                                  int n, const int32_t* n_dev) {
    if (n_dev) {
        const int c = *n_dev;
        n = c < 0 ? 0 : (c < n ? c : n);
    }
    copy_pairs<NT_LOAD, NT_STORE>(a, dst_pages, src_pages, n);
}

// Exclusive sum of x over the workgroup's threads; total: the whole sum.
template <int THREADS>
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
    for (int w = 0; w < THREADS / 64; ++w) {
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
struct ForkArgs {
    int n_pages, n, m;
    const int32_t *table, *parent, *spare;
    int32_t *new_table, *left;
};
// Returns the number of copies, listed in src and dst; write: also the new
// table and the pages left. lowest[n] and waves in LDS.
template <int THREADS>
__device__ int fork_plan(const ForkArgs& f, int32_t* src, int32_t* dst, bool write, int* lowest, int* waves) {
    const int n = f.n, m = f.m, n_pages = f.n_pages, tid = threadIdx.x;
    const int32_t *table = f.table, *parent = f.parent, *spare = f.spare;
    for (int i = tid; i < n; i += THREADS) lowest[i] = n;
    if (write)
        for (int i = tid; i < n + m; i += THREADS) f.left[i] = -1;
    __syncthreads();
    auto source = [&](int i) {   // the slot that i continues, or -1
        const int p = parent[i];
        return p >= 0 && p < n && is_page(table[p], n_pages) ? p : -1;
    };
    for (int i = tid; i < n; i += THREADS) {
        const int p = source(i);
        if (p >= 0) atomicMin(&lowest[p], i);
    }
    __syncthreads();
    const int per = (n + THREADS - 1) / THREADS, lo = min(tid * per, n), hi = min(lo + per, n);
    const int mper = (m + THREADS - 1) / THREADS, mlo = min(tid * mper, m), mhi = min(mlo + mper, m);
    int extra = 0, dead = 0, spares = 0;
    for (int i = lo; i < hi; ++i) {
        const int p = source(i);
        extra += p >= 0 && lowest[p] != i;
        dead += lowest[i] == n && is_page(table[i], n_pages);
    }
    for (int i = mlo; i < mhi; ++i) spares += is_page(spare[i], n_pages);
    int n_extra, n_dead, n_spare;
    int e = block_scan<THREADS>(extra, &n_extra, waves);
    int d = block_scan<THREADS>(dead, &n_dead, waves);
    int sp = n_dead + block_scan<THREADS>(spares, &n_spare, waves);
    const int copies = min(n_extra, n_dead + n_spare);
    // the free pages in order: the first `copies` are destinations, the rest is left
    auto free_page = [&](int rank, int page) {
        if (rank < copies) dst[rank] = page;
        else if (write) f.left[rank - copies] = page;
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
        if (write) f.new_table[i] = page;
    }
    return copies;
}

__global__ __launch_bounds__(PT) void fork_plan_kernel(ForkArgs f, int32_t* ws) {
    __shared__ int lowest[FORK_MAX];
    __shared__ int waves[PT / 64];
    const int copies = fork_plan<PT>(f, ws + 1, ws + 1 + f.n, true, lowest, waves);
    if (threadIdx.x == 0) ws[0] = copies;
}

// The same for at most THREADS slots and spare pages, one of each a thread:
// all is read from memory at once, and the three counts are one sum of fields
// of 10 bits (80 MB, 20 slots: 8.1 to 6.6 us a call; 384 MB, 32: 30.0 to 27.9).
template <int THREADS>
__device__ int fork_plan_small(const ForkArgs& f, int32_t* src, int32_t* dst, bool write, int* lowest, int* table,
                               int* waves) {
    static_assert(THREADS < 1024, "");
    const int n = f.n, m = f.m, n_pages = f.n_pages, i = threadIdx.x;
    const int p = i < n ? f.parent[i] : -1, page = i < n ? f.table[i] : -1, free = i < m ? f.spare[i] : -1;
    lowest[i] = n;
    table[i] = page;
    if (write)
        for (int j = i; j < n + m; j += THREADS) f.left[j] = -1;
    __syncthreads();
    const bool child = p >= 0 && p < n && is_page(table[p], n_pages);
    if (child) atomicMin(&lowest[p], i);
    __syncthreads();
    const bool extra = child && lowest[p] != i, dead = lowest[i] == n && is_page(page, n_pages);
    const bool spare = is_page(free, n_pages);
    int all;
    const int before = block_scan<THREADS>(extra | dead << 10 | spare << 20, &all, waves);
    const int n_dead = all >> 10 & 1023, copies = min(all & 1023, n_dead + (all >> 20));
    auto free_page = [&](int rank, int x) {
        if (rank < copies) dst[rank] = x;
        else if (write) f.left[rank - copies] = x;
    };
    if (dead) free_page(before >> 10 & 1023, page);
    if (spare) free_page(n_dead + (before >> 20), free);
    const int e = before & 1023;
    const bool copied = extra && e < copies;
    if (copied) src[e] = table[p];
    __syncthreads();
    if (write && i < n) f.new_table[i] = copied ? dst[e] : child && !extra ? table[p] : -1;
    return copies;
}

// At most FORK_SMALL slots and spare pages: one kernel for two (8 slots, 8 MB:
// 8.1 to 5.6 us)
constexpr int FORK_SMALL = NT;
template <bool NT_STORE>
__global__ __launch_bounds__(NT) void fork_kernel(PoolArgs a, ForkArgs f) {
    __shared__ int lowest[FORK_SMALL], table[FORK_SMALL], src[FORK_SMALL], dst[FORK_SMALL];
    __shared__ int waves[NT / 64];
    const int copies = fork_plan_small<NT>(f, src, dst, blockIdx.x == 0, lowest, table, waves);
    copy_pairs<false, NT_STORE>(a, dst, src, copies);
}


// A bit for each used page; a page's rank among the pages that move, and a
// hole's rank among the holes, are counts of bits before it.
struct CompactArgs {
    int n_pages, n;
    const int32_t* table;
    int32_t *new_table, *count;
};
// Returns the number of moves, listed in src and dst; write: also the new
// table and the count. used[], movers_before[] (a word for 32 pages) and
// waves in LDS.
template <int THREADS>
__device__ int compact_plan(const CompactArgs& f, int32_t* src, int32_t* dst, bool write, uint32_t* used,
                            int* movers_before, int* waves) {
    const int n_pages = f.n_pages, n = f.n, tid = threadIdx.x, words = (n_pages + 31) / 32;
    const int32_t* table = f.table;
    for (int w = tid; w < words; w += THREADS) used[w] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
        const int p = table[i];
        if (is_page(p, n_pages)) atomicOr(&used[p >> 5], 1u << (p & 31));
    }
    __syncthreads();
    const int per = (words + THREADS - 1) / THREADS, lo = min(tid * per, words), hi = min(lo + per, words);
    int mine = 0, total;
    for (int w = lo; w < hi; ++w) mine += __popc(used[w]);
    block_scan<THREADS>(mine, &total, waves);
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
    int mv = block_scan<THREADS>(movers, &n_movers, waves);
    int ho = block_scan<THREADS>(holes, &n_holes, waves);
    for (int w = lo; w < hi; ++w) {
        movers_before[w] = mv;
        for (uint32_t b = used[w] & ~below(w); b; b &= b - 1) src[mv++] = 32 * w + __ffs(b) - 1;
        for (uint32_t b = ~used[w] & below(w); b; b &= b - 1) dst[ho++] = 32 * w + __ffs(b) - 1;
    }
    __syncthreads();
    if (write) {
        for (int i = tid; i < n; i += THREADS) {
            int p = table[i];
            if (!is_page(p, n_pages)) {
                p = -1;
            } else if (p >= total) {
                const int w = p >> 5;
                p = dst[movers_before[w] + __popc(used[w] & ~below(w) & ((1u << (p & 31)) - 1u))];
            }
            f.new_table[i] = p;
        }
        if (tid == 0) *f.count = total;
    }
    return n_movers;
}

__global__ __launch_bounds__(PT) void compact_plan_kernel(CompactArgs f, int32_t* ws) {
    __shared__ uint32_t used[COMPACT_MAX / 32];
    __shared__ int movers_before[COMPACT_MAX / 32];
    __shared__ int waves[PT / 64];
    const int moves = compact_plan<PT>(f, ws + 1, ws + 1 + f.n_pages, true, used, movers_before, waves);
    if (threadIdx.x == 0) ws[0] = moves;
}

// At most COMPACT_SMALL pages and slots
constexpr int COMPACT_SMALL = 1024;
template <bool AROUND>
__global__ __launch_bounds__(NT) void compact_kernel(PoolArgs a, CompactArgs f) {
    __shared__ uint32_t used[COMPACT_SMALL / 32];
    __shared__ int movers_before[COMPACT_SMALL / 32], src[COMPACT_SMALL], dst[COMPACT_SMALL];
    __shared__ int waves[NT / 64];
    const int moves = compact_plan<NT>(f, src, dst, blockIdx.x == 0, used, movers_before, waves);
    __syncthreads();
    copy_pairs<AROUND, AROUND>(a, dst, src, moves);
}

}  // namespace

namespace {

// Whether the pages that a call walks through exceed the last-level cache: a
// fork's and a compaction's slots, both lists of a copy. Not the pool's size:
// copies of a few pages of a large one stay in the caches for the next step
// that reads them (slots of 16.8 MB in 3.4 GB, forked or compacted and then
// read and written by a step of every layer: 8 of them 98 us through the
// caches and 100 around, 134 and 140; 16 of them 156 and 154, 222 and 221; 24
// 250 and 242, 345 and 329).
bool beyond_caches(const PoolArgs& pool, int64_t pages) {
    return pages * pool.n_layers * pool.page_bytes > LAST_LEVEL_BYTES;
}
// Workgroups for at most n pairs: four a compute unit, each making the plan
// once; beyond the caches, where copying takes far longer than a plan, four
// times as many, which even out (3.2 GB, 128 slots: 284 to 259 us forked, 313
// to 273 compacted; 80 MB, 20 slots: 8.0 us at 1024, 9.9 at 4096).
unsigned copy_blocks(const PoolArgs& pool, int n, bool beyond) {
    const int64_t items = (pool.page_bytes + PIECE - 1) / PIECE * pool.n_layers * n;
    const int64_t most = beyond ? 4096 : 1024;
    return (unsigned)(items < most ? items : most);
}

// read_once: no page is the source of several
hipError_t copy_listed(const PoolArgs& pool, const int32_t* dst_pages, const int32_t* src_pages, int n,
                       const int32_t* n_dev, bool beyond, bool read_once, hipStream_t s) {
    const unsigned blocks = copy_blocks(pool, n, beyond);
    if (blocks == 0) return hipSuccess;
    if (!beyond) copy_kernel<false, false><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    else if (read_once) copy_kernel<true, true><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    else copy_kernel<false, true><<<blocks, NT, 0, s>>>(pool, dst_pages, src_pages, n, n_dev);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pages_copy(const PoolArgs& pool, const int32_t* dst_pages, const int32_t* src_pages, int n,
                             hipStream_t s) {
    return copy_listed(pool, dst_pages, src_pages, n, nullptr, beyond_caches(pool, 2 * (int64_t)n), false, s);
}

hipError_t launch_fork(const PoolArgs& pool, const int32_t* table, const int32_t* parent, int n, const int32_t* spare,
                       int m, int32_t* new_table, int32_t* left, int32_t* ws, hipStream_t s) {
    const ForkArgs f{pool.src_pages, n, m, table, parent, spare, new_table, left};
    const bool beyond = beyond_caches(pool, n);
    if (n <= FORK_SMALL && m <= FORK_SMALL) {
        const unsigned blocks = copy_blocks(pool, n, beyond);
        if (beyond) fork_kernel<true><<<blocks ? blocks : 1, NT, 0, s>>>(pool, f);
        else fork_kernel<false><<<blocks ? blocks : 1, NT, 0, s>>>(pool, f);
        return hipGetLastError();
    }
    fork_plan_kernel<<<1, PT, 0, s>>>(f, ws);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : copy_listed(pool, ws + 1 + n, ws + 1, n, ws, beyond, false, s);
}

hipError_t launch_compact(const PoolArgs& pool, const int32_t* table, int n, int32_t* new_table, int32_t* count,
                          int32_t* ws, hipStream_t s) {
    const int n_pages = pool.src_pages;
    const CompactArgs f{n_pages, n, table, new_table, count};
    const int moves = n < n_pages ? n : n_pages;   // at most
    const bool beyond = beyond_caches(pool, moves);
    if (n_pages <= COMPACT_SMALL && n <= COMPACT_SMALL) {
        const unsigned blocks = copy_blocks(pool, moves, beyond);
        if (beyond) compact_kernel<true><<<blocks ? blocks : 1, NT, 0, s>>>(pool, f);
        else compact_kernel<false><<<blocks ? blocks : 1, NT, 0, s>>>(pool, f);
        return hipGetLastError();
    }
    compact_plan_kernel<<<1, PT, 0, s>>>(f, ws);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : copy_listed(pool, ws + 1 + n_pages, ws + 1, moves, ws, beyond, true, s);
}

}  // namespace gdn
