// Pages that requests share: forking, freeing and compacting on the block table, and the copies
// of whole pages that follow from it (gdn_paged_fork, gdn_paged_free, gdn_paged_compact,
// gdn_paged_copy).
//
// Page: [LA-Infra] "深度解析线性注意力机制演进与 AI Infra 实现", sections on the prefix cache of
// hybrid models (a block table per request, null blocks).
#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int PG_THREADS = 256;
constexpr int PG_CHUNK = 1024;  // table entries a workgroup takes at a time

__device__ __forceinline__ int relaxed_load(const int32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive sum over the workgroup; `total` receives the sum of all. Two barriers.
template <int THREADS>
__device__ __forceinline__ int block_scan(int x, int* total) {
    __shared__ int part[THREADS / WAVE];
    int upto = x;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int t = __shfl_up(upto, off, WAVE);
        if (lane_id() >= off) upto += t;
    }
    __syncthreads();  // `part` of an earlier call has been read
    if (lane_id() == WAVE - 1) part[wave_id()] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / WAVE; w++) {
        if (w < wave_id()) before += part[w];
        all += part[w];
    }
    *total = all;
    return before + upto - x;
}

// Table entries that a request of `len` tokens holds.
__device__ __forceinline__ int held_entries(int len, int block_size, int max_blocks) {
    const uint32_t x = (uint32_t)max(len, 0), bs = (uint32_t)block_size;
    return (int)min(x / bs + (x % bs != 0), (uint32_t)max_blocks);
}

// Workgroups for n rows of up to max_blocks entries: a workgroup takes PG_CHUNK entries of a row
// at a time, and goes on to the next such piece by the number of workgroups.
inline unsigned row_pieces_grid(int64_t n, int max_blocks) {
    const int64_t items = n * ((max_blocks + PG_CHUNK - 1) / PG_CHUNK);
    return (unsigned)(items < 1 ? 1 : items > 16384 ? 16384 : items);
}

// ------------------------------------------------------------------------------------ fork
// Fork i: with x = lens[i], whole = floor(x / b), the entries 0 .. whole - 1 of row src are
// entered into row dst and each page named by one has a holder more; with x mod b > 0 entry
// `whole` becomes the next page of the free list, and (source page, new page) a copy to make.
//
// Bound: launch latency (8 bytes an entry). Measured: 4 forks of 1000 tokens 3.3 us; 256 forks of 100
// to 20000 tokens 5.2 us beside 49 for their copies. So one launch: the first workgroup deals out the
// free pages, which takes a prefix sum over the forks; the others share whole pages, which takes none.
// The counts are atomic additions of whole numbers, whose order does not matter.
__global__ __launch_bounds__(PG_THREADS) void paged_fork_kernel(ForkArgs a) {
    const int tid = threadIdx.x;
    const int64_t most = (int64_t)a.max_blocks * a.block_size;
    auto fork = [&](int i, int* src, int* dst, int* len) {
        *src = a.src_rows[i];
        *dst = a.dst_rows[i];
        *len = (int)min((int64_t)max(a.lens[i], 0), most);
        return *src >= 0 && *src < a.n_rows && *dst >= 0 && *dst < a.n_rows && *src != *dst;
    };
    if (blockIdx.x > 0) {
        const int chunks = (a.max_blocks + PG_CHUNK - 1) / PG_CHUNK;
        const int64_t items = (int64_t)a.n * chunks;
        for (int64_t x = blockIdx.x - 1; x < items; x += gridDim.x - 1) {
            const int i = (int)(x / chunks), p0 = (int)(x - (int64_t)i * chunks) * PG_CHUNK;
            int src, dst, len;
            if (!fork(i, &src, &dst, &len)) continue;
            const int whole = (int)((uint32_t)len / (uint32_t)a.block_size);
            const int32_t* from = a.table + (size_t)src * a.max_blocks;
            int32_t* to = a.table + (size_t)dst * a.max_blocks;
            for (int p = p0 + tid; p < min(whole, p0 + PG_CHUNK); p += PG_THREADS) {
                const int page = from[p];
                to[p] = page;
                if (page >= 0 && page < a.n_blocks) atomicAdd(a.shares + page, 1);
            }
        }
        return;
    }
    const int per = (a.n + PG_THREADS - 1) / PG_THREADS;
    const int i0 = min((int64_t)tid * per, (int64_t)a.n), i1 = min((int64_t)i0 + per, (int64_t)a.n);
    // the page that fork i has to copy, -1 for none; *entry: where its copy is entered
    auto partial = [&](int i, int32_t** entry) {
        int src, dst, len;
        *entry = nullptr;
        if (!fork(i, &src, &dst, &len)) return -1;
        const int whole = (int)((uint32_t)len / (uint32_t)a.block_size);
        if (len - whole * a.block_size == 0) return -1;
        *entry = a.table + (size_t)dst * a.max_blocks + whole;
        const int page = a.table[(size_t)src * a.max_blocks + whole];
        return page >= 0 && page < a.n_blocks ? page : -1;
    };
    int asks = 0;
    int32_t* entry;
    for (int i = i0; i < i1; i++) asks += partial(i, &entry) >= 0;
    int asked;
    int rank = block_scan<PG_THREADS>(asks, &asked);
    for (int i = i0; i < i1; i++) {
        const int page = partial(i, &entry);
        int got = -1;
        if (page >= 0) {
            if (rank < a.n_free) got = a.free_blocks[rank];
            rank++;
        }
        if (entry != nullptr) *entry = got;
        a.copy_src[i] = got >= 0 ? page : -1;
        a.copy_dst[i] = got;
    }
    if (tid == 0) {
        a.counts[0] = asked;
        a.counts[1] = min(asked, a.n_free);
    }
}

// ------------------------------------------------------------------------------------ free
// Every entry of a row that ends is taken out of the table (by an exchange, so that a row listed
// twice ends once) and its page has a holder less. A page whose count falls below zero had no
// other holder: it is free, and the count itself marks it until the listing kernels, which read
// all counts in the order of the ids, set it to zero again.
//
// Bound: launch latency, and the pool's counts (4 bytes a page). Measured: 256 requests, 70000 entries,
// a pool of 300000 pages 7.2 + 2.8 + 4.4 us; one request of 9000 tokens, 9000 pages 7.4.
__device__ __forceinline__ void drop_entry(const FreeArgs& a, int32_t* entry) {
    const int page = atomicExch(entry, -1);
    if (page >= 0 && page < a.n_blocks) atomicSub(a.shares + page, 1);
}

__global__ __launch_bounds__(PG_THREADS) void paged_drop_kernel(FreeArgs a) {
    const int chunks = (a.max_blocks + PG_CHUNK - 1) / PG_CHUNK;
    const int64_t items = (int64_t)a.n * chunks;
    for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
        const int i = (int)(x / chunks), p0 = (int)(x - (int64_t)i * chunks) * PG_CHUNK;
        const int row = a.rows[i];
        if (row < 0 || row >= a.n_rows) continue;
        const int held = held_entries(a.lens[i], a.block_size, a.max_blocks);
        int32_t* entries = a.table + (size_t)row * a.max_blocks;
        for (int p = p0 + (int)threadIdx.x; p < min(held, p0 + PG_CHUNK); p += PG_THREADS)
            drop_entry(a, entries + p);
    }
}

// Marks among the FREE_PER counts of a thread from id `at` on, one bit each.
constexpr int FREE_PER = 16;
constexpr int FREE_SEG = PG_THREADS * FREE_PER;
__device__ __forceinline__ uint32_t free_marks(const FreeArgs& a, int64_t at) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    uint32_t m = 0;
    if (at + FREE_PER <= a.n_blocks) {
#pragma unroll
        for (int k = 0; k < FREE_PER; k += 4) {
            const i32x4 x = *reinterpret_cast<const i32x4*>(a.shares + at + k);
#pragma unroll
            for (int e = 0; e < 4; e++) m |= (uint32_t)(x[e] < 0) << (k + e);
        }
    } else {
        for (int k = 0; k < FREE_PER && at + k < a.n_blocks; k++)
            m |= (uint32_t)(a.shares[at + k] < 0) << k;
    }
    return m;
}
__device__ __forceinline__ void list_marks(const FreeArgs& a, int64_t at, uint32_t m, int rank) {
    for (; m != 0; m &= m - 1, rank++) {
        const int id = (int)at + __builtin_ctz(m);
        a.shares[id] = 0;
        if (rank < a.max_freed) a.freed[rank] = id;
    }
}

__global__ __launch_bounds__(PG_THREADS) void paged_count_kernel(FreeArgs a) {
    int total;
    const uint32_t m = free_marks(a, (int64_t)blockIdx.x * FREE_SEG + threadIdx.x * FREE_PER);
    block_scan<PG_THREADS>(__popc(m), &total);
    if (threadIdx.x == 0) a.seg_count[blockIdx.x] = total;
}

__global__ __launch_bounds__(PG_THREADS) void paged_list_kernel(FreeArgs a, int segs) {
    const int tid = threadIdx.x;
    int before = 0, all = 0, base, total, unused;
    for (int s = tid; s < segs; s += PG_THREADS) {
        const int c = a.seg_count[s];
        all += c;
        before += s < (int)blockIdx.x ? c : 0;
    }
    block_scan<PG_THREADS>(before, &base);
    block_scan<PG_THREADS>(all, &total);
    const int64_t at = (int64_t)blockIdx.x * FREE_SEG + tid * FREE_PER;
    const uint32_t m = free_marks(a, at);
    const int rank = base + block_scan<PG_THREADS>(__popc(m), &unused);
    list_marks(a, at, m, rank);
    for (int64_t i = (int64_t)total + blockIdx.x * PG_THREADS + tid; i < a.max_freed;
         i += (int64_t)gridDim.x * PG_THREADS)
        a.freed[i] = -1;
    if (blockIdx.x == 0 && tid == 0) a.counts[0] = total;
}

// All of it by one workgroup, where there is little to do: one launch instead of three. Each
// thread lists what lies in its own run of ids. A call from Python by one workgroup and by three
// launches: 256 entries, 8000 pages 9.7 and 15.8 us, 32000 pages 10.6 and 15.8, 64000 pages 14.0 and
// 15.7 (14.0 and 9.3 in a graph); 8192 entries, 8000 pages 27.5 and 15.6. The entries of all rows are
// taken at once: 48 rows of up to 2 entries one row after the other 32.4 us, at once 12.1.
constexpr int FREE_ONE_THREADS = 1024;
constexpr int64_t FREE_ONE_ENTRIES = 1024;
constexpr int FREE_ONE_POOL = 2 * FREE_ONE_THREADS * FREE_PER;
__global__ __launch_bounds__(FREE_ONE_THREADS) void paged_free_one_kernel(FreeArgs a) {
    const int tid = threadIdx.x;
    for (int x = tid; x < a.n * a.max_blocks; x += FREE_ONE_THREADS) {
        const int i = x / a.max_blocks, p = x - i * a.max_blocks, row = a.rows[i];
        if (row >= 0 && row < a.n_rows && p < held_entries(a.lens[i], a.block_size, a.max_blocks))
            drop_entry(a, a.table + (size_t)row * a.max_blocks + p);
    }
    __threadfence();
    __syncthreads();
    int listed = 0;
    for (int64_t first = 0; first < a.n_blocks; first += FREE_ONE_THREADS * FREE_PER) {
        const int64_t at = first + tid * FREE_PER;
        const uint32_t m = free_marks(a, at);
        int total;
        const int rank = listed + block_scan<FREE_ONE_THREADS>(__popc(m), &total);
        list_marks(a, at, m, rank);
        listed += total;
    }
    for (int64_t i = (int64_t)listed + tid; i < a.max_freed; i += FREE_ONE_THREADS)
        a.freed[i] = -1;
    if (tid == 0) a.counts[0] = listed;
}

// --------------------------------------------------------------------------------- compact
// With U the pages that the table's held entries name and n = |U|: the pages of U from id n on
// (the movers) go to the ids below n that are not in U (the holes), the k-th of both in the order
// of their ids. With r(x) = |{u in U : u < x}|, r0 = r(n): mover u is number r(u) - r0, hole h
// number h - r(h), and there are n - r0 of each. Sources lie at n and above, destinations below:
// the copies do not depend on each other.
//
// Bound: launch latency and the table (4 bytes an entry, read twice). Measured: 120 rows, 29000 pages
// 4.3 + 6 + 5.7 + 4.8 us in the four launches below (least 1.8 + 5.6 + 5.2 + 3.8); 10 rows, 600 pages 8.3
// in one. U is a bit per page in the
// workspace: cleared, marked from the table, counted and listed, and the table rewritten, each in
// a launch of its own, since each needs all of the one before.
__global__ __launch_bounds__(PG_THREADS) void compact_clear_kernel(CompactArgs a) {
    for (int64_t w = blockIdx.x * PG_THREADS + threadIdx.x; w < a.words;
         w += (int64_t)gridDim.x * PG_THREADS)
        a.bits[w] = 0;
}

__device__ __forceinline__ void mark_page(uint32_t* bits, int page) {
    uint32_t* word = bits + (page >> 5);
    const uint32_t bit = 1u << (page & 31);
    // (a shared page is named by many entries: most of them find its bit set)
    if (!(__hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & bit))
        atomicOr(word, bit);
}

// fn(entry) for every held entry of every row.
template <typename Fn>
__device__ __forceinline__ void held_pages(const CompactArgs& a, Fn fn) {
    const int chunks = (a.max_blocks + PG_CHUNK - 1) / PG_CHUNK;
    const int64_t items = (int64_t)a.n_rows * chunks;
    for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
        const int i = (int)(x / chunks), p0 = (int)(x - (int64_t)i * chunks) * PG_CHUNK;
        const int held = held_entries(a.seq_lens[i], a.block_size, a.max_blocks);
        int32_t* entries = a.table + (size_t)i * a.max_blocks;
        for (int p = p0 + (int)threadIdx.x; p < min(held, p0 + PG_CHUNK); p += PG_THREADS)
            fn(entries + p);
    }
}

__global__ __launch_bounds__(PG_THREADS) void compact_mark_kernel(CompactArgs a) {
    held_pages(a, [&](int32_t* entry) {
        const int page = *entry;
        if (page >= 0 && page < a.n_blocks) mark_page(a.bits, page);
    });
}

__device__ __forceinline__ int bits_below(uint32_t bits, int b) {
    return __popc(bits & ((1u << b) - 1));
}

// Page id's place in the lists, r(id) being `rank`.
__device__ __forceinline__ void list_page(const CompactArgs& a, int id, bool live, int rank, int n,
                                          int r0) {
    if (live) {
        if (id >= n && rank - r0 < a.max_copies) a.copy_src[rank - r0] = id;
    } else if (id < n && id - rank < a.max_copies) {
        a.copy_dst[id - rank] = id;
    }
}

// A workgroup lists the pages of LIST_WORDS words, and counts all words itself (4 KB of them for
// 32768 pages, out of the L2) instead of waiting for a launch that would: reads that grow with the
// square of the pool, for a million pages 512 workgroups of 128 KB. A thread takes a page at a
// time: a word at a time, its pages one after another, 29000 pages took 8.5 us.
constexpr int LIST_WORDS = 64;
__global__ __launch_bounds__(PG_THREADS) void compact_list_kernel(CompactArgs a) {
    const int tid = threadIdx.x;
    __shared__ uint32_t word[LIST_WORDS];
    __shared__ int word_rank[LIST_WORDS];
    const int64_t w0 = (int64_t)blockIdx.x * LIST_WORDS;
    int mine = 0, all = 0, base, n, below = 0, r0, unused;
    for (int64_t w = tid; w < a.words; w += PG_THREADS) {
        const int c = __popc(a.bits[w]);
        all += c;
        mine += w < w0 ? c : 0;
    }
    block_scan<PG_THREADS>(mine, &base);
    block_scan<PG_THREADS>(all, &n);
    for (int64_t w = tid; w <= n >> 5 && w < a.words; w += PG_THREADS)
        below += w < n >> 5 ? __popc(a.bits[w]) : bits_below(a.bits[w], n & 31);
    block_scan<PG_THREADS>(below, &r0);
    const int64_t w = w0 + tid;
    const uint32_t bits = tid < LIST_WORDS && w < a.words ? a.bits[w] : 0;
    const int rank = base + block_scan<PG_THREADS>(__popc(bits), &unused);
    if (tid < LIST_WORDS) {
        word[tid] = bits;
        word_rank[tid] = rank;
        if (w < a.words) a.rank[w] = rank;
    }
    __syncthreads();
    for (int i = tid; i < LIST_WORDS * 32; i += PG_THREADS) {
        const int64_t id = w0 * 32 + i;
        if (id >= a.n_blocks) break;
        const uint32_t x = word[i >> 5];
        list_page(a, (int)id, (x >> (i & 31)) & 1, word_rank[i >> 5] + bits_below(x, i & 31), n, r0);
    }
    for (int64_t k = (int64_t)(n - r0) + blockIdx.x * PG_THREADS + tid; k < a.max_copies;
         k += (int64_t)gridDim.x * PG_THREADS) {
        a.copy_src[k] = -1;
        a.copy_dst[k] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.counts[0] = n;
        a.counts[1] = n - r0;
    }
}

__device__ __forceinline__ void move_share(const CompactArgs& a, int src, int dst) {
    a.shares[dst] = a.shares[src];
    a.shares[src] = 0;
}

__global__ __launch_bounds__(PG_THREADS) void compact_rewrite_kernel(CompactArgs a) {
    const int n = a.counts[0], moves = min(a.counts[1], a.max_copies);
    const int r0 = n - a.counts[1];
    for (int64_t k = blockIdx.x * PG_THREADS + threadIdx.x; k < moves;
         k += (int64_t)gridDim.x * PG_THREADS)
        move_share(a, a.copy_src[k], a.copy_dst[k]);
    held_pages(a, [&](int32_t* entry) {
        const int page = *entry;
        if (page < n || page >= a.n_blocks) return;
        const int k = a.rank[page >> 5] + bits_below(a.bits[page >> 5], page & 31) - r0;
        if (k < moves) *entry = a.copy_dst[k];
    });
}

// All of it by one workgroup with the bits in LDS, where there is little to do: one launch
// instead of four. A call from Python by one workgroup and by four launches: 256 entries, 1000 pages
// 10.2 and 19.7 us, 32000 pages 16.7 and 19.5; 8192 entries, 8000 pages 20.9 and 20.8, 32000 pages
// 28.6 and 22.3.
constexpr int COMPACT_ONE_THREADS = 1024;
constexpr int64_t COMPACT_ONE_ENTRIES = 4096;
constexpr int COMPACT_ONE_WORDS = COMPACT_ONE_THREADS;
__global__ __launch_bounds__(COMPACT_ONE_THREADS) void compact_one_kernel(CompactArgs a) {
    __shared__ uint32_t bits[COMPACT_ONE_WORDS];
    __shared__ int ranks[COMPACT_ONE_WORDS];
    const int tid = threadIdx.x;
    bits[tid] = 0;
    __syncthreads();
    const int entries = a.n_rows * a.max_blocks;  // at most COMPACT_ONE_ENTRIES
    auto held = [&](int x, int* page) {
        const int i = x / a.max_blocks, p = x - i * a.max_blocks;
        if (p >= held_entries(a.seq_lens[i], a.block_size, a.max_blocks)) return false;
        *page = a.table[x];
        return *page >= 0 && *page < a.n_blocks;
    };
    int page = 0;
    for (int x = tid; x < entries; x += COMPACT_ONE_THREADS)
        if (held(x, &page)) atomicOr(&bits[page >> 5], 1u << (page & 31));
    __syncthreads();
    const uint32_t mine = bits[tid];
    int n, r0;
    const int rank = block_scan<COMPACT_ONE_THREADS>(__popc(mine), &n);
    const int first = tid * 32;
    block_scan<COMPACT_ONE_THREADS>(
        first + 32 <= n ? __popc(mine) : first < n ? bits_below(mine, n & 31) : 0, &r0);
    ranks[tid] = rank;
    __syncthreads();
    for (int id = tid; id < a.n_blocks; id += COMPACT_ONE_THREADS) {
        const uint32_t x = bits[id >> 5];
        list_page(a, id, (x >> (id & 31)) & 1, ranks[id >> 5] + bits_below(x, id & 31), n, r0);
    }
    for (int64_t k = (int64_t)(n - r0) + tid; k < a.max_copies; k += COMPACT_ONE_THREADS) {
        a.copy_src[k] = -1;
        a.copy_dst[k] = -1;
    }
    if (tid == 0) {
        a.counts[0] = n;
        a.counts[1] = n - r0;
    }
    __threadfence();
    __syncthreads();
    const int moves = min(n - r0, a.max_copies);
    for (int k = tid; k < moves; k += COMPACT_ONE_THREADS)
        move_share(a, relaxed_load(a.copy_src + k), relaxed_load(a.copy_dst + k));
    for (int x = tid; x < entries; x += COMPACT_ONE_THREADS) {
        if (!held(x, &page) || page < n) continue;
        const int k = ranks[page >> 5] + bits_below(bits[page >> 5], page & 31) - r0;
        if (k < moves) a.table[x] = relaxed_load(a.copy_dst + k);
    }
}

// ------------------------------------------------------------------------------------ copy
// Pages copied within each of up to COPY_CACHES pools, 16 bytes a thread at a time. Bound: HBM.
// Measured: 6300 pages of 16 KiB in 4 pools (826 MB read and written) 152-160 us, 5.2-5.4 TB/s, which is
// what a large copy reaches.
constexpr int COPY_PER = 4;                              // 16-byte pieces of a thread on their way
constexpr int COPY_PIECES = PG_THREADS * COPY_PER;       // pieces a workgroup takes at a time

__global__ __launch_bounds__(PG_THREADS) void paged_copy_kernel(CopyArgs a, int chunks) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const int n = a.count == nullptr ? a.n : min(max(*a.count, 0), a.n);
    const int64_t items = (int64_t)n * chunks;
    char* pool = static_cast<char*>(a.caches[blockIdx.y]);
    for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
        const int i = (int)(x / chunks);
        const int src = a.src[i], dst = a.dst[i];
        // (a page onto itself is left alone: another pair may be writing it)
        if (src < 0 || src >= a.n_blocks || dst < 0 || dst >= a.n_blocks || src == dst) continue;
        const int64_t p0 = (x - (int64_t)i * chunks) * COPY_PIECES + threadIdx.x;
        const i32x4* from = reinterpret_cast<const i32x4*>(pool + src * a.page_bytes);
        i32x4* to = reinterpret_cast<i32x4*>(pool + dst * a.page_bytes);
        const int64_t pieces = a.page_bytes / 16;
        i32x4 v[COPY_PER];
#pragma unroll
        for (int k = 0; k < COPY_PER; k++)
            if (p0 + k * PG_THREADS < pieces) v[k] = from[p0 + k * PG_THREADS];
#pragma unroll
        for (int k = 0; k < COPY_PER; k++)
            if (p0 + k * PG_THREADS < pieces) to[p0 + k * PG_THREADS] = v[k];
    }
}

}  // namespace

hipError_t launch_paged_fork(const ForkArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    hipLaunchKernelGGL(paged_fork_kernel, dim3(1u + row_pieces_grid(a.n, a.max_blocks)),
                       dim3(PG_THREADS), 0, s, a);
    return hipGetLastError();
}

size_t paged_free_layout(FreeArgs* a, void* ws) {
    a->seg_count = static_cast<int32_t*>(ws);
    return ((size_t)a->n_blocks + FREE_SEG - 1) / FREE_SEG * sizeof(int32_t);
}

hipError_t launch_paged_free(const FreeArgs& a, hipStream_t s) {
    (void)hipGetLastError();
    if ((int64_t)a.n * a.max_blocks <= FREE_ONE_ENTRIES && a.n_blocks <= FREE_ONE_POOL) {
        hipLaunchKernelGGL(paged_free_one_kernel, dim3(1), dim3(FREE_ONE_THREADS), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(paged_drop_kernel, dim3(row_pieces_grid(a.n, a.max_blocks)),
                       dim3(PG_THREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int segs = (int)(((int64_t)a.n_blocks + FREE_SEG - 1) / FREE_SEG);
    hipLaunchKernelGGL(paged_count_kernel, dim3((unsigned)segs), dim3(PG_THREADS), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(paged_list_kernel, dim3((unsigned)segs), dim3(PG_THREADS), 0, s, a, segs);
    return hipGetLastError();
}

size_t paged_compact_layout(CompactArgs* a, void* ws) {
    a->words = ((int64_t)a->n_blocks + 31) / 32;
    const size_t part = ((size_t)a->words * 4 + 15) & ~(size_t)15;
    a->bits = static_cast<uint32_t*>(ws);
    a->rank = ws == nullptr ? nullptr
                            : reinterpret_cast<int32_t*>(static_cast<char*>(ws) + part);
    return 2 * part;
}

hipError_t launch_paged_compact(const CompactArgs& a, hipStream_t s) {
    (void)hipGetLastError();
    if ((int64_t)a.n_rows * a.max_blocks <= COMPACT_ONE_ENTRIES && a.words <= COMPACT_ONE_WORDS) {
        hipLaunchKernelGGL(compact_one_kernel, dim3(1), dim3(COMPACT_ONE_THREADS), 0, s, a);
        return hipGetLastError();
    }
    const dim3 block(PG_THREADS);
    const unsigned by_word = (unsigned)((a.words + PG_THREADS - 1) / PG_THREADS);
    const unsigned by_row = row_pieces_grid(a.n_rows, a.max_blocks);
    hipLaunchKernelGGL(compact_clear_kernel, dim3(by_word), block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_mark_kernel, dim3(by_row), block, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_list_kernel, dim3((unsigned)((a.words + LIST_WORDS - 1) / LIST_WORDS)),
                       block, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_rewrite_kernel, dim3(by_row), block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_paged_copy(const CopyArgs& a, int n_caches, hipStream_t s) {
    (void)hipGetLastError();
    const int chunks = (int)((a.page_bytes / 16 + COPY_PIECES - 1) / COPY_PIECES);
    const int64_t items = (int64_t)a.n * chunks, most = 16 * (int64_t)device_cu_count();
    const unsigned grid = (unsigned)(items < most ? items : most);
    hipLaunchKernelGGL(paged_copy_kernel, dim3(grid, (unsigned)n_caches), dim3(PG_THREADS), 0, s, a,
                       chunks);
    return hipGetLastError();
}

}  // namespace gdn
