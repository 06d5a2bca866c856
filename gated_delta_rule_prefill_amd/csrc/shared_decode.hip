// Decode attention for a batch in which groups of requests share a prefix (gdn_paged_shared_decode).
//
//   o[b, p, h] = sum_j softmax_j(scale q[b, p, h] . k_j) v_j,   j < len_b - n_pos + p + 1,
// as gdn_paged_decode, but the first P tokens of the requests of a group lie in the same pages. A
// decode step is bound by reading keys, so the prefix is attended for all query rows of a group
// at once (size x n_pos x heads of a key/value head: a matrix product, paged_attend.h), each
// request's own keys behind it as in a decode step (paged_decode.hip), and the two joined:
//   o = (e^{m1 - M} acc1 + e^{m2 - M} acc2) / (e^{m1 - M} l1 + e^{m2 - M} l2).
// Four launches: tables, prefixes, own keys, join.
//
// Bound: the prefixes by their steps (paged_attend.h), the own keys by HBM and their units' starts,
// the join by its parts. 128 requests, 32 heads, 4 KV heads, d = 128, behind one prefix of 32000
// tokens, 30 to 2000 tokens of their own, bf16: 6 + 89 + 40 + 21 us (least 5 + 84 + 38 + 18), 145-153 a
// call; gdn_paged_decode 619.
// (Own keys of up to 128 or 256 tokens taken by a wave alone, without a cut or a merge: no quicker.)
// 48 requests of 4 positions, 16 heads of 256, in 8 groups behind 500 to 16000 tokens: 6 + 53 + 20 + 13
// us, 88-90 a call; gdn_paged_decode 105.
#include "paged_attend.h"

namespace gdn {

namespace {

// Workgroups of the joining launch a CU, and groups of lanes that share a row of up to 32 parts (128
// requests, 17 parts a row: 148 us a call with 8 and 4, 157 with 16 and 4, 153 with 8 and 2, 151 with
// 16 and 8; rows of other numbers of parts were not measured).
constexpr int JOIN_WGS = 8, JOIN_ROW_GROUPS = 4;

// Prefixes are attended apart where that spares reads of so many bytes in all: the prefix kernel's
// start and the parts that it leaves cost as much as reading a prefix again out of the caches, which
// a plain decode mostly does. Spared MB, us a call apart and not, bf16, 60 own tokens each: 8 requests,
// 4 heads of 128, 59 MB 29 and 23, 235 MB 36 and 49; 4 groups of 2, 134 MB 49 and 53; 64 requests, 4
// heads, 132 MB 42 and 23, 529 MB 49 and 49, 2114 MB 62 and 156; 7 requests, 4 heads of 64, 101 MB 27
// and 28. fp32: 8 requests, 8 heads of 128, 235 MB 49 and 48, 940 MB 100 and 146.
// Bytes alone do not tell the two apart: what many requests read again comes out of the caches
// faster, so that 32 to 128 requests are better apart from about 250 to 500 MB on only, and are up to
// 1.4 times slower by this rule in between (4 heads of 128: 32 requests behind 4096 tokens 40 and 39,
// 64 behind 2048 46 and 34, 128 behind 1024 43 and 36; 64, 2 heads of 256, behind 2048 43 and 40). A caller
// that knows its batch names min_bytes. Not apart, a call takes 5 to 7 us more than gdn_paged_decode
// (tables, an empty prefix launch, a join of units that need none: 8 requests behind 512 tokens 17
// and 11, 64 behind 4096 50 and 44).
constexpr int64_t SHARED_LEAST_BF16 = (int64_t)128 << 20, SHARED_LEAST_F32 = (int64_t)256 << 20;
// In fp32 a wave's 16 rows take as long as the reads of several requests: 4 groups of 2 requests (16
// rows), 268 MB, 166 us apart, 92 not; 8 requests (64 rows), 470 MB, 69 and 82.
constexpr int SHARED_ROWS_F32 = 64;

// A group whose prefix is attended apart. One request alone has nothing to share: its prefix is
// left to the decode kernel.
struct SharedGroup {
    int first, size, prefix;
};
__device__ __forceinline__ SharedGroup shared_group(const SharedDecodeArgs& a, int g) {
    const int b0 = min(max(a.group_cu[g], 0), a.batch), b1 = min(max(a.group_cu[g + 1], 0), a.batch);
    const int prefix = min(max(a.prefix_lens[g], 0), a.at.max_keys);
    const int least_rows = a.min_bytes < 0 && a.at.dtype == 0 ? SHARED_ROWS_F32 : 0;
    const bool apart = b1 - b0 >= 2 && prefix > 0 &&
                       (int64_t)(b1 - b0) * a.at.n_pos * a.at.group >= least_rows;
    return {b0, apart ? b1 - b0 : 0, apart ? prefix : 0};
}

template <typename T, int D>
__global__ __launch_bounds__(AT_TABLE_THREADS) void shared_tables_kernel(SharedDecodeArgs a) {
    using X = AttendTile<T, D>;
    constexpr int ROWS = ATTEND_ROWS<T, D>;
    const int per_request = a.at.n_pos * a.at.group, groups = a.at.n_seqs;
    // keys that need not be read again; every workgroup comes to the same decision
    __shared__ int64_t part[AT_TABLE_THREADS / WAVE];
    int64_t spared = 0;
    for (int g = threadIdx.x; g < groups; g += AT_TABLE_THREADS) {
        const SharedGroup s = shared_group(a, g);
        spared += (int64_t)max(s.size - 1, 0) * s.prefix;
    }
#pragma unroll
    for (int off = WAVE / 2; off > 0; off >>= 1) spared += __shfl_xor(spared, off, WAVE);
    if (lane_id() == 0) part[wave_id()] = spared;
    __syncthreads();
    spared = 0;
#pragma unroll
    for (int w = 0; w < AT_TABLE_THREADS / WAVE; w++) spared += part[w];
    const int64_t least = a.min_bytes >= 0 ? a.min_bytes
                          : sizeof(T) == 2 ? SHARED_LEAST_BF16 : SHARED_LEAST_F32;
    const bool apart = spared * a.at.kv_heads * (2 * D * (int)sizeof(T)) >= least;
    if (blockIdx.x == 0) {
        attend_tables(
            a.at, ROWS, X::KB, [&](int g) { return apart ? shared_group(a, g).size * per_request : 0; },
            [&](int g, int row0) {
                const SharedGroup s = shared_group(a, g);
                const int rows = s.size * per_request;
                // The tile reads the table row of its first request that holds the whole prefix, or
                // of its longest one, behind whose tokens none of the tile's rows sees a key: a
                // request that ended has no pages any more.
                const int b0 = s.first + row0 / per_request;
                const int b1 = s.first + (row0 + min(ROWS, rows - row0) - 1) / per_request;
                int holder = b0, held = 0;
                constexpr int U = 8;  // lengths on their way
                for (int b = b0; b <= b1 && held < s.prefix; b += U) {
                    int n[U];
#pragma unroll
                    for (int k = 0; k < U; k++) n[k] = a.at.seq_lens[min(b + k, b1)];
#pragma unroll
                    for (int k = 0; k < U; k++) {
                        n[k] = min(max(n[k], 0), s.prefix);
                        if (n[k] > held) {
                            holder = min(b + k, b1);
                            held = n[k];
                        }
                    }
                }
                return AttendUnit{holder, s.first * a.at.n_pos, row0, rows, max(held, 1), 0};
            });
        return;
    }
    // which group each request is in, and what it has to attend itself
    __shared__ int near_cu[AT_TABLE_SEQS];
    const bool near = groups <= AT_TABLE_SEQS;
    for (int g = threadIdx.x; near && g < groups; g += AT_TABLE_THREADS) near_cu[g] = a.group_cu[g];
    __syncthreads();
    const int b = (int)(blockIdx.x - 1) * AT_TABLE_THREADS + threadIdx.x;
    if (b >= a.batch) return;
    const int lo = last_at(groups, b, [&](int g) { return near ? near_cu[g] : a.group_cu[g]; });
    int start = 0;
    int2 place = make_int2(-1, 0);
    if (groups > 0 && apart) {
        const SharedGroup s = shared_group(a, lo);
        if (b >= s.first && b < s.first + s.size) {
            start = s.prefix;
            place = make_int2(lo, (b - s.first) * per_request);
        }
    }
    a.start[b] = start;
    a.own_keys[b] = max(min(max(a.at.seq_lens[b], 0), a.at.max_keys) - start, 0);
    a.place[b] = place;
}

// A workgroup per (request, key/value head) and share of its rows: the parts of the prefix's tiles
// first, then those of the request's own keys. Parts lie in one array: the decode kernel's slots,
// then the prefix kernel's.
template <typename T, int D>
__global__ __launch_bounds__(JOIN_THREADS) void shared_join_kernel(SharedDecodeArgs a) {
    constexpr int ROWS = ATTEND_ROWS<T, D>;
    const JoinShape& j = a.own.join;
    const int unit = (int)blockIdx.x / j.share, b = unit / a.at.kv_heads;
    const int kvh = unit - b * a.at.kv_heads;
    const int4 note = j.notes[unit];
    if (note.w < 0) return;  // no prefix, and one worker took all of its keys
    const int2 place = a.place[b];
    const int t0 = place.x < 0 ? 0 : a.at.seq_tile[place.x];
    const int t1 = place.x < 0 ? 0 : a.at.seq_tile[place.x + 1];
    auto tile_parts = [&](int t) {
        if (t >= t1) return 0;
        const int2 n = a.prefix_notes[kvh * a.at.tiles + t];
        return n.y - n.x + 1;
    };
    int most = 0;
    for (int t = t0 + place.y / ROWS; t <= t0 + (place.y + j.rows - 1) / ROWS && t < t1; t++)
        most = max(most, tile_parts(t));
    auto parts_of = [&](int r) { return note.x + tile_parts(t0 + (place.y + r) / ROWS); };
    const size_t own_rows = (size_t)j.row_tiles * j.tile;
    const size_t prefix0 = ((size_t)2 * a.own.workers + (size_t)a.batch * a.at.kv_heads) * own_rows;
    auto at = [&](int i, int r) {
        if (i < note.x) return (size_t)(i == 0 ? note.z : 2 * (note.y + i)) * own_rows + r;
        i -= note.x;
        const int row = place.y + r, t = t0 + row / ROWS;
        const int w0 = a.prefix_notes[kvh * a.at.tiles + t].x;
        const int64_t slot = i == 0 ? (int64_t)a.at.workers + kvh * a.at.tiles + t : w0 + i;
        return prefix0 + (size_t)slot * ROWS + row % ROWS;
    };
    join_rows<D, (D + 127) / 128, 4, JOIN_ROW_GROUPS>(
        j, note.x + most, parts_of, at, (int)blockIdx.x % j.share, 0,
        [&](int row, int col, const float x[4]) {
            const int p = row / a.at.group, h = row - p * a.at.group;
            store4<T>(reinterpret_cast<T*>(a.own.o) +
                          (((size_t)b * a.at.n_pos + p) * a.at.H + kvh * a.at.group + h) * D + col,
                      x);
        });
}

template <typename T, int D>
hipError_t run_shared(const SharedDecodeArgs& a, hipStream_t s) {
    using X = AttendTile<T, D>;
    const unsigned tables = 1u + (unsigned)((a.batch + AT_TABLE_THREADS - 1) / AT_TABLE_THREADS);
    hipLaunchKernelGGL((shared_tables_kernel<T, D>), dim3(tables), dim3(AT_TABLE_THREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.at.n_seqs > 0) {
        hipLaunchKernelGGL((paged_attend_kernel<T, D, true>), dim3((unsigned)a.at.workers),
                           dim3(X::WAVES * WAVE), 0, s, a.at);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    e = launch_own_keys(a.own, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((shared_join_kernel<T, D>), dim3(join_grid(a.own.join)), dim3(JOIN_THREADS),
                       0, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t pick_dim(const SharedDecodeArgs& a, hipStream_t s) {
    switch (a.at.d) {
        case 64: return run_shared<T, 64>(a, s);
        case 128: return run_shared<T, 128>(a, s);
        case 256: return run_shared<T, 256>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t shared_decode_layout(SharedDecodeArgs* a, void* ws) {
    AttendArgs& at = a->at;
    PagedDecodeArgs& own = a->own;
    const int rows = attend_tile_rows(at.dtype, at.d), cus = device_cu_count();
    at.group = at.H / at.kv_heads;
    at.by_group = FastDiv::of((uint32_t)at.group);
    at.by_pos = FastDiv::of((uint32_t)at.n_pos);
    const int64_t all = (int64_t)a->batch * at.n_pos * at.group;
    // a group has two requests at least
    const int64_t groups = at.n_seqs < a->batch / 2 ? at.n_seqs : a->batch / 2;
    at.tiles = (int)((all + groups * (rows - 1)) / rows);
    at.workers = split_workers(cus < JOIN_MAX_WORKERS / 2 ? cus : JOIN_MAX_WORKERS / 2, 1);
    (void)paged_decode_layout(&own, nullptr);  // row tiles and workers
    if (own.workers > JOIN_MAX_WORKERS / 2) own.workers = JOIN_MAX_WORKERS / 2;
    Layout l(ws);
    attend_table_layout(&at, &l);
    a->start = l.take<int32_t>((size_t)a->batch);
    a->own_keys = l.take<int32_t>((size_t)a->batch);
    a->place = l.take<int2>((size_t)a->batch);
    a->prefix_notes = l.take<int2>((size_t)at.kv_heads * at.tiles);
    JoinShape& j = own.join;
    const int64_t units = (int64_t)a->batch * at.kv_heads;
    j.count = (int)units;
    j.per_unit = 1;
    const int64_t share = units > 0 ? JOIN_WGS * (int64_t)cus / units : 1;
    j.share = share < 1 ? 1 : share < j.rows ? (int)share : j.rows;
    j.slices = 1;
    const size_t own_rows = ((size_t)2 * own.workers + (size_t)units) * own.row_tiles * j.tile;
    const size_t prefix_rows = ((size_t)at.workers + (size_t)at.kv_heads * at.tiles) * rows;
    j.part_o = l.take<float>((own_rows + prefix_rows) * at.d);
    j.part_ml = l.take<float>((own_rows + prefix_rows) * 2);
    j.notes = l.take<int4>((size_t)units);
    at.join.part_o = ws == nullptr ? nullptr : j.part_o + own_rows * at.d;
    at.join.part_ml = ws == nullptr ? nullptr : j.part_ml + own_rows * 2;
    at.prefix_notes = a->prefix_notes;
    own.start = a->start;
    own.split.seq_lens = a->own_keys;
    return l.size;
}

hipError_t launch_shared_decode(const SharedDecodeArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    return a.at.dtype == 1 ? pick_dim<bf16>(a, s) : pick_dim<float>(a, s);
}

}  // namespace gdn
