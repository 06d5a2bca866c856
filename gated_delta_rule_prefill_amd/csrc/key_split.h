// Work split of the paged decode kernels: the keys of all (request, head group) units laid end
// to end in chunks of KB keys, and cut into equal runs of chunks, one per worker. Lengths are
// device data, so every workgroup derives the cut from them; nothing is read on the host.
//
// A unit that one worker covers whole is finished by it. A unit cut between workers leaves one
// partial result (unnormalised output, running maximum and sum, per row) per worker that touched
// it, and a second kernel joins them (key_join.h). A worker can touch at most two cut units (its
// first and its last), so it owns two partial slots: 2 w for the unit it starts with, 2 w + 1
// for a later one. Work is even to one chunk whatever the lengths, the slots are as many as the
// workers, and the sums run in a fixed order. With fewer chunks than workers each chunk gets one
// worker and the rest have nothing to do, so every worker between the first and the last of a
// unit holds a part of it.
//
// Starting and ending a unit (queries, first keys, results) takes as long as some chunks do, and
// a run of many short units would be the last to end: each unit is followed by `extra` chunks
// that exist for the cut only.
//
// Query rows beyond one row tile: a worker is then one workgroup per row tile, side by side on
// the same XCD at the same time, so that the tiles after the first find the keys in its L2.
#pragma once
#include "gdn_common.h"

namespace gdn {

// n / d for n < 2^31 by a multiplication (d fixed for a call): q = (hi(n m) + n) >> s with
// s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.
struct FastDiv {
    uint32_t mul, shift, div;
    static FastDiv of(uint32_t d) {
        uint32_t s = 0;
        while ((1ull << s) < d) s++;
        return {(uint32_t)(((((1ull << s) - d) << 32) / d) + 1), s, d};
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

struct SplitShape {
    const int32_t* seq_lens;
    int batch;
    int units;      // head groups of a request
    int max_keys;   // keys a table row can address
    int extra;      // chunks that a unit counts for beyond its own, at most SPLIT_EXTRA
    int halve;      // 1: half of the workers, where units have SPLIT_LONG chunks on average
};
constexpr int SPLIT_EXTRA = 6;
constexpr int SPLIT_LONG = 8;  // (the extra ones among them)

// Keys of request b that the table can address.
__device__ __forceinline__ int split_keys(const SplitShape& s, int b) {
    return min(max(s.seq_lens[b], 0), s.max_keys);
}
// Chunks of a unit of request b in the cut: its own and the extra ones (none without keys).
template <int KB>
__device__ __forceinline__ int split_chunks(const SplitShape& s, int b) {
    const int n = (split_keys(s, b) + KB - 1) / KB;
    return n > 0 ? n + s.extra : 0;
}

// Which worker and row tile a workgroup is. Workgroups are dealt to the 8 XCDs in turn; n is a
// multiple of 8.
struct SplitPlace {
    int worker, row_tile;
};
__device__ __forceinline__ SplitPlace split_place(int block, int row_tiles) {
    const int round = block / (8 * row_tiles), rest = block - round * 8 * row_tiles;
    return {round * 8 + (rest & 7), rest >> 3};
}
inline int split_workers(int workgroups, int row_tiles) {
    const int n = workgroups / row_tiles / 8 * 8;
    return n < 8 ? 8 : n > 1024 ? 1024 : n;
}

// `total` chunks over at most n workers: the first `more` take each + 1, the others `each`.
struct SplitCut {
    int total, n, each, more;
    __device__ __forceinline__ static SplitCut of(int total, int workers) {
        const int n = total < workers ? total : workers;
        if (n == 0) return {0, 0, 0, 0};
        return {total, n, total / n, total % n};
    }
    __device__ __forceinline__ int start(int w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int owner(int x) const {
        const int big = more * (each + 1);
        return x < big ? x / (each + 1) : more + (x - big) / each;
    }
};

// Workgroup-uniform values moved to scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// A worker's run of chunks [pos, end), and the request that chunk `pos` lies in, whose first
// chunk is `base`. `pos` may be one of a unit's extra chunks. All threads of the workgroup call
// it.
struct SplitRun {
    int pos, end, base, b;
    SplitCut cut;
    // On to chunk `to`; behind the request's last the next request with keys follows.
    __device__ __forceinline__ void advance(const SplitShape& s, int to, int request_end) {
        pos = to;
        if (pos < end && pos == request_end) {
            base = pos;
            do b++;
            while (b + 1 < s.batch && uniform(split_keys(s, b)) == 0);
        }
    }
};
template <int KB, int THREADS>
__device__ SplitRun split_run(const SplitShape& s, int w, int workers) {
    __shared__ int wave_tot[THREADS / WAVE];
    __shared__ int found_base, found_b;
    const int tid = threadIdx.x;
    const int per = (s.batch + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, s.batch), b1 = min(b0 + per, s.batch);
    int mine = 0;
    for (int b = b0; b < b1; b++) mine += split_chunks<KB>(s, b);
    mine *= s.units;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int t = __shfl_up(upto, off, WAVE);
        if (lane_id() >= off) upto += t;
    }
    if (lane_id() == WAVE - 1) wave_tot[wave_id()] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / WAVE; i++) {
        if (i < wave_id()) upto += wave_tot[i];
        total += wave_tot[i];
    }
    const bool fewer = s.halve && total / SPLIT_LONG >= s.batch * s.units;
    const SplitCut cut = SplitCut::of(uniform(total), fewer ? workers / 2 : workers);
    SplitRun r = {0, 0, 0, 0, cut};
    if (w >= cut.n) return r;
    r.pos = cut.start(w);
    r.end = cut.start(w + 1);
    const int before = upto - mine;
    if (before <= r.pos && r.pos < upto) {  // exactly one thread
        int at = before, b = b0;
        for (; b + 1 < b1; b++) {
            const int c = split_chunks<KB>(s, b) * s.units;
            if (r.pos < at + c) break;
            at += c;
        }
        found_base = at;
        found_b = b;
    }
    __syncthreads();
    r.base = uniform(found_base);
    r.b = uniform(found_b);
    return r;
}

}  // namespace gdn
