// Work split of the paged decode kernels: the keys of all (request, head group) units laid end
// to end in chunks of KB keys, and cut into equal runs of chunks, one per workgroup. Lengths
// are device data, so every workgroup derives the cut from them; nothing is read on the host.
//
// A unit that one workgroup covers whole is finished by it. A unit cut between workgroups
// leaves one partial result (unnormalised output, running maximum and sum, per row) per
// workgroup that touched it, and a second kernel joins them (key_join.h). A workgroup can touch at most two
// cut units (its first and its last), so it owns two partial slots: 2 w for the unit it starts
// with, 2 w + 1 for a later one. Work is even to one chunk whatever the lengths, the slots are
// as many as the grid is wide, and the sums run in a fixed order.
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
    int units;      // per request: head groups x row tiles
    int max_keys;   // keys a table row can address
};

// Keys of request b that the table can address.
__device__ __forceinline__ int split_keys(const SplitShape& s, int b) {
    return min(max(s.seq_lens[b], 0), s.max_keys);
}
template <int KB>
__device__ __forceinline__ int split_chunks(const SplitShape& s, int b) {
    return (split_keys(s, b) + KB - 1) / KB;
}

// Workgroups that get work, the first chunk of workgroup w, and the owner of chunk x.
__device__ __forceinline__ int split_wgs(int64_t total, int n_wg) {
    return total < n_wg ? (int)total : n_wg;
}
__device__ __forceinline__ int64_t split_start(int w, int64_t total, int n) {
    return (int64_t)((uint64_t)w * (uint64_t)total / (uint32_t)n);
}
__device__ __forceinline__ int split_owner(int64_t x, int64_t total, int n) {
    return (int)(((uint64_t)(x + 1) * (uint32_t)n - 1) / (uint64_t)total);
}

// Workgroup-uniform values moved to scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 | lo);
}

// This workgroup's run of chunks [pos, end), and the request that chunk `pos` lies in, whose
// first chunk is `base`. All threads of the workgroup call it.
struct SplitRun {
    int64_t pos, end, base;
    int b;
};
template <int KB, int THREADS>
__device__ SplitRun split_run(const SplitShape& s, int w, int n_wg) {
    __shared__ int64_t wave_tot[THREADS / WAVE];
    __shared__ int64_t found_base;
    __shared__ int found_b;
    const int tid = threadIdx.x;
    const int per = (s.batch + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, s.batch), b1 = min(b0 + per, s.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; b++) mine += split_chunks<KB>(s, b);
    mine *= s.units;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int64_t t = __shfl_up(upto, off, WAVE);
        if (lane_id() >= off) upto += t;
    }
    if (lane_id() == WAVE - 1) wave_tot[wave_id()] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / WAVE; i++) {
        if (i < wave_id()) upto += wave_tot[i];
        total += wave_tot[i];
    }
    SplitRun r;
    const int n = split_wgs(total, n_wg);
    r.pos = w < n ? split_start(w, total, n) : 0;
    r.end = w < n ? split_start(w + 1, total, n) : 0;
    const int64_t before = upto - mine;
    if (before <= r.pos && r.pos < upto) {  // exactly one thread when pos < total
        int64_t at = before;
        int b = b0;
        for (; b + 1 < b1; b++) {
            const int64_t c = (int64_t)split_chunks<KB>(s, b) * s.units;
            if (r.pos < at + c) break;
            at += c;
        }
        found_base = at;
        found_b = b;
    }
    __syncthreads();
    // (found_* are unset when there is nothing to do)
    const bool any = r.pos < r.end;
    r.base = uniform(any ? found_base : 0);
    r.b = uniform(any ? found_b : 0);
    r.pos = uniform(r.pos);
    r.end = uniform(r.end);
    return r;
}

}  // namespace gdn
