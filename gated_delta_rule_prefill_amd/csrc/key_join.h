// Joins the partial results that key_split.h's cut leaves: for each row of a cut unit
//   o = sum_w e^{m_w - M} acc_w / sum_w e^{m_w - M} l_w,   M = max_w m_w
// over the workgroups w that hold a part of it (exponentials to base 2, as the parts keep
// their maxima).
//
// Only cut units have work, and a launch cannot know which those are, so every workgroup lists
// them for itself (one look-up per worker boundary of the split: a boundary inside a unit cuts
// it, and the first such boundary stands for the unit) and takes its share of the list. A group
// of 32 lanes reads a whole row of one part at a time; a row with many parts gets up to eight
// groups (its sums meet in LDS in a fixed order), rows with few parts run side by side. Bound by
// latency (two dependent reads), so the grid is a few workgroups per CU and each makes few
// passes.
#pragma once
#include "key_split.h"

namespace gdn {

constexpr int JOIN_THREADS = 256;
constexpr int JOIN_GROUPS = JOIN_THREADS / 32;
constexpr int JOIN_MAX_WORKERS = 1024;

struct JoinShape {
    SplitShape split;
    int workers;
    int row_tiles, tile;   // row tiles of a worker, rows of a tile
    int rows;              // live rows of a unit, over its row tiles
    const float* part_o;   // [2 workers][row_tiles][tile][COLS]
    const float* part_ml;  // [2 workers][row_tiles][tile][2]
};

// store(b, unit, row, col, x[4]) takes 4 columns of a row of request b's unit; zero(b) is called
// by all threads of one workgroup for every request without keys.
template <int KB, int COLS, typename Store, typename Zero>
__device__ __forceinline__ void join_parts(const JoinShape& s, Store store, Zero zero) {
    constexpr int NC = (COLS + 127) / 128;  // 16-byte pieces of a row per lane
    __shared__ int first[JOIN_THREADS + 1];  // chunks before each thread's requests
    __shared__ int wave_tot[JOIN_THREADS / WAVE];
    __shared__ int cut_b[JOIN_MAX_WORKERS], cut_unit[JOIN_MAX_WORKERS];
    __shared__ int cut_w0[JOIN_MAX_WORKERS];  // 2 (first worker) + (its part is in the late slot)
    __shared__ int cut_w1[JOIN_MAX_WORKERS];  // last worker
    __shared__ int wave_cuts[JOIN_THREADS / WAVE];
    __shared__ float red[JOIN_GROUPS][NC * 128 + 4];
    __shared__ float red_l[JOIN_GROUPS];
    const int tid = threadIdx.x;
    const int per = (s.split.batch + JOIN_THREADS - 1) / JOIN_THREADS;
    const int b0 = min(tid * per, s.split.batch), b1 = min(b0 + per, s.split.batch);
    int mine = 0;
    for (int b = b0; b < b1; b++) mine += split_chunks<KB>(s.split, b);
    mine *= s.split.units;
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
    for (int i = 0; i < JOIN_THREADS / WAVE; i++) {
        if (i < wave_id()) upto += wave_tot[i];
        total += wave_tot[i];
    }
    first[tid + 1] = upto;
    if (tid == 0) first[0] = 0;
    __syncthreads();

    for (int b = blockIdx.x; b < s.split.batch; b += gridDim.x)
        if (split_keys(s.split, b) == 0) zero(b);

    const SplitCut split = SplitCut::of(uniform(total), s.workers);
    int cuts = 0;
    for (int w_base = 1; w_base < split.n; w_base += JOIN_THREADS) {
        const int w = w_base + tid;
        bool cut = false;
        int b = 0, unit = 0, last = 0, late = 0;
        if (w < split.n) {
            const int x = split.start(w);
            int lo = 0, hi = JOIN_THREADS;  // last slice that starts at or before x
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= x) lo = mid; else hi = mid;
            }
            int base = first[lo], nch = 0;
            for (b = lo * per;; b++) {
                nch = split_chunks<KB>(s.split, b);
                const int c = nch * s.split.units;
                if (x < base + c || b + 1 >= s.split.batch) break;
                base += c;
            }
            unit = (x - base) / nch;
            const int u0 = base + unit * nch, before = split.start(w - 1);
            cut = before <= u0 && u0 < x;
            late = before < u0;
            last = split.owner(u0 + nch - 1);
        }
        const uint64_t ballot = __ballot(cut);
        if (lane_id() == 0) wave_cuts[wave_id()] = __popcll(ballot);
        __syncthreads();
        int at = cuts + __popcll(ballot & ((1ull << lane_id()) - 1));
#pragma unroll
        for (int i = 0; i < JOIN_THREADS / WAVE; i++) {
            if (i < wave_id()) at += wave_cuts[i];
            cuts += wave_cuts[i];
        }
        if (cut) {
            cut_b[at] = b;
            cut_unit[at] = unit;
            cut_w0[at] = 2 * (w - 1) + late;
            cut_w1[at] = last;
        }
        __syncthreads();
    }
    if (cuts == 0) return;

    // With at least one workgroup per cut unit, `share` of them take turns at its steps of
    // JOIN_GROUPS / gpr rows (the grid's remainder has nothing to do); with fewer, each takes
    // whole units.
    const int share = max((int)gridDim.x / cuts, 1);
    if ((int)blockIdx.x >= cuts * share) return;
    const int group = tid >> 5, lane = tid & 31;
    const size_t rows_per_part = (size_t)s.row_tiles * s.tile;
    for (int u = (int)blockIdx.x % cuts; u < cuts; u += gridDim.x) {
        const int b = cut_b[u], unit = cut_unit[u];
        const int w0 = cut_w0[u] >> 1, late = cut_w0[u] & 1, w1 = cut_w1[u];
        const int parts = w1 - w0 + 1;
        int gpr = 1;  // groups per row
        while (gpr < JOIN_GROUPS && gpr < parts) gpr *= 2;
        const int rows_here = JOIN_GROUPS / gpr, turn = group & (gpr - 1);
        for (int step = (int)blockIdx.x / cuts; step * rows_here < s.rows; step += share) {
            const int row = step * rows_here + group / gpr;
            const bool live = row < s.rows;
            const int r = live ? row : 0;
            auto at = [&](int w) {
                return (size_t)(2 * w + (w == w0 ? late : 0)) * rows_per_part + r;
            };
            float top = -INFINITY;
            for (int w = w0 + lane; w <= w1; w += 32) top = fmaxf(top, s.part_ml[at(w) * 2]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 32));
            const float ref = top == -INFINITY ? 0.f : top;
            f32x4 x[NC];
#pragma unroll
            for (int c = 0; c < NC; c++) x[c] = zero4();
            float sum = 0.f;
#pragma unroll 2
            for (int w = w0 + turn; w <= w1; w += gpr) {
                const size_t e = at(w);
                const float f = __builtin_amdgcn_exp2f(s.part_ml[e * 2] - ref);
                sum = fmaf(f, s.part_ml[e * 2 + 1], sum);
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int col = c * 128 + lane * 4;
                    if (COLS % 128 != 0 && col >= COLS) continue;
                    const f32x4 y = *reinterpret_cast<const f32x4*>(s.part_o + e * COLS + col);
#pragma unroll
                    for (int i = 0; i < 4; i++) x[c][i] = fmaf(f, y[i], x[c][i]);
                }
            }
            if (gpr > 1) {  // uniform over the workgroup
#pragma unroll
                for (int c = 0; c < NC; c++)
                    *reinterpret_cast<f32x4*>(&red[group][c * 128 + lane * 4]) = x[c];
                if (lane == 0) red_l[group] = sum;
                __syncthreads();
                if (turn == 0)
                    for (int g = 1; g < gpr; g++) {
#pragma unroll
                        for (int c = 0; c < NC; c++) {
                            const f32x4 y = *reinterpret_cast<const f32x4*>(
                                &red[group + g][c * 128 + lane * 4]);
#pragma unroll
                            for (int i = 0; i < 4; i++) x[c][i] += y[i];
                        }
                        sum += red_l[group + g];
                    }
                __syncthreads();
            }
            if (turn == 0 && live) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int col = c * 128 + lane * 4;
                    if (COLS % 128 != 0 && col >= COLS) continue;
                    const float y[4] = {x[c][0] * inv, x[c][1] * inv, x[c][2] * inv, x[c][3] * inv};
                    store(b, unit, row, col, y);
                }
            }
        }
    }
}

}  // namespace gdn
