// Joins the partial results that key_split.h's cut leaves: for each row of a cut unit
//   o = sum_w e^{m_w - M} acc_w / sum_w e^{m_w - M} l_w,   M = max_w m_w
// over the workgroups w that hold a part of it (exponentials to base 2, as the parts keep
// their maxima).
//
// Only cut units have work, and a launch cannot know which those are, so every workgroup lists
// them for itself (one look-up per workgroup boundary of the split: a boundary inside a unit
// cuts it, and the first such boundary stands for the unit) and takes its share of the list. A
// group of 32 lanes reads 128 columns of one part at a time; a row with many parts gets up to
// eight groups (its sums meet in LDS in a fixed order), rows with few parts run side by side.
// Bound by latency (two dependent reads), so the grid is a few workgroups per CU and each
// makes few passes.
#pragma once
#include "key_split.h"

namespace gdn {

constexpr int JOIN_THREADS = 256;
constexpr int JOIN_GROUPS = JOIN_THREADS / 32;
constexpr int JOIN_COLS = 128;     // columns of a pass: 32 lanes x 4
constexpr int JOIN_MAX_WG = 1024;  // most workgroups of a split that can be joined

struct JoinShape {
    SplitShape split;
    int n_wg;
    int tile;            // rows of a unit's tile in the parts
    int rows;            // most live rows of a unit
    int cols;            // columns of a row
    const float* part_o;  // [2 n_wg][tile][cols]
    const float* part_ml;  // [2 n_wg][tile][2]
};

// rows_of(unit): live rows of that unit; store(b, unit, row, col, x[4]); zero(b) is called by
// all threads of one workgroup for every request without keys.
template <int KB, typename Rows, typename Store, typename Zero>
__device__ __forceinline__ void join_parts(const JoinShape& s, Rows rows_of, Store store,
                                           Zero zero) {
    __shared__ int64_t first[JOIN_THREADS + 1];  // chunks before each thread's requests
    __shared__ int64_t wave_tot[JOIN_THREADS / WAVE];
    __shared__ int cut_b[JOIN_MAX_WG], cut_unit[JOIN_MAX_WG];
    __shared__ int cut_w0[JOIN_MAX_WG];  // 2 (first workgroup) + (its part is in the late slot)
    __shared__ int cut_w1[JOIN_MAX_WG];  // last workgroup
    __shared__ int wave_cuts[JOIN_THREADS / WAVE];
    __shared__ float red[JOIN_GROUPS][JOIN_COLS + 4];
    __shared__ float red_l[JOIN_GROUPS];
    const int tid = threadIdx.x;
    const int per = (s.split.batch + JOIN_THREADS - 1) / JOIN_THREADS;
    const int b0 = min(tid * per, s.split.batch), b1 = min(b0 + per, s.split.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; b++) mine += split_chunks<KB>(s.split, b);
    mine *= s.split.units;
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
    for (int i = 0; i < JOIN_THREADS / WAVE; i++) {
        if (i < wave_id()) upto += wave_tot[i];
        total += wave_tot[i];
    }
    first[tid + 1] = upto;
    if (tid == 0) first[0] = 0;
    __syncthreads();

    for (int b = blockIdx.x; b < s.split.batch; b += gridDim.x)
        if (split_keys(s.split, b) == 0) zero(b);

    const int n = split_wgs(total, s.n_wg);
    int cuts = 0;
    for (int w_base = 1; w_base < n; w_base += JOIN_THREADS) {
        const int w = w_base + tid;
        bool cut = false;
        int b = 0, unit = 0, last = 0, late = 0;
        if (w < n) {
            const int64_t x = split_start(w, total, n);
            int lo = 0, hi = JOIN_THREADS;  // last slice that starts at or before x
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= x) lo = mid; else hi = mid;
            }
            int64_t base = first[lo];
            int nch = 0;
            for (b = lo * per;; b++) {
                nch = split_chunks<KB>(s.split, b);
                const int64_t c = (int64_t)nch * s.split.units;
                if (x < base + c || b + 1 >= s.split.batch) break;
                base += c;
            }
            unit = (int)((x - base) / nch);
            const int64_t u0 = base + (int64_t)unit * nch;
            const int64_t before = split_start(w - 1, total, n);
            cut = before <= u0 && u0 < x;
            late = before < u0;
            last = split_owner(u0 + nch - 1, total, n);
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

    const int slices = (s.cols + JOIN_COLS - 1) / JOIN_COLS;
    const int group = tid >> 5, lane = tid & 31;
    // a pass: one cut unit, one column slice, JOIN_GROUPS / gpr of its rows (passes are numbered
    // as if gpr were JOIN_GROUPS; surplus numbers fall through). Neighbouring workgroups take
    // different units.
    const int64_t passes = (int64_t)cuts * slices * s.rows;
    for (int64_t pass = blockIdx.x; pass < passes; pass += gridDim.x) {
        const int u = (int)(pass % cuts), rest = (int)(pass / cuts);
        const int slice = rest % slices, step = rest / slices;
        const int b = cut_b[u], unit = cut_unit[u];
        const int w0 = cut_w0[u] >> 1, late = cut_w0[u] & 1, w1 = cut_w1[u];
        const int parts = w1 - w0 + 1;
        int gpr = 1;  // groups per row
        while (gpr < JOIN_GROUPS && gpr < parts) gpr *= 2;
        const int rows_here = JOIN_GROUPS / gpr;
        const int rows = rows_of(unit);
        if (step * rows_here >= rows) continue;  // uniform over the workgroup
        const int row = step * rows_here + group / gpr, turn = group % gpr;
        const bool live = row < rows;
        const int r = live ? row : 0;
        auto at = [&](int w) { return (size_t)(2 * w + (w == w0 ? late : 0)) * s.tile + r; };
        float top = -INFINITY;
        for (int w = w0 + lane; w <= w1; w += 32) top = fmaxf(top, s.part_ml[at(w) * 2]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 32));
        const float ref = top == -INFINITY ? 0.f : top;
        const int col = slice * JOIN_COLS + lane * 4;
        const bool in_row = col < s.cols;
        f32x4 x = zero4();
        float sum = 0.f;
#pragma unroll 4
        for (int w = w0 + turn; w <= w1; w += gpr) {
            const size_t e = at(w);
            const float f = __builtin_amdgcn_exp2f(s.part_ml[e * 2] - ref);
            sum = fmaf(f, s.part_ml[e * 2 + 1], sum);
            const f32x4 y = in_row ? *reinterpret_cast<const f32x4*>(s.part_o + e * s.cols + col)
                                   : zero4();
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] = fmaf(f, y[i], x[i]);
        }
        if (gpr > 1) {
            *reinterpret_cast<f32x4*>(&red[group][lane * 4]) = x;
            if (lane == 0) red_l[group] = sum;
            __syncthreads();
            if (turn == 0)
                for (int g = 1; g < gpr; g++) {
                    const f32x4 y = *reinterpret_cast<const f32x4*>(&red[group + g][lane * 4]);
#pragma unroll
                    for (int i = 0; i < 4; i++) x[i] += y[i];
                    sum += red_l[group + g];
                }
            __syncthreads();
        }
        if (turn == 0 && live && in_row) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = x[i] * inv;
            store(b, unit, row, col, y);
        }
    }
}

}  // namespace gdn
