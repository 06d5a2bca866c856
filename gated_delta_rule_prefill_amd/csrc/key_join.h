// Joins the partial results that key_split.h's cut leaves: for each row of a cut unit
//   o = sum_w e^{m_w - M} acc_w / sum_w e^{m_w - M} l_w,   M = max_w m_w
// over the workers w that hold a part of it (exponentials to base 2, as the parts keep their
// maxima).
//
// Which units were cut only the device knows. The worker that starts a unit writes down whether
// it ended it too (JoinNote); notes are kept per unit when the call has no more units than
// workers, else per worker (a worker leaves at most one unit unfinished, its last). Each note
// gets `share` workgroups of the joining launch: a note of a whole unit costs them one read.
// A group of 32 lanes reads a whole row of one part at a time; a row with many parts gets up to
// eight groups (its sums meet in LDS in a fixed order), rows with few parts run side by side.
// Bound by latency: three dependent reads (note, maxima, parts). Measured: one request over 256
// workers, 20 rows of 512 columns, 7 us (12.4 with a row's parts read one after another); 80
// requests, 128 rows of 512 columns, 14 us; 128 requests, 32 rows of 128 columns, 5 us.
#pragma once
#include "key_split.h"

namespace gdn {

constexpr int JOIN_THREADS = 256;
constexpr int JOIN_GROUPS = JOIN_THREADS / 32;
constexpr int JOIN_MAX_WORKERS = 1024;  // most parts of a unit

struct JoinShape {
    int4* notes;          // [count]
    int count, share;     // share workgroups per note (and column slice)
    int slices;           // workgroups side by side along a row's columns
    int per_unit;         // notes are kept per unit (else per worker)
    int row_tiles, tile;  // row tiles of a worker, rows of a tile
    int rows;             // live rows of a unit, over its row tiles
    float* part_o;        // [2 workers][row_tiles][tile][COLS]
    float* part_ml;       // [2 workers][row_tiles][tile][2]
};
// Notes of a call and their workgroups: about 4 per CU, no more for a note than it has rows,
// and the columns split up too where that leaves CUs idle (one long request).
inline void join_layout(JoinShape* j, int64_t units, int workers, int cus, int cols) {
    j->per_unit = units <= workers;
    j->count = j->per_unit ? (int)units : workers;
    const int share = j->count > 0 ? 4 * cus / j->count : 1;
    j->share = share < 1 ? 1 : share < j->rows ? share : j->rows;
    const int slices = (cols + 127) / 128;
    j->slices = share >= j->rows * slices ? slices : 1;
}
inline unsigned join_grid(const JoinShape& j) { return (unsigned)(j.count * j.share * j.slices); }

// A note: request, unit, 2 (first worker) + (its part is in the late slot), last worker; -1 for
// the last worker of a unit that needs no joining.
__device__ __forceinline__ void join_none(const JoinShape& j, int note) {
    j.notes[note] = make_int4(0, 0, 0, -1);
}

// By one thread, at a unit's first chunk: [c0 = 0, c1) of nch chunks by this worker.
__device__ __forceinline__ void join_note(const JoinShape& j, const SplitShape& s,
                                          const SplitRun& run, int worker, int b, int unit,
                                          int c1, int nch, bool late) {
    if (c1 < nch)
        j.notes[j.per_unit ? b * s.units + unit : worker] =
            make_int4(b, unit, 2 * worker + (late ? 1 : 0), run.cut.owner(run.pos + nch - 1));
    else if (j.per_unit)
        join_none(j, b * s.units + unit);
}

// One workgroup's share of a note's rows, NC pieces of 128 columns from column `first` on, U
// parts on their way at a time per group.
template <int COLS, int NC, int U, typename Store>
__device__ __forceinline__ void join_rows(const JoinShape& s, int4 note, int step0, int first,
                                          Store store) {
    __shared__ float red[JOIN_GROUPS][NC * 128 + 4];
    __shared__ float weight[JOIN_MAX_WORKERS];
    __shared__ float wave_part[JOIN_THREADS / WAVE];
    const int b = note.x, unit = note.y, w0 = note.z >> 1, late = note.z & 1, w1 = note.w;
    const int tid = threadIdx.x, group = tid >> 5, lane = tid & 31;
    const size_t rows_per_part = (size_t)s.row_tiles * s.tile;
    const int parts = w1 - w0 + 1;
    int gpr = 1;  // groups per row: U parts each, if there are groups enough
    while (gpr < JOIN_GROUPS && gpr * U < parts) gpr *= 2;
    const int rows_here = JOIN_GROUPS / gpr, turn = group & (gpr - 1);
    for (int step = step0; step * rows_here < s.rows; step += s.share) {
        const int row = step * rows_here + group / gpr;
        const bool live = row < s.rows;
        const int r = live ? row : 0;
        auto at = [&](int i) {  // part i of the unit
            return (size_t)(2 * (w0 + i) + (i == 0 ? late : 0)) * rows_per_part + r;
        };
        // the parts' weights: lane i's is part i's, or all of them in LDS where a row has so
        // many that the whole workgroup shares it
        float f = 0.f, sum = 0.f;
        if (gpr < JOIN_GROUPS) {  // at most JOIN_GROUPS / 2 x U <= 32 parts
            float m = -INFINITY, l = 0.f;
            if (lane < parts) {
                m = s.part_ml[at(lane) * 2];
                l = s.part_ml[at(lane) * 2 + 1];
            }
            float top = m;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 32));
            f = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.f : top));
            sum = f * l;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 32);
        } else {
            constexpr int PER = JOIN_MAX_WORKERS / JOIN_THREADS;
            float m[PER], l[PER], top = -INFINITY;
#pragma unroll
            for (int k = 0; k < PER; k++) {
                const int i = k * JOIN_THREADS + tid;
                m[k] = i < parts ? s.part_ml[at(i) * 2] : -INFINITY;
                l[k] = i < parts ? s.part_ml[at(i) * 2 + 1] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < PER; k++) top = fmaxf(top, m[k]);
#pragma unroll
            for (int off = WAVE / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, WAVE));
            if (lane_id() == 0) wave_part[wave_id()] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < JOIN_THREADS / WAVE; i++) top = fmaxf(top, wave_part[i]);
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int k = 0; k < PER; k++) {
                const float w = __builtin_amdgcn_exp2f(m[k] - ref);
                weight[k * JOIN_THREADS + tid] = w;
                sum = fmaf(w, l[k], sum);
            }
#pragma unroll
            for (int off = WAVE / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, WAVE);
            __syncthreads();
            if (lane_id() == 0) wave_part[wave_id()] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < JOIN_THREADS / WAVE; i++) sum += wave_part[i];
        }
        f32x4 x[NC];
#pragma unroll
        for (int c = 0; c < NC; c++) x[c] = zero4();
        for (int i0 = turn; i0 < parts; i0 += U * gpr) {
            f32x4 y[U][NC];
            float g[U];
#pragma unroll
            for (int k = 0; k < U; k++) {  // (the surplus ones weigh nothing)
                const int i = i0 + k * gpr;
                g[k] = gpr < JOIN_GROUPS ? __shfl(f, i & 31, 32)
                                         : weight[min(i, JOIN_MAX_WORKERS - 1)];
                if (i >= parts) g[k] = 0.f;
                const float* src = s.part_o + at(min(i, parts - 1)) * COLS;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int col = first + c * 128 + lane * 4;
                    y[k][c] = COLS % 128 == 0 || col < COLS
                                  ? *reinterpret_cast<const f32x4*>(src + col) : zero4();
                }
            }
#pragma unroll
            for (int k = 0; k < U; k++)
#pragma unroll
                for (int c = 0; c < NC; c++)
#pragma unroll
                    for (int e = 0; e < 4; e++) x[c][e] = fmaf(g[k], y[k][c][e], x[c][e]);
        }
        if (gpr > 1) {  // uniform over the workgroup
#pragma unroll
            for (int c = 0; c < NC; c++)
                *reinterpret_cast<f32x4*>(&red[group][c * 128 + lane * 4]) = x[c];
            __syncthreads();
            if (turn == 0)
                for (int g = 1; g < gpr; g++)
#pragma unroll
                    for (int c = 0; c < NC; c++) {
                        const f32x4 y =
                            *reinterpret_cast<const f32x4*>(&red[group + g][c * 128 + lane * 4]);
#pragma unroll
                        for (int e = 0; e < 4; e++) x[c][e] += y[e];
                    }
            __syncthreads();
        }
        if (turn == 0 && live) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int col = first + c * 128 + lane * 4;
                if (COLS % 128 != 0 && col >= COLS) continue;
                const float y[4] = {x[c][0] * inv, x[c][1] * inv, x[c][2] * inv, x[c][3] * inv};
                store(b, unit, row, col, y);
            }
        }
    }
}

// store(b, unit, row, col, x[4]) takes 4 columns of a row of request b's unit.
template <int COLS, typename Store>
__device__ __forceinline__ void join_parts(const JoinShape& s, Store store) {
    constexpr int NC = (COLS + 127) / 128;
    const int per_note = s.share * s.slices;
    const int4 note = s.notes[blockIdx.x / per_note];
    if (note.w < 0) return;
    const int rest = blockIdx.x % per_note;
    if (s.slices == 1) {
        join_rows<COLS, NC, 4>(s, note, rest, 0, store);
    } else if constexpr (NC > 1) {
        join_rows<COLS, 1, 8>(s, note, rest / s.slices, rest % s.slices * 128, store);
    }
}

}  // namespace gdn
