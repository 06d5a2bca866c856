// Attention of many query rows over a paged key/value cache, grouped heads: the kernel of
// gdn_paged_prefill (packed prompts, causal) and of the shared part of gdn_paged_shared_decode.
//
// Query rows that share a key/value head (tokens x group) are packed into tiles of 128 or 256, so
// that the keys are read once for all heads of a group, and a causal tile of few tokens reaches
// little beyond its own diagonal. A tile and a key/value head make a unit; the 64-key steps
// (32 in fp32) of all units are laid end to end and cut into equal runs, one per worker, one
// worker a CU: work is even to a few steps whatever the lengths, which are device data. A unit
// cut between workers leaves partial results (key_join.h's form) that a joining launch combines.
//
// Per step and wave, for its 32 rows (16 in fp32):
//   S^T = K Q^T     queries in registers as the MFMA's B operand, so that a query is an accumulator
//                   column: a lane's scores are reduced in registers, then over its partners;
//   O^T += V^T P^T  the accumulator layout of S^T is the B operand's with the keys renumbered, so
//                   weights stay in registers; V^T comes from transposing LDS reads (bf16) or
//                   column reads (fp32).
// Keys and values go from their pages straight into LDS, two or three buffers each, the keys one
// step ahead of the values: a step's scores (matrix pipe) are formed beside the previous step's
// softmax (vector pipe), with one barrier a step. Rows that do not exist are loaded from a row of
// zeros: a zero weight would not cancel what a page's unused rows hold.
//
// Bound (bf16): by no unit alone. 12000 tokens, 32 heads, 8 KV heads, d = 128 (1.18 TFLOP): 1250-1360
// us, 0.87-0.94 PFLOP/s (a 16384^3 product on the same chips 1.37-1.57); counters: matrix pipe busy for
// 49 % of the cycles, the vector pipe for 47 %, LDS for 39 %. A step is 2048 cycles of matrix work a SIMD
// and takes 4200 (2.28 us at the 1.8 GHz of a full chip; with a quarter of the CUs at work 1.84 us, which
// is as many at 2.3 GHz): both waves of a SIMD pass the same barrier and are in the same phase, so that
// a step's scores, softmax and values wait for each other. Leaving work out therefore moves the time little: no
// tile loads 10 %, no exponentials 5 %, no score products 15 %; more of it adds its part (products for
// the rests of the weights 16 %, forming those 7 %). 24 turns of 3 to 1500 tokens behind up to 16000,
// 32 heads, 4 KV heads: 610-665 us, 0.70-0.77 PFLOP/s; 128 requests behind 32000 shared tokens 84-89
// us, 0.8 (matrix pipe 40 %); groups of 6 behind 500 to 16000 tokens, 16 heads of 256, 52-53 us (18 %: one
// wave a SIMD, and second tiles of few rows that take a whole unit's steps). fp32 is bound by its
// matrix instructions (a step of 32 keys 1.8 us at d = 64 and full tiles, by their rate).
#pragma once
#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"
#include "key_join.h"
#include "lds_tile.h"

namespace gdn {

constexpr uint32_t AT_NO_ROW = 0xffffffffu;
constexpr float AT_LOG2E = 1.4426950408889634f;

static __device__ __align__(16) char at_zero_row[1024];  // the longest row

typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------ one wave's arithmetic
// A step's pieces in LDS lie row by row, 16-byte pieces turned by a function of their row.
template <typename T, int D> struct AttendTile;

template <int D> struct AttendTile<bf16, D> {
    // One wave a SIMD at d = 256 (outputs and queries alone take 192 registers), else two. (Waves
    // of 64 rows, one a SIMD, halve the LDS reads, and lose more: a prompt of 12000 tokens, 32
    // heads, 1860 us in steps of 32 keys, and 3160 with 64, where registers spill; 1290 with two.)
    static constexpr int WAVE_ROWS = 32, KB = 64;
    static constexpr int WAVES = D == 256 ? 4 : 8, WAVES_PER_SIMD = WAVES / 4;
    static constexpr int ROW = D * 2, PIECES = ROW / 16;
    // Steps that keys and values are loaded ahead of the one that waits for them: the first pieces
    // of a step's keys can then be read before its barrier. (Three buffers each; at d = 256 two
    // fit.)
    static constexpr int LEAD = D == 256 ? 0 : 1;
    static constexpr int NQ = D / 16, NO = D / 32, NV = KB / 16 * NO;
    static constexpr int AHEAD = D == 256 ? 3 : 2;  // pieces on their way (3 spill at d = 128)
    static constexpr bool INTERLEAVED = true;
    struct Scores {
        f32x16 v[2];
        __device__ __forceinline__ float get(int n) const { return v[n >> 4][n & 15]; }
        __device__ __forceinline__ void set(int n, float z) { v[n >> 4][n & 15] = z; }
    };
    static constexpr int N = 32;  // scores of a lane
    bf16x8 q[NQ];
    f32x16 acc[NO];
    bf16x8 kf[AHEAD + 1][2], vf[AHEAD + 1];

    __device__ __forceinline__ static int k_turn(int r) { return D >= 128 ? r & 15 : (r >> 1) & 7; }
    // (pairs of pieces: a transposing read takes 32 bytes of each of 8 rows, twice side by side)
    __device__ __forceinline__ static int v_turn(int r) {
        return (D >= 128 ? r & 7 : (r >> 1) & 3) << 1;
    }
    __device__ __forceinline__ static int row_of_lane(int lane) { return lane & 31; }
    __device__ __forceinline__ static int first_key(int lane) { return (lane >> 5) * 4; }
    __device__ __forceinline__ static int key(int n) {  // of score n, + first_key
        return (n >> 4) * 32 + ((n & 15) >> 2) * 8 + (n & 3);
    }
    __device__ __forceinline__ static float max_partners(float x) { return max_halves(x); }
    __device__ __forceinline__ static float sum_partners(float x) {
        return x + __shfl_xor(x, 32, WAVE);
    }
    __device__ __forceinline__ void load_q(const bf16* src, int lane, float sign) {
#pragma unroll
        for (int f = 0; f < NQ; f++) q[f] = Mma<bf16>::load(src + f * 16 + (lane >> 5) * 8);
        if (sign != 1.f) {
#pragma unroll
            for (int f = 0; f < NQ; f++)
#pragma unroll
                for (int i = 0; i < 8; i++) q[f][i] = (bf16)(sign == 0.f ? 0.f : -(float)q[f][i]);
        }
        arrived(q);
    }
    __device__ __forceinline__ static f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // Places of this lane's first pieces in the tiles at `kt` and `vt`.
    __device__ __forceinline__ static uint32_t key_place(uint32_t kt, int lane) {
        const int r = lane & 31;
        uint32_t at = kt + r * ROW + (((lane >> 5) ^ k_turn(r)) << 4);
        asm volatile("" : "+v"(at));  // (formed here: one register, not one for each piece)
        return at;
    }
    __device__ __forceinline__ static uint32_t value_place(uint32_t vt, int lane) {
        // lanes 0-15 and 16-31 read 16 columns each of 4 keys, the upper half of the next 4
        const int r = (lane >> 5) * 4 + ((lane >> 2) & 3);
        uint32_t at = vt + r * ROW + ((((lane >> 4) & 1) << 5) ^ (v_turn(r) << 4)) + (lane & 3) * 8;
        asm volatile("" : "+v"(at));
        return at;
    }
    __device__ __forceinline__ void load_key(uint32_t at, int f) {
#pragma unroll
        for (int x = 0; x < 2; x++)  // (32 rows on, the pieces are turned alike)
            kf[f % (AHEAD + 1)][x] = lds_get<bf16x8>((at ^ (f << 5)) + x * 32 * ROW);
    }
    __device__ __forceinline__ void load_value(uint32_t at, int n) {
        // keys 16 g + r and 16 g + 8 + r: rows 8 on are turned alike
        const uint32_t x = (at ^ (n % NO << 6)) + n / NO * 16 * ROW;
        vf[n % (AHEAD + 1)] = join(lds_read_tr(x), lds_read_tr(x + 8 * ROW));
    }
    // The first pieces of a tile, ahead of scores() and values().
    __device__ __forceinline__ void start_keys(uint32_t kt, int lane) {
        const uint32_t at = key_place(kt, lane);
#pragma unroll
        for (int f = 0; f < AHEAD; f++) load_key(at, f);
    }
    __device__ __forceinline__ void start_values(uint32_t vt, int lane) {
        const uint32_t at = value_place(vt, lane);
#pragma unroll
        for (int n = 0; n < AHEAD; n++) load_value(at, n);
    }
    // Scores of the keys at `kt`. beside(m) is other work for the time of MFMA m (32 cycles, in
    // which the wave can issue eight vector instructions); the fences keep the compiler from taking
    // the two apart again.
    static constexpr int SCORE_MFMAS = NQ * 2, VALUE_MFMAS = NV;
    template <typename Beside>
    __device__ __forceinline__ void scores(uint32_t kt, int lane, Scores& s, Beside beside) {
        const uint32_t at = key_place(kt, lane);
        f32x16 zero;
#pragma unroll
        for (int i = 0; i < 16; i++) zero[i] = 0.f;
#pragma unroll
        for (int f = 0; f < NQ; f++) {
            if (f + AHEAD < NQ) load_key(at, f + AHEAD);
#pragma unroll
            for (int x = 0; x < 2; x++) {
                s.v[x] = mma(kf[f % (AHEAD + 1)][x], q[f], f == 0 ? zero : s.v[x]);
                beside(f * 2 + x);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // l + the weights p.
    __device__ __forceinline__ static float add(const bf16x8& p, float l) {
        typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 ones = {(bf16)1.f, (bf16)1.f};
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{p[i], p[i + 1]}, ones, l, false);
        return l;
    }
    // acc += V^T P^T for the weights s, l += their sum. The weights are rounded to bf16 (2^-8 of
    // each at most) as the MFMA's operand, and the sum takes them as rounded: what is left of the
    // roundings is weighted by a value's distance from the output, so that a weight that outweighs
    // the others has none (relative 2-norm errors 0.0017-0.0021 where one rounding of the outputs
    // leaves 0.0016-0.0017, 0.0017-0.0022 with the sum of the weights before rounding; 1 % of a
    // call's time). To keep all of a weight costs more than it gives: as the sum of two bf16
    // numbers 0.00165, but 12000 tokens take 1670 us instead of 1303, 128 requests behind 32000
    // tokens 172 instead of 151; with the second part in 6 bits, whose products are a quarter as
    // dear but want the values in 6 bits too, 1641 and 176.
    // Weights of the second half of the keys may be formed in beside(m) until m = VALUE_MFMAS * 5 / 8.
    template <typename Beside>
    __device__ __forceinline__ void values(uint32_t vt, int lane, Scores& s, float& l,
                                           Beside beside) {
        const uint32_t at = value_place(vt, lane);
        bf16x8 p;
#pragma unroll
        for (int n = 0; n < NV; n++) {
            if (n + AHEAD < NV) load_value(at, n + AHEAD);
            if (n % NO == 0)
#pragma unroll
                for (int i = 0; i < 8; i++) p[i] = (bf16)s.get(n / NO * 8 + i);
            if (n % NO == NO - 1) l = add(p, l);
            acc[n % NO] = mma(vf[n % (AHEAD + 1)], p, acc[n % NO]);
            beside(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < NO; j++)
#pragma unroll
            for (int i = 0; i < 16; i++) acc[j][i] = 0.f;
    }
    __device__ __forceinline__ void shrink(float f) {
#pragma unroll
        for (int j = 0; j < NO; j++)
#pragma unroll
            for (int i = 0; i < 16; i++) acc[j][i] *= f;
    }
    // store(column, x[4]) for this lane's pieces of its row, times f
    template <typename Store>
    __device__ __forceinline__ void results(int lane, float f, Store store) const {
#pragma unroll
        for (int j = 0; j < NO; j++)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float y[4] = {acc[j][i] * f, acc[j][i + 1] * f, acc[j][i + 2] * f,
                                    acc[j][i + 3] * f};
                store(j * 32 + (i >> 2) * 8 + (lane >> 5) * 4, y);
            }
    }
};

template <int D> struct AttendTile<float, D> {
    static constexpr int WAVES = 8, WAVES_PER_SIMD = 2;
    static constexpr int WAVE_ROWS = 16, KB = 32;
    static constexpr int ROW = D * 4, PIECES = ROW / 16;
    static constexpr int LEAD = 0;
    static constexpr int NQ = D / 16, NO = D / 16;
    static constexpr bool INTERLEAVED = false;
    struct Scores {
        f32x4 v[2];
        __device__ __forceinline__ float get(int n) const { return v[n >> 2][n & 3]; }
        __device__ __forceinline__ void set(int n, float z) { v[n >> 2][n & 3] = z; }
    };
    static constexpr int N = 8;
    f32x4 q[NQ];
    f32x4 acc[NO];

    __device__ __forceinline__ static int k_turn(int r) { return r & 15; }
    // (a column read takes 64 bytes of each of 4 rows 4 apart)
    __device__ __forceinline__ static int v_turn(int r) { return ((r >> 2) & 3) << 2; }
    __device__ __forceinline__ static int row_of_lane(int lane) { return lane & 15; }
    __device__ __forceinline__ static int first_key(int lane) { return (lane >> 4) * 4; }
    __device__ __forceinline__ static int key(int n) { return (n >> 2) * 16 + (n & 3); }
    __device__ __forceinline__ static float max_partners(float x) { return max_groups(x); }
    __device__ __forceinline__ static float sum_partners(float x) {
        x += __shfl_xor(x, 16, WAVE);
        return x + __shfl_xor(x, 32, WAVE);
    }
    __device__ __forceinline__ void load_q(const float* src, int lane, float sign) {
#pragma unroll
        for (int f = 0; f < NQ; f++)
            q[f] = sign == 0.f ? zero4()
                               : *reinterpret_cast<const f32x4*>(src + f * 16 + (lane >> 4) * 4) * sign;
#pragma unroll
        for (int f = 0; f < NQ; f++) asm volatile("" : "+v"(q[f]));  // as arrived()
    }
    __device__ __forceinline__ void start_keys(uint32_t, int) {}
    template <typename Beside>
    __device__ __forceinline__ void scores(uint32_t kt, int lane, Scores& s, Beside) {
        const int r = lane & 15;
        uint32_t at = kt + r * ROW + (((lane >> 4) ^ k_turn(r)) << 4);
        asm volatile("" : "+v"(at));
        s.v[0] = zero4();
        s.v[1] = zero4();
#pragma unroll
        for (int f = 0; f < NQ; f++)
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const f32x4 k = lds_get<f32x4>((at ^ (f << 6)) + x * 16 * ROW);
#pragma unroll
                for (int e = 0; e < 4; e++) s.v[x] = Mma<float>::mma(k[e], q[f][e], s.v[x]);
            }
    }
    // A step's sums are formed by themselves and added once: a long sequence is then summed in
    // two levels, and the roundings of n / 32 additions reach a result instead of those of n / 4.
    template <typename Beside>
    __device__ __forceinline__ void values(uint32_t vt, int lane, Scores& s, float& l, Beside) {
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < N; n++) sum += s.get(n);
        l += sum;
        constexpr int JN = 2;  // columns of tiles on their way
        const uint32_t at = vt + (lane >> 4) * 4 * ROW + (lane & 15) * 4;
#pragma unroll
        for (int j0 = 0; j0 < NO; j0 += JN) {
            f32x4 sum[JN];
#pragma unroll
            for (int j = 0; j < JN; j++) sum[j] = zero4();
#pragma unroll
            for (int n = 0; n < N; n++)
#pragma unroll
                for (int j = 0; j < JN; j++)
                    sum[j] = Mma<float>::mma(
                        lds_get<float>(at + key(n) * ROW +
                                       ((((j0 + j) << 2) ^ v_turn((lane >> 4) * 4)) << 4)),
                        s.get(n), sum[j]);
#pragma unroll
            for (int j = 0; j < JN; j++) acc[j0 + j] += sum[j];
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < NO; j++) acc[j] = zero4();
    }
    __device__ __forceinline__ void shrink(float f) {
#pragma unroll
        for (int j = 0; j < NO; j++) acc[j] *= f;
    }
    template <typename Store>
    __device__ __forceinline__ void results(int lane, float f, Store store) const {
#pragma unroll
        for (int j = 0; j < NO; j++) {
            const float y[4] = {acc[j][0] * f, acc[j][1] * f, acc[j][2] * f, acc[j][3] * f};
            store(j * 16 + (lane >> 4) * 4, y);
        }
    }
};

template <typename T, int D>
constexpr int ATTEND_ROWS = AttendTile<T, D>::WAVES * AttendTile<T, D>::WAVE_ROWS;

// ------------------------------------------------------------------------------- the units
// Positions in the stream that a unit has beyond its steps: its start and end take as long.
constexpr int ATTEND_EXTRA = 2;
// No worker is given fewer positions than this: a run's start, and the parts that a cut leaves to
// be joined, cost as much (three turns of 5 to 200 tokens, fp32: 29.7 us a call with 1, 25.7 with 2,
// 28.4 with 3, 30.7 with 4, 42.5 with 8; not measured elsewhere: longer streams have longer runs).
constexpr int ATTEND_MIN_RUN = 2;
static_assert(ATTEND_MIN_RUN <= ATTEND_EXTRA, "a stream of one unit has a run");

// The stream of all units (total positions) cut over the workers, the longer runs spread evenly
// among them: where units are equally long and their number divides the workers', as with one
// prefix that all share, the tiles of a head are cut alike, and the workers that read the same
// keys do so at the same time.
struct AttendCut {
    int64_t total;
    int n;
    __device__ __forceinline__ static AttendCut of(int64_t total, int workers) {
        const int64_t n = total / ATTEND_MIN_RUN;  // (a unit alone has ATTEND_EXTRA positions)
        return {total, (int)(n < workers ? n : workers)};
    }
    __device__ __forceinline__ int64_t start(int w) const { return w * total / n; }
    // the last w with start(w) <= x
    __device__ __forceinline__ int owner(int64_t x) const {
        return (int)(((x + 1) * n - 1) / total);
    }
};

// Rows of a tile, for the host.
inline int attend_tile_rows(int dtype, int d) { return dtype == 0 || d == 256 ? 128 : 256; }

// Sections of a workspace, 256 bytes apart.
struct Layout {
    char* base;
    size_t size = 0;
    explicit Layout(void* ws) : base(static_cast<char*>(ws)) {}
    template <typename V> V* take(size_t n) {
        V* p = base == nullptr ? nullptr : reinterpret_cast<V*>(base + size);
        size += (n * sizeof(V) + 255) & ~(size_t)255;
        return p;
    }
};
inline void attend_table_layout(AttendArgs* a, Layout* l) {
    a->head = l->take<int32_t>(1);
    a->total = l->take<int64_t>(1);
    a->seq_tile = l->take<int32_t>((size_t)a->n_seqs + 1);
    a->first = l->take<int64_t>((size_t)a->tiles + 1);
    a->tile = l->take<AttendUnit>((size_t)a->tiles);
}

// One workgroup lays out the tiles: rows_of(i) of each sequence, then each tile's unit.
// Sums that the host's bound does not hold (lengths that break the contract) are cut off there.
constexpr int AT_TABLE_THREADS = 1024;
constexpr int AT_TABLE_SEQS = 2048;  // sequences whose bounds are kept in LDS for the searches

// The last i < n with first(i) <= x.
template <typename First>
__device__ __forceinline__ int last_at(int n, int x, First first) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
}

template <typename RowsOf, typename UnitOf>
__device__ __forceinline__ void attend_tables(const AttendArgs& a, int rows_a_tile, int kb,
                                              RowsOf rows_of, UnitOf unit_of) {
    __shared__ int64_t part[AT_TABLE_THREADS / WAVE];
    __shared__ int near_tile[AT_TABLE_SEQS];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const bool near = a.n_seqs <= AT_TABLE_SEQS;
    auto scan = [&](int64_t x, int64_t* total) {  // exclusive
        int64_t upto = x;
#pragma unroll
        for (int off = 1; off < WAVE; off <<= 1) {
            const int64_t t = __shfl_up(upto, off, WAVE);
            if (lane >= off) upto += t;
        }
        __syncthreads();
        if (lane == WAVE - 1) part[wave] = upto;
        __syncthreads();
        int64_t before = 0, all = 0;
        for (int w = 0; w < AT_TABLE_THREADS / WAVE; w++) {
            if (w < wave) before += part[w];
            all += part[w];
        }
        *total = all;
        return before + upto - x;
    };
    auto tiles_of = [&](int i) {
        return ((int64_t)rows_of(i) + rows_a_tile - 1) / rows_a_tile;
    };
    const int per = (a.n_seqs + AT_TABLE_THREADS - 1) / AT_TABLE_THREADS;
    const int i0 = (int)min((int64_t)tid * per, (int64_t)a.n_seqs), i1 = min(i0 + per, a.n_seqs);
    int64_t mine = 0, all;
    for (int i = i0; i < i1; i++) mine += tiles_of(i);
    int64_t at = scan(mine, &all);
    for (int i = i0; i < i1; i++) {
        const int t = (int)min(at, (int64_t)a.tiles);
        a.seq_tile[i] = t;
        if (near) near_tile[i] = t;
        if (i + 1 < i1) at += tiles_of(i);
    }
    const int n_tiles = (int)min(all, (int64_t)a.tiles);
    if (tid == 0) a.seq_tile[a.n_seqs] = n_tiles;
    if (!near) __threadfence();
    __syncthreads();
    int64_t base = 0;
    for (int t0 = 0; t0 < n_tiles; t0 += AT_TABLE_THREADS) {
        const int t = t0 + tid;
        int64_t len = 0;
        if (t < n_tiles) {
            auto tile_of = [&](int i) { return near ? near_tile[i] : a.seq_tile[i]; };
            const int i = last_at(a.n_seqs, t, tile_of);
            const AttendUnit u = unit_of(i, (t - tile_of(i)) * rows_a_tile);
            a.tile[t] = u;
            len = (u.reach + kb - 1) / kb + ATTEND_EXTRA;
        }
        int64_t block;
        const int64_t first = base + scan(len, &block);
        if (t < n_tiles) a.first[t] = first;
        base += block;
    }
    if (tid == 0) {
        a.first[n_tiles] = base;
        a.head[0] = n_tiles;
        a.total[0] = base;
    }
}

// ------------------------------------------------------------------------------ the kernel
// SHARED: the rows are decode positions of a group's requests, whose results are always parts;
// else tokens of a prompt, causal.
template <typename T, int D, bool SHARED>
__global__ __launch_bounds__((AttendTile<T, D>::WAVES * WAVE), (AttendTile<T, D>::WAVES_PER_SIMD))
void paged_attend_kernel(AttendArgs a) {
    using X = AttendTile<T, D>;
    using Scores = typename X::Scores;
    constexpr int THREADS = X::WAVES * WAVE, KB = X::KB, ROW = X::ROW, N = X::N;
    constexpr int ROWS = ATTEND_ROWS<T, D>, LEAD = X::LEAD, NB = 2 + LEAD;
    constexpr int LOADS = KB * ROW / 1024 / X::WAVES;  // 1 KiB loads of a wave per tile
    constexpr int ROWS_A_LOAD = 1024 / ROW;
    constexpr uint64_t ALL = KB == 64 ? ~0ull : (1ull << (KB & 63)) - 1;
    __shared__ __align__(1024) char k_tile[NB][KB * ROW];
    __shared__ __align__(1024) char v_tile[NB][KB * ROW];
    __shared__ uint32_t key_row[8][KB];  // cache rows of the next steps' keys
    __shared__ uint64_t key_exists[8];   // a bit per key
    __shared__ int found;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(wave_id());
    // neighbours in the stream read the same keys: they sit on one XCD
    const int w = (int)(blockIdx.x & 7) * (a.workers >> 3) + (int)(blockIdx.x >> 3);
    const int n_tiles = a.head[0];
    const int64_t total = a.total[0];
    const AttendCut cut = AttendCut::of(total * a.kv_heads, a.workers);
    if constexpr (!SHARED)
        if (tid == 0) join_none(a.join, w);
    if (w >= cut.n) return;
    int64_t pos = cut.start(w);
    const int64_t run_start = pos, end = cut.start(w + 1);
    int kvh = (int)(pos / total);
    {
        const int64_t x = pos - kvh * total;
        for (int t = tid; t < n_tiles; t += THREADS)
            if (a.first[t] <= x && x < a.first[t + 1]) found = t;
        __syncthreads();
    }
    int t = uniform(found);
    const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
    // The scale enters the exponent's multiplication; a negative one is moved into the queries, so
    // that the largest score is the largest weight (and zero makes the queries zero).
    const float cs = a.scale == 0.f ? 1.f : fabsf(a.scale) * AT_LOG2E;
    const T* k_cache = reinterpret_cast<const T*>(a.k_cache);
    const T* v_cache = reinterpret_cast<const T*>(a.v_cache);
    auto keys_at = [&](int c) { return lds_offset(k_tile[LEAD ? c % NB : c & 1]); };
    auto values_at = [&](int c) { return lds_offset(v_tile[LEAD ? c % NB : c & 1]); };

    for (; pos < end; t + 1 < n_tiles ? t++ : (t = 0, kvh++)) {
        const AttendUnit u = a.tile[t];
        const int64_t unit_start = kvh * total + a.first[t];
        const int reach = uniform(u.reach);
        const int nch = (reach + KB - 1) / KB;
        const int c0 = (int)(pos - unit_start);
        const int64_t unit_next = unit_start + nch + ATTEND_EXTRA;
        if (c0 >= nch && c0 > 0) {  // the run starts behind the unit's own steps
            pos = unit_next;
            continue;
        }
        const int c1 = (int)min((int64_t)nch, c0 + (end - pos));
        const int32_t* table = a.block_table + (size_t)uniform(u.seq) * a.max_blocks;
        const bool late = pos != run_start;

        X x;
        const int tile_row = wave * X::WAVE_ROWS + X::row_of_lane(lane);  // of this lane
        const bool live = u.row0 + tile_row < u.rows;
        const int row = live ? u.row0 + tile_row : u.rows - 1;
        const int tok = (int)a.by_group((uint32_t)row);
        const size_t q_row = (size_t)(u.token0 + tok) * a.H + kvh * a.group + (row - tok * a.group);
        x.load_q(reinterpret_cast<const T*>(a.q) + q_row * D, lane, sign);
        int lim;  // keys that the row sees
        if constexpr (SHARED) {
            const int b = (int)a.by_pos((uint32_t)(u.token0 + tok));
            lim = max(a.seq_lens[b], 0) - a.n_pos + (u.token0 + tok - b * a.n_pos) + 1;
        } else {
            lim = u.pos0 + tok + 1;
        }
        int low = lim, high = lim;
#pragma unroll
        for (int off = X::WAVE_ROWS / 2; off > 0; off >>= 1) {
            low = min(low, __shfl_xor(low, off, WAVE));
            high = max(high, __shfl_xor(high, off, WAVE));
        }
        low = uniform(low);
        // steps that this wave's rows see
        const bool any = u.row0 + wave * X::WAVE_ROWS < u.rows;
        const int mine = uniform(any ? min(c1, (max(min(high, reach), 0) + KB - 1) / KB) : 0);

        // The waves take turns in looking up the pages of a step: a table entry is asked for in one
        // step, its keys' rows put down in the next, read in the one after, and loaded from in the
        // fourth.
        auto page_of = [&](int c) {
            const uint32_t key = (uint32_t)(c * KB + lane);
            return table[min(a.block(key), (uint32_t)a.max_blocks - 1)];
        };
        auto put_rows = [&](int c, int page) {
            const uint32_t key = (uint32_t)(c * KB + lane), off = key - a.block(key) * a.block.div;
            const bool ok = lane < KB && (int)key < reach && page >= 0 && page < a.n_blocks;
            const uint32_t r = ((uint32_t)page * a.kv_heads + kvh) * a.block.div + off;
            if (lane < KB) key_row[c & 7][lane] = ok ? r : AT_NO_ROW;
            const uint64_t exist = __ballot(ok);
            if (lane == 0) key_exists[c & 7] = exist;
        };
        // Cache rows of the loads to come, read a step ahead where they are few registers.
        constexpr bool ROWS_EARLY = LOADS <= 4;
        uint32_t k_rows[LOADS], v_rows[LOADS];
        auto rows_of = [&](int c, uint32_t (&rows)[LOADS]) {
#pragma unroll
            for (int i = 0; i < LOADS; i++)
                rows[i] = key_row[c & 7][(wave * LOADS + i) * ROWS_A_LOAD + lane / X::PIECES];
        };
        auto load = [&](const T* cache, uint32_t from, int i, uint32_t lds, auto turn) {
            const int r = (wave * LOADS + i) * ROWS_A_LOAD + lane / X::PIECES;
            const int piece = (lane % X::PIECES) ^ turn(r);
            const char* base = from == AT_NO_ROW
                ? at_zero_row : reinterpret_cast<const char*>(cache + (size_t)from * D);
            load_to_lds(base + piece * 16, lds + (wave * LOADS + i) * 1024);
        };
        auto load_key = [&](int c, int i) {
            load(k_cache, k_rows[i], i, keys_at(c), [](int r) { return X::k_turn(r); });
        };
        auto load_value = [&](int c, int i) {
            load(v_cache, v_rows[i], i, values_at(c), [](int r) { return X::v_turn(r); });
        };
        auto load_keys = [&](int c) {
#pragma unroll
            for (int i = 0; i < LOADS; i++) load_key(c, i);
        };
        auto load_values = [&](int c) {
#pragma unroll
            for (int i = 0; i < LOADS; i++) load_value(c, i);
        };
        auto mask = [&](int c, Scores& s) {
            const uint64_t exist = key_exists[c & 7];
            const int key0 = c * KB;
            if (exist == ALL && key0 + KB <= low) return;
            int first = X::first_key(lane);
            asm volatile("" : "+v"(first));  // formed here, not kept across the key loop
            const uint64_t here = exist >> first;
            const int left = lim - key0 - first;
#pragma unroll
            for (int n = 0; n < N; n++) {
                const int k = X::key(n);
                s.set(n, ((here >> k) & 1) && k < left ? s.get(n) : -INFINITY);
            }
        };

        x.clear();
        // the exponents' reference (scaled), and what is taken off them; the sum
        float ref = -INFINITY, shift = 0.f, l = 0.f;
        auto weight = [&](Scores& s, int n) {
            float z = __builtin_amdgcn_exp2f(fmaf(s.get(n), cs, -shift));
            if constexpr (X::INTERLEAVED) asm volatile("" : "+v"(z));  // formed here
            s.set(n, z);
        };
        // The reference for scores whose largest is `top`: sums are taken along. A row without a key
        // so far has sums of zero, and shift 0.
        auto refer = [&](float top) {
            const bool grown = top > ref + LAG;
            if (!__any(grown)) return;
            const float f = grown ? __builtin_amdgcn_exp2f(ref - top) : 1.f;
            ref = grown ? top : ref;
            shift = grown ? top : shift;
            l *= f;
            x.shrink(f);
        };
        auto largest = [&](const Scores& s, int n0, int n1, float top) {
#pragma unroll
            for (int n = n0; n < n1; n++) top = fmaxf(top, s.get(n));
            return top;
        };
        int page = 0;
        // One step: the weights of s (masked, their references known), its values added; meanwhile
        // the next step's scores and their maximum. Beside the MFMAs of the scores go 5 in 8 of the
        // weights, beside those of the values the others, the sums and the maximum: about as many
        // cycles of the vector pipe as of the matrix pipe in both halves.
        auto step = [&](int c, Scores& s, Scores& next) {
            lds_loads_done();
            // keys c + 1 + LEAD and values c + LEAD are whole; all are done with what comes next
            lds_barrier();
            if (!ROWS_EARLY) rows_of(c + 2 + LEAD, k_rows);
            if (c + 2 + LEAD < c1) load_keys(c + 2 + LEAD);
            if (!ROWS_EARLY) rows_of(c + 1 + LEAD, v_rows);
            if (c + 1 + LEAD < c1) load_values(c + 1 + LEAD);
            if (ROWS_EARLY) {
                rows_of(c + 3 + LEAD, k_rows);
                rows_of(c + 2 + LEAD, v_rows);
            }
            if (wave == (c & (X::WAVES - 1)) && c + 4 + LEAD < c1) {
                arrived(page);
                put_rows(c + 4 + LEAD, page);
            }
            if (wave == ((c + 1) & (X::WAVES - 1)) && c + 5 + LEAD < c1) {
                page = page_of(c + 5 + LEAD);
                sched_fence();
            }
            if (c >= mine) return;
            const uint32_t kt = keys_at(c + 1), vt = values_at(c);
            float top = -INFINITY;
            if constexpr (X::INTERLEAVED) {
                constexpr int FIRST = N * 5 / 8, REST = N - FIRST;
                constexpr int MS = X::SCORE_MFMAS, MV = X::VALUE_MFMAS;
                if constexpr (LEAD == 0) x.start_keys(kt, lane);
                x.scores(kt, lane, next, [&](int m) {
#pragma unroll
                    for (int n = m * FIRST / MS; n < (m + 1) * FIRST / MS; n++) weight(s, n);
                    if (m == MS - 2) x.start_values(vt, lane);
                });
                if (c + 1 < mine) mask(c + 1, next);
                x.values(vt, lane, s, l, [&](int m) {
                    constexpr int L = MV * 5 / 8, HALF = MV / 2;
                    if (m < L)
#pragma unroll
                        for (int n = m * REST / L; n < (m + 1) * REST / L; n++) weight(s, FIRST + n);
                    if (m < HALF) {
                        top = largest(next, m * N / HALF, (m + 1) * N / HALF, top);
                        asm volatile("" : "+v"(top));
                    }
                    if (m == HALF + 1) top = X::max_partners(top) * cs;
                    if (LEAD > 0 && m == MV - 2) x.start_keys(keys_at(c + 2), lane);
                });
            } else {
#pragma unroll
                for (int n = 0; n < N; n++) weight(s, n);
                x.scores(kt, lane, next, [](int) {});
                if (c + 1 < mine) mask(c + 1, next);
                x.values(vt, lane, s, l, [](int) {});
                top = X::max_partners(largest(next, 0, N, top)) * cs;
            }
            if (c + 1 < mine) refer(top);
        };
        if (c1 > c0) {
            Scores s0, s1;
            __syncthreads();  // the unit before is done with its tiles and rows
            for (int i = wave; i < 4 + LEAD; i += X::WAVES) put_rows(c0 + i, page_of(c0 + i));
            lds_barrier();
            rows_of(c0, k_rows);
            load_keys(c0);
            if (LEAD > 0 && c0 + 1 < c1) {
                rows_of(c0 + 1, k_rows);
                load_keys(c0 + 1);
            }
            lds_loads_done();
            lds_barrier();
            if (wave == (c0 & (X::WAVES - 1)) && c0 + 4 + LEAD < c1) {
                page = page_of(c0 + 4 + LEAD);
                sched_fence();
            }
            rows_of(c0 + 1 + LEAD, k_rows);
            rows_of(c0, v_rows);
            if (c0 + 1 + LEAD < c1) load_keys(c0 + 1 + LEAD);
            load_values(c0);
            if (LEAD > 0 && c0 + 1 < c1) {
                rows_of(c0 + 1, v_rows);
                load_values(c0 + 1);
            }
            if (ROWS_EARLY) {
                rows_of(c0 + 2 + LEAD, k_rows);
                rows_of(c0 + 1 + LEAD, v_rows);
            }
            if (c0 < mine) {
                x.start_keys(keys_at(c0), lane);
                x.scores(keys_at(c0), lane, s0, [](int) {});
                mask(c0, s0);
                refer(X::max_partners(largest(s0, 0, N, -INFINITY)) * cs);
                if constexpr (LEAD > 0) x.start_keys(keys_at(c0 + 1), lane);
            }
            for (int c = c0; c < c1; c += 2) {
                step(c, s0, s1);
                if (c + 1 < c1) step(c + 1, s1, s0);
            }
        }
        const bool whole = c0 == 0 && c1 == nch;
        int64_t slot = 0;
        if (SHARED || !whole) {
            const int last = cut.owner(unit_start + nch - 1);
            if constexpr (SHARED) {  // one slot per unit, and one per worker that goes on with one
                const int unit = kvh * a.tiles + t;
                slot = c0 == 0 ? (int64_t)a.workers + unit : w;
                if (c0 == 0 && tid == 0) a.prefix_notes[unit] = make_int2(w, last);
            } else {
                slot = 2 * w + (late ? 1 : 0);
                if (c0 == 0 && tid == 0) a.join.notes[w] = make_int4(t, kvh, (int)slot, last);
            }
        }
        const float sum = X::sum_partners(l);
        if (live && !SHARED && whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
            T* out = reinterpret_cast<T*>(a.o) + q_row * D;
            x.results(lane, inv, [&](int col, const float z[4]) { store4<T>(out + col, z); });
        } else if (live) {
            const size_t at = (size_t)slot * ROWS + tile_row;
            float* out = a.join.part_o + at * D;
            x.results(lane, 1.f, [&](int col, const float z[4]) { store4<float>(out + col, z); });
            if (X::first_key(lane) == 0) {
                a.join.part_ml[at * 2] = ref;
                a.join.part_ml[at * 2 + 1] = sum;
            }
        }
        pos = c1 == nch ? unit_next : end;
    }
}

}  // namespace gdn
