// Attention of the newest n_pos tokens of each request over a paged key/value cache, grouped
// heads (gdn_paged_decode).
//
//   o[b, p, h] = sum_j softmax_j(scale q[b, p, h] . k_j) v_j,   j < len_b - n_pos + p + 1,
// k_j and v_j the rows of head h / group in the request's pages. The n_pos x group query rows
// that share a key/value head form the 16-row MFMA tiles, so the cache is read once for all of
// them; the keys are split over workgroups by key_split.h and joined by a second kernel.
//
// One wave takes KW keys at a time and keeps everything of them in registers:
//   S^T = K Q^T   keys are the rows of the MFMA's A operand, read from the cache row by row in
//                 16-byte pieces straight into registers (no LDS);
//   softmax       running maximum and sum per query row, i.e. per accumulator column: a lane's
//                 KW / 4 scores are reduced in registers, then over the four lane groups;
//   O^T += V^T P^T  the accumulator layout of S^T is the B operand's with the keys renumbered
//                 (lane group g holds keys 4 g .. 4 g + 3 of each 16), so P stays in registers.
//                 V^T is the one operand that needs a transpose: V rows go through a per-wave
//                 LDS tile and come back by transposing reads (bf16) or column reads (fp32).
// Waves never wait for each other inside the key loop; the four partial results of a workgroup
// are merged through LDS at the end of a unit.
//
// Bound: HBM, each key and value being read once. Measured (bf16): one request of 250001 tokens,
// 8 KV heads, d = 128 (1.02 GB) 173 us, 5.9 TB/s; 128 requests of 30 to 30000 tokens, 4 KV heads
// (1.11 GB) 192 us, 5.8 TB/s; 40 requests x 4 positions, 2 KV heads, d = 256 (0.35 GB) 79 us,
// 4.4 TB/s, where a step's registers leave fewer loads on their way.
#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"
#include "key_join.h"
#include "lds_tile.h"

namespace gdn {

namespace {

constexpr int PD_THREADS = 256;
constexpr int PD_WAVES = PD_THREADS / WAVE;
constexpr float LOG2E = 1.4426950408889634f;

// Per element type: keys per wave step, fragments, and the two products.
template <typename T, int D> struct PdTile;

template <int D> struct PdTile<bf16, D> {
    // Keys of a wave step: a contraction of P V. With 32 at d = 256 the step's keys and values
    // alone take 128 registers beside 96 for queries and outputs, one wave fits a SIMD and spills.
    static constexpr int KW = D == 256 ? 16 : 32;
    static constexpr int NSUB = KW / 16;
    static constexpr int NF = D / 32;        // 16-byte pieces per lane of a key or query row
    static constexpr int ROW = D * 2;        // bytes of an LDS row
    static constexpr int CPR = D * 2 / 16;   // 16-byte pieces per row
    typedef bf16x8 frag;
    __device__ __forceinline__ static int piece(int f, int g) { return f * 4 + g; }
    __device__ __forceinline__ static f32x4 qk(const frag* k, const frag* q) {
        f32x4 s = zero4();
#pragma unroll
        for (int f = 0; f < NF; f++) s = Mma<bf16>::mma(k[f], q[f], s);
        return s;
    }
    // LDS position of piece c of row r: pairs of pieces (the 32 bytes a transposing read takes
    // from a row) are rotated over the banks by the row, so that its 16 rows do not collide
    __device__ __forceinline__ static int turn(int r) { return D >= 128 ? r & 7 : (r >> 1) & 3; }
    __device__ __forceinline__ static int place(int r, int c) {
        return r * ROW + ((c ^ (turn(r) << 1)) << 4);
    }
    // o[j] += V^T(16 dims from 16 j) P^T
    template <int NS>
    __device__ __forceinline__ static void pv(f32x4* o, const char* v, const float (*p)[4],
                                              int lane) {
        const int r = (lane >> 4) * 4 + ((lane >> 2) & 3);
        const char* row = v + r * ROW + (lane & 3) * 8;
        const int turned = turn(r) << 5;
        bf16x4 pb[NSUB];
#pragma unroll
        for (int t = 0; t < NSUB; t++)
#pragma unroll
            for (int i = 0; i < 4; i++) pb[t][i] = (bf16)p[t][i];
#pragma unroll
        for (int j = 0; j < D / 16; j++) {
            const char* at = row + ((j << 5) ^ turned);
            if constexpr (NSUB == 2)
                o[j] = Mma<bf16>::mma(join(lds_read_tr(at), lds_read_tr(at + 16 * ROW)),
                                      join(pb[0], pb[1]), o[j]);
            else
                o[j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                    __builtin_bit_cast(s16x4, lds_read_tr(at)), __builtin_bit_cast(s16x4, pb[0]),
                    o[j], 0, 0, 0);
        }
    }
};

template <int D> struct PdTile<float, D> {
    static constexpr int KW = 16;
    static constexpr int NSUB = 1;
    static constexpr int NF = D / 16;
    static constexpr int ROW = D * 4 + 16;   // 4 floats of padding: rows 4 apart on other banks
    static constexpr int CPR = D * 4 / 16;
    typedef f32x4 frag;
    __device__ __forceinline__ static int piece(int f, int g) { return f * 4 + g; }
    __device__ __forceinline__ static f32x4 qk(const frag* k, const frag* q) {
        f32x4 s = zero4();
#pragma unroll
        for (int f = 0; f < NF; f++)
#pragma unroll
            for (int e = 0; e < 4; e++) s = Mma<float>::mma(k[f][e], q[f][e], s);
        return s;
    }
    __device__ __forceinline__ static int place(int r, int c) { return r * ROW + c * 16; }
    template <int NS>
    __device__ __forceinline__ static void pv(f32x4* o, const char* v, const float (*p)[4],
                                              int lane) {
        const float* row = reinterpret_cast<const float*>(v + (lane >> 4) * 4 * ROW) + (lane & 15);
#pragma unroll
        for (int j = 0; j < D / 16; j++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                o[j] = Mma<float>::mma(row[i * (ROW / 4) + j * 16], p[0][i], o[j]);
    }
};

template <typename T, int D, int RT>
struct PdLds {
    static constexpr int VTILE = PdTile<T, D>::KW * PdTile<T, D>::ROW;
    static constexpr int MROW = D + 4;  // floats: merge rows on different banks
    static constexpr int MERGE = PD_WAVES * 16 * MROW * 4;
    static constexpr int BYTES = VTILE * PD_WAVES > MERGE ? VTILE * PD_WAVES : MERGE;
};

constexpr uint32_t NO_ROW = 0xffffffffu;

// Two waves per SIMD (256 registers each) where one row tile fits beside a step's keys and
// values: the loads of one wave then fill the time the other computes.
template <typename T, int D, int RT>
constexpr int PD_WAVES_PER_SIMD = RT == 1 && (sizeof(T) == 2 || D <= 128) ? 2 : 1;

// BEHIND: the keys behind a shared prefix (a.start of them), whose results join those of the
// prefix: a unit of a request that has one leaves parts also where one worker covers it whole.
template <typename T, int D, int RT, bool BEHIND>
__global__ __launch_bounds__(PD_THREADS, (PD_WAVES_PER_SIMD<T, D, RT>)) void paged_decode_kernel(
    PagedDecodeArgs a) {
    using X = PdTile<T, D>;
    using L = PdLds<T, D, RT>;
    typedef typename X::frag frag;
    constexpr int KW = X::KW, NSUB = X::NSUB, NF = X::NF, CPR = X::CPR;
    constexpr int KB = KW * PD_WAVES;
    constexpr int NV = KW * CPR / WAVE;  // 16-byte pieces of V per lane
    __shared__ __align__(16) char smem[L::BYTES];
    __shared__ float ml[PD_WAVES][16][2];
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(wave_id());
    const int col = lane & 15, grp = lane >> 4;
    const SplitPlace me = split_place(blockIdx.x, a.row_tiles);
    int own_keys = me.worker < a.split.batch ? split_keys(a.split, me.worker) : 1;
    SplitRun run = split_run<KB, PD_THREADS>(a.split, me.worker, a.workers);
    const int run_start = run.pos;
    const int row0 = me.row_tile * 16 * RT;
    if (me.row_tile == 0) {
        // requests without keys: zeros, and nothing to join
        for (int b = me.worker; b < a.split.batch; b += a.workers) {
            if (b != me.worker) own_keys = split_keys(a.split, b);
            if (uniform(own_keys) != 0) continue;
            if constexpr (BEHIND) {
                const bool joined = uniform(a.start[b]) > 0;
                for (int u = tid; u < a.kv_heads; u += PD_THREADS)
                    a.join.notes[b * a.kv_heads + u] = make_int4(0, 0, 0, joined ? 0 : -1);
                if (joined) continue;
            }
            const size_t n = (size_t)a.n_pos * a.H * D;
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            for (size_t i = tid * 4; i < n; i += PD_THREADS * 4)
                store4<T>(reinterpret_cast<T*>(a.o) + (size_t)b * n + i, z);
            if (!BEHIND && a.join.per_unit)
                for (int u = tid; u < a.kv_heads; u += PD_THREADS)
                    join_none(a.join, b * a.kv_heads + u);
        }
        if (!BEHIND && !a.join.per_unit && tid == 0) join_none(a.join, me.worker);
    }
    char* vlds = smem + wave * L::VTILE;
    const float cs = a.scale * LOG2E;

    while (run.pos < run.end) {
        const int b = run.b;
        const int nkeys = uniform(split_keys(a.split, b));
        const int nch = (nkeys + KB - 1) / KB;
        const int per_unit = nch + a.split.extra;
        const int kvh = (run.pos - run.base) / per_unit;
        const int c0 = run.pos - run.base - kvh * per_unit;
        const int next_unit = run.base + (kvh + 1) * per_unit;
        const int request_end = run.base + a.split.units * per_unit;
        if (c0 >= nch) {  // the run starts behind the unit's own chunks
            run.advance(a.split, next_unit, request_end);
            continue;
        }
        const int c1 = min(nch, c0 + (run.end - run.pos));
        const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
        const int skip = BEHIND ? uniform(a.start[b]) : 0;
        // keys that position 0 sees
        const int seen0 = uniform((BEHIND ? a.seq_lens : a.split.seq_lens)[b]) - skip - a.n_pos + 1;

        frag q[RT][NF];
        int lim[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            const int r = row0 + rt * 16 + col;
            const bool live = r < a.rows;
            const int p = live ? r / a.group : 0, h = live ? r - p * a.group : 0;
            lim[rt] = live ? seen0 + p : 0;
            const T* src = reinterpret_cast<const T*>(a.q) +
                           (((size_t)b * a.n_pos + p) * a.H + (size_t)kvh * a.group + h) * D;
#pragma unroll
            for (int f = 0; f < NF; f++)
                q[rt][f] = reinterpret_cast<const frag*>(src)[X::piece(f, grp)];
        }

        f32x4 acc[RT][D / 16];
        float m[RT], l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            m[rt] = -INFINITY;
            l[rt] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; j++) acc[rt][j] = zero4();
        }

        // table entry of this lane's key of each 16-key group of wave step c (lanes 16.. repeat
        // 0..15); keys past the end read the table's last entry, and find_rows() drops them
        int page[NSUB];
        auto load_pages = [&](int c) {
#pragma unroll
            for (int t = 0; t < NSUB; t++) {
                const uint32_t key = (uint32_t)(c * KB + wave * KW + t * 16 + col + skip);
                page[t] = table[min(a.block(key), (uint32_t)a.max_blocks - 1)];
            }
        };
        uint32_t row[NSUB];
        auto find_rows = [&](int c) {
#pragma unroll
            for (int t = 0; t < NSUB; t++) {
                arrived(page[t]);
                const uint32_t key = (uint32_t)(c * KB + wave * KW + t * 16 + col + skip);
                const uint32_t off = key - a.block(key) * a.block.div;
                const bool ok = (int)key < nkeys + skip && page[t] >= 0 && page[t] < a.n_blocks;
                row[t] = ok ? ((uint32_t)page[t] * a.kv_heads + kvh) * a.block.div + off : NO_ROW;
            }
        };
        frag kf[NSUB][NF];
        auto load_k = [&]() {
#pragma unroll
            for (int t = 0; t < NSUB; t++) {
                const uint32_t r = row[t] == NO_ROW ? 0u : row[t];
                const frag* src = reinterpret_cast<const frag*>(
                    reinterpret_cast<const T*>(a.k_cache) + (size_t)r * D);
#pragma unroll
                for (int f = 0; f < NF; f++) kf[t][f] = src[X::piece(f, grp)];
            }
        };
        f32x4 vf[NV];
        auto load_v = [&]() {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int x = i * WAVE + lane, r = x / CPR, c = x % CPR;
                uint32_t at = __shfl(row[0], r & 15, WAVE);
                if constexpr (NSUB > 1) {
                    const uint32_t at1 = __shfl(row[1], r & 15, WAVE);
                    at = r < 16 ? at : at1;
                }
                at = at == NO_ROW ? 0u : at;
                vf[i] = reinterpret_cast<const f32x4*>(reinterpret_cast<const T*>(a.v_cache) +
                                                       (size_t)at * D)[c];
            }
        };
        load_pages(c0);
        find_rows(c0);
        load_pages(c0 + 1);
        load_k();
        load_v();

        for (int c = c0; c < c1; c++) {
            float s[RT][NSUB][4];
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                for (int t = 0; t < NSUB; t++) {
                    const f32x4 x = X::qk(kf[t], q[rt]);
#pragma unroll
                    for (int i = 0; i < 4; i++) s[rt][t][i] = x[i] * cs;
                }
            // keys of this step that exist, one bit each
            uint32_t exist = 0;
#pragma unroll
            for (int t = 0; t < NSUB; t++)
                exist |= (uint32_t)(__ballot(row[t] != NO_ROW) & 0xffff) << (16 * t);
            constexpr uint32_t ALL = (uint32_t)((1ull << KW) - 1);
            const int key0 = c * KB + wave * KW;
            if (exist != ALL || key0 + KW > seen0) {
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int t = 0; t < NSUB; t++)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int k = t * 16 + grp * 4 + i;
                            const bool keep = ((exist >> k) & 1) && key0 + k < lim[rt];
                            s[rt][t][i] = keep ? s[rt][t][i] : -INFINITY;
                        }
            }
            // V to LDS, absent keys as zeros (a zero weight does not cancel what their rows hold)
            if (exist != ALL) {
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    const int r = (i * WAVE + lane) / CPR;
                    if (!((exist >> r) & 1)) vf[i] = zero4();
                }
            }
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int x = i * WAVE + lane;
                *reinterpret_cast<f32x4*>(vlds + X::place(x / CPR, x % CPR)) = vf[i];
            }
            if (c + 1 < c1) {
                find_rows(c + 1);
                load_pages(c + 2);  // first: the wait for it must not be behind the others
                load_k();
                load_v();
            }
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                float top = s[rt][0][0];
#pragma unroll
                for (int t = 0; t < NSUB; t++)
#pragma unroll
                    for (int i = 0; i < 4; i++) top = fmaxf(top, s[rt][t][i]);
                top = max_groups(top);
                const bool grown = top > m[rt] + LAG;
                if (__any(grown)) {
                    const float shrink = grown ? __builtin_amdgcn_exp2f(m[rt] - top) : 1.f;
                    l[rt] *= shrink;
#pragma unroll
                    for (int j = 0; j < D / 16; j++)
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[rt][j][i] *= shrink;
                    m[rt] = grown ? top : m[rt];
                }
                const float ref = m[rt] == -INFINITY ? 0.f : m[rt];  // a row with no key so far
#pragma unroll
                for (int t = 0; t < NSUB; t++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        s[rt][t][i] = __builtin_amdgcn_exp2f(s[rt][t][i] - ref);
                        l[rt] += s[rt][t][i];
                    }
                X::template pv<NSUB>(acc[rt], vlds, s[rt], lane);
            }
        }

        // merge the four waves, one 16-row tile at a time
        const bool covered = c0 == 0 && c1 == nch, whole = covered && (!BEHIND || skip == 0);
        const int unit = b * a.kv_heads + kvh;
        int slot = 2 * me.worker + (run.pos == run_start ? 0 : 1);
        if (BEHIND && covered) slot = 2 * a.workers + unit;
        if (c0 == 0 && me.row_tile == 0 && tid == 0) {
            if constexpr (BEHIND) {  // (parts, the first one's slot; the others' are 2 w)
                const int parts = covered ? 1 : run.cut.owner(run.pos + nch - 1) - me.worker + 1;
                a.join.notes[unit] = make_int4(parts, me.worker, slot, whole ? -1 : 0);
            } else {
                join_note(a.join, a.split, run, me.worker, b, kvh, c1, nch, run.pos != run_start);
            }
        }
        const size_t part_row = ((size_t)slot * a.row_tiles + me.row_tile) * (16 * RT);
        float* mrow = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            __syncthreads();
            float lt = l[rt];
            lt += __shfl_xor(lt, 16, WAVE);
            lt += __shfl_xor(lt, 32, WAVE);
            if (grp == 0) {
                ml[wave][col][0] = m[rt];
                ml[wave][col][1] = lt;
            }
#pragma unroll
            for (int j = 0; j < D / 16; j++)
                *reinterpret_cast<f32x4*>(mrow + (wave * 16 + col) * L::MROW + j * 16 + grp * 4) =
                    acc[rt][j];
            __syncthreads();
            const int r = tid >> 4, rr = row0 + rt * 16 + r;
            if (rr < a.rows) {
                float top = ml[0][r][0];
#pragma unroll
                for (int w = 1; w < PD_WAVES; w++) top = fmaxf(top, ml[w][r][0]);
                const float ref = top == -INFINITY ? 0.f : top;
                float wt[PD_WAVES], sum = 0.f;
#pragma unroll
                for (int w = 0; w < PD_WAVES; w++) {
                    wt[w] = __builtin_amdgcn_exp2f(ml[w][r][0] - ref);
                    sum += wt[w] * ml[w][r][1];
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
                const int p = rr / a.group, h = rr - p * a.group;
                T* dst = reinterpret_cast<T*>(a.o) +
                         (((size_t)b * a.n_pos + p) * a.H + (size_t)kvh * a.group + h) * D;
                float* part = a.join.part_o + (part_row + rt * 16 + r) * D;
#pragma unroll
                for (int j = 0; j < D / 64; j++) {
                    const int d = j * 64 + (tid & 15) * 4;
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < PD_WAVES; w++) {
                        const f32x4 y = *reinterpret_cast<const f32x4*>(
                            mrow + (w * 16 + r) * L::MROW + d);
#pragma unroll
                        for (int i = 0; i < 4; i++) x[i] = fmaf(wt[w], y[i], x[i]);
                    }
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 4; i++) x[i] *= inv;
                        store4<T>(dst + d, x);
                    } else {
                        store4<float>(part + d, x);
                    }
                }
                if (!whole && (tid & 15) == 0) {
                    float* pm = a.join.part_ml + (part_row + rt * 16 + r) * 2;
                    pm[0] = top;
                    pm[1] = sum;
                }
            }
        }
        __syncthreads();  // the merge rows are the next unit's V tiles

        run.advance(a.split, c1 == nch ? next_unit : run.pos + c1 - c0, request_end);
    }
}

// Results of the units that were cut.
template <typename T, int D>
__global__ __launch_bounds__(JOIN_THREADS) void paged_join_kernel(PagedDecodeArgs a) {
    join_parts<D>(a.join, [&](int b, int kvh, int row, int col, const float x[4]) {
        const int p = row / a.group, h = row - p * a.group;
        store4<T>(reinterpret_cast<T*>(a.o) +
                      (((size_t)b * a.n_pos + p) * a.H + (size_t)kvh * a.group + h) * D + col,
                  x);
    });
}

template <typename T, int D, int RT, bool BEHIND>
hipError_t run_decode(const PagedDecodeArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((paged_decode_kernel<T, D, RT, BEHIND>),
                       dim3((unsigned)(a.workers * a.row_tiles)), dim3(PD_THREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || BEHIND) return e;
    hipLaunchKernelGGL((paged_join_kernel<T, D>), dim3(join_grid(a.join)), dim3(JOIN_THREADS),
                       0, s, a);
    return hipGetLastError();
}

template <typename T, int D, bool BEHIND>
hipError_t pick_rows(const PagedDecodeArgs& a, hipStream_t s) {
    switch (a.rt) {
        case 1: return run_decode<T, D, 1, BEHIND>(a, s);
        case 2:
            if constexpr (sizeof(T) == 2 && D <= 128) return run_decode<T, D, 2, BEHIND>(a, s);
            break;
        case 4:
            if constexpr (sizeof(T) == 2 && D == 64) return run_decode<T, D, 4, BEHIND>(a, s);
            break;
    }
    return hipErrorInvalidValue;
}

template <typename T, bool BEHIND>
hipError_t pick_dim(const PagedDecodeArgs& a, hipStream_t s) {
    switch (a.d) {
        case 64: return pick_rows<T, 64, BEHIND>(a, s);
        case 128: return pick_rows<T, 128, BEHIND>(a, s);
        case 256: return pick_rows<T, 256, BEHIND>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t paged_decode_layout(PagedDecodeArgs* a, void* ws) {
    a->group = a->H / a->kv_heads;
    a->rows = a->group * a->n_pos;
    // Rows of a tile: as many as the registers hold beside the head dim, so that a workgroup
    // reads the keys for all of them (48 rows at d = 128: 57 us with two tiles, 79 with one at a
    // time; 64 rows at d = 64: 45 us with four, 46 with two, 54 with one).
    const int most = a->dtype == 0 || a->d == 256 ? 1 : a->d == 128 ? 2 : 4;
    const int tiles = (a->rows + 15) / 16;
    a->rt = tiles >= 4 && most >= 4 ? 4 : tiles >= 2 && most >= 2 ? 2 : 1;
    a->row_tiles = (tiles + a->rt - 1) / a->rt;
    a->split.units = a->kv_heads;
    // (128 requests of 30 to 30000 tokens, 4 KV heads: 204 us a call with 0, 201 with 1, 200
    // with 2; 1 and 2 are within the spread of runs)
    a->split.extra = 2;
    const int cus = device_cu_count();
    // Two workgroups a CU hide each other's starts, where they fit; with long units, whose starts
    // are few, one a CU leaves fewer parts to write and join. 4 KV heads, d = 128: 300 requests of
    // 300 tokens 37 us with two, 41 with one; of 1000 tokens 123 and 117; 128 requests of 30 to
    // 30000 tokens 203 and 197; one of 100000 tokens (8 KV heads) 81 and 78. (Two row tiles side
    // by side read the same keys, and two of them a CU stay ahead: 40 requests of 200 to 20000
    // tokens, 32 rows at d = 256, 86 us and 88.)
    const bool two = a->rt == 1 && (a->dtype == 1 || a->d <= 128);
    a->split.halve = two && a->row_tiles == 1 ? 1 : 0;
    a->workers = split_workers(two ? 2 * cus : cus, a->row_tiles);
    JoinShape& j = a->join;
    j.row_tiles = a->row_tiles;
    j.tile = 16 * a->rt;
    j.rows = a->rows;
    join_layout(&j, (int64_t)a->split.batch * a->split.units, a->workers, cus, a->d);
    const size_t rows = (size_t)2 * a->workers * a->row_tiles * j.tile;
    j.part_o = static_cast<float*>(ws);
    j.part_ml = ws == nullptr ? nullptr : j.part_o + rows * a->d;
    j.notes = ws == nullptr ? nullptr : reinterpret_cast<int4*>(j.part_ml + rows * 2);
    return rows * (a->d + 2) * sizeof(float) + (size_t)j.count * sizeof(int4);
}

hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    return a.dtype == 1 ? pick_dim<bf16, false>(a, s) : pick_dim<float, false>(a, s);
}

hipError_t launch_own_keys(const PagedDecodeArgs& a, hipStream_t s) {
    return a.dtype == 1 ? pick_dim<bf16, true>(a, s) : pick_dim<float, true>(a, s);
}

}  // namespace gdn
