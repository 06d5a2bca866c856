// Latent attention of the newest n_pos tokens of each request, absorbed form
// (gdn_latent_decode), bf16.
//
// A token's cache row is a latent c_j (rank elements) shared by all heads and a rotary key r_j
// (64). Head h's key is (W_uk,h c_j, r_j) and its value W_uv,h c_j, so with
//   q'_h = W_uk,h^T q_nope,h      (absorb)
//   s_j = scale (q'_h . c_j + q_pe,h . r_j),  p = softmax(s),  u_h = sum_j p_j c_j   (core)
//   o_h = W_uv,h u_h              (up)
// no key or value of a head is ever written out: the core reads each cache row once for all
// heads. Three launches; the core's work split and its join are key_split.h's, the join runs at
// the start of `up`.
#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"
#include "lds_tile.h"

namespace gdn {

namespace {

constexpr int LD_THREADS = 256;
constexpr int LD_WAVES = LD_THREADS / WAVE;
constexpr int LD_ROPE = 64;
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ uint64_t bits4(const float x[4]) {
    bf16x4 v;
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = (bf16)x[i];
    return __builtin_bit_cast(uint64_t, v);
}

// ---------------------------------------------------------------------------------- absorb
// q'^T (rank x rows) = W_uk^T q_nope^T per head: a workgroup takes 128 rank columns of one
// head's W_uk (LDS, read back transposed into the MFMA's A operand and kept in registers) and
// runs over its share of the (request, position) rows, 16 at a time. Bound by reading the
// weights once. q' is rounded to bf16 as the core's MFMA operand.
constexpr int AB_COLS = 128;

// LDS position of the 16-byte piece c of row n (rows of AB_COLS elements = 16 pieces): the 16
// rows of a transposing read are 8 g + (0..3), so pairs of pieces turn by those bits
__device__ __forceinline__ int ab_place(int n, int c) {
    const int turn = (n & 3) | ((n >> 1) & 4);
    return n * (AB_COLS * 2) + ((c ^ (turn << 1)) << 4);
}

template <int DN>
__global__ __launch_bounds__(LD_THREADS) void latent_absorb_kernel(LatentDecodeArgs a,
                                                                   int tiles_per_wg) {
    __shared__ __align__(16) char w[DN * AB_COLS * 2];
    const int h = blockIdx.x, r0 = blockIdx.y * AB_COLS;
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const bf16* W = reinterpret_cast<const bf16*>(a.w_kv) +
                    (size_t)h * (a.d_nope + a.d_v) * a.rank + r0;
#pragma unroll
    for (int i = 0; i < DN * 16 / LD_THREADS; i++) {
        const int x = i * LD_THREADS + tid, n = x >> 4, c = x & 15;
        *reinterpret_cast<f32x4*>(w + ab_place(n, c)) =
            *reinterpret_cast<const f32x4*>(W + (size_t)n * a.rank + c * 8);
    }
    __syncthreads();
    const int col = lane & 15, grp = lane >> 4;
    bf16x8 A[2][DN / 32];  // 2 x 16 rank columns of this wave
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int k = 0; k < DN / 32; k++) {
            const int n = k * 32 + grp * 8 + ((lane >> 2) & 3);
            const int c = (wave * 2 + t) * 2 + ((lane & 3) >> 1);
            A[t][k] = join(lds_read_tr(w + ab_place(n, c) + (lane & 1) * 8),
                           lds_read_tr(w + ab_place(n + 4, c) + (lane & 1) * 8));
        }
    const int rows = a.split.batch * a.n_pos;
    const int t0 = blockIdx.z * tiles_per_wg;
    for (int t = t0; t < t0 + tiles_per_wg && t * 16 < rows; t++) {
        const int row = t * 16 + col;
        const bf16* q = reinterpret_cast<const bf16*>(a.q_nope) +
                        ((size_t)min(row, rows - 1) * a.H + h) * DN;
        bf16x8 B[DN / 32];
#pragma unroll
        for (int k = 0; k < DN / 32; k++) B[k] = Mma<bf16>::load(q + k * 32 + grp * 8);
        bf16* out = reinterpret_cast<bf16*>(a.q_lat) + ((size_t)row * a.H + h) * a.rank + r0;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            f32x4 d = zero4();
#pragma unroll
            for (int k = 0; k < DN / 32; k++) d = Mma<bf16>::mma(A[x][k], B[k], d);
            float y[4] = {d[0], d[1], d[2], d[3]};
            if (row < rows) store4<bf16>(out + (wave * 2 + x) * 16 + grp * 4, y);
        }
    }
}

// ------------------------------------------------------------------------------------ core
// A workgroup of 4 RH waves holds one row tile (16 RT RH query rows) and walks 64 keys at a time:
//   S^T = K Q^T   wave w takes keys 16 (w & 3) .. + 15 of the tile for the 16 RT rows of part
//                 w >> 2; the queries stay in registers, K fragments come from LDS;
//   softmax       the row maximum goes over the waves through LDS, weights go back as bf16;
//   U^T += C^T P^T  wave w takes rank / (4 RH) of the output columns for all rows; C^T by
//                 transposing LDS reads of the very tile the scores came from.
// So each cache row is read once from memory per row tile; from LDS a tile is read RH times as
// keys and once as values. The next tile loads straight into the other LDS buffer meanwhile.
constexpr int LD_KB = 64;

template <int R>
struct LdTile {
    static constexpr int LAT = R * 2;                  // bytes of a latent
    static constexpr int PIECES = LAT / 16;            // 16-byte pieces
    static constexpr int ROPE_AT = LD_KB * LAT;        // rotary keys behind the latents
    static constexpr int BYTES = LD_KB * (LAT + LD_ROPE * 2);
    static constexpr int ROW = (R + LD_ROPE) * 2;      // bytes of a cache row
    // Piece c of key row r lies at piece c ^ turn(r). Key fragments read one piece of 16
    // consecutive rows: turn takes 16 values over them. Transposing reads take a pair of pieces
    // of rows 8 g + (0..3): turn >> 1 takes 8 values, twice each, over those.
    __device__ __forceinline__ static int turn(int r) {
        return ((r & 3) << 1) | (r & 8) | ((r >> 2) & 1);
    }
    __device__ __forceinline__ static int lat(int r, int c) { return r * LAT + ((c ^ turn(r)) << 4); }
    __device__ __forceinline__ static int rope(int r, int c) {
        return ROPE_AT + r * (LD_ROPE * 2) + ((c ^ ((r >> 1) & 7)) << 4);
    }
};

// Weights [16 RT rows][64 keys] bf16, pieces of 8 keys turned by the row.
__device__ __forceinline__ int ld_weight(int row, int piece) {
    return row * (LD_KB * 2) + ((piece ^ ((row >> 1) & 7)) << 4);
}

template <int R, int RT, int RH>
__global__ __launch_bounds__(LD_THREADS * RH) void latent_core_kernel(LatentDecodeArgs a) {
    using X = LdTile<R>;
    constexpr int WAVES = 4 * RH;
    constexpr int TILES = RT * RH, ROWS = 16 * TILES;
    constexpr int NL = R / 32, NF = NL + LD_ROPE / 32;  // key fragments: latent, then rotary
    constexpr int NT = R / 16 / WAVES;                  // 16-column output tiles per wave
    constexpr int OWN = 16 / RH;                        // rows of a tile that a wave loads
    __shared__ __align__(16) char tile[2 * X::BYTES];
    __shared__ __align__(16) char wt[ROWS * LD_KB * 2];
    __shared__ float tops[4][ROWS];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int col = lane & 15, grp = lane >> 4;
    const int kq = wave & 3, part = wave >> 2;  // key quarter; row part of the scores
    SplitRun run = split_run<LD_KB, LD_THREADS * RH>(a.split, blockIdx.x, a.n_wg);
    const int64_t run_start = run.pos;
    const float cs = a.scale * LOG2E;
    const char* cache = reinterpret_cast<const char*>(a.cache);

    while (run.pos < run.end) {
        const int b = run.b;
        const int nkeys = split_keys(a.split, b);
        const int nch = (nkeys + LD_KB - 1) / LD_KB;
        const int unit = (int)((run.pos - run.base) / nch);
        const int c0 = (int)(run.pos - run.base - (int64_t)unit * nch);
        const int c1 = (int)min((int64_t)nch, c0 + (run.end - run.pos));
        const int row0 = unit * ROWS;
        const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
        const int seen0 = a.split.seq_lens[b] - a.n_pos + 1;  // keys that position 0 sees

        // this wave's 16 keys of a chunk: the page of lane's key (16 lanes, repeated)
        int page;
        auto load_pages = [&](int c) {
            const int key = c * LD_KB + kq * 16 + col;
            page = key < nkeys ? table[a.block((uint32_t)key)] : -1;
        };
        uint32_t exist, exist_next = 0;
        auto load_tile = [&](int c, int buf) {
            const uint32_t key = (uint32_t)(c * LD_KB + kq * 16 + col);
            const uint32_t off = key - a.block(key) * a.block.div;
            const bool ok = page >= 0 && page < a.n_blocks;
            const uint32_t slot = ok ? (uint32_t)page * a.block.div + off : 0u;
            exist_next = (uint32_t)(__ballot(ok) & 0xffff);
            const uint32_t at = lds_offset(tile) + buf * X::BYTES;
            const int first = part * OWN;
            if constexpr (X::PIECES == 64) {
#pragma unroll
                for (int i = 0; i < OWN; i++) {
                    const int r = first + i;
                    const uint32_t s = __builtin_amdgcn_readlane(slot, r);
                    load_to_lds(cache + (size_t)s * X::ROW, (uint32_t)((lane ^ X::turn(r)) << 4),
                                at + (kq * 16 + r) * X::LAT);
                }
            } else {  // two rows per load
#pragma unroll
                for (int i = 0; i < OWN; i += 2) {
                    const int r = first + i, rr = r + (lane >> 5);
                    const uint32_t s = __shfl(slot, rr, WAVE);
                    load_to_lds(cache + (size_t)s * X::ROW + (((lane & 31) ^ X::turn(rr)) << 4),
                                at + (kq * 16 + r) * X::LAT);
                }
            }
#pragma unroll
            for (int i = 0; i < OWN; i += 8) {
                const int r = first + i, rr = r + (lane >> 3);
                const uint32_t s = __shfl(slot, rr, WAVE);
                load_to_lds(cache + (size_t)s * X::ROW + X::LAT +
                                (((lane & 7) ^ ((rr >> 1) & 7)) << 4),
                            at + X::ROPE_AT + (kq * 16 + r) * (LD_ROPE * 2));
            }
        };
        load_pages(c0);
        load_tile(c0, 0);
        load_pages(c0 + 1 < c1 ? c0 + 1 : c0);

        bf16x8 q[RT][NF];
        int lim[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            const int r = row0 + (part * RT + rt) * 16 + col;
            const bool live = r < a.rows;
            lim[rt] = live ? seen0 + r / a.H : 0;
            const size_t at = (size_t)b * a.rows + (live ? r : 0);
            const bf16* ql = reinterpret_cast<const bf16*>(a.q_lat) + at * R;
            const bf16* qp = reinterpret_cast<const bf16*>(a.q_pe) + at * LD_ROPE;
#pragma unroll
            for (int f = 0; f < NF; f++)
                q[rt][f] = Mma<bf16>::load(f < NL ? ql + f * 32 + grp * 8
                                                  : qp + (f - NL) * 32 + grp * 8);
        }
        f32x4 acc[TILES][NT];
        float m[TILES], l[RT];  // running maxima; this lane's share of its rows' running sums
#pragma unroll
        for (int t = 0; t < TILES; t++) {
            m[t] = -INFINITY;
            if (t < RT) l[t] = 0.f;
#pragma unroll
            for (int j = 0; j < NT; j++) acc[t][j] = zero4();
        }

        for (int c = c0; c < c1; c++) {
            const int buf = (c - c0) & 1;
            const char* kt = tile + buf * X::BYTES;
            exist = exist_next;
            lds_loads_done();
            if (exist != 0xffff) {
                // latents of absent keys as zeros: a zero weight does not cancel what they hold
                for (int r = part * OWN; r < part * OWN + OWN; r++)
                    if (!((exist >> r) & 1) && lane < X::PIECES)
                        *reinterpret_cast<f32x4*>(tile + buf * X::BYTES + (kq * 16 + r) * X::LAT +
                                                  lane * 16) = zero4();
            }
            lds_barrier();  // tile c is whole; all waves are done with the other buffer
            if (c + 1 < c1) {
                load_tile(c + 1, buf ^ 1);
                load_pages(c + 2 < c1 ? c + 2 : c + 1);
            }
            f32x4 s[RT];
#pragma unroll
            for (int rt = 0; rt < RT; rt++) s[rt] = zero4();
#pragma unroll
            for (int f = 0; f < NF; f++) {
                const int r = kq * 16 + col;
                const bf16x8 k = *reinterpret_cast<const bf16x8*>(
                    kt + (f < NL ? X::lat(r, f * 4 + grp) : X::rope(r, (f - NL) * 4 + grp)));
#pragma unroll
                for (int rt = 0; rt < RT; rt++) s[rt] = Mma<bf16>::mma(k, q[rt][f], s[rt]);
            }
            const int key0 = c * LD_KB + kq * 16;
            const bool mask = exist != 0xffff || key0 + 16 > seen0;
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    s[rt][i] *= cs;
                    if (mask) {
                        const int k = grp * 4 + i;
                        const bool keep = ((exist >> k) & 1) && key0 + k < lim[rt];
                        s[rt][i] = keep ? s[rt][i] : -INFINITY;
                    }
                    top = fmaxf(top, s[rt][i]);
                }
                top = fmaxf(top, __shfl_xor(top, 16, WAVE));
                top = fmaxf(top, __shfl_xor(top, 32, WAVE));
                if (grp == 0) tops[kq][(part * RT + rt) * 16 + col] = top;
            }
            lds_barrier();
#pragma unroll
            for (int t = 0; t < TILES; t++) {
                float m1 = m[t];
#pragma unroll
                for (int w = 0; w < 4; w++) m1 = fmaxf(m1, tops[w][t * 16 + col]);
                const float ref = m1 == -INFINITY ? 0.f : m1;  // a row with no key so far
                const int rt = t - part * RT;
                const bool own = RH == 1 || (rt >= 0 && rt < RT);
                if (__any(m1 > m[t])) {
                    const float shrink = __builtin_amdgcn_exp2f(m[t] - ref);
#pragma unroll
                    for (int x = 0; x < RT; x++)
                        if (x == rt) l[x] *= shrink;
#pragma unroll
                    for (int j = 0; j < NT; j++)
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[t][j][i] *= shrink;
                    m[t] = m1;
                }
                if (own) {
#pragma unroll
                    for (int x = 0; x < RT; x++)
                        if (x == rt) {
                            float p[4];
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                p[i] = __builtin_amdgcn_exp2f(s[x][i] - ref);
                                l[x] += p[i];
                            }
                            *reinterpret_cast<uint64_t*>(
                                wt + ld_weight(t * 16 + col, kq * 2 + (grp >> 1)) + (grp & 1) * 8) =
                                bits4(p);
                        }
                }
            }
            lds_barrier();
#pragma unroll
            for (int ks = 0; ks < LD_KB / 32; ks++) {
                bf16x8 pb[TILES];
#pragma unroll
                for (int t = 0; t < TILES; t++)
                    pb[t] = *reinterpret_cast<const bf16x8*>(
                        wt + ld_weight(t * 16 + col, ks * 4 + grp));
                const int r = ks * 32 + grp * 8 + ((lane >> 2) & 3);
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const int pc = (wave * NT + j) * 2 + ((lane & 3) >> 1);
                    const bf16x8 v = join(lds_read_tr(kt + X::lat(r, pc) + (lane & 1) * 8),
                                          lds_read_tr(kt + X::lat(r + 4, pc) + (lane & 1) * 8));
#pragma unroll
                    for (int t = 0; t < TILES; t++)
                        acc[t][j] = Mma<bf16>::mma(v, pb[t], acc[t][j]);
                }
            }
        }

        // total of the running sums over lanes and waves
        const bool whole = c0 == 0 && c1 == nch;
        const int slot = 2 * (int)blockIdx.x + (run.pos == run_start ? 0 : 1);
        lds_barrier();
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            float t = l[rt];
            t += __shfl_xor(t, 16, WAVE);
            t += __shfl_xor(t, 32, WAVE);
            if (grp == 0) tops[kq][(part * RT + rt) * 16 + col] = t;
        }
        lds_barrier();
#pragma unroll
        for (int t = 0; t < TILES; t++) {
            const int rr = t * 16 + col, r = row0 + rr;
            if (r < a.rows) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < 4; w++) sum += tops[w][rr];
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
                bf16* dst = reinterpret_cast<bf16*>(a.o_lat) + ((size_t)b * a.rows + r) * R;
                float* out = a.part_o + ((size_t)slot * ROWS + rr) * R;
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const int d = (wave * NT + j) * 16 + grp * 4;
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) x[i] = whole ? acc[t][j][i] * inv : acc[t][j][i];
                    if (whole) store4<bf16>(dst + d, x);
                    else store4<float>(out + d, x);
                }
                if (!whole && wave == 0 && grp == 0) {
                    float* pm = a.part_ml + ((size_t)slot * ROWS + rr) * 2;
                    pm[0] = m[t];
                    pm[1] = sum;
                }
            }
        }
        lds_barrier();  // the next unit writes tops and the tiles

        run.pos += c1 - c0;
        if (run.pos < run.end && run.pos == run.base + (int64_t)nch * a.split.units) {
            run.base = run.pos;
            do run.b++;
            while (run.b + 1 < a.split.batch && split_chunks<LD_KB>(a.split, run.b) == 0);
        }
    }
}

// -------------------------------------------------------------------------------------- up
// o = W_uv u for one head and 16 (request, position) rows. u is staged in LDS: copied where the
// core finished the row, joined from the parts where its unit was cut, zeros where the request
// has no key.
template <int R, int DV>
__global__ __launch_bounds__(LD_THREADS) void latent_up_kernel(LatentDecodeArgs a) {
    constexpr int PITCH = R * 2 + 16;
    constexpr int PER = R / WAVE;
    __shared__ __align__(16) char u[16 * PITCH];
    const int h = blockIdx.x, base_row = blockIdx.y * 16;
    const int lane = lane_id(), wave = wave_id();
    const int n_rows = a.split.batch * a.n_pos;
    const int tile = 16 * a.rt;
    for (int k = 0; k < 16 / LD_WAVES; k++) {
        const int rr = wave * (16 / LD_WAVES) + k, bp = base_row + rr;
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; i++) x[i] = 0.f;
        bool copy = false;
        if (bp < n_rows) {
            const int b = bp / a.n_pos, row = (bp - b * a.n_pos) * a.H + h;
            const int unit = row / tile, r = row - unit * tile;
            const int nch = split_chunks<LD_KB>(a.split, b);
            if (nch > 0) {
                int64_t base, total;
                split_base<LD_KB>(a.split, b, &base, &total);
                const int64_t u0 = base + (int64_t)unit * nch;
                const int n = split_wgs(total, a.n_wg);
                const int w0 = split_owner(u0, total, n), w1 = split_owner(u0 + nch - 1, total, n);
                copy = w0 == w1;
                if (copy) {
                    const bf16* src = reinterpret_cast<const bf16*>(a.o_lat) +
                                      ((size_t)bp * a.H + h) * R;
#pragma unroll
                    for (int i = 0; i < PER; i++) x[i] = (float)src[lane * PER + i];
                } else {
                    const int late = split_start(w0, total, n) < u0 ? 1 : 0;
                    auto at = [&](int w) {
                        return (size_t)(2 * w + (w == w0 ? late : 0)) * tile + r;
                    };
                    float top = -INFINITY;
                    for (int w = w0 + lane; w <= w1; w += WAVE)
                        top = fmaxf(top, a.part_ml[at(w) * 2]);
#pragma unroll
                    for (int off = WAVE / 2; off > 0; off >>= 1)
                        top = fmaxf(top, __shfl_xor(top, off, WAVE));
                    const float ref = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
#pragma unroll 4
                    for (int w = w0; w <= w1; w++) {
                        const size_t e = at(w);
                        const float f = __builtin_amdgcn_exp2f(a.part_ml[e * 2] - ref);
                        sum = fmaf(f, a.part_ml[e * 2 + 1], sum);
#pragma unroll
                        for (int i = 0; i < PER; i++)
                            x[i] = fmaf(f, a.part_o[e * R + lane * PER + i], x[i]);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                    for (int i = 0; i < PER; i++) x[i] *= inv;
                }
            }
        }
        bf16* dst = reinterpret_cast<bf16*>(u + rr * PITCH) + lane * PER;
#pragma unroll
        for (int i = 0; i < PER; i++) dst[i] = (bf16)x[i];
    }
    __syncthreads();
    const int col = lane & 15, grp = lane >> 4;
    const bf16* W = reinterpret_cast<const bf16*>(a.w_kv) +
                    ((size_t)h * (a.d_nope + DV) + a.d_nope) * R;
    const int bp = base_row + col;
#pragma unroll
    for (int j = 0; j < DV / 16 / LD_WAVES; j++) {
        const int t = j * LD_WAVES + wave;
        f32x4 d = zero4();
#pragma unroll
        for (int k = 0; k < R / 32; k++)
            d = Mma<bf16>::mma(Mma<bf16>::load(W + (size_t)(t * 16 + col) * R + k * 32 + grp * 8),
                               *reinterpret_cast<const bf16x8*>(u + col * PITCH + k * 64 + grp * 16),
                               d);
        float y[4] = {d[0], d[1], d[2], d[3]};
        if (bp < n_rows)
            store4<bf16>(reinterpret_cast<bf16*>(a.o) + ((size_t)bp * a.H + h) * DV + t * 16 +
                             grp * 4, y);
    }
}

template <int DN>
void run_absorb(const LatentDecodeArgs& a, hipStream_t s) {
    const int tiles = (a.split.batch * a.n_pos + 15) / 16;
    const int per = tiles < 8 ? tiles : 8;
    hipLaunchKernelGGL(latent_absorb_kernel<DN>,
                       dim3((unsigned)a.H, (unsigned)(a.rank / AB_COLS),
                            (unsigned)((tiles + per - 1) / per)),
                       dim3(LD_THREADS), 0, s, a, per);
}

template <int R>
hipError_t run_core(const LatentDecodeArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.n_wg), block(LD_THREADS);
    switch (a.rt) {
        case 1: hipLaunchKernelGGL((latent_core_kernel<R, 1, 1>), grid, block, 0, s, a); break;
        case 2: hipLaunchKernelGGL((latent_core_kernel<R, 2, 1>), grid, block, 0, s, a); break;
        case 4:
            hipLaunchKernelGGL((latent_core_kernel<R, 2, 2>), grid, dim3(2 * LD_THREADS), 0, s, a);
            break;
        default: return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 up((unsigned)a.H, (unsigned)((a.split.batch * a.n_pos + 15) / 16));
    if (a.d_v == 128) hipLaunchKernelGGL((latent_up_kernel<R, 128>), up, block, 0, s, a);
    else hipLaunchKernelGGL((latent_up_kernel<R, 64>), up, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t latent_decode_layout(LatentDecodeArgs* a, void* ws) {
    a->rows = a->H * a->n_pos;
    const int tiles = (a->rows + 15) / 16;
    a->rt = tiles >= 3 ? 4 : tiles;
    a->row_tiles = (tiles + a->rt - 1) / a->rt;
    a->split.units = a->row_tiles;
    a->n_wg = device_cu_count();
    const size_t part = (size_t)2 * a->n_wg * 16 * a->rt;
    const size_t lat = (size_t)a->split.batch * a->rows * a->rank;  // bf16 elements
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = ws == nullptr ? nullptr : static_cast<char*>(ws) + off;
        off += (bytes + 255) & ~(size_t)255;
        return p;
    };
    a->part_o = reinterpret_cast<float*>(take(part * a->rank * sizeof(float)));
    a->part_ml = reinterpret_cast<float*>(take(part * 2 * sizeof(float)));
    a->q_lat = take(lat * 2);
    a->o_lat = take(lat * 2);
    return off;
}

hipError_t launch_latent_decode(const LatentDecodeArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    if (a.d_nope == 128) run_absorb<128>(a, s);
    else run_absorb<64>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return a.rank == 512 ? run_core<512>(a, s) : run_core<256>(a, s);
}

}  // namespace gdn
