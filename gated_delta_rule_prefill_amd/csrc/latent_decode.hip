// Latent attention of the newest n_pos tokens of each request, absorbed form
// (gdn_latent_decode), bf16.
//
// A token's cache row is a latent c_j (rank elements) shared by all heads and a rotary key r_j
// (64). Head h's key is (W_uk,h c_j, r_j) and its value W_uv,h c_j, so with
//   q'_h = W_uk,h^T q_nope,h      (absorb)
//   s_j = scale (q'_h . c_j + q_pe,h . r_j),  p = softmax(s),  u_h = sum_j p_j c_j   (core)
//   o_h = W_uv,h u_h              (up)
// no key or value of a head is ever written out: the core reads each cache row once for all
// heads. Four launches; the core's work split is key_split.h's, the join between core and up
// key_join.h's.
#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"
#include "key_join.h"
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

// The absorbed queries enter the core's products as the sum of two numbers: their rounding to bf16
// and what that leaves, the rest, in 4 bits (fp4, e2m1) times a unit that 128 columns of a row
// share, 2^-10 of the binade of the largest: a rest is 4 units at most, held to half a unit, to a
// quarter where it is small. One bf16 number moves a row's scores by its rounding of q', and
// outputs were off by 0.0025 to 0.0029 (relative 2-norm; their own rounding leaves 0.0017); with
// the rests by 0.0019, the weights' rounding. A second bf16 number would take 64 registers, which
// the tile of 64 rows does not have. The rests cost a product for each one of the latents' scores:
// 80 requests, 128 heads 136 -> 157 us a call, one request of 40003 tokens, 20 heads 33.7 -> 36 us.
// Until the core writes a row's outputs, its rests lie in their place: only workers that hold a part
// of a unit read them, and one that writes there holds all of it.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int R>
struct LdRest {
    static constexpr int PER_GROUP = R / 32;  // words of 8 codes that a lane group reads
    static constexpr int UNITS_AT = R / 8;    // float offset of the units
    __device__ __forceinline__ static uint32_t* word(float* o_row, int grp, int f) {
        return reinterpret_cast<uint32_t*>(o_row) + grp * PER_GROUP + f;
    }
};
// The unit of 128 columns, by the largest: 2^-10 of its binade.
__device__ __forceinline__ float rest_unit(float top) {
    return __uint_as_float((max(__float_as_uint(top) >> 23, 11u) - 10u) << 23);
}
// 8 numbers to codes of a unit, and back.
__device__ __forceinline__ uint32_t to_fp4(const float (&x)[8], float unit) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], unit, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], unit, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], unit, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], unit, 3);
    return c;
}
__device__ __forceinline__ bf16x8 from_fp4(uint32_t c, float unit) {
    return __builtin_bit_cast(
        bf16x8,
        u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, unit, 0)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, unit, 1)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, unit, 2)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, unit, 3))});
}

// ---------------------------------------------------------------------------------- absorb
// q'^T (rank x rows) = W_uk^T q_nope^T per head: a workgroup takes 128 rank columns of one
// head's W_uk (through LDS, read back transposed as the MFMA's A operand) and 64 (request,
// position) rows, all loads issued at once: one trip to memory. Bound: that trip, and for many rows
// the weights (16.8 MB at 128 heads, d = 128, rank 512). Measured: 80 rows, 128 heads 14 us; one
// row, 20 heads 3.7 us.
constexpr int AB_COLS = 128, AB_TILES = 4;

// LDS position of the 16-byte piece c of row n (rows of AB_COLS elements = 16 pieces): the 16
// rows of a transposing read are 8 g + (0..3), so pairs of pieces turn by those bits
__device__ __forceinline__ int ab_place(int n, int c) {
    const int turn = (n & 3) | ((n >> 1) & 4);
    return n * (AB_COLS * 2) + ((c ^ (turn << 1)) << 4);
}

template <int DN, int R>
__global__ __launch_bounds__(LD_THREADS) void latent_absorb_kernel(LatentDecodeArgs a) {
    __shared__ __align__(16) char w[DN * AB_COLS * 2];
    __shared__ float tops[LD_WAVES][AB_TILES * 16];  // largest |q'| of a wave's columns of a row
    const int h = blockIdx.x, r0 = blockIdx.y * AB_COLS;
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int col = lane & 15, grp = lane >> 4;
    const int rows = a.split.batch * a.n_pos, row0 = blockIdx.z * (AB_TILES * 16);
    const bf16* W = reinterpret_cast<const bf16*>(a.w_kv) +
                    (size_t)h * (a.d_nope + a.d_v) * R + r0;
    f32x4 in[DN * 16 / LD_THREADS];
#pragma unroll
    for (int i = 0; i < DN * 16 / LD_THREADS; i++) {
        const int x = i * LD_THREADS + tid;
        in[i] = *reinterpret_cast<const f32x4*>(W + (size_t)(x >> 4) * R + (x & 15) * 8);
    }
    bf16x8 B[AB_TILES][DN / 32];
#pragma unroll
    for (int t = 0; t < AB_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
        const bf16* q = reinterpret_cast<const bf16*>(a.q_nope) +
                        ((size_t)min(row0 + t * 16 + col, rows - 1) * a.H + h) * DN;
#pragma unroll
        for (int k = 0; k < DN / 32; k++) B[t][k] = Mma<bf16>::load(q + k * 32 + grp * 8);
    }
    sched_fence();
#pragma unroll
    for (int i = 0; i < DN * 16 / LD_THREADS; i++) {
        const int x = i * LD_THREADS + tid;
        *reinterpret_cast<f32x4*>(w + ab_place(x >> 4, x & 15)) = in[i];
    }
    __syncthreads();
    // Two MFMA rows tiles of 16 rank columns each, dealt out so that a lane's four rows of both
    // are 8 consecutive columns (a transposing read takes any four columns per lane): 8 g + 4 x.
    bf16x8 A[2][DN / 32];
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
        for (int k = 0; k < DN / 32; k++) {
            const int n = k * 32 + grp * 8 + ((lane >> 2) & 3), c = wave * 4 + (lane & 3);
            A[x][k] = join(lds_read_tr(w + ab_place(n, c) + x * 8),
                           lds_read_tr(w + ab_place(n + 4, c) + x * 8));
        }
    float y[AB_TILES][8];
#pragma unroll
    for (int t = 0; t < AB_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
        float top = 0.f;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            f32x4 d = zero4();
#pragma unroll
            for (int k = 0; k < DN / 32; k++) d = Mma<bf16>::mma(A[x][k], B[t][k], d);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                y[t][x * 4 + i] = d[i];
                top = fmaxf(top, fabsf(d[i]));
            }
        }
        top = max_groups(top);
        if (grp == 0) tops[wave][t * 16 + col] = top;
    }
    __syncthreads();
    // words of the rests through LDS (where the weights were), stored 16 bytes a lane
    uint32_t* words = reinterpret_cast<uint32_t*>(w);  // [row][lane group][wave]
    auto unit_of = [&](int r) {
        return rest_unit(fmaxf(fmaxf(tops[0][r], tops[1][r]), fmaxf(tops[2][r], tops[3][r])));
    };
#pragma unroll
    for (int t = 0; t < AB_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
        const int row = row0 + t * 16 + col;
        float rest[8];
#pragma unroll
        for (int i = 0; i < 8; i++) rest[i] = y[t][i] - (float)(bf16)y[t][i];
        words[(t * 16 + col) * 16 + grp * 4 + wave] = to_fp4(rest, unit_of(t * 16 + col));
        if (row < rows)
            store8<bf16>(reinterpret_cast<bf16*>(a.q_lat) + ((size_t)row * a.H + h) * R + r0 +
                             wave * 32 + grp * 8, y[t]);
    }
    __syncthreads();
    static_assert(AB_TILES * 16 * 4 == LD_THREADS && LD_WAVES == 4, "a thread for each 16 bytes");
    const int r = tid >> 2, row = row0 + r;
    if (row < rows) {
        float* o_row = a.o_lat + ((size_t)row * a.H + h) * R;
        *reinterpret_cast<u32x4*>(LdRest<R>::word(o_row, tid & 3, r0 / 32)) =
            *reinterpret_cast<const u32x4*>(words + tid * 4);
        if ((tid & 3) == 0) o_row[LdRest<R>::UNITS_AT + r0 / AB_COLS] = unit_of(r);
    }
}

// ------------------------------------------------------------------------------------ core
// A workgroup holds one row tile (16 RH query rows) and walks 64 keys at a time:
//   S^T = K Q^T   each wave takes 16 KS of the keys for 16 of the rows; the queries stay in
//                 registers, K fragments come from LDS;
//   softmax       weights go to LDS as bf16; the waves of a row share its running reference;
//   U^T += C^T P^T  each wave takes its share of the rank for all rows; C^T by transposing LDS
//                 reads of the very tile the scores came from.
// So each cache row is read once from memory per row tile; from LDS a tile is read RH times as
// keys and once as values. The next tile loads straight into the other LDS buffer meanwhile.
// Bound: a unit's start and end (queries, the first tile's trip, results: as long as 6 tiles) and,
// for 64 rows, a tile's matrix work, LDS reads and conversions of rests.
// Measured at rank 512: 80 requests of 100 to 12000 tokens (223 MB), 128 heads 113 us, 2.0 TB/s; one
// request of 40003 tokens (46 MB), 20 heads 19 us.
// (64 rows with 32 rows a wave read the keys twice only, but their queries take 144 registers:
// the compiler then spills inside the key loop, and a reload from scratch memory waits for the
// tile loads issued before it. As it is, 11 registers of the kernel for 64 rows of rank 512 are
// spilled before its first unit and come back at the end of one: none inside the key loop.)
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
    __device__ __forceinline__ static int lat(int r, int c) {
        return r * LAT + ((c ^ turn(r)) << 4);
    }
    __device__ __forceinline__ static int rope(int r, int c) {
        return ROPE_AT + r * (LD_ROPE * 2) + ((c ^ ((r >> 1) & 7)) << 4);
    }
};

// Weights [16 RT rows][64 keys] bf16, pieces of 8 keys turned by the row.
__device__ __forceinline__ int ld_weight(int row, int piece) {
    return row * (LD_KB * 2) + ((piece ^ ((row >> 1) & 7)) << 4);
}

// Four keys of 16 that rows 4 a .. of a key fragment are: 0, 2, 3, 1. A 16-byte LDS read takes
// lanes 0-3, 12-15, 20-23 and 24-27 at a time (then 4-11, 16-19, 28-31; then those 32 on), and in
// this order their pieces lie in 16 different bank groups (in memory order a tile's key reads took
// twice as long; 80 requests, 128 heads: 143.5 and 137.5 us a call).
__device__ __forceinline__ int ld_quad(int a) { return ((a ^ a >> 1) & 1) << 1 | a >> 1; }

template <int RH, int KS>
struct LdWaves {
    static constexpr int KEYS = 16 * KS;            // keys of a wave
    static constexpr int GROUPS = LD_KB / KEYS;     // waves side by side along the keys
    static constexpr int WAVES = GROUPS * RH;
    static constexpr int OWN = LD_KB / WAVES;       // tile rows that a wave loads
};

template <int R, int RH, int KS>
__global__ __launch_bounds__((LdWaves<RH, KS>::WAVES * WAVE)) void latent_core_kernel(
    LatentDecodeArgs a) {
    using X = LdTile<R>;
    using Y = LdWaves<RH, KS>;
    constexpr int WAVES = Y::WAVES, KEYS = Y::KEYS, OWN = Y::OWN;
    constexpr uint64_t ALL = (1ull << KEYS) - 1;
    constexpr int ROWS = 16 * RH;
    constexpr int NL = R / 32, NF = NL + LD_ROPE / 32;  // key fragments: latent, then rotary
    constexpr int NT = R / 16 / WAVES;                  // 16-column output tiles per wave
    __shared__ __align__(1024) char tile[2 * X::BYTES];
    __shared__ __align__(1024) char wt[ROWS * LD_KB * 2];
    __shared__ float tops[Y::GROUPS][ROWS];  // row maxima of a tile per key group; then row sums
    __shared__ float shrinks[ROWS];          // what a new reference scales older sums by
    __shared__ int flags[WAVES];             // a wave's rows have outgrown their reference
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int col = lane & 15, grp = lane >> 4;
    const int kg = wave / RH, part = wave % RH;  // key group and 16-row part of the scores
    const int key_row = kg * KEYS;               // first tile row of this wave's keys
    const SplitPlace me = split_place(blockIdx.x, a.row_tiles);
    int own_keys = me.worker < a.split.batch ? split_keys(a.split, me.worker) : 1;
    SplitRun run = split_run<LD_KB, WAVES * WAVE>(a.split, me.worker, a.workers);
    const int run_start = run.pos;
    const int row0 = me.row_tile * ROWS;
    if (me.row_tile == 0) {
        // requests without keys: zeros, and nothing to join
        for (int b = me.worker; b < a.split.batch; b += a.workers) {
            if (b != me.worker) own_keys = split_keys(a.split, b);
            if (uniform(own_keys) != 0) continue;
            const size_t n = (size_t)a.rows * R;
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            for (size_t i = threadIdx.x * 4; i < n; i += WAVES * WAVE * 4)
                store4<float>(a.o_lat + (size_t)b * n + i, z);
            if (a.join.per_unit && threadIdx.x == 0) join_none(a.join, b);
        }
        if (!a.join.per_unit && threadIdx.x == 0) join_none(a.join, me.worker);
    }
    // The scale enters the exponent's multiplication; a negative one is moved into the queries,
    // so that the largest score is the largest weight (and zero makes the queries zero).
    const float cs = a.scale == 0.f ? 1.f : fabsf(a.scale) * LOG2E;
    const char* cache = reinterpret_cast<const char*>(a.cache);

    // LDS byte offsets of this lane's reads and writes within a tile or the weights. A piece
    // index is xored with a function of the row, so its constant part can be xored in last, and
    // one offset serves all pieces of a kind.
    const int key_of = ld_quad(col >> 2) * 4 + (col & 3);
    const uint32_t k_at = X::lat(key_row + key_of, grp), pe_at = X::rope(key_row + key_of, grp);
    const uint32_t p_at = ld_weight(col, grp);
    const uint32_t p_put = ld_weight(col, kg * KS * 2 + (ld_quad(grp) >> 1)) +
                           (ld_quad(grp) & 1) * 8;
    const uint32_t v_at = X::lat(grp * 8 + ((lane >> 2) & 3), wave * NT * 2 + ((lane & 3) >> 1)) +
                          (lane & 1) * 8;

    while (run.pos < run.end) {
        const int b = run.b;
        const int nkeys = uniform(split_keys(a.split, b));
        const int nch = (nkeys + LD_KB - 1) / LD_KB;
        const int c0 = run.pos - run.base;
        const int next_unit = run.base + nch + a.split.extra;
        if (c0 >= nch) {  // the run starts behind the unit's own chunks
            run.advance(a.split, next_unit, next_unit);
            continue;
        }
        const int c1 = min(nch, c0 + (run.end - run.pos));
        const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
        const int seen0 = uniform(a.split.seq_lens[b]) - a.n_pos + 1;  // keys that position 0 sees

        // the table entry of lane's key among this wave's keys of a chunk (KEYS lanes, repeated);
        // keys past the end read the table's last entry, and load_tile() drops them
        int page;
        auto load_pages = [&](int c) {
            const uint32_t key = (uint32_t)(c * LD_KB + key_row + lane % KEYS);
            page = table[min(a.block(key), (uint32_t)a.max_blocks - 1)];
        };
        uint64_t exist, exist_next = 0;
        // Tile c into a buffer, its pages being in `page`, which then takes those of chunk `next`.
        // (That load goes first: the compiler's wait for it must not be behind the tile's.)
        auto load_tile = [&](int c, int buf, int next) {
            arrived(page);
            const uint32_t key = (uint32_t)(c * LD_KB + key_row + lane % KEYS);
            const uint32_t off = key - a.block(key) * a.block.div;
            const bool ok = (int)key < nkeys && page >= 0 && page < a.n_blocks;
            const uint32_t slot = ok ? (uint32_t)page * a.block.div + off : 0u;
            exist_next = __ballot(ok) & ALL;
            load_pages(next);
            sched_fence();
            const uint32_t at = lds_offset(tile) + buf * X::BYTES;
            const int first = part * OWN;
            if constexpr (X::PIECES == 64) {
                // turn(first + i) = turn(first) ^ turn(i); the lane part is hidden from the
                // compiler, which would keep one register per row alive across the key loop
                int piece = lane ^ X::turn(first);
                asm volatile("" : "+v"(piece));
#pragma unroll
                for (int i = 0; i < OWN; i++) {
                    const int r = first + i;
                    const uint32_t s = __builtin_amdgcn_readlane(slot, r);
                    load_to_lds(cache + (size_t)s * X::ROW, (uint32_t)((piece ^ X::turn(i)) << 4),
                                at + (key_row + r) * X::LAT);
                }
            } else {  // two rows per load
#pragma unroll
                for (int i = 0; i < OWN; i += 2) {
                    const int r = first + i, rr = r + (lane >> 5);
                    const uint32_t s = __shfl(slot, rr, WAVE);
                    load_to_lds(cache + (size_t)s * X::ROW + (((lane & 31) ^ X::turn(rr)) << 4),
                                at + (key_row + r) * X::LAT);
                }
            }
#pragma unroll
            for (int i = 0; i < OWN; i += 8) {
                const int r = first + i, rr = r + (lane >> 3);
                const uint32_t s = __shfl(slot, rr, WAVE);
                load_to_lds(cache + (size_t)s * X::ROW + X::LAT +
                                (((lane & 7) ^ ((rr >> 1) & 7)) << 4),
                            at + X::ROPE_AT + (key_row + r) * (LD_ROPE * 2));
            }
        };
        load_pages(c0);
        load_tile(c0, 0, c0 + 1);

        bf16x8 q[NF];
        uint32_t rest[NL];  // of the absorbed query
        float unit[NL / 4];
        const int q_row = row0 + part * 16 + col;
        const bool live = q_row < a.rows;
        const int lim = live ? seen0 + q_row / a.H : 0;
        {
            const size_t at = (size_t)b * a.rows + (live ? q_row : row0);
            const bf16* ql = reinterpret_cast<const bf16*>(a.q_lat) + at * R;
            const bf16* qp = reinterpret_cast<const bf16*>(a.q_pe) + at * LD_ROPE;
#pragma unroll
            for (int f = 0; f < NF; f++)
                q[f] = Mma<bf16>::load(f < NL ? ql + f * 32 + grp * 8
                                              : qp + (f - NL) * 32 + grp * 8);
            float* o_row = a.o_lat + at * R;
            typedef float units __attribute__((ext_vector_type(NL / 4)));
#pragma unroll
            for (int f = 0; f < NL; f += 4) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(LdRest<R>::word(o_row, grp, f));
#pragma unroll
                for (int i = 0; i < 4; i++) rest[f + i] = x[i];
            }
            const units u = *reinterpret_cast<const units*>(o_row + LdRest<R>::UNITS_AT);
#pragma unroll
            for (int i = 0; i < NL / 4; i++) unit[i] = u[i];
        }
        if (a.scale <= 0.f) {
#pragma unroll
            for (int f = 0; f < NL; f++) rest[f] = a.scale < 0.f ? rest[f] ^ 0x88888888u : 0u;
#pragma unroll
            for (int f = 0; f < NF; f++)
#pragma unroll
                for (int i = 0; i < 8; i++) q[f][i] = a.scale < 0.f ? -q[f][i] : (bf16)0.f;
        }
        arrived(q);
#pragma unroll
        for (int f = 0; f < NL; f++) asm volatile("" : "+v"(rest[f]));
#pragma unroll
        for (int f = 0; f < NL / 4; f++) asm volatile("" : "+v"(unit[f]));
        f32x4 acc[RH][NT];
        float ref = -INFINITY, l = 0.f;  // this lane's row: reference, share of the sum
#pragma unroll
        for (int t = 0; t < RH; t++)
#pragma unroll
            for (int j = 0; j < NT; j++) acc[t][j] = zero4();

        for (int c = c0; c < c1; c++) {
            const int buf = (c - c0) & 1;
            const uint32_t kt = lds_offset(tile) + buf * X::BYTES;
            // (copies that the compiler cannot take for constant over the key loop: it would keep
            // every sum below in a register of its own and spill for it)
            uint32_t k_here = kt + k_at, pe_here = kt + pe_at, v_here = kt + v_at;
            uint32_t p_here = p_at, put_here = p_put;
            asm volatile("" : "+v"(k_here), "+v"(pe_here), "+v"(v_here), "+v"(p_here),
                              "+v"(put_here));
            auto weights = [&](int t) {  // of the 16 rows of row tile t
                return lds_offset(wt) + t * (16 * LD_KB * 2);
            };
            exist = exist_next;
            lds_loads_done();
            if (exist != ALL) {
                // latents of absent keys as zeros: a zero weight does not cancel what they hold
#pragma unroll 1
                for (int r = part * OWN; r < part * OWN + OWN; r++)
                    if (!((exist >> r) & 1) && lane < X::PIECES)
                        lds_put(kt + (key_row + r) * X::LAT + lane * 16, zero4());
            }
            lds_barrier();  // tile c is whole; all waves are done with the other buffer
            if (c + 1 < c1) load_tile(c + 1, buf ^ 1, c + 2);
            f32x4 s[KS];
#pragma unroll
            for (int x = 0; x < KS; x++) s[x] = zero4();
            // key fragments SF steps of the contraction at a time, the next ones on their way; rests
            // one step ahead
            constexpr int SF = KS == 1 ? 2 : 1;
            bf16x8 k[2][SF][KS];
            auto load_k = [&](int f, bf16x8 (&to)[KS]) {
#pragma unroll
                for (int x = 0; x < KS; x++)  // (16 rows on, the pieces are turned alike)
                    to[x] = lds_get<bf16x8>(
                        f < NL ? (k_here ^ (f & 3) << 6) + (f >> 2) * 256 + x * (16 * X::LAT)
                               : (pe_here ^ (f - NL) << 6) + x * (16 * LD_ROPE * 2));
            };
#pragma unroll
            for (int e = 0; e < SF; e++) load_k(e, k[0][e]);
            auto rest_at = [&](int f) {
                // (converted anew for every tile: the compiler would keep all of them)
                asm volatile("" : "+v"(rest[f]));
                return from_fp4(rest[f], unit[f / 4]);
            };
            bf16x8 low_next = rest_at(0);
#pragma unroll
            for (int f = 0; f < NF; f += SF) {
                const int now = f / SF & 1;
                if (f + SF < NF) {
#pragma unroll
                    for (int e = 0; e < SF; e++) load_k(f + SF + e, k[now ^ 1][e]);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < SF; e++) {
                    const bf16x8 low = low_next;
                    if (f + e + 1 < NL) low_next = rest_at(f + e + 1);
#pragma unroll
                    for (int x = 0; x < KS; x++) s[x] = Mma<bf16>::mma(k[now][e][x], q[f + e], s[x]);
                    if (f + e < NL) {
#pragma unroll
                        for (int x = 0; x < KS; x++)
                            s[x] = Mma<bf16>::mma(k[now][e][x], low, s[x]);
                    }
                }
            }
            const int key0 = c * LD_KB + key_row;
            if (exist != ALL || key0 + KEYS > seen0) {
                // this lane's keys are key0 + first + 16 x + i (`first` hidden from the compiler, which
                // would keep what depends on it in registers across the key loop)
                int first = ld_quad(grp) * 4;
                asm volatile("" : "+v"(first));
                const uint64_t here = exist >> first;
                const int left = lim - key0 - first;
#pragma unroll
                for (int x = 0; x < KS; x++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const bool keep = ((here >> (x * 16 + i)) & 1) && x * 16 + i < left;
                        s[x][i] = keep ? s[x][i] : -INFINITY;
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int x = 0; x < KS; x++)
#pragma unroll
                for (int i = 0; i < 4; i++) top = fmaxf(top, s[x][i]);
            top = max_groups(top) * cs;
            float p[KS][4];
            auto weigh = [&]() {
                const float shift = ref == -INFINITY ? 0.f : ref;  // a row with no key so far
#pragma unroll
                for (int x = 0; x < KS; x++) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        p[x][i] = __builtin_amdgcn_exp2f(fmaf(s[x][i], cs, -shift));
                    lds_put((weights(part) + put_here) ^ x << 5, bits4(p[x]));
                }
            };
            // Weights by the reference so far. If a row's maximum has outgrown it in any wave (all
            // see the flags behind the barrier), the waves of a row agree on a new reference and
            // weigh again: a few tiles of a request, which saves the others a barrier.
            weigh();
            const int grew = __any(top > ref + LAG);
            if (lane == 0) flags[wave] = grew;
            lds_barrier();
            if (__any(flags[lane % WAVES])) {
                if (grp == 0) tops[kg][part * 16 + col] = top;
                lds_barrier();
                float most = tops[0][part * 16 + col];
#pragma unroll
                for (int g = 1; g < Y::GROUPS; g++) most = fmaxf(most, tops[g][part * 16 + col]);
                const bool grown = most > ref + LAG;
                const float shrink = grown ? __builtin_amdgcn_exp2f(ref - most) : 1.f;
                ref = grown ? most : ref;
                l *= shrink;
                if (kg == 0 && grp == 0) shrinks[part * 16 + col] = shrink;
                weigh();
                lds_barrier();
#pragma unroll
                for (int t = 0; t < RH; t++) {
                    const float f = shrinks[t * 16 + col];
#pragma unroll
                    for (int j = 0; j < NT; j++)
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[t][j][i] *= f;
                }
            }
#pragma unroll
            for (int x = 0; x < KS; x++)
#pragma unroll
                for (int i = 0; i < 4; i++) l += p[x][i];
            // values VB fragments at a time, the next ones on their way
            constexpr int VB = RH == 4 ? 2 : NT < 4 ? NT : 4, NB = LD_KB / 32 * (NT / VB);
            bf16x8 v[2][VB];
            auto load_v = [&](int n) {
                const int ks = n / (NT / VB), j0 = n % (NT / VB) * VB;
#pragma unroll
                for (int j = 0; j < VB; j++) {
                    // the second half lies 4 rows on, where the lowest piece bit is turned
                    const uint32_t at = v_here ^ (j0 + j) << 5;
                    v[n & 1][j] = join(lds_read_tr(at + ks * (32 * X::LAT)),
                                       lds_read_tr((at ^ 16) + ks * (32 * X::LAT) + 4 * X::LAT));
                }
            };
            load_v(0);
            bf16x8 w[RH];
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const int ks = n / (NT / VB), j0 = n % (NT / VB) * VB;
                if (j0 == 0) {
#pragma unroll
                    for (int t = 0; t < RH; t++)
                        w[t] = lds_get<bf16x8>((weights(t) + p_here) ^ ks << 6);
                }
                if (n + 1 < NB) load_v(n + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < RH; t++)
#pragma unroll
                    for (int j = 0; j < VB; j++)
                        acc[t][j0 + j] = Mma<bf16>::mma(v[n & 1][j], w[t], acc[t][j0 + j]);
            }
        }

        // total of the running sums over lanes and waves
        const bool whole = c0 == 0 && c1 == nch;
        if (c0 == 0 && me.row_tile == 0 && threadIdx.x == 0)
            join_note(a.join, a.split, run, me.worker, b, 0, c1, nch, run.pos != run_start);
        const int slot = 2 * me.worker + (run.pos == run_start ? 0 : 1);
        const size_t part_row = ((size_t)slot * a.row_tiles + me.row_tile) * ROWS;
        lds_barrier();
        l += __shfl_xor(l, 16, WAVE);
        l += __shfl_xor(l, 32, WAVE);
        if (grp == 0) tops[kg][part * 16 + col] = l;
        lds_barrier();
#pragma unroll
        for (int t = 0; t < RH; t++) {
            const int rr = t * 16 + col, r = row0 + rr;
            if (r < a.rows) {
                float sum = 0.f;
#pragma unroll
                for (int g = 0; g < Y::GROUPS; g++) sum += tops[g][rr];
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
                float* out = whole ? a.o_lat + ((size_t)b * a.rows + r) * R
                                   : a.join.part_o + (part_row + rr) * R;
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const int d = (wave * NT + j) * 16 + grp * 4;
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) x[i] = whole ? acc[t][j][i] * inv : acc[t][j][i];
                    store4<float>(out + d, x);
                }
                if (!whole && wave == 0 && grp == 0) a.join.part_ml[(part_row + rr) * 2 + 1] = sum;
            }
        }
        if (!whole && kg == 0 && grp == 0 && live)
            a.join.part_ml[(part_row + part * 16 + col) * 2] = ref;
        lds_barrier();  // the next unit writes tops and the tiles

        run.advance(a.split, c1 == nch ? next_unit : run.pos + c1 - c0, next_unit);
    }
}

// ------------------------------------------------------------------------------------ join
// Weighted latents of the units that were cut.
template <int R>
__global__ __launch_bounds__(JOIN_THREADS) void latent_join_kernel(LatentDecodeArgs a) {
    join_parts<R>(a.join, [&](int b, int, int row, int col, const float x[4]) {
        store4<float>(a.o_lat + ((size_t)b * a.rows + row) * R + col, x);
    });
}

// -------------------------------------------------------------------------------------- up
// o = W_uv u for one head and 32 (request, position) rows. u is taken as the sum of two bf16
// numbers, its rounding and the rounding of what that leaves (which leaves 2^-16 of it): one more
// MFMA each, in a kernel that waits for memory, for an output error that is a third smaller.
// Everything is requested at once (the weights as the MFMA's A operand into registers, the rows
// of u into LDS), so a workgroup pays one trip to memory. Measured: 80 rows, 128 heads, rank 512,
// d = 128 15 us (38 MB); one row, 20 heads 5.7 us. (Joining the parts of a unit here where they
// are few costs more than the join's pass saves: 20.6 us, the join 10 instead of 14.)
constexpr int UP_TILES = 2;

template <int R, int DV>
__global__ __launch_bounds__(LD_THREADS, 2) void latent_up_kernel(LatentDecodeArgs a) {
    constexpr int NJ = DV / 16 / LD_WAVES;
    constexpr int PITCH = R * 2 + 16;                    // LDS row: 16-byte pieces on all banks
    constexpr int PER = 16 * R / 4 / LD_THREADS;         // 4-column pieces of a tile per thread
    __shared__ __align__(16) char lds[UP_TILES][2][16 * PITCH];  // the two parts of u
    const int h = blockIdx.x, lane = lane_id(), wave = wave_id();
    const int col = lane & 15, grp = lane >> 4;
    const int rows = a.split.batch * a.n_pos, row0 = blockIdx.y * (UP_TILES * 16);
    const bf16* W = reinterpret_cast<const bf16*>(a.w_kv) +
                    ((size_t)h * (a.d_nope + DV) + a.d_nope) * R;
    f32x4 u[UP_TILES][PER];
#pragma unroll
    for (int t = 0; t < UP_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int x = i * LD_THREADS + threadIdx.x, r = x / (R / 4), c = x % (R / 4);
            u[t][i] = *reinterpret_cast<const f32x4*>(
                a.o_lat + ((size_t)min(row0 + t * 16 + r, rows - 1) * a.H + h) * R + c * 4);
        }
    }
    bf16x8 w[NJ][R / 32];
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
        for (int k = 0; k < R / 32; k++)
            w[j][k] = Mma<bf16>::load(W + (size_t)((wave * NJ + j) * 16 + col) * R + k * 32 +
                                      grp * 8);
    sched_fence();
#pragma unroll
    for (int t = 0; t < UP_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int x = i * LD_THREADS + threadIdx.x, r = x / (R / 4), c = x % (R / 4);
            float hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                hi[e] = (float)(bf16)u[t][i][e];
                lo[e] = u[t][i][e] - hi[e];
            }
            *reinterpret_cast<uint64_t*>(lds[t][0] + r * PITCH + c * 8) = bits4(hi);
            *reinterpret_cast<uint64_t*>(lds[t][1] + r * PITCH + c * 8) = bits4(lo);
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < UP_TILES; t++) {
        if (row0 + t * 16 >= rows) break;
        f32x4 d[NJ];
#pragma unroll
        for (int j = 0; j < NJ; j++) d[j] = zero4();
#pragma unroll
        for (int k = 0; k < R / 32; k++)
#pragma unroll
            for (int part = 0; part < 2; part++) {
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(lds[t][part] + col * PITCH +
                                                                  k * 64 + grp * 16);
#pragma unroll
                for (int j = 0; j < NJ; j++) d[j] = Mma<bf16>::mma(w[j][k], x, d[j]);
            }
        const int row = row0 + t * 16 + col;
        bf16* out = reinterpret_cast<bf16*>(a.o) + ((size_t)row * a.H + h) * DV;
#pragma unroll
        for (int j = 0; j < NJ; j++) {
            const float y[4] = {d[j][0], d[j][1], d[j][2], d[j][3]};
            if (row < rows) store4<bf16>(out + (wave * NJ + j) * 16 + grp * 4, y);
        }
    }
}

template <int DN, int R>
void run_absorb(const LatentDecodeArgs& a, hipStream_t s) {
    const int tiles = (a.split.batch * a.n_pos + 16 * AB_TILES - 1) / (16 * AB_TILES);
    hipLaunchKernelGGL((latent_absorb_kernel<DN, R>),
                       dim3((unsigned)a.H, (unsigned)(R / AB_COLS), (unsigned)tiles),
                       dim3(LD_THREADS), 0, s, a);
}

template <int R, int RH, int KS>
void core_launch(const LatentDecodeArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((latent_core_kernel<R, RH, KS>), dim3((unsigned)(a.workers * a.row_tiles)),
                       dim3(LdWaves<RH, KS>::WAVES * WAVE), 0, s, a);
}

template <int R>
hipError_t run_core(const LatentDecodeArgs& a, hipStream_t s) {
    switch (a.rt) {
        case 1: core_launch<R, 1, 1>(a, s); break;
        case 2: core_launch<R, 2, 1>(a, s); break;
        case 4: core_launch<R, 4, 2>(a, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int R, int DV>
hipError_t run_up(const LatentDecodeArgs& a, hipStream_t s) {
    const int tiles = (a.split.batch * a.n_pos + 16 * UP_TILES - 1) / (16 * UP_TILES);
    hipLaunchKernelGGL((latent_up_kernel<R, DV>), dim3((unsigned)a.H, (unsigned)tiles),
                       dim3(LD_THREADS), 0, s, a);
    return hipGetLastError();
}

template <int R>
hipError_t run_rank(const LatentDecodeArgs& a, hipStream_t s) {
    if (a.d_nope == 128) run_absorb<128, R>(a, s);
    else run_absorb<64, R>(a, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = run_core<R>(a, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(latent_join_kernel<R>, dim3(join_grid(a.join)), dim3(JOIN_THREADS),
                       0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return a.d_v == 128 ? run_up<R, 128>(a, s) : run_up<R, 64>(a, s);
}

}  // namespace

size_t latent_decode_layout(LatentDecodeArgs* a, void* ws) {
    a->rows = a->H * a->n_pos;
    const int tiles = (a->rows + 15) / 16;
    // Rows of a tile, up to 64 (16 requests of 8000 tokens: 128 heads 85 us with 64 rows, 96 with
    // 32; 16 heads 46 us with 16 rows, 49.5 with 64).
    a->rt = tiles > 2 ? 4 : tiles;
    a->row_tiles = (tiles + a->rt - 1) / a->rt;
    a->split.units = 1;
    // A unit's queries, first tile and results take as long as about 6 chunks (10 us) for tiles of
    // 64 rows at rank 512: 80 requests of 100 to 12000 tokens, 128 heads, took 175 us a call with
    // 0, 164 with 1, 149 with 4, 144.5 with 6, 151 with 8 and 150 with 12 (one product a score
    // then). Smaller tiles and rank 256 start and end sooner; they were not measured and use the
    // same number.
    a->split.extra = SPLIT_EXTRA;
    a->split.halve = 0;  // a tile's buffers leave room for one workgroup a CU
    const int cus = device_cu_count();
    a->workers = split_workers(cus, a->row_tiles);
    JoinShape& j = a->join;
    j.row_tiles = a->row_tiles;
    j.tile = 16 * a->rt;
    j.rows = a->rows;
    join_layout(&j, a->split.batch, a->workers, cus, a->rank);
    const size_t part = (size_t)2 * a->workers * a->row_tiles * j.tile;
    const size_t lat = (size_t)a->split.batch * a->rows * a->rank;  // bf16 elements
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = ws == nullptr ? nullptr : static_cast<char*>(ws) + off;
        off += (bytes + 255) & ~(size_t)255;
        return p;
    };
    j.part_o = reinterpret_cast<float*>(take(part * a->rank * sizeof(float)));
    j.part_ml = reinterpret_cast<float*>(take(part * 2 * sizeof(float)));
    j.notes = reinterpret_cast<int4*>(take((size_t)j.count * sizeof(int4)));
    a->q_lat = take(lat * 2);
    a->o_lat = reinterpret_cast<float*>(take(lat * sizeof(float)));
    return off;
}

hipError_t launch_latent_decode(const LatentDecodeArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    return a.rank == 512 ? run_rank<512>(a, s) : run_rank<256>(a, s);
}

}  // namespace gdn
