// Latent attention of packed prompts, expanded form, causal (gdn_latent_prefill), bf16.
//
// Per head h: k_j = (W_uk,h c_j, r_j), v_j = W_uv,h c_j written out once (expand), then
//   o_i = sum_{j <= pos_i} softmax_j(scale q_i . k_j) v_j   (attend)
// with the running maximum and sum of a softmax over 64-key tiles. Against many queries per key
// the written-out form needs 2 (2 d + 64) operations per (query, key, head) where the absorbed
// form needs 2 (2 rank + 64).
//
// Three launches: the tile tables (prefix sums of the device-resident lengths), expand, attend.
#include <type_traits>

#include "attn_launch.h"
#include "gdn_common.h"
#include "gdn_launch.h"
#include "lds_tile.h"

namespace gdn {

namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WAVES = LP_THREADS / WAVE;
constexpr int LP_ROPE = 64;
constexpr int LP_KB = 64;    // keys of a tile
constexpr int LP_QB = 128;   // query rows of a tile
constexpr float LOG2E = 1.4426950408889634f;

typedef float f32x16 __attribute__((ext_vector_type(16)));

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Written-out keys and values, and the softmax weights, are the roundings that this form makes
// between its inputs and its outputs. They are kept in fp16 (11 significant bits): with bf16
// outputs were off by 0.0030 (relative 2-norm; 0.0017 is their own rounding), with fp16 by 0.0017.
// A call takes 5 % longer, mostly because the matrix pipe draws more power (a library product of
// 8192^3 reaches 1.41 PFLOP/s in bf16 and 1.34 in fp16). fp16's range is made to do by exact
// scalings by powers of two. With |c| < 2^(t + 6) for the latents of a key tile, t a multiple of 8,
// and |w| < 2^(x + 1) for a head's rows of w_kv, a key or value is below rank 2^(t + x + 7); it is
// written times 2^(s - t) with s = 8 - log2 rank - x, that is below 2^15. Tiles whose largest
// latent lies between 2^-2 and 2^6 (a normalised one does) have t = 0, and with weights of about
// rank^-1/2 s is about 2. A tile's typical number (2^-8.5 of the bound) is then 2^-2 at least, and
// one 2^12 times smaller still has as many bits as in bf16.
//   scores   2^(a - s + t) (q 2^-a . k 2^(s - t) + q_pe 2^(s - a) . r 2^-t), 2^a by a row's largest
//            |q|: its fp16 numbers are below 2
//   outputs  a row's sums are kept at the t of the last tile added; a tile whose t the range of the
//            sums does not reach could not add 2^-64 of them, and is left out
constexpr int LP_T_MIN = -48, LP_T_MAX = 64;

__device__ __forceinline__ float exp2i(int e) { return ldexpf(1.f, e); }
// Larger magnitudes of two pairs of bf16 numbers, as bits.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t most, uint32_t x) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t,
                              __builtin_elementwise_max(__builtin_bit_cast(u16x2, most),
                                                        __builtin_bit_cast(u16x2, x & 0x7fff7fffu)));
}
// x without infinities and NaN: they make up what they reach, and must not take the others' bits.
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t x) {
    x &= 0x7fff7fffu;
    uint32_t no;  // from 0x7f80 on, 0x80 more are negative
    asm("v_pk_ashrrev_i16 %0, %1, %2" : "=v"(no) : "s"(0x000f000fu), "v"(x + 0x00800080u));
    return x & ~no;
}
template <bool FINITE, typename V>
__device__ __forceinline__ uint32_t max_magnitudes_of(uint32_t most, V eight) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 x = __builtin_bit_cast(u32x4, eight);
#pragma unroll
    for (int i = 0; i < 4; i++)
        most = max_magnitudes(most, FINITE ? finite_magnitudes(x[i]) : x[i]);
    return most;
}
__device__ __forceinline__ int larger_half(uint32_t most) {
    return (int)max(most & 0xffffu, most >> 16);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
    for (int off = WAVE / 2; off > 0; off >>= 1) x = max(x, __shfl_xor(x, off, WAVE));
    return x;
}
// t by the largest magnitude of a tile's latents (bf16 bits).
__device__ __forceinline__ int lp_shift(int bits) {
    if (bits == 0) return 0;
    const int t = ((bits >> 7) - 127 + 2) & ~7;
    return min(max(t, LP_T_MIN), LP_T_MAX);
}

// Length of request i without the tokens that lie behind total_tokens: those have no rows here
// (a step that overflowed its buffers), and the rows before them keep their positions.
__device__ __forceinline__ int lp_len(const LatentPrefillArgs& a, int i) {
    return max(a.seq_lens[i], 0) - (max(a.cu_seqlens[i + 1], a.total_tokens) - a.total_tokens);
}
// Keys of it that its table can address, and its new tokens.
__device__ __forceinline__ int lp_keys(const LatentPrefillArgs& a, int i) {
    return min(max(lp_len(a, i), 0), a.max_keys);
}
__device__ __forceinline__ int lp_new(const LatentPrefillArgs& a, int i) {
    const int s = min(max(a.cu_seqlens[i], 0), a.total_tokens);
    return max(min(a.cu_seqlens[i + 1], a.total_tokens) - s, 0);
}

// Last i < n with first[i] <= t.
__device__ __forceinline__ int lp_find(const int32_t* first, int n, int t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Key tiles that query tile qt of request i sees.
__device__ __forceinline__ int lp_key_tiles(const LatentPrefillArgs& a, int i, int qt) {
    const int fresh = lp_new(a, i), q0 = (qt - a.q_tile[i]) * LP_QB;
    const int keys = min(lp_keys(a, i), (a.key_tile[i + 1] - a.key_tile[i]) * LP_KB);
    const int reach = min(keys, lp_len(a, i) - fresh + min(q0 + LP_QB, fresh));
    return reach > 0 ? (reach + LP_KB - 1) / LP_KB : 0;
}

// ---------------------------------------------------------------------------------- tables
// Prefix sums of each request's key and query tiles, cut off at the host's bounds (lengths
// that break the contract then lose keys or rows, never memory): the first workgroup. 3 us.
// The others: s of a head's keys or values, from its largest weight; 7 us in all.
__device__ __forceinline__ void lp_head_shift(const LatentPrefillArgs& a, int n) {
    __shared__ int most[LP_WAVES];
    const int rows = a.d * a.rank / 8;  // pieces of 8 weights
    const f32x4* w = reinterpret_cast<const f32x4*>(a.w_kv) + (size_t)n * rows;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < rows; i += 8 * LP_THREADS) {  // (2048 pieces or a multiple)
        f32x4 x[8];
#pragma unroll
        for (int k = 0; k < 8; k++) x[k] = w[i + k * LP_THREADS];
#pragma unroll
        for (int k = 0; k < 8; k++) m = max_magnitudes_of<true>(m, x[k]);
    }
    const int mine = wave_max(larger_half(m));
    if (lane_id() == 0) most[wave_id()] = mine;
    __syncthreads();
    if (threadIdx.x != 0) return;
    int x = most[0];
#pragma unroll
    for (int i = 1; i < LP_WAVES; i++) x = max(x, most[i]);
    x = min(max((x >> 7) - 127, -80), 80);
    a.head_shift[n] = 8 - (a.rank == 512 ? 9 : 8) - x;
}
__global__ __launch_bounds__(LP_THREADS) void latent_tiles_kernel(LatentPrefillArgs a) {
    __shared__ int64_t part[LP_WAVES][2];
    if (blockIdx.x > 0) {
        lp_head_shift(a, blockIdx.x - 1);
        return;
    }
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int per = (a.n_seqs + LP_THREADS - 1) / LP_THREADS;
    const int i0 = min(tid * per, a.n_seqs), i1 = min(i0 + per, a.n_seqs);
    int64_t k = 0, q = 0;
    for (int i = i0; i < i1; i++) {
        k += (lp_keys(a, i) + LP_KB - 1) / LP_KB;
        q += (lp_new(a, i) + LP_QB - 1) / LP_QB;
    }
    int64_t ks = k, qs = q;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int64_t x = __shfl_up(ks, off, WAVE), y = __shfl_up(qs, off, WAVE);
        if (lane >= off) {
            ks += x;
            qs += y;
        }
    }
    if (lane == WAVE - 1) {
        part[wave][0] = ks;
        part[wave][1] = qs;
    }
    __syncthreads();
    for (int w = 0; w < wave; w++) {
        ks += part[w][0];
        qs += part[w][1];
    }
    ks -= k;
    qs -= q;
    for (int i = i0; i < i1; i++) {
        a.key_tile[i] = (int)min(ks, (int64_t)a.key_tiles);
        a.q_tile[i] = (int)min(qs, (int64_t)a.q_tiles);
        ks += (lp_keys(a, i) + LP_KB - 1) / LP_KB;
        qs += (lp_new(a, i) + LP_QB - 1) / LP_QB;
    }
    if (tid == LP_THREADS - 1) {
        a.key_tile[a.n_seqs] = (int)min(ks, (int64_t)a.key_tiles);
        a.q_tile[a.n_seqs] = (int)min(qs, (int64_t)a.q_tiles);
    }
}

// An order of the query tiles by their keys, most first: a tile's time goes with its keys, and
// one with many that starts late is the call's end. Tiles are sorted by their number of key tiles
// to a sixteenth of a power of two; among equals the order is open, and no result depends on it.
// One workgroup of the expanding launch does this beside the others (28 requests of 3 to 1500 new
// tokens, up to 7500 keys, 20 heads: 557 -> 516 us a call against the order of the batch from its
// end; as part of the prefix sums' launch 525; one prompt of 8192 tokens loses 1%).
constexpr int LP_CLASSES = 512;
__device__ __forceinline__ int lp_class(int key_tiles) {  // 0 for the most keys
    const int x = (int)(__float_as_uint((float)key_tiles) >> 19) - (127 << 4);  // 2^25: 400
    return LP_CLASSES - 1 - max(x + 1, 0);
}
__device__ void lp_order(const LatentPrefillArgs& a, int tid, int threads) {
    __shared__ int place[LP_CLASSES];
    const int n = a.q_tile[a.n_seqs];
    auto place_of = [&](int i, int t) { return &place[lp_class(lp_key_tiles(a, i, t))]; };
    if (tid < LP_CLASSES) place[tid] = 0;
    __syncthreads();
    for (int t = tid; t < n; t += threads)
        atomicAdd(place_of(lp_find(a.q_tile, a.n_seqs, t), t), 1);
    __syncthreads();
    int before = 0;
    if (tid < LP_CLASSES)
        for (int c = 0; c < tid; c++) before += place[c];
    __syncthreads();
    if (tid < LP_CLASSES) place[tid] = before;
    __syncthreads();
    for (int t = tid; t < n; t += threads) {
        const int i = lp_find(a.q_tile, a.n_seqs, t);
        a.order[atomicAdd(place_of(i, t), 1)] = make_int2(i, t);
    }
}

// ---------------------------------------------------------------------------------- expand
// Keys and values of 128 cache rows (two key tiles). The rows come through the block table into
// LDS once, whole (128 KiB at rank 512), and stay; then each of the eight waves forms 128 x 64
// products with 64 rows of w_kv at a time, read straight into registers as MFMA fragments
// (w_kv lies in the L2: every workgroup reads all its rows). No barrier after the first one.
// A wave's 64 columns are all of one kind: for keys the weights are the MFMA's A operand, so
// that a lane holds 4 dims of a key; for values the latents are, so that it holds 4 keys of a
// dim: each is stored along its rows in memory order, and the values come out transposed. Keys
// that do not exist are stored as zeros.
// Bound: its two waves a SIMD wait for weights and for room to store. Without its stores (2 d x 2
// bytes a key and head) a call takes a fifth less time, without its weight loads a fifth less,
// without its LDS reads the same; the matrix pipe is busy a third of the time. Measured at rank
// 512, d = 128: 8192 keys, 32 heads (69 GFLOP) 91-107 us, 30124 keys of 28 requests, 20 heads (158
// GFLOP) 207-239 us: 640-760 TFLOP/s.
constexpr int EX_THREADS = 512, EX_WAVES = EX_THREADS / WAVE;
constexpr int EX_M = 128;              // keys of a workgroup
constexpr int EX_N = 64;               // columns of a wave
constexpr int EX_COLS = EX_WAVES * EX_N;

// LDS piece (16 bytes) c of row r of a tile with 128-byte rows
__device__ __forceinline__ int row128(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

template <int R>
__global__ __launch_bounds__(EX_THREADS, 2) void latent_expand_kernel(LatentPrefillArgs a,
                                                                      int units_per_wg) {
    constexpr int ROW = R * 2, PIECES = ROW / 16;
    __shared__ __align__(1024) char lat[EX_M * ROW];
    __shared__ uint32_t slot_of[EX_M];
    __shared__ int most[EX_WAVES];  // largest magnitude of 16 rows' latents
    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    static_assert(LP_CLASSES <= EX_THREADS, "lp_order has a thread per class");
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0) lp_order(a, tid, EX_THREADS);
        return;
    }
    const int t0 = (blockIdx.x - 1) * 2;
    const int used = a.key_tile[a.n_seqs];
    if (t0 >= used) return;
    constexpr size_t CACHE_ROW = (R + LP_ROPE) * 2;
    const char* cache = reinterpret_cast<const char*>(a.cache);

    bool ok = false;
    if (tid < EX_M) {
        const int t = t0 + tid / LP_KB;
        uint32_t slot = 0;
        if (t < used) {
            const int i = lp_find(a.key_tile, a.n_seqs, t);
            const int key = (t - a.key_tile[i]) * LP_KB + tid % LP_KB;
            if (key < lp_keys(a, i)) {
                const uint32_t p = a.block((uint32_t)key);
                const int page = a.block_table[(size_t)i * a.max_blocks + p];
                ok = page >= 0 && page < a.n_blocks;
                if (ok) slot = (uint32_t)page * a.block.div + ((uint32_t)key - p * a.block.div);
            }
        }
        slot_of[tid] = slot | (ok ? 0u : 0x80000000u);  // slots stay below 2^31
    }
    __syncthreads();
    const uint32_t flagged = slot_of[wave * 16 + (lane & 15)];
    {
        // 16 rows per wave; piece c of row r lies at piece c ^ ((r & 7) | (r >> 4 & 1) << 3), which
        // takes 16 values over the rows that a fragment's lanes read (below)
        const int odd = (wave & 1) << 3;
        const uint32_t mine = flagged & 0x7fffffffu;
        const uint32_t at = lds_offset(lat) + wave * 16 * ROW;
        if constexpr (PIECES == 64) {
#pragma unroll
            for (int r = 0; r < 16; r++)
                load_to_lds(cache + __builtin_amdgcn_readlane(mine, r) * CACHE_ROW,
                            (uint32_t)((lane ^ (r & 7) ^ odd) << 4), at + r * ROW);
        } else {  // two rows per load
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const int rr = r + (lane >> 5);
                load_to_lds(cache + __shfl(mine, rr, WAVE) * CACHE_ROW +
                                (((lane & 31) ^ (rr & 7) ^ odd) << 4),
                            at + r * ROW);
            }
        }
    }
    bf16x8 pe[EX_M * 8 / EX_THREADS];  // rotary keys of the pair: tile i, row tid / 8
    static_assert(EX_M * 8 / EX_THREADS == 2 && EX_THREADS / 8 == LP_KB, "a tile a step");
    if (blockIdx.y == 0) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            pe[i] = *reinterpret_cast<const bf16x8*>(
                cache + (size_t)(slot_of[i * LP_KB + (tid >> 3)] & 0x7fffffffu) * CACHE_ROW + ROW +
                (tid & 7) * 16);
    }
    lds_loads_done();
    {
        // this wave's 16 rows are here; what absent keys' slots hold does not count
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 16; r += 64 / PIECES) {
            const uint32_t row = r + lane / PIECES;
            const bool absent = __shfl(flagged, row, WAVE) >> 31;
            const uint32_t x = max_magnitudes_of<true>(
                0, lds_get<f32x4>(lds_offset(lat) + (wave * 16 + row) * ROW + lane % PIECES * 16));
            m = max_magnitudes(m, absent ? 0u : x);
        }
        const int x = wave_max(larger_half(m));
        if (lane == 0) most[wave] = x;
    }
    lds_barrier();
    int shift[2];  // t of the two tiles
#pragma unroll
    for (int i = 0; i < 2; i++)
        shift[i] = uniform(lp_shift(max(max(most[4 * i], most[4 * i + 1]),
                                        max(most[4 * i + 2], most[4 * i + 3]))));
    if (blockIdx.y == 0) {
        // the pair's existence bits, shifts and rotary keys, once for all heads
        if (wave < 2) {
            const uint64_t bits = __ballot(ok);
            if (lane == 0 && t0 + wave < used)
                a.tile[t0 + wave] = make_int4((int)bits, (int)(bits >> 32), shift[wave], 0);
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (t0 + i >= used) break;
            if (shift[i] != 0) {
                const float f = exp2i(-shift[i]);
#pragma unroll
                for (int e = 0; e < 8; e++) pe[i][e] = (bf16)((float)pe[i][e] * f);
            }
            *reinterpret_cast<bf16x8*>(reinterpret_cast<char*>(a.k_pe) +
                                       (size_t)(t0 + i) * LP_KB * 128 + tid * 16) = pe[i];
        }
    }
    const int col = lane & 15, grp = lane >> 4;
    const int columns = a.H * 2 * a.d;
    // Which rows make up a fragment is free, and chosen so that two fragments give a lane 8
    // neighbours in memory, one 16-byte store. Keys: lane c of fragments i = 2 p + e reads row
    // 32 p + 16 (c >> 3) + 8 e + (c & 7); with the values' key order (keys 4 h + (0..3) and
    // 8 + 4 h + (0..3) of each 16 make up its half h) lane group g then holds places
    // 32 p + 8 g + 4 e + (0..3). Dims of a key: rows 32 p + 8 (c >> 2) + 4 e + (c & 3) of w_kv.
    const uint32_t x_at = lds_offset(lat) + (16 * (col >> 3) + (col & 7)) * ROW +
                          (((grp * 2) ^ col) << 4);
    // The contraction's order is free. Two steps take 128 bytes of a row of w_kv: lane group g 32
    // of them, the first 16 in one step and the others in the next. Weights of two steps are
    // requested together, two steps ahead, so that a cache line is fetched once; the first ones
    // of a unit while the one before it ends.
    uint32_t w_at[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        w_at[j] = ((j >> 1) * 32 + (col >> 2) * 8 + (j & 1) * 4 + (col & 3)) * ROW + grp * 32;
    bf16x8 w[4][4];
    auto load_w = [&](const char* from, int k) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            asm volatile("" : "+v"(w_at[j]));  // (else 64-bit sums of it are kept)
            w[k][j] = *reinterpret_cast<const bf16x8*>(from + (k >> 1) * 128 + (k & 1) * 16 +
                                                       (size_t)w_at[j]);
        }
    };
    // 64 columns, of one kind, of weights at `block`; after them those at `next`
    auto unit = [&](auto kind, int h, int in_head, const char* block, const char* next) {
        constexpr bool VALUE = decltype(kind)::value;
        const int s = a.head_shift[h * 2 + VALUE];
        // (copies that the compiler cannot take for the same in every unit: it would work out all
        // addresses of the stores before the first one and keep them)
        int col = lane & 15, grp = lane >> 4;
        asm volatile("" : "+v"(col), "+v"(grp));
        f32x4 acc[8][4];  // [key fragment][weight fragment]
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = zero4();
        bf16x8 x[4];
        uint32_t base[2], at = x_at;
        // fragment n & 7 of step n >> 3 of the block at `at`; an LDS instruction's immediate
        // offset reaches 64 KiB
        auto load_x = [&](uint32_t from, int n) {
            const int k = n >> 3 & 3, i = n & 7;
            if (i == 0) {
                base[0] = from ^ ((k & 2) << 6 | (k & 1) << 4);
                base[1] = base[0] + 64 * ROW;
                asm volatile("" : "+v"(base[0]), "+v"(base[1]));
            }
            x[n & 3] = lds_get<bf16x8>(base[i >> 2] + ((i >> 1 & 1) * 32 + (i & 1) * 8) * ROW);
        };
        load_x(at, 0);
        load_x(at, 1);
#pragma unroll 1
        for (int left = R / 128; left > 0; left--) {  // four steps
#pragma unroll
            for (int n = 0; n < 32; n++) {
                const int k = n >> 3, i = n & 7;
                if (n == 0) {
                    load_w(block, 2);
                    load_w(block, 3);
                }
                if (n == 16) {
                    block = left > 1 ? block + 256 : next;
                    load_w(block, 0);
                    load_w(block, 1);
                }
                // (the last block's look-ahead reads LDS behind its rows, and is not used)
                load_x(n + 2 < 32 ? at : at + 256, n + 2);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    acc[i][j] = VALUE ? Mma<bf16>::mma(x[n & 3], w[k][j], acc[i][j])
                                      : Mma<bf16>::mma(w[k][j], x[n & 3], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            at += 256;
        }
        asm volatile("" : "+v"(col), "+v"(grp));
#pragma unroll
        for (int half = 0; half < 2; half++) {
            if (t0 + half >= used) break;
            const size_t head_tile = (size_t)h * a.key_tiles + t0 + half;
            const float f = exp2i(s - shift[half]);
            auto store = [&](_Float16* to, const float (&y)[8]) {
                f16x8 v;
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = (_Float16)y[e];
                *reinterpret_cast<f16x8*>(to) = v;
            };
            if constexpr (VALUE) {
                _Float16* out = reinterpret_cast<_Float16*>(a.vt) + head_tile * a.d * LP_KB;
#pragma unroll
                for (int p = 0; p < 2; p++) {
                    // the lane's 8 keys: 32 p + 16 (g >> 1) + 4 (g & 1) + 8 e + (0..3)
                    const int key = half * LP_KB + p * 32 + (grp >> 1) * 16 + (grp & 1) * 4;
                    bool absent[8];
#pragma unroll
                    for (int y = 0; y < 8; y++)
                        absent[y] = slot_of[key + (y >> 2) * 8 + (y & 3)] >> 31;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            y[e] = absent[e] ? 0.f : acc[half * 4 + 2 * p + (e >> 2)][j][e & 3] * f;
                        const int dim = (j >> 1) * 32 + (col >> 2) * 8 + (j & 1) * 4 + (col & 3);
                        store(out + (size_t)(in_head - a.d + dim) * LP_KB + p * 32 + grp * 8, y);
                    }
                }
            } else {
                _Float16* out = reinterpret_cast<_Float16*>(a.k) + head_tile * LP_KB * a.d;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int key = (i >> 1) * 32 + 16 * (col >> 3) + (i & 1) * 8 + (col & 7);
                    const bool absent = slot_of[half * LP_KB + key] >> 31;
#pragma unroll
                    for (int p = 0; p < 2; p++) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            y[e] = absent ? 0.f : acc[half * 4 + i][2 * p + (e >> 2)][e & 3] * f;
                        store(out + (size_t)key * a.d + in_head + p * 32 + grp * 8, y);
                    }
                }
            }
        }
    };
    int col0 = (int)blockIdx.y * units_per_wg * EX_COLS + wave * EX_N;
    if (col0 >= columns) return;
    const char* block = reinterpret_cast<const char*>(a.w_kv) + (size_t)col0 * ROW;
    load_w(block, 0);
    load_w(block, 1);
    for (int u = 0; u < units_per_wg && col0 < columns; u++, col0 += EX_COLS) {
        const int h = col0 / (2 * a.d), in_head = col0 - h * 2 * a.d;
        // (behind the last unit the same weights again, which are not used)
        const bool more = u + 1 < units_per_wg && col0 + EX_COLS < columns;
        const char* next = block + (more ? (size_t)EX_COLS * ROW : 0);
        if (in_head >= a.d) unit(std::true_type(), h, in_head, block, next);
        else unit(std::false_type(), h, in_head, block, next);
        block = next;
    }
}

// ---------------------------------------------------------------------------------- attend
// A workgroup takes 128 query rows of one head, 32 a wave; all four waves walk the same key
// tiles, loaded straight into LDS, one barrier a tile. With 32 x 32 x 16 MFMAs:
//   S^T = K Q^T     queries in registers as the B operand, so a query is an accumulator column:
//                   its scores lie in two lanes, and its statistics need one exchange a tile;
//   O^T += V^T P^T  the accumulator layout of S^T is the B operand's with the keys of each 16
//                   renumbered, and V^T was written out in that order: weights never leave the
//                   registers.
// A tile's scores (matrix pipe) are formed beside the previous tile's softmax (vector pipe): keys
// and values have two LDS buffers each, and the keys run one tile ahead of the values.
// Bound: the matrix pipe beside the softmax's vector work at two waves a SIMD (2.5 us a tile).
// Measured at d = 128: one prompt of 8192 tokens, 32 heads (687 GFLOP) 654-725 us, 0.95-1.05
// PFLOP/s (a large bf16 product reaches 1.57); 28 ragged prompts, 20 heads 299-332 us.
template <int D>
struct LpTile {
    static constexpr int K_BYTES = LP_KB * (D + LP_ROPE) * 2;     // [64][D] keys, [64][64] rotary
    static constexpr int PE_AT = LP_KB * D * 2;
    static constexpr int V_BYTES = D * LP_KB * 2;                 // [D][64] values
    // pieces of a key row turned by the row (256-byte rows: 16 pieces)
    __device__ __forceinline__ static int turn(int r) { return D == 128 ? r & 15 : (r >> 1) & 7; }
    __device__ __forceinline__ static int key(int r, int c) {
        return r * (D * 2) + ((c ^ turn(r)) << 4);
    }
};

template <int D>
__global__ __launch_bounds__(LP_THREADS, 2) void latent_attend_kernel(LatentPrefillArgs a) {
    using X = LpTile<D>;
    constexpr int NK = D / 16, NR = LP_ROPE / 16;  // contraction steps of a score
    constexpr int NO = D / 32;                     // 32-column output tiles
    __shared__ __align__(1024) char k_tile[2][X::K_BYTES];
    __shared__ __align__(1024) char v_tile[2][X::V_BYTES];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int h = blockIdx.x % a.H;
    const int n_qt = a.q_tile[a.n_seqs];
    const int nth = (int)(blockIdx.x / a.H);
    if (nth >= n_qt) return;
    const int2 who = a.order[nth];
    const int seq = uniform(who.x), qt = uniform(who.y);
    const int q0 = (qt - a.q_tile[seq]) * LP_QB;
    const int fresh = lp_new(a, seq);
    const int first_pos = lp_len(a, seq) - fresh;       // of the request's first new token
    const int kt0 = a.key_tile[seq];
    const int nt = uniform(lp_key_tiles(a, seq, qt));

    const int col = lane & 31, half = lane >> 5;
    const int row = q0 + wave * 32 + col;               // this lane's query row
    const bool live = row < fresh;
    const int pos = first_pos + row;
    const int wave_first = uniform(first_pos + q0 + wave * 32);  // position of the wave's first row
    // tiles that this wave's rows see
    const int mine = wave_first + 31 < 0 ? 0 : min(nt, (wave_first + 31) / LP_KB + 1);
    const size_t token = (size_t)min(max(a.cu_seqlens[seq], 0), a.total_tokens) +
                         (live ? row : q0);
    // The scale enters the exponent's multiplication; a negative one is moved into the queries,
    // so that the largest score is the largest weight (and zero makes the queries zero).
    bf16x8 q[NK + NR];  // (the first NK hold fp16)
    {
        const bf16* qn = reinterpret_cast<const bf16*>(a.q_nope) + (token * a.H + h) * D;
        const bf16* qp = reinterpret_cast<const bf16*>(a.q_pe) + (token * a.H + h) * LP_ROPE;
#pragma unroll
        for (int f = 0; f < NK; f++) q[f] = Mma<bf16>::load(qn + f * 16 + half * 8);
#pragma unroll
        for (int f = 0; f < NR; f++) q[NK + f] = Mma<bf16>::load(qp + f * 16 + half * 8);
    }
    if (a.scale <= 0.f) {
#pragma unroll
        for (int f = 0; f < NK + NR; f++)
#pragma unroll
            for (int i = 0; i < 8; i++) q[f][i] = a.scale < 0.f ? -q[f][i] : (bf16)0.f;
    }
    const int key_s = uniform(a.head_shift[h * 2]), value_s = uniform(a.head_shift[h * 2 + 1]);
    float cs;  // of this lane's row, for tiles with t = 0
    {
        uint32_t m = 0;
#pragma unroll
        for (int f = 0; f < NK; f++) m = max_magnitudes_of<false>(m, q[f]);
        int x = larger_half(m);
        x = max(x, __shfl_xor(x, 32, WAVE)) >> 7;
        // (the rotary part's 2^(s - a) is kept in range: by then the rest of a score is nothing)
        const int row_a = min(max(x == 0 ? 0 : x - 127, key_s - 60), 127);
        const float down = exp2i(-row_a), pe_down = exp2i(key_s - row_a);
#pragma unroll
        for (int f = 0; f < NK; f++) {
            f16x8 to;
#pragma unroll
            for (int i = 0; i < 8; i++) to[i] = (_Float16)((float)q[f][i] * down);
            q[f] = __builtin_bit_cast(bf16x8, to);
        }
#pragma unroll
        for (int f = NK; f < NK + NR; f++)
#pragma unroll
            for (int i = 0; i < 8; i++) q[f][i] = (bf16)((float)q[f][i] * pe_down);
        cs = ldexpf(a.scale == 0.f ? 1.f : fabsf(a.scale) * LOG2E, row_a - key_s);
    }
    arrived(q);
    const char* ksrc = reinterpret_cast<const char*>(a.k) +
                       ((size_t)h * a.key_tiles + kt0) * (LP_KB * D * 2);
    const char* vsrc = reinterpret_cast<const char*>(a.vt) +
                       ((size_t)h * a.key_tiles + kt0) * (LP_KB * D * 2);
    const char* psrc = reinterpret_cast<const char*>(a.k_pe) + (size_t)kt0 * (LP_KB * LP_ROPE * 2);
    // Byte offsets of this lane within a tile. Pieces are xored with a function of their row, so
    // the constant part of a piece index is xored in last and one offset serves all of them;
    // fixed() hides it from the compiler, which would keep every result of that across the loop.
    auto fixed = [](uint32_t x) {
        asm volatile("" : "+v"(x));
        return x;
    };
    const uint32_t k_at = X::key(col, half), r_at = row128(col, half);
    const uint32_t load128 = row128(lane >> 3, lane & 7);       // 8 rows of 128 bytes per load
    const uint32_t load_k = D == 128 ? X::key(lane >> 4, lane & 15) : load128;
    constexpr int KI = LP_KB * D * 2 / 1024 / LP_WAVES;         // 1 KiB loads per wave
    auto load_keys = [&](int t) {
        const uint32_t at = lds_offset(k_tile[t & 1]), off = fixed(load_k), pe = fixed(load128);
        const char* src = ksrc + ((size_t)t * LP_WAVES + wave) * (KI * 1024);
#pragma unroll
        for (int i = 0; i < KI; i++)  // 1 KiB on, the rows' turn is off by 4 i (128-byte rows: 4)
            load_to_lds(src + i * 1024, off ^ (D == 128 ? i << 6 : (i & 1) << 6),
                        at + (wave * KI + i) * 1024);
        const char* psrc_t = psrc + ((size_t)t * LP_WAVES + wave) * 2048;
#pragma unroll
        for (int i = 0; i < 2; i++)
            load_to_lds(psrc_t + i * 1024, pe ^ i << 6, at + X::PE_AT + (wave * 2 + i) * 1024);
    };
    auto load_values = [&](int t) {
        const uint32_t at = lds_offset(v_tile[t & 1]), off = fixed(load128);
        const char* src = vsrc + ((size_t)t * LP_WAVES + wave) * (KI * 1024);
#pragma unroll
        for (int i = 0; i < KI; i++)
            load_to_lds(src + i * 1024, off ^ (i & 1) << 6, at + (wave * KI + i) * 1024);
    };
    f32x16 acc[NO];
#pragma unroll
    for (int j = 0; j < NO; j++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc[j][i] = 0.f;
    float ref = -INFINITY, l = 0.f;  // the exponents' reference (scaled); the sum
    int sums_t = 0;                  // t that this row's sums of values are kept at
    // Weights are taken 2^7 times as large: up to 2^(7 + LAG), and down to 2^-31 in fp16.
    constexpr float WEIGHT_SHIFT = 7.f;

    // Scores of tile t, unscaled, and beside each pair of MFMAs a slice of other work: the
    // matrix pipe takes 32 cycles for one MFMA, in which the wave can issue eight vector
    // instructions. The fences keep the compiler from taking the two apart again.
    constexpr int NF = NK + NR, AHEAD = 3;
    auto scores = [&](int t, f32x16 (&s)[2], auto beside) {
        const uint32_t kt = lds_offset(k_tile[t & 1]);
        const uint32_t key = fixed(kt + k_at), pe = fixed(kt + X::PE_AT + r_at);
        bf16x8 k[AHEAD + 1][2];
        auto load = [&](int f) {
#pragma unroll
            for (int x = 0; x < 2; x++)  // (32 rows on, the pieces are turned alike)
                k[f % (AHEAD + 1)][x] = lds_get<bf16x8>(
                    f < NK ? (key ^ f << 5) + x * (32 * D * 2)
                           : (pe ^ (f - NK) << 5) + x * (32 * 128));
        };
#pragma unroll
        for (int f = 0; f < AHEAD; f++) load(f);
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int i = 0; i < 16; i++) s[x][i] = 0.f;
#pragma unroll
        for (int f = 0; f < NF; f++) {
            if (f + AHEAD < NF) load(f + AHEAD);
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const bf16x8 y = k[f % (AHEAD + 1)][x];
                s[x] = f < NK ? mma32(__builtin_bit_cast(f16x8, y), __builtin_bit_cast(f16x8, q[f]),
                                      s[x])
                              : mma32(y, q[f], s[x]);
            }
            beside(f);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto mask = [&](int t, uint64_t exist, f32x16 (&s)[2]) {
        const int key0 = t * LP_KB;
        if (exist == ~0ull && key0 + LP_KB - 1 <= wave_first) return;
        // this lane's keys are key0 + first + ..: hidden from the compiler, which would keep
        // what depends on it in registers across the key loop
        int first = half * 4;
        asm volatile("" : "+v"(first));
        const uint64_t here = exist >> first;
        const int left = pos - key0 - first;
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int k = x * 32 + (i >> 2) * 8 + (i & 3);
                s[x][i] = ((here >> k) & 1) && k <= left ? s[x][i] : -INFINITY;
            }
    };
    int4 tile_next = make_int4(0, 0, 0, 0);
    struct Tile {
        uint64_t exist;
        int t;
    };
    auto take_tile = [&]() -> Tile {
        // moved to scalar registers where nothing else is in flight: a wait for the ordinary
        // load further down would also wait for the tile loads issued behind it
        return {(uint64_t)(uint32_t)uniform(tile_next.y) << 32 | (uint32_t)uniform(tile_next.x),
                uniform(tile_next.z)};
    };
    int now_t = 0;  // of the tile whose weights come next
    // One tile: its weights from s (masked), its values added; meanwhile the next tile's scores.
    auto step = [&](int t, f32x16 (&s)[2], f32x16 (&next)[2]) {
        lds_loads_done();
        const Tile after = take_tile();  // tile t + 1
        const int tile_t = now_t;
        now_t = after.t;
        lds_barrier();  // keys t + 1 and values t are whole; all are done with what they replace
        if (t + 2 < nt) {
            tile_next = a.tile[kt0 + t + 2];
            sched_fence();
            load_keys(t + 2);
        }
        if (t + 1 < nt) load_values(t + 1);
        if (t >= mine) return;
        float top = -INFINITY, shift = 0.f;
        bool grown = false;
        const float cs_t = ldexpf(cs, tile_t);
        // slices 0 and 1: the tile's maximum; 2: over both halves; from 3 on: the weights
        constexpr int PER = (32 + NF - 4) / (NF - 3);
        // (behind this wave's last tile the scores are nobody's: that buffer is not being filled,
        // tile t's may be)
        scores(t + 1, next, [&](int f) {
            if (f < 2) {
#pragma unroll
                for (int i = 0; i < 16; i++) top = fmaxf(top, s[f][i]);
            } else if (f == 2) {
                top = max_halves(top) * cs_t;
                grown = top > ref + LAG;
                const float to = grown ? top : ref;
                shift = to == -INFINITY ? 0.f : to;  // a row with no key so far
            } else {
                const float up = WEIGHT_SHIFT - shift;
#pragma unroll
                for (int i = (f - 3) * PER; i < (f - 2) * PER && i < 32; i++) {
                    float w = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], cs_t, up));
                    asm volatile("" : "+v"(w));  // formed here, not where it is used
                    s[i >> 4][i & 15] = w;
                }
            }
        });
        if (__any(grown)) {
            // (a row without a reference so far has sums of zero)
            const float shrink = grown ? __builtin_amdgcn_exp2f(ref - shift) : 1.f;
            ref = grown ? shift : ref;
            l *= shrink;
#pragma unroll
            for (int j = 0; j < NO; j++)
#pragma unroll
                for (int i = 0; i < 16; i++) acc[j][i] *= shrink;
        }
        if (__any(sums_t != tile_t)) {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < NO; j++)
#pragma unroll
                for (int i = 0; i < 16; i++) most = fmaxf(most, fabsf(acc[j][i]));
            const int to = ldexpf(max_halves(most), sums_t - tile_t) < 0x1p100f ? tile_t : sums_t;
            const float f = exp2i(sums_t - to);
#pragma unroll
            for (int j = 0; j < NO; j++)
#pragma unroll
                for (int i = 0; i < 16; i++) acc[j][i] *= f;
            if (to != tile_t) {  // this tile's share would be lost in the sums
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    l += s[i >> 4][i & 15];
                    s[i >> 4][i & 15] = 0.f;
                }
            }
            sums_t = to;
        }
        const uint32_t value = fixed(lds_offset(v_tile[t & 1]) + r_at);
        auto weights = [&](int n) {  // 8 of them, an operand
            f16x8 w;
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = (_Float16)s[n >> 1][(n & 1) * 8 + i];
            return w;
        };
        f16x8 p[4] = {weights(0), weights(1), weights(2), weights(3)};
        f16x8 v[AHEAD + 1];
        constexpr int NV = LP_KB / 16 * NO;
        auto load = [&](int n) {
            v[n % (AHEAD + 1)] = lds_get<f16x8>((value ^ (n / NO) << 5) + n % NO * (32 * 128));
        };
#pragma unroll
        for (int n = 0; n < AHEAD; n++) load(n);
#pragma unroll
        for (int n = 0; n < NV; n++) {
            if (n + AHEAD < NV) load(n + AHEAD);
            acc[n % NO] = mma32(v[n % (AHEAD + 1)], p[n / NO], acc[n % NO]);
#pragma unroll
            for (int i = n * 32 / NV; i < (n + 1) * 32 / NV; i++) l += s[i >> 4][i & 15];
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t + 1 < mine) mask(t + 1, after.exist, next);
    };
    if (nt > 0) {
        f32x16 s0[2], s1[2];
        tile_next = a.tile[kt0];
        sched_fence();
        load_keys(0);
        lds_loads_done();
        const Tile first = take_tile();
        now_t = first.t;
        lds_barrier();
        if (nt > 1) {
            tile_next = a.tile[kt0 + 1];
            sched_fence();
            load_keys(1);
        }
        load_values(0);
        if (mine > 0) {
            scores(0, s0, [](int) {});
            mask(0, first.exist, s0);
        }
        for (int t = 0; t < nt; t += 2) {
            step(t, s0, s1);
            if (t + 1 < nt) step(t + 1, s1, s0);
        }
    }
    l += __shfl_xor(l, 32, WAVE);
    // no key: zeros. (The sum holds 2^7 as the weights do.)
    const float inv = l == 0.f ? 0.f : ldexpf(1.f / l, sums_t - value_s);
    if (live) {
        bf16* out = reinterpret_cast<bf16*>(a.o) + (token * a.H + h) * D;
#pragma unroll
        for (int j = 0; j < NO; j++)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; e++) y[e] = acc[j][i + e] * inv;
                store4<bf16>(out + j * 32 + (i >> 2) * 8 + half * 4, y);
            }
    }
}

}  // namespace

size_t latent_prefill_layout(LatentPrefillArgs* a, int64_t total_keys, void* ws) {
    // sum_i ceil(len_i / B) <= (sum len_i + n (B - 1)) / B
    a->key_tiles = (int)((total_keys + (int64_t)a->n_seqs * (LP_KB - 1)) / LP_KB);
    a->q_tiles = (int)((a->total_tokens + (int64_t)a->n_seqs * (LP_QB - 1)) / LP_QB);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = ws == nullptr ? nullptr : static_cast<char*>(ws) + off;
        off += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t tiles = (size_t)a->key_tiles;
    a->key_tile = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * (size_t)(a->n_seqs + 1)));
    a->q_tile = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * (size_t)(a->n_seqs + 1)));
    a->order = reinterpret_cast<int2*>(take(sizeof(int2) * (size_t)a->q_tiles));
    a->head_shift = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * 2 * (size_t)a->H));
    a->tile = reinterpret_cast<int4*>(take(sizeof(int4) * tiles));
    a->k_pe = take(tiles * LP_KB * LP_ROPE * 2);
    a->k = take(tiles * LP_KB * a->d * 2 * a->H);
    a->vt = take(tiles * LP_KB * a->d * 2 * a->H);
    return off;
}

hipError_t launch_latent_prefill(const LatentPrefillArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    const dim3 block(LP_THREADS);
    hipLaunchKernelGGL(latent_tiles_kernel, dim3(1u + 2u * (unsigned)a.H), block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.q_tiles == 0) return e;
    // The columns in equal runs of units, a workgroup each (one fits a CU): as many runs as end
    // soonest, a workgroup's start (its latents) counted as a third of a unit. (28 requests with
    // 250 key blocks, 10 units: one run 239 us, three 265.)
    const int blocks = (a.key_tiles + 1) / 2, cus = device_cu_count();
    const int units = (a.H * 2 * a.d + EX_COLS - 1) / EX_COLS;
    int per = units;
    int64_t best = INT64_MAX;
    for (int runs = 1; runs <= units; runs++) {
        const int n = (units + runs - 1) / runs;
        const int64_t cost = (((int64_t)blocks * runs + cus - 1) / cus) * (3 * n + 1);
        if (cost < best) {
            best = cost;
            per = n;
        }
    }
    const dim3 expand((unsigned)blocks + 1, (unsigned)((units + per - 1) / per));
    if (a.rank == 512)
        hipLaunchKernelGGL(latent_expand_kernel<512>, expand, dim3(EX_THREADS), 0, s, a, per);
    else
        hipLaunchKernelGGL(latent_expand_kernel<256>, expand, dim3(EX_THREADS), 0, s, a, per);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)a.q_tiles * (unsigned)a.H);
    if (a.d == 128) hipLaunchKernelGGL(latent_attend_kernel<128>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(latent_attend_kernel<64>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace gdn
