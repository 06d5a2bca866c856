// Bookkeeping of a paged cache on the GPU: block tables, slot maps, positions and cu_seqlens
// from request lengths (gdn_paged_plan), and the rows of new tokens written through a slot map
// (gdn_paged_append, gdn_latent_append).
//
// Page: [LA-Infra] "深度解析线性注意力机制演进与 AI Infra 实现", sections on the prefix cache of
// hybrid models (a block table per request, null blocks, pages of a fixed number of tokens).
#include "attn_launch.h"
#include "gdn_common.h"

namespace gdn {

// ------------------------------------------------------------------------------------ plan
// With c_i cached and w_i new tokens of request i and pages of b tokens:
//   held_i = ceil(c_i / b),  need_i = max(0, min(ceil((c_i + w_i) / b), max_blocks) - held_i),
//   first_i = sum_{j<i} need_j,  cu_i = sum_{j<i} w_j;
//   page p of request i is free_blocks[first_i + p - held_i] for held_i <= p < held_i + need_i;
//   token t in [cu_i, cu_{i+1}) sits at position c_i + t - cu_i.
//
// Bound: launch latency (12 bytes written per token: 131072 tokens are 1.6 MB). So one launch
// does it all: every workgroup repeats the prefix sums over the n requests (8 n bytes, out of
// the L2 after the first) and then maps its own PLAN_TOK tokens, instead of a scan kernel
// followed by a mapping kernel. A page's table entry is written by the thread of its first
// token: a page that is new starts at a new token, so each entry has exactly one writer and no
// workgroup reads an entry that another one writes. Measured: 24 requests of one token 4.4 us,
// 320 prompts of 169418 tokens 6.5 us.
constexpr int PLAN_THREADS = 256;
constexpr int PLAN_PER = 4;  // consecutive tokens of a thread (two 16-byte slot stores)
constexpr int PLAN_TOK = PLAN_THREADS * PLAN_PER;

struct PlanReq {
    int64_t ctx, held;
    int fresh, need;
};

__device__ __forceinline__ PlanReq plan_req(const PlanArgs& a, int i) {
    PlanReq r;
    r.ctx = max(a.ctx_lens[i], 0);
    r.fresh = max(a.new_lens[i], 0);
    const uint32_t bs = (uint32_t)a.block_size;
    // ctx + fresh < 2^32: unsigned division
    r.held = ((uint32_t)r.ctx + bs - 1) / bs;
    const int64_t all = ((uint32_t)r.ctx + (uint32_t)r.fresh) / bs +
                        (((uint32_t)r.ctx + (uint32_t)r.fresh) % bs != 0);
    const int64_t last = all < a.max_blocks ? all : a.max_blocks;
    r.need = last > r.held ? (int)(last - r.held) : 0;
    return r;
}

__global__ __launch_bounds__(PLAN_THREADS) void paged_plan_kernel(PlanArgs a) {
    __shared__ int tok0[PLAN_THREADS + 1];   // new tokens before each thread's requests
    __shared__ int page0[PLAN_THREADS + 1];  // new pages before them
    __shared__ int wave_tok[PLAN_THREADS / WAVE], wave_page[PLAN_THREADS / WAVE];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int per = (a.n + PLAN_THREADS - 1) / PLAN_THREADS;
    const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
    int tok = 0, page = 0;
    for (int i = i0; i < i1; i++) {
        const PlanReq r = plan_req(a, i);
        tok += r.fresh;
        page += r.need;
    }
    // inclusive sums over the wave, then over the waves
    int ts = tok, ps = page;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int t = __shfl_up(ts, off, WAVE), p = __shfl_up(ps, off, WAVE);
        if (lane >= off) {
            ts += t;
            ps += p;
        }
    }
    if (lane == WAVE - 1) {
        wave_tok[wave] = ts;
        wave_page[wave] = ps;
    }
    __syncthreads();
    for (int w = 0; w < wave; w++) {
        ts += wave_tok[w];
        ps += wave_page[w];
    }
    tok0[tid + 1] = ts;
    page0[tid + 1] = ps;
    if (tid == 0) {
        tok0[0] = 0;
        page0[0] = 0;
    }
    __syncthreads();
    const int total = tok0[PLAN_THREADS];
    if (blockIdx.x == 0) {
        int t = tok0[tid];
        for (int i = i0; i < i1; i++) {
            const PlanReq r = plan_req(a, i);
            a.cu_seqlens[i] = t;
            a.seq_lens[i] = (int)(r.ctx + r.fresh);
            t += r.fresh;
        }
        if (tid == 0) {
            a.cu_seqlens[a.n] = total;
            a.counts[0] = total;
            a.counts[1] = page0[PLAN_THREADS];
        }
    }
    const int64_t t0 = (int64_t)blockIdx.x * PLAN_TOK + tid * PLAN_PER;
    if (t0 >= a.max_tokens) return;
    int64_t slot[PLAN_PER];
    int pos[PLAN_PER];
#pragma unroll
    for (int k = 0; k < PLAN_PER; k++) {
        slot[k] = -1;
        pos[k] = 0;
    }
    if (t0 < total) {
        // the thread slice that holds token t0 (last s with tok0[s] <= t0), then the request in it
        int lo = 0, hi = PLAN_THREADS;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tok0[mid] <= t0) lo = mid; else hi = mid;
        }
        int i = lo * per;
        const int end = a.n;
        int cu = tok0[lo], first = page0[lo];
        PlanReq r = plan_req(a, i);
#pragma unroll
        for (int k = 0; k < PLAN_PER; k++) {
            const int64_t t = t0 + k;
            if (t >= total || t >= a.max_tokens) break;
            while (t >= (int64_t)cu + r.fresh && i + 1 < end) {
                cu += r.fresh;
                first += r.need;
                i++;
                r = plan_req(a, i);
            }
            const int64_t p = r.ctx + (t - cu);
            const int64_t b = (uint32_t)p / (uint32_t)a.block_size;
            const int off = (int)(p - b * a.block_size);
            int blk = -1;
            if (b < a.max_blocks) {
                int32_t* entry = a.block_table + (size_t)i * a.max_blocks + b;
                if (b < r.held) {
                    blk = *entry;
                } else {
                    const int64_t f = first + (b - r.held);
                    if (f >= 0 && f < a.n_free) blk = a.free_blocks[f];
                    if (off == 0) *entry = blk;
                }
            }
            slot[k] = blk >= 0 ? (int64_t)blk * a.block_size + off : -1;
            pos[k] = (int)p;
        }
    }
    if (t0 + PLAN_PER <= a.max_tokens) {
        typedef long long i64x2 __attribute__((ext_vector_type(2)));
        typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int k = 0; k < PLAN_PER; k += 2)
            *reinterpret_cast<i64x2*>(a.slot_map + t0 + k) = i64x2{slot[k], slot[k + 1]};
        *reinterpret_cast<i32x4*>(a.positions + t0) = i32x4{pos[0], pos[1], pos[2], pos[3]};
    } else {
        for (int k = 0; k < PLAN_PER && t0 + k < a.max_tokens; k++) {
            a.slot_map[t0 + k] = slot[k];
            a.positions[t0 + k] = pos[k];
        }
    }
}

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    const unsigned grid = a.max_tokens > 0 ? (unsigned)((a.max_tokens - 1) / PLAN_TOK + 1) : 1u;
    hipLaunchKernelGGL(paged_plan_kernel, dim3(grid), dim3(PLAN_THREADS), 0, s, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------- append
// A copy: cache[slot_map[t]] = row t, in 16-byte pieces; a slot outside the cache skips the
// token. Bound: HBM (each row read and written once). Consecutive threads take consecutive
// pieces of a token, so both sides move in whole rows. Measured: 65000 rows of 1152 bytes 33 us
// (4.5 TB/s; a large copy reaches 5.0), 24 us out of the last-level cache; 96 tokens 2.6 us.
constexpr int APP_THREADS = 256;

template <bool SPLIT>
__global__ __launch_bounds__(APP_THREADS) void append_kernel(AppendArgs a, int tokens_per_wg) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const uint32_t an = (uint32_t)(a.heads * a.a_row), n = an + (uint32_t)(a.heads * a.b_row);
    const int64_t base = (int64_t)blockIdx.x * tokens_per_wg;
    const uint32_t here = (uint32_t)min((int64_t)tokens_per_wg, a.tokens - base);
    const int64_t slots = (int64_t)a.n_blocks * a.block_size;
    for (uint32_t x = threadIdx.x; x < here * n; x += APP_THREADS) {
        const uint32_t tt = x / n, piece = x - tt * n;
        const int64_t t = base + tt;
        const int64_t slot = a.slot_map[t];
        if (slot < 0 || slot >= slots) continue;
        const bool in_a = piece < an;
        const uint32_t p = in_a ? piece : piece - an;
        const i32x4* src = reinterpret_cast<const i32x4*>(in_a ? a.a : a.b) +
                           t * (in_a ? a.a_stride : a.b_stride) + p;
        i32x4* dst;
        if constexpr (SPLIT) {
            const uint32_t row = (uint32_t)(in_a ? a.a_row : a.b_row);
            const uint32_t h = p / row, c = p - h * row;
            const uint32_t blk = (uint32_t)slot / (uint32_t)a.block_size;
            const uint32_t off = (uint32_t)slot - blk * (uint32_t)a.block_size;
            dst = reinterpret_cast<i32x4*>(in_a ? a.a_cache : a.b_cache) +
                  (((size_t)blk * a.heads + h) * a.block_size + off) * row + c;
        } else {
            dst = reinterpret_cast<i32x4*>(a.a_cache) + (size_t)slot * n + piece;
        }
        *dst = *src;
    }
}

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    // four pieces per thread once there are tokens enough for that
    const int n = a.heads * (a.a_row + a.b_row);
    const int per = n < 4 * APP_THREADS ? 4 * APP_THREADS / n : 1;
    const int few = (a.tokens + 1023) / 1024;
    const int tpw = per < few ? per : few;
    const dim3 grid((unsigned)((a.tokens + tpw - 1) / tpw)), block(APP_THREADS);
    if (a.b_cache != nullptr) hipLaunchKernelGGL(append_kernel<true>, grid, block, 0, s, a, tpw);
    else hipLaunchKernelGGL(append_kernel<false>, grid, block, 0, s, a, tpw);
    return hipGetLastError();
}

}  // namespace gdn
