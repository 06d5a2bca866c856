// Attention of packed prompts over a paged key/value cache, grouped heads, causal
// (gdn_paged_prefill).
//
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j,   j <= pos_t,
// k_j and v_j the rows of head h / group in the request's pages, pos_t the token's position in its
// request. Three launches: the tile tables (prefix sums of the device-resident lengths), the
// attention (paged_attend.h), the joining of units that were cut between workers (key_join.h).
// 12000 tokens of one prompt, 32 heads of 128, bf16: 5 + 1357 + 23 us (least 4.5 + 1251 + 22); three
// turns of 5 to 200 tokens, 8 heads of 64, fp32: 4 + 15.4 + 6.4 us.
#include "paged_attend.h"

namespace gdn {

namespace {

// Length of request i without the tokens that lie behind total_tokens: those have no rows here
// (a step that overflowed its buffers), and the rows before them keep their positions.
__device__ __forceinline__ int pp_len(const PagedPrefillArgs& a, int i) {
    return max(a.at.seq_lens[i], 0) - (max(a.cu_seqlens[i + 1], a.total_tokens) - a.total_tokens);
}
__device__ __forceinline__ int pp_start(const PagedPrefillArgs& a, int i) {
    return min(max(a.cu_seqlens[i], 0), a.total_tokens);
}
__device__ __forceinline__ int pp_new(const PagedPrefillArgs& a, int i) {
    return max(min(a.cu_seqlens[i + 1], a.total_tokens) - pp_start(a, i), 0);
}

template <typename T, int D>
__global__ __launch_bounds__(AT_TABLE_THREADS) void prefill_tables_kernel(PagedPrefillArgs a) {
    using X = AttendTile<T, D>;
    constexpr int ROWS = ATTEND_ROWS<T, D>;
    attend_tables(
        a.at, ROWS, X::KB, [&](int i) { return pp_new(a, i) * a.at.group; },
        [&](int i, int row0) {
            const int fresh = pp_new(a, i), len = pp_len(a, i), pos0 = len - fresh;
            const int rows = fresh * a.at.group;
            const int upto = (min(row0 + ROWS, rows) + a.at.group - 1) / a.at.group;
            const int reach = max(min(min(len, a.at.max_keys), pos0 + upto), 0);
            return AttendUnit{i, pp_start(a, i), row0, rows, reach, pos0};
        });
}

template <typename T, int D>
__global__ __launch_bounds__(JOIN_THREADS) void prefill_join_kernel(AttendArgs a) {
    join_parts<D>(a.join, [&](int t, int kvh, int row, int col, const float x[4]) {
        const AttendUnit u = a.tile[t];
        const int r = u.row0 + row;
        if (r >= u.rows) return;
        const int tok = (int)a.by_group((uint32_t)r), h = r - tok * a.group;
        store4<T>(reinterpret_cast<T*>(a.o) +
                      ((size_t)(u.token0 + tok) * a.H + kvh * a.group + h) * D + col, x);
    });
}

template <typename T, int D>
hipError_t run_prefill(const PagedPrefillArgs& a, hipStream_t s) {
    using X = AttendTile<T, D>;
    hipLaunchKernelGGL((prefill_tables_kernel<T, D>), dim3(1), dim3(AT_TABLE_THREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((paged_attend_kernel<T, D, false>), dim3((unsigned)a.at.workers),
                       dim3(X::WAVES * WAVE), 0, s, a.at);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prefill_join_kernel<T, D>), dim3(join_grid(a.at.join)), dim3(JOIN_THREADS),
                       0, s, a.at);
    return hipGetLastError();
}

template <typename T>
hipError_t pick_dim(const PagedPrefillArgs& a, hipStream_t s) {
    switch (a.at.d) {
        case 64: return run_prefill<T, 64>(a, s);
        case 128: return run_prefill<T, 128>(a, s);
        case 256: return run_prefill<T, 256>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t paged_prefill_layout(PagedPrefillArgs* a, void* ws) {
    AttendArgs& at = a->at;
    const int rows = attend_tile_rows(at.dtype, at.d);
    at.group = at.H / at.kv_heads;
    at.by_group = FastDiv::of((uint32_t)at.group);
    // sum_i ceil(rows_i / R) <= (sum rows_i + n (R - 1)) / R
    at.tiles = (int)(((int64_t)a->total_tokens * at.group + (int64_t)at.n_seqs * (rows - 1)) / rows);
    at.workers = split_workers(device_cu_count(), 1);
    Layout l(ws);
    attend_table_layout(&at, &l);
    JoinShape& j = at.join;
    j.row_tiles = 1;
    j.tile = j.rows = rows;
    j.per_unit = 0;
    j.count = at.workers;
    // Workgroups of a note: a short prompt (three turns of 5 to 200 tokens) 39.7 us a call with 4,
    // 30.7 with 16, 29.8 with 32; long ones do not mind.
    j.share = 16;
    j.slices = 1;
    j.part_o = l.take<float>((size_t)2 * at.workers * rows * at.d);
    j.part_ml = l.take<float>((size_t)2 * at.workers * rows * 2);
    j.notes = l.take<int4>((size_t)at.workers);
    return l.size;
}

hipError_t launch_paged_prefill(const PagedPrefillArgs& a, hipStream_t s) {
    (void)hipGetLastError();  // report only errors raised by this call's launches
    return a.at.dtype == 1 ? pick_dim<bf16>(a, s) : pick_dim<float>(a, s);
}

}  // namespace gdn
