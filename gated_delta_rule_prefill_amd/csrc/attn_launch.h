// Host-side launch interface between the C ABI layer (gdn_api.cpp) and the kernels of the
// softmax-attention layers (paged.hip, paged_decode.hip, latent_decode.hip,
// latent_prefill.hip). Arguments arrive here already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "key_join.h"

namespace gdn {

struct PlanArgs {
    const int32_t *ctx_lens, *new_lens;
    int n, block_size;
    int32_t* block_table;
    int max_blocks;
    const int32_t* free_blocks;
    int n_free, max_tokens;
    int32_t *cu_seqlens, *seq_lens;
    int64_t* slot_map;
    int32_t* positions;
    int32_t* counts;
};
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream);

// Rows of two sources written to cache slots. All sizes in 16-byte pieces.
//   split caches (b_cache != null): source a [tokens][heads][row] to a_cache
//     [n_blocks][heads][block_size][row], b to b_cache likewise
//   one cache (b_cache == null, heads == 1): a_cache row = a's row followed by b's
struct AppendArgs {
    const void *a, *b;
    int64_t a_stride, b_stride;
    const int64_t* slot_map;
    int tokens, heads, a_row, b_row;
    void *a_cache, *b_cache;
    int n_blocks, block_size;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t stream);

// Paged decode: rows of one unit are the n_pos x (num_heads / kv_heads) query rows that share
// a key/value head, cut into row tiles of 16 * rt rows.
struct PagedDecodeArgs {
    int dtype, H, kv_heads, d, n_pos, max_blocks, n_blocks;
    float scale;
    const void *q, *k_cache, *v_cache;
    const int32_t* block_table;
    FastDiv block;       // by the page size
    SplitShape split;    // units = kv_heads
    int group, rows, rt, row_tiles, workers;
    JoinShape join;
    void* o;
};
// Row tiles, workers and workspace bytes of a call (fills what lies between q and o).
size_t paged_decode_layout(PagedDecodeArgs* a, void* ws);
hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t stream);

// Latent decode (bf16): a request's n_pos x H query rows all read the same latents; they are
// cut into row tiles of 16 * rt rows.
struct LatentDecodeArgs {
    int H, rank, d_nope, d_v, n_pos, max_blocks, n_blocks;
    float scale;
    const void *q_nope, *q_pe, *w_kv, *cache;
    const int32_t* block_table;
    FastDiv block;       // by the page size
    SplitShape split;    // units = 1
    int rows, rt, row_tiles, workers;
    JoinShape join;
    void* o;
    void* q_lat;         // [batch n_pos][H][rank] bf16: queries in the latent space
    float* o_lat;        // [batch n_pos][H][rank]: outputs there
};
size_t latent_decode_layout(LatentDecodeArgs* a, void* ws);
hipError_t launch_latent_decode(const LatentDecodeArgs& a, hipStream_t stream);

// Latent prefill (bf16). Keys are laid out in the workspace request after request, each
// starting at a new 64-key tile; queries in tiles of 128 rows of one request.
struct LatentPrefillArgs {
    int H, rank, d, n_seqs, total_tokens, max_blocks, n_blocks, max_keys;
    float scale;
    const void *q_nope, *q_pe, *w_kv, *cache;
    const int32_t *block_table, *cu_seqlens, *seq_lens;
    FastDiv block;       // by the page size
    int key_tiles, q_tiles;  // bounds from the host's totals
    void* o;
    int32_t* key_tile;   // [n_seqs + 1] first key tile of each request
    int2* order;         // [q_tiles] (request, query tile) in the order of their start
    int32_t* q_tile;     // [n_seqs + 1] first query tile
    int32_t* head_shift; // [H][2] powers of two that its keys and values are written times
    int4* tile;          // [key_tiles] x, y: a bit per existing key; z: power of two below 1 / that
    void* k_pe;          // [key_tiles][64][64] rotary keys (bf16)
    void* k;             // [H][key_tiles][64][d] (fp16)
    void* vt;            // [H][key_tiles][d][64] (fp16), keys of each 16 in the order of the weights
};
size_t latent_prefill_layout(LatentPrefillArgs* a, int64_t total_keys, void* ws);
hipError_t launch_latent_prefill(const LatentPrefillArgs& a, hipStream_t stream);

}  // namespace gdn
