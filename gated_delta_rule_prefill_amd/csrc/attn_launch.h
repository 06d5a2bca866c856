// Host-side launch interface between the C ABI layer (gdn_api.cpp) and the kernels of the
// softmax-attention layers (paged.hip, pages.hip, paged_decode.hip, paged_prefill.hip,
// shared_decode.hip, latent_decode.hip, latent_prefill.hip). Arguments arrive here already
// validated.
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

// Pages that requests share (pages.hip).
struct ForkArgs {
    const int32_t *src_rows, *dst_rows, *lens;
    int n;
    int32_t* table;
    int n_rows, max_blocks, block_size;
    int32_t* shares;
    int n_blocks;
    const int32_t* free_blocks;
    int n_free;
    int32_t *copy_src, *copy_dst, *counts;
};
hipError_t launch_paged_fork(const ForkArgs& a, hipStream_t stream);

struct FreeArgs {
    const int32_t *rows, *lens;
    int n;
    int32_t* table;
    int n_rows, max_blocks, block_size;
    int32_t* shares;
    int n_blocks;
    int32_t* freed;
    int max_freed;
    int32_t* counts;
    int32_t* seg_count;  // workspace: freed pages of each segment of the pool
};
size_t paged_free_layout(FreeArgs* a, void* ws);
hipError_t launch_paged_free(const FreeArgs& a, hipStream_t stream);

struct CompactArgs {
    const int32_t* seq_lens;
    int n_rows;
    int32_t* table;
    int max_blocks, block_size;
    int32_t* shares;
    int n_blocks;
    int32_t *copy_src, *copy_dst;
    int max_copies;
    int32_t* counts;
    int64_t words;   // of 32 pages
    uint32_t* bits;  // workspace: a bit per live page
    int32_t* rank;   // workspace: live pages before each word
};
size_t paged_compact_layout(CompactArgs* a, void* ws);
hipError_t launch_paged_compact(const CompactArgs& a, hipStream_t stream);

constexpr int COPY_CACHES = 128;
struct CopyArgs {
    void* caches[COPY_CACHES];
    int64_t page_bytes;
    int n_blocks;
    const int32_t *src, *dst;
    int n;
    const int32_t* count;  // or null: pairs from *count on are not looked at
};
hipError_t launch_paged_copy(const CopyArgs& a, int n_caches, hipStream_t stream);

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
    // behind a shared prefix (gdn_paged_shared_decode): split.seq_lens counts a request's own keys
    const int32_t* start;     // [batch] keys of the prefix, which another kernel attends
    const int32_t* seq_lens;  // [batch] the whole lengths
};
// Row tiles, workers and workspace bytes of a call (fills what lies between q and o).
size_t paged_decode_layout(PagedDecodeArgs* a, void* ws);
hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t stream);

// Attention of many query rows over a paged cache (paged_attend.h).
// A tile of query rows: those rows of a sequence that share a key/value head.
struct AttendUnit {
    int seq;     // its row of the block table
    int token0;  // packed token (request x position) of the sequence's first query row
    int row0;    // the tile's first row in the sequence
    int rows;    // rows of the sequence
    int reach;   // keys that the tile's last row sees, at most
    int pos0;    // causal: position of the sequence's first query token
};
struct AttendArgs {
    int dtype, H, kv_heads, d, group, n_pos, max_blocks, n_blocks, max_keys;
    float scale;
    const void *q, *k_cache, *v_cache;
    const int32_t *block_table, *seq_lens;
    FastDiv block, by_group, by_pos;  // by the page size, the heads of a group, n_pos
    int n_seqs;        // sequences that share a table row's keys: prompts, or groups of requests
    int tiles;         // bound from the host's totals
    int workers;
    int32_t* head;     // [1] tiles
    int64_t* total;    // [1] positions in the stream of one key/value head
    int32_t* seq_tile; // [n_seqs + 1] first tile of each sequence
    int64_t* first;    // [tiles + 1] first position of each tile
    AttendUnit* tile;  // [tiles]
    JoinShape join;
    int2* prefix_notes;  // shared prefixes: [kv_heads x tiles] first and last worker of a unit
    void* o;
};

// Prompts: sequence i's query tokens are its last cu_seqlens[i + 1] - cu_seqlens[i].
struct PagedPrefillArgs {
    AttendArgs at;
    const int32_t* cu_seqlens;
    int total_tokens;
};
size_t paged_prefill_layout(PagedPrefillArgs* a, void* ws);
hipError_t launch_paged_prefill(const PagedPrefillArgs& a, hipStream_t stream);

// Decode behind shared prefixes: `at` attends each group's prefix for all its requests, `own` the
// rest of each request; then both are joined.
struct SharedDecodeArgs {
    AttendArgs at;        // n_seqs: groups
    PagedDecodeArgs own;
    const int32_t *group_cu, *prefix_lens;
    int batch;
    int64_t min_bytes;    // spared reads from which on prefixes are attended apart; < 0: by rule
    int32_t *start, *own_keys;  // [batch] keys of the prefix, and behind it
    int2* place;          // [batch] group (-1: none), first row in it
    int2* prefix_notes;   // [kv_heads x tiles] first and last worker of a unit
};
size_t shared_decode_layout(SharedDecodeArgs* a, void* ws);
hipError_t launch_shared_decode(const SharedDecodeArgs& a, hipStream_t stream);
// Its second half, in paged_decode.hip.
hipError_t launch_own_keys(const PagedDecodeArgs& a, hipStream_t stream);

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
