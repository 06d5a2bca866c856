// C ABI of libgdn.so: host-side validation, workspace sizing and launches.
// Every check happens before the first HIP call, so a rejected call launches nothing and
// touches no memory; errors are reported as status codes plus a thread-local message.
#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "../../include/gdn.h"
#include "attn_launch.h"
#include "gdn_launch.h"

namespace {

thread_local char g_err[512] = "";

int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return status;
}

int ok() {
    g_err[0] = '\0';
    return GDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

int check_dims(const gdn_dims_t* d) {
    if (d == nullptr) return fail(GDN_ERR_NULL, "dims is NULL");
    if (d->num_heads < 1) return fail(GDN_ERR_SHAPE, "num_heads must be >= 1 (got %d)", d->num_heads);
    if (!dim_ok(d->d_k) || !dim_ok(d->d_v))
        return fail(GDN_ERR_UNSUPPORTED, "d_k, d_v must be in {16,32,64,128} (got %d, %d)",
                    d->d_k, d->d_v);
    if (d->d_k != d->d_v)
        return fail(GDN_ERR_UNSUPPORTED, "d_k must equal d_v (got %d, %d)", d->d_k, d->d_v);
    if (d->dtype != GDN_DTYPE_F32 && d->dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype must be 0 (fp32) or 1 (bf16), got %d", d->dtype);
    if (d->gate != GDN_GATE_SCALAR && d->gate != GDN_GATE_PER_KEY)
        return fail(GDN_ERR_UNSUPPORTED, "gate must be 0 (scalar) or 1 (per key), got %d", d->gate);
    if (d->qk_l2norm != 0 && d->qk_l2norm != 1)
        return fail(GDN_ERR_UNSUPPORTED, "qk_l2norm must be 0 or 1, got %d", d->qk_l2norm);
    return GDN_OK;
}

#define REQUIRE_PTR(p)                                                         \
    do {                                                                       \
        if ((p) == nullptr) return fail(GDN_ERR_NULL, "%s is NULL", #p);       \
        if (!aligned16(p)) return fail(GDN_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
    } while (0)

// Lists that kernels read one entry at a time, so that a part of a longer one will do.
#define REQUIRE_LIST(p)                                                        \
    do {                                                                       \
        if ((p) == nullptr) return fail(GDN_ERR_NULL, "%s is NULL", #p);       \
        if (reinterpret_cast<uintptr_t>(p) % sizeof(*(p)) != 0)                \
            return fail(GDN_ERR_ALIGN, "%s is not aligned to its entries", #p); \
    } while (0)

#define OPT_PTR(p)                                                                   \
    do {                                                                             \
        if ((p) != nullptr && !aligned16(p))                                         \
            return fail(GDN_ERR_ALIGN, "%s is not 16-byte aligned", #p);             \
    } while (0)

// Debug builds (GDN_DEBUG_CHECKS) also verify what the kernels assume but the host cannot
// see without reading device memory: the valid slot indices of one call are distinct. The
// check copies the slot arrays to the host, which synchronises `stream`; release builds
// skip it. A repeated slot returns GDN_ERR_SHAPE before any launch.
#ifdef GDN_DEBUG_CHECKS
int debug_distinct_slots(std::initializer_list<std::pair<const int32_t*, int64_t>> lists,
                         int32_t n_slots, void* stream, const char* what) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    std::vector<char> seen((size_t)n_slots, 0);
    for (const auto& l : lists) {
        if (l.first == nullptr || l.second <= 0) continue;
        std::vector<int32_t> h((size_t)l.second);
        if (hipMemcpyAsync(h.data(), l.first, sizeof(int32_t) * h.size(), hipMemcpyDeviceToHost,
                           s) != hipSuccess ||
            hipStreamSynchronize(s) != hipSuccess) {
            (void)hipGetLastError();
            return fail(GDN_ERR_LAUNCH, "%s: debug check could not read the slot indices", what);
        }
        for (int32_t v : h) {
            if (v < 0 || v >= n_slots) continue;
            if (seen[(size_t)v]) return fail(GDN_ERR_SHAPE, "%s: slot %d used twice", what, v);
            seen[(size_t)v] = 1;
        }
    }
    return GDN_OK;
}
#define DEBUG_DISTINCT_SLOTS(lists, n_slots, what)                                  \
    do {                                                                            \
        int st_ = debug_distinct_slots(lists, n_slots, stream, what);               \
        if (st_) return st_;                                                        \
    } while (0)
#else
#define DEBUG_DISTINCT_SLOTS(lists, n_slots, what) \
    do {                                           \
    } while (0)
#endif
#define SLOT_LISTS(...) (std::initializer_list<std::pair<const int32_t*, int64_t>>{__VA_ARGS__})

// Workspace of the allocation-free prefill (gdn_prefill_chunked_noalloc): one copy per GPU,
// created with the library's code object on that GPU. Host code never uses the array's name
// as an address (on the host it is only a stand-in for the symbol); the device address of
// each GPU's copy comes from hipGetSymbolAddress with that GPU current, kept per device.
static __device__ __align__(256) unsigned char scratch[GDN_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// The current device's copy of `scratch`, resolved on the first call with that device
// current. The caller's stream must belong to that device.
int scratch_for_stream(void* stream, void** out, const char* what) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return fail(GDN_ERR_LAUNCH, "%s: no current HIP device", what);
    }
    if (dev < 0 || dev >= kMaxDevices)
        return fail(GDN_ERR_UNSUPPORTED, "%s: device %d beyond the %d the library tracks", what,
                    dev, kMaxDevices);
    if (stream != nullptr) {
        hipDevice_t sdev = -1;
        if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev) != hipSuccess) {
            (void)hipGetLastError();
            return fail(GDN_ERR_LAUNCH, "%s: cannot query the stream's device", what);
        }
        if (sdev != dev)
            return fail(GDN_ERR_UNSUPPORTED, "%s: the stream belongs to device %d, device %d is "
                                             "current", what, (int)sdev, dev);
    }
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        void* p = nullptr;
        const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || p == nullptr) {
            (void)hipGetLastError();
            return fail(GDN_ERR_LAUNCH, "%s: hipGetSymbolAddress(scratch) failed: %s", what,
                        hipGetErrorString(e));
        }
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return GDN_OK;
}

int launch_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(GDN_ERR_LAUNCH, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

int prefill_common_checks(const gdn_dims_t* dims, int32_t n_seqs, int32_t total_tokens,
                          int32_t chunk) {
    int st = check_dims(dims);
    if (st) return st;
    if (n_seqs < 0 || total_tokens < 0)
        return fail(GDN_ERR_SHAPE, "n_seqs and total_tokens must be >= 0 (got %d, %d)", n_seqs,
                    total_tokens);
    if (chunk != 16 && chunk != 32 && chunk != 64)
        return fail(GDN_ERR_UNSUPPORTED, "chunk must be 16, 32 or 64 (got %d)", chunk);
    return GDN_OK;
}

int deltalog_pool_checks(const gdn_deltalog_pool_t* pool) {
    if (pool == nullptr) return fail(GDN_ERR_NULL, "pool is NULL");
    REQUIRE_PTR(pool->base);
    REQUIRE_PTR(pool->lbar);
    REQUIRE_PTR(pool->klog);
    REQUIRE_PTR(pool->ulog);
    REQUIRE_PTR(pool->lamlog);
    REQUIRE_PTR(pool->len);
    if (pool->M < 2 || pool->M > 17)
        return fail(GDN_ERR_UNSUPPORTED, "merge interval M must be in [2, 17] (got %d)", pool->M);
    return GDN_OK;
}

// Raw projection and short-convolution operands of the conv-fused prefill.
struct ConvIn {
    const void* x;
    const float* w;
    int32_t width;
    void* state;
};

// Shared by gdn_prefill_chunked (no checkpoints), gdn_prefill_chunked_ckpt and, with conv
// set (q, k, v then unused), gdn_prefill_chunked_conv.
int prefill_run(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
                const float* g, const float* beta, const int32_t* cu_seqlens, int32_t n_seqs,
                int32_t total_tokens, int32_t chunk, float* state_pool, int32_t n_slots,
                const int32_t* slots, const int32_t* has_init, const int32_t* ckpt_cu,
                const int32_t* ckpt_pos, const int32_t* ckpt_slots, int32_t n_ckpt, void* o,
                void* workspace, size_t ws_bytes, void* stream, const char* what,
                const ConvIn* conv = nullptr, bool noalloc = false) {
    int st = prefill_common_checks(dims, n_seqs, total_tokens, chunk);
    if (st) return st;
    if (conv != nullptr && (conv->width < 2 || conv->width > 4))
        return fail(GDN_ERR_UNSUPPORTED, "conv_width must be 2, 3 or 4 (got %d)", conv->width);
    if (n_seqs == 0) return ok();
    REQUIRE_PTR(cu_seqlens);
    REQUIRE_PTR(slots);
    OPT_PTR(has_init);
    REQUIRE_PTR(state_pool);
    if (n_slots < 1) return fail(GDN_ERR_SHAPE, "n_slots must be >= 1 (got %d)", n_slots);
    if (n_ckpt < 0) return fail(GDN_ERR_SHAPE, "n_ckpt must be >= 0 (got %d)", n_ckpt);
    if (n_ckpt > 0) {
        REQUIRE_PTR(ckpt_cu);
        REQUIRE_PTR(ckpt_pos);
        REQUIRE_PTR(ckpt_slots);
    }
    if (conv != nullptr) {
        const void* x = conv->x;
        const float* conv_w = conv->w;
        void* conv_state = conv->state;
        if (total_tokens > 0) REQUIRE_PTR(x);
        REQUIRE_PTR(conv_w);
        OPT_PTR(conv_state);
    }
    if (total_tokens > 0) {
        if (conv == nullptr) {
            REQUIRE_PTR(q);
            REQUIRE_PTR(k);
            REQUIRE_PTR(v);
        }
        REQUIRE_PTR(g);
        REQUIRE_PTR(beta);
        REQUIRE_PTR(o);
    }
    if (noalloc) {
        const size_t need = gdn::prefill_ws_layout(dims->dtype, dims->num_heads, dims->d_k,
                                                   dims->d_v, chunk, n_seqs, total_tokens,
                                                   nullptr, nullptr);
        if (need > GDN_NOALLOC_SCRATCH_BYTES)
            return fail(GDN_ERR_WORKSPACE, "%s: the call needs %zu bytes of workspace, the "
                                           "library's per-GPU scratch holds %zu", what, need,
                        GDN_NOALLOC_SCRATCH_BYTES);
        st = scratch_for_stream(stream, &workspace, what);
        if (st) return st;
        ws_bytes = GDN_NOALLOC_SCRATCH_BYTES;
    }
    REQUIRE_PTR(workspace);
    gdn::PrefillWs ws;
    const size_t need = gdn::prefill_ws_layout(dims->dtype, dims->num_heads, dims->d_k,
                                               dims->d_v, chunk, n_seqs, total_tokens,
                                               workspace, &ws);
    if (ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    gdn::PrefillArgs a;
    a.dtype = dims->dtype;
    a.gate = dims->gate;
    a.H = dims->num_heads;
    a.dk = dims->d_k;
    a.dv = dims->d_v;
    a.chunk = chunk;
    a.cp = gdn::prefill_cp(dims->dtype, chunk);
    a.l2norm = dims->qk_l2norm;
    a.scale = dims->scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.cu_seqlens = cu_seqlens;
    a.n_seqs = n_seqs;
    a.total_tokens = total_tokens;
    a.state_pool = state_pool;
    a.n_slots = n_slots;
    a.slots = slots;
    a.has_init = has_init;
    a.o = o;
    a.ckpt_cu = n_ckpt > 0 ? ckpt_cu : nullptr;
    a.ckpt_pos = n_ckpt > 0 ? ckpt_pos : nullptr;
    a.ckpt_slots = n_ckpt > 0 ? ckpt_slots : nullptr;
    a.n_ckpt = n_ckpt;
    a.x = conv != nullptr ? conv->x : nullptr;
    a.conv_w = conv != nullptr ? conv->w : nullptr;
    a.conv_state = conv != nullptr ? conv->state : nullptr;
    a.conv_width = conv != nullptr ? conv->width : 0;
    a.ws = ws;
    DEBUG_DISTINCT_SLOTS(SLOT_LISTS({slots, n_seqs}, {a.ckpt_slots, (int64_t)n_ckpt}), n_slots,
                         what);
    return launch_status(gdn::launch_prefill(a, static_cast<hipStream_t>(stream)), what);
}

// Shared by gdn_decode_step (spec = false: one token, num_accepted unused) and
// gdn_decode_spec (spec = true: n_pos tokens per request, num_accepted required).
int decode_run(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
               const float* g, const float* beta, float* state_pool, int32_t n_slots,
               const int32_t* slots, bool spec, const int32_t* num_accepted, int32_t batch,
               int32_t n_pos, void* o, void* stream, const char* what) {
    int st = check_dims(dims);
    if (st) return st;
    if (batch < 0) return fail(GDN_ERR_SHAPE, "batch must be >= 0 (got %d)", batch);
    if (batch == 0) return ok();
    REQUIRE_PTR(q);
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
    REQUIRE_PTR(state_pool);
    REQUIRE_PTR(slots);
    REQUIRE_PTR(o);
    if (spec) REQUIRE_PTR(num_accepted);
    if (n_slots < 1) return fail(GDN_ERR_SHAPE, "n_slots must be >= 1 (got %d)", n_slots);
    gdn::DecodeArgs a;
    a.dtype = dims->dtype;
    a.gate = dims->gate;
    a.H = dims->num_heads;
    a.dk = dims->d_k;
    a.dv = dims->d_v;
    a.l2norm = dims->qk_l2norm;
    a.scale = dims->scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.pool = state_pool;
    a.n_slots = n_slots;
    a.slots = slots;
    a.batch = batch;
    a.o = o;
    a.num_accepted = spec ? num_accepted : nullptr;
    a.n_pos = n_pos;
    DEBUG_DISTINCT_SLOTS(SLOT_LISTS({slots, (int64_t)batch * (spec ? n_pos : 1)}), n_slots, what);
    return launch_status(gdn::launch_decode(a, static_cast<hipStream_t>(stream)), what);
}

// ------------------------------------------------- paged softmax attention: shared checks

bool paged_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// A cache of n_blocks pages of block_size rows per head. Rows are numbered in 32 bits inside
// the kernels (byte offsets in 64).
int check_cache(int32_t dtype, int32_t kv_heads, int32_t n_blocks, int32_t block_size) {
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype must be 0 (fp32) or 1 (bf16), got %d", dtype);
    if (kv_heads < 1 || n_blocks < 1 || block_size < 1)
        return fail(GDN_ERR_SHAPE, "heads, n_blocks and block_size must be >= 1 (got %d, %d, %d)",
                    kv_heads, n_blocks, block_size);
    const uint64_t slots = (uint64_t)n_blocks * (uint32_t)block_size;
    if (slots > 0x7fffffffull || slots * (uint32_t)kv_heads > 0xfffffffeull)
        return fail(GDN_ERR_UNSUPPORTED, "a cache holds at most 2^31 - 1 tokens and 2^32 - 2 rows "
                                         "(got %d blocks of %d tokens, %d heads)", n_blocks,
                    block_size, kv_heads);
    return GDN_OK;
}

// The keys that a block table row can address are counted in 32 bits.
int check_table(int32_t max_blocks, int32_t block_size) {
    if (max_blocks < 1) return fail(GDN_ERR_SHAPE, "max_blocks must be >= 1 (got %d)", max_blocks);
    if ((int64_t)max_blocks * block_size > 0x3fffffff)
        return fail(GDN_ERR_UNSUPPORTED, "a block table row addresses at most 2^30 - 1 tokens "
                                         "(got %d blocks of %d)", max_blocks, block_size);
    return GDN_OK;
}

// The split of a decode call counts its key chunks (64 keys at least, and SPLIT_EXTRA for a head
// group of a request) in 32 bits.
int check_chunks(int32_t batch, int32_t units, int32_t max_blocks, int32_t block_size) {
    const int64_t chunks = ((int64_t)max_blocks * block_size + 63) / 64 + gdn::SPLIT_EXTRA;
    if (chunks * units > 0x3fffffffll / (batch > 0 ? batch : 1))
        return fail(GDN_ERR_UNSUPPORTED, "batch x heads x table row are too many key chunks (%d x "
                                         "%d x %lld): split the batch", batch, units,
                    (long long)chunks);
    return GDN_OK;
}

// Source rows of an append: `width` elements each, `stride` elements apart, 16-byte aligned.
int check_rows(int32_t dtype, int32_t tokens, int64_t stride, int64_t width, const char* name) {
    if (tokens < 0) return fail(GDN_ERR_SHAPE, "tokens must be >= 0 (got %d)", tokens);
    if (width > (1 << 24))
        return fail(GDN_ERR_UNSUPPORTED, "%s: rows of %lld elements", name, (long long)width);
    if (tokens == 0) return GDN_OK;
    if (stride < width)
        return fail(GDN_ERR_SHAPE, "%s: row stride %lld is smaller than the row (%lld)", name,
                    (long long)stride, (long long)width);
    if (stride % (dtype == GDN_DTYPE_BF16 ? 8 : 4) != 0)
        return fail(GDN_ERR_ALIGN, "%s: row stride %lld is not a multiple of 16 bytes", name,
                    (long long)stride);
    return GDN_OK;
}

int check_batch(int32_t batch, int32_t n_pos) {
    if (batch < 0) return fail(GDN_ERR_SHAPE, "batch must be >= 0 (got %d)", batch);
    if (n_pos < 1 || n_pos > GDN_SPEC_MAX_POS)
        return fail(GDN_ERR_UNSUPPORTED, "n_pos must be in [1, %d] (got %d)", GDN_SPEC_MAX_POS,
                    n_pos);
    return GDN_OK;
}

int check_paged_dims(const gdn_paged_dims_t* d, int32_t batch, int32_t n_pos) {
    if (d == nullptr) return fail(GDN_ERR_NULL, "dims is NULL");
    if (d->num_heads < 1 || d->num_kv_heads < 1 || d->num_heads % d->num_kv_heads != 0)
        return fail(GDN_ERR_SHAPE, "num_heads (%d) must be a positive multiple of num_kv_heads "
                                   "(%d)", d->num_heads, d->num_kv_heads);
    if (d->num_heads > GDN_ATTN_MAX_HEADS)
        return fail(GDN_ERR_UNSUPPORTED, "num_heads must be <= %d (got %d)", GDN_ATTN_MAX_HEADS,
                    d->num_heads);
    if (!paged_dim_ok(d->d))
        return fail(GDN_ERR_UNSUPPORTED, "d must be 64, 128 or 256 (got %d)", d->d);
    if (d->dtype != GDN_DTYPE_F32 && d->dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype must be 0 (fp32) or 1 (bf16), got %d", d->dtype);
    return check_batch(batch, n_pos);
}

gdn::PagedDecodeArgs paged_args(const gdn_paged_dims_t* d, int32_t batch, int32_t n_pos) {
    gdn::PagedDecodeArgs a = {};
    a.dtype = d->dtype;
    a.H = d->num_heads;
    a.kv_heads = d->num_kv_heads;
    a.d = d->d;
    a.n_pos = n_pos;
    a.scale = d->scale;
    a.split.batch = batch;
    return a;
}

int check_latent_dims(const gdn_latent_dims_t* d) {
    if (d == nullptr) return fail(GDN_ERR_NULL, "dims is NULL");
    if (d->num_heads < 1) return fail(GDN_ERR_SHAPE, "num_heads must be >= 1 (got %d)", d->num_heads);
    if (d->num_heads > GDN_ATTN_MAX_HEADS)
        return fail(GDN_ERR_UNSUPPORTED, "num_heads must be <= %d (got %d)", GDN_ATTN_MAX_HEADS,
                    d->num_heads);
    if (d->dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "latent attention takes bf16 (dtype 1), got %d", d->dtype);
    if (d->rank != 256 && d->rank != 512)
        return fail(GDN_ERR_UNSUPPORTED, "rank must be 256 or 512 (got %d)", d->rank);
    if (d->d_rope != 64)
        return fail(GDN_ERR_UNSUPPORTED, "d_rope must be 64 (got %d)", d->d_rope);
    if ((d->d_nope != 64 && d->d_nope != 128) || d->d_v != d->d_nope)
        return fail(GDN_ERR_UNSUPPORTED, "d_nope and d_v must be equal, 64 or 128 (got %d, %d)",
                    d->d_nope, d->d_v);
    return GDN_OK;
}

// The row counts of a call are kept in 32 bits.
int check_latent_rows(const gdn_latent_dims_t* d, int64_t tokens) {
    if (tokens * d->num_heads > 0x7fffffffll)
        return fail(GDN_ERR_UNSUPPORTED, "tokens x heads must stay below 2^31 (got %lld x %d)",
                    (long long)tokens, d->num_heads);
    return GDN_OK;
}

// A decode call's projections have a workgroup row per 32 (request, position) rows.
int check_latent_batch(const gdn_latent_dims_t* d, int32_t batch, int32_t n_pos) {
    const int st = check_batch(batch, n_pos);
    if (st) return st;
    if ((int64_t)batch * n_pos > (1 << 20))
        return fail(GDN_ERR_UNSUPPORTED, "batch x n_pos must be <= 2^20 (got %d x %d): split the "
                                         "batch", batch, n_pos);
    return check_latent_rows(d, (int64_t)batch * n_pos);
}

gdn::LatentDecodeArgs latent_decode_args(const gdn_latent_dims_t* d, int32_t batch,
                                         int32_t n_pos) {
    gdn::LatentDecodeArgs a = {};
    a.H = d->num_heads;
    a.rank = d->rank;
    a.d_nope = d->d_nope;
    a.d_v = d->d_v;
    a.n_pos = n_pos;
    a.scale = d->scale;
    a.split.batch = batch;
    return a;
}

int check_latent_prefill(const gdn_latent_dims_t* d, int32_t n_seqs, int32_t total_tokens,
                         int64_t total_keys) {
    int st = check_latent_dims(d);
    if (st) return st;
    if (n_seqs < 0 || total_tokens < 0 || total_keys < 0)
        return fail(GDN_ERR_SHAPE, "n_seqs, total_tokens and total_keys must be >= 0 (got %d, %d, "
                                   "%lld)", n_seqs, total_tokens, (long long)total_keys);
    // tile counts, grids and their products stay in 32 bits
    if (total_keys + (int64_t)n_seqs * 64 > 0x3fffffff ||
        ((int64_t)total_tokens / 128 + n_seqs + 1) * d->num_heads > 0x7fffff)
        return fail(GDN_ERR_UNSUPPORTED, "%lld keys, %d tokens in %d sequences, %d heads: split the "
                                         "call", (long long)total_keys, total_tokens, n_seqs,
                    d->num_heads);
    return check_latent_rows(d, total_tokens);
}

gdn::LatentPrefillArgs latent_prefill_args(const gdn_latent_dims_t* d, int32_t n_seqs,
                                           int32_t total_tokens) {
    gdn::LatentPrefillArgs a = {};
    a.H = d->num_heads;
    a.rank = d->rank;
    a.d = d->d_nope;
    a.n_seqs = n_seqs;
    a.total_tokens = total_tokens;
    a.scale = d->scale;
    return a;
}

// Debug builds: valid cache slots of one append are distinct (as DEBUG_DISTINCT_SLOTS).
#ifdef GDN_DEBUG_CHECKS
int debug_distinct_cache_slots(const int64_t* slot_map, int32_t tokens, int64_t n_slots,
                               void* stream, const char* what) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    std::vector<int64_t> h;
    std::vector<bool> seen;
    try {
        h.resize((size_t)tokens);
        seen.resize((size_t)n_slots);
    } catch (const std::bad_alloc&) {  // no exception leaves a C entry point
        return fail(GDN_ERR_LAUNCH, "%s: debug check: out of host memory", what);
    }
    if (hipMemcpyAsync(h.data(), slot_map, sizeof(int64_t) * h.size(), hipMemcpyDeviceToHost, s) !=
            hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess) {
        (void)hipGetLastError();
        return fail(GDN_ERR_LAUNCH, "%s: debug check could not read the slot map", what);
    }
    for (int64_t v : h) {
        if (v < 0 || v >= n_slots) continue;
        if (seen[(size_t)v])
            return fail(GDN_ERR_SHAPE, "%s: cache slot %lld used twice", what, (long long)v);
        seen[(size_t)v] = true;
    }
    return GDN_OK;
}
#define DEBUG_DISTINCT_CACHE_SLOTS(map, tokens, n_slots, what)                            \
    do {                                                                                  \
        int st_ = debug_distinct_cache_slots(map, tokens, n_slots, stream, what);         \
        if (st_) return st_;                                                              \
    } while (0)
#else
#define DEBUG_DISTINCT_CACHE_SLOTS(map, tokens, n_slots, what) \
    do {                                                       \
        (void)(what);                                          \
    } while (0)
#endif

}  // namespace

extern "C" {

int gdn_prefill_workspace_bytes(const gdn_dims_t* dims, int32_t n_seqs, int32_t total_tokens,
                                int32_t chunk, size_t* bytes) {
    int st = prefill_common_checks(dims, n_seqs, total_tokens, chunk);
    if (st) return st;
    if (bytes == nullptr) return fail(GDN_ERR_NULL, "bytes is NULL");
    *bytes = gdn::prefill_ws_layout(dims->dtype, dims->num_heads, dims->d_k, dims->d_v, chunk,
                                    n_seqs, total_tokens, nullptr, nullptr);
    return ok();
}

int gdn_prefill_chunked(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, const int32_t* cu_seqlens,
                        int32_t n_seqs, int32_t total_tokens, int32_t chunk,
                        float* state_pool, int32_t n_slots, const int32_t* slots,
                        const int32_t* has_init, void* o, void* workspace, size_t ws_bytes,
                        void* stream) {
    return prefill_run(dims, q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, chunk,
                       state_pool, n_slots, slots, has_init, nullptr, nullptr, nullptr, 0, o,
                       workspace, ws_bytes, stream, "gdn_prefill_chunked");
}

int gdn_prefill_chunked_ckpt(const gdn_dims_t* dims, const void* q, const void* k,
                             const void* v, const float* g, const float* beta,
                             const int32_t* cu_seqlens, int32_t n_seqs, int32_t total_tokens,
                             int32_t chunk, float* state_pool, int32_t n_slots,
                             const int32_t* slots, const int32_t* has_init,
                             const int32_t* ckpt_cu, const int32_t* ckpt_pos,
                             const int32_t* ckpt_slots, int32_t n_ckpt, void* o,
                             void* workspace, size_t ws_bytes, void* stream) {
    return prefill_run(dims, q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, chunk,
                       state_pool, n_slots, slots, has_init, ckpt_cu, ckpt_pos, ckpt_slots,
                       n_ckpt, o, workspace, ws_bytes, stream, "gdn_prefill_chunked_ckpt");
}

int gdn_prefill_chunked_conv(const gdn_dims_t* dims, const void* x, const float* conv_w,
                             int32_t conv_width, void* conv_state, const float* g,
                             const float* beta, const int32_t* cu_seqlens, int32_t n_seqs,
                             int32_t total_tokens, int32_t chunk, float* state_pool,
                             int32_t n_slots, const int32_t* slots, const int32_t* has_init,
                             void* o, void* workspace, size_t ws_bytes, void* stream) {
    const ConvIn conv{x, conv_w, conv_width, conv_state};
    return prefill_run(dims, nullptr, nullptr, nullptr, g, beta, cu_seqlens, n_seqs,
                       total_tokens, chunk, state_pool, n_slots, slots, has_init, nullptr,
                       nullptr, nullptr, 0, o, workspace, ws_bytes, stream,
                       "gdn_prefill_chunked_conv", &conv);
}

int gdn_prefill_chunked_noalloc(const gdn_dims_t* dims, const void* q, const void* k,
                                const void* v, const float* g, const float* beta,
                                const int32_t* cu_seqlens, int32_t n_seqs,
                                int32_t total_tokens, int32_t chunk, float* state_pool,
                                int32_t n_slots, const int32_t* slots, const int32_t* has_init,
                                void* o, void* stream) {
    return prefill_run(dims, q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, chunk,
                       state_pool, n_slots, slots, has_init, nullptr, nullptr, nullptr, 0, o,
                       nullptr, 0, stream, "gdn_prefill_chunked_noalloc", nullptr, true);
}

int gdn_decode_step(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, float* state_pool, int32_t n_slots,
                    const int32_t* slots, int32_t batch, void* o, void* stream) {
    return decode_run(dims, q, k, v, g, beta, state_pool, n_slots, slots, false, nullptr, batch,
                      1, o, stream, "gdn_decode_step");
}

int gdn_decode_spec(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, float* state_pool, int32_t n_slots,
                    const int32_t* spec_slots, const int32_t* num_accepted, int32_t batch,
                    int32_t n_pos, void* o, void* stream) {
    if (n_pos < 1 || n_pos > GDN_SPEC_MAX_POS)
        return fail(GDN_ERR_UNSUPPORTED, "n_pos must be in [1, %d] (got %d)", GDN_SPEC_MAX_POS,
                    n_pos);
    return decode_run(dims, q, k, v, g, beta, state_pool, n_slots, spec_slots, true,
                      num_accepted, batch, n_pos, o, stream, "gdn_decode_spec");
}

int gdn_decode_fused(const gdn_dims_t* dims, const void* x, const float* conv_w,
                     int32_t conv_width, void* conv_state, const float* forget_b,
                     const float* write_logit, const float* A_log, const float* dt_bias,
                     float lower_bound, float* state_pool, int32_t n_slots,
                     const int32_t* slots, int32_t batch, void* o, void* stream) {
    int st = check_dims(dims);
    if (st) return st;
    if (dims->gate != GDN_GATE_PER_KEY)
        return fail(GDN_ERR_UNSUPPORTED, "the fused decode step forms per-key (KDA) gates; "
                                         "gate must be GDN_GATE_PER_KEY");
    if (conv_width < 2 || conv_width > 4)
        return fail(GDN_ERR_UNSUPPORTED, "conv_width must be 2, 3 or 4 (got %d)", conv_width);
    if (!(lower_bound < 0.f) || lower_bound < -1e30f)
        return fail(GDN_ERR_UNSUPPORTED, "lower_bound must be finite and < 0 (got %g)",
                    (double)lower_bound);
    if (batch < 0) return fail(GDN_ERR_SHAPE, "batch must be >= 0 (got %d)", batch);
    if (batch == 0) return ok();
    REQUIRE_PTR(x);
    REQUIRE_PTR(conv_w);
    REQUIRE_PTR(conv_state);
    REQUIRE_PTR(forget_b);
    REQUIRE_PTR(write_logit);
    REQUIRE_PTR(A_log);
    REQUIRE_PTR(dt_bias);
    REQUIRE_PTR(state_pool);
    REQUIRE_PTR(slots);
    REQUIRE_PTR(o);
    if (n_slots < 1) return fail(GDN_ERR_SHAPE, "n_slots must be >= 1 (got %d)", n_slots);
    gdn::FusedDecodeArgs a;
    a.dtype = dims->dtype;
    a.H = dims->num_heads;
    a.dk = dims->d_k;
    a.dv = dims->d_v;
    a.l2norm = dims->qk_l2norm;
    a.width = conv_width;
    a.scale = dims->scale;
    a.lower_bound = lower_bound;
    a.x = x;
    a.conv_w = conv_w;
    a.conv_state = conv_state;
    a.forget_b = forget_b;
    a.write_logit = write_logit;
    a.A_log = A_log;
    a.dt_bias = dt_bias;
    a.pool = state_pool;
    a.n_slots = n_slots;
    a.slots = slots;
    a.batch = batch;
    a.o = o;
    DEBUG_DISTINCT_SLOTS(SLOT_LISTS({slots, batch}), n_slots, "gdn_decode_fused");
    return launch_status(gdn::launch_fused_decode(a, static_cast<hipStream_t>(stream)),
                         "gdn_decode_fused");
}

int gdn_deltalog_workspace_bytes(const gdn_dims_t* dims, int32_t batch, int32_t M,
                                 size_t* bytes) {
    int st = check_dims(dims);
    if (st) return st;
    if (batch < 0) return fail(GDN_ERR_SHAPE, "batch must be >= 0 (got %d)", batch);
    if (M < 2 || M > 17) return fail(GDN_ERR_UNSUPPORTED, "M must be in [2, 17] (got %d)", M);
    if (bytes == nullptr) return fail(GDN_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    return ok();
}

static gdn::DeltaLogArgs dl_args(const gdn_dims_t* dims, const gdn_deltalog_pool_t* pool,
                                 int32_t n_slots, const int32_t* slots, int32_t n) {
    gdn::DeltaLogArgs a = {};
    a.dtype = dims->dtype;
    a.gate = dims->gate;
    a.H = dims->num_heads;
    a.dk = dims->d_k;
    a.dv = dims->d_v;
    a.l2norm = dims->qk_l2norm;
    a.M = pool->M;
    a.scale = dims->scale;
    a.base = pool->base;
    a.lbar = pool->lbar;
    a.klog = pool->klog;
    a.ulog = pool->ulog;
    a.lamlog = pool->lamlog;
    a.len = pool->len;
    a.n_slots = n_slots;
    a.slots = slots;
    a.batch = n;
    return a;
}

int gdn_decode_deltalog(const gdn_dims_t* dims, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, const gdn_deltalog_pool_t* pool,
                        int32_t n_slots, const int32_t* slots, int32_t batch, void* o,
                        void* ws, size_t ws_bytes, void* stream) {
    (void)ws;
    (void)ws_bytes;
    int st = check_dims(dims);
    if (st) return st;
    if (batch < 0) return fail(GDN_ERR_SHAPE, "batch must be >= 0 (got %d)", batch);
    st = deltalog_pool_checks(pool);
    if (st) return st;
    if (batch == 0) return ok();
    REQUIRE_PTR(q);
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
    REQUIRE_PTR(slots);
    REQUIRE_PTR(o);
    if (n_slots < 1) return fail(GDN_ERR_SHAPE, "n_slots must be >= 1 (got %d)", n_slots);
    gdn::DeltaLogArgs a = dl_args(dims, pool, n_slots, slots, batch);
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.o = o;
    DEBUG_DISTINCT_SLOTS(SLOT_LISTS({slots, batch}), n_slots, "gdn_decode_deltalog");
    return launch_status(gdn::launch_deltalog(a, static_cast<hipStream_t>(stream)),
                         "gdn_decode_deltalog");
}

static int deltalog_maint(const gdn_dims_t* dims, const gdn_deltalog_pool_t* pool,
                          int32_t n_slots, const int32_t* slots, int32_t n, void* stream,
                          int mode, const char* what) {
    int st = check_dims(dims);
    if (st) return st;
    st = deltalog_pool_checks(pool);
    if (st) return st;
    if (n < 0) return fail(GDN_ERR_SHAPE, "n must be >= 0 (got %d)", n);
    if (n == 0) return ok();
    REQUIRE_PTR(slots);
    if (n_slots < 1) return fail(GDN_ERR_SHAPE, "n_slots must be >= 1 (got %d)", n_slots);
    gdn::DeltaLogArgs a = dl_args(dims, pool, n_slots, slots, n);
    DEBUG_DISTINCT_SLOTS(SLOT_LISTS({slots, n}), n_slots, what);
    return launch_status(gdn::launch_deltalog_maint(a, mode, static_cast<hipStream_t>(stream)),
                         what);
}

int gdn_deltalog_reset(const gdn_dims_t* dims, const gdn_deltalog_pool_t* pool,
                       int32_t n_slots, const int32_t* slots, int32_t n, void* stream) {
    return deltalog_maint(dims, pool, n_slots, slots, n, stream, 0, "gdn_deltalog_reset");
}

int gdn_deltalog_materialize(const gdn_dims_t* dims, const gdn_deltalog_pool_t* pool,
                             int32_t n_slots, const int32_t* slots, int32_t n, void* stream) {
    return deltalog_maint(dims, pool, n_slots, slots, n, stream, 1, "gdn_deltalog_materialize");
}

int gdn_conv1d_silu(const void* x, const float* w, const int32_t* cu_seqlens, int32_t n_seqs,
                    int32_t total_tokens, int32_t channels, int32_t width, int32_t planes,
                    int32_t dtype, void* y, void* stream) {
    if (n_seqs < 0 || total_tokens < 0 || channels < 1)
        return fail(GDN_ERR_SHAPE, "bad sizes (n_seqs %d, total_tokens %d, channels %d)", n_seqs,
                    total_tokens, channels);
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype must be 0 or 1 (got %d)", dtype);
    if (width < 2 || width > 4)
        return fail(GDN_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %d)", width);
    if (planes < 1 || channels % (8 * planes) != 0)
        return fail(GDN_ERR_SHAPE, "channels (%d) must be a multiple of 8 * planes (%d)", channels,
                    planes);
    if (n_seqs == 0 || total_tokens == 0) return ok();
    REQUIRE_PTR(x);
    REQUIRE_PTR(w);
    REQUIRE_PTR(cu_seqlens);
    REQUIRE_PTR(y);
    gdn::ConvArgs a;
    a.dtype = dtype;
    a.channels = channels;
    a.width = width;
    a.planes = planes;
    a.n_seqs = n_seqs;
    a.total_tokens = total_tokens;
    a.x = x;
    a.w = w;
    a.cu_seqlens = cu_seqlens;
    a.y = y;
    return launch_status(gdn::launch_conv1d(a, static_cast<hipStream_t>(stream)),
                         "gdn_conv1d_silu");
}

// ---------------------------------------------------------------- paged softmax attention

int gdn_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int32_t n,
                   int32_t block_size, int32_t* block_table, int32_t max_blocks,
                   const int32_t* free_blocks, int32_t n_free, int32_t max_tokens,
                   int32_t* cu_seqlens, int32_t* seq_lens, int64_t* slot_map,
                   int32_t* positions, int32_t* counts, void* stream) {
    if (n < 0 || max_blocks < 0 || n_free < 0 || max_tokens < 0)
        return fail(GDN_ERR_SHAPE, "n, max_blocks, n_free and max_tokens must be >= 0 (got %d, "
                                   "%d, %d, %d)", n, max_blocks, n_free, max_tokens);
    if (block_size < 1) return fail(GDN_ERR_SHAPE, "block_size must be >= 1 (got %d)", block_size);
    if (n > 0) {
        REQUIRE_PTR(ctx_lens);
        REQUIRE_PTR(new_lens);
        REQUIRE_PTR(seq_lens);
        if (max_blocks > 0) REQUIRE_PTR(block_table);
        if (seq_lens == ctx_lens || seq_lens == new_lens)
            return fail(GDN_ERR_SHAPE, "seq_lens must not be ctx_lens or new_lens");
    }
    if (n_free > 0) REQUIRE_LIST(free_blocks);
    REQUIRE_PTR(cu_seqlens);
    REQUIRE_PTR(counts);
    if (max_tokens > 0) {
        REQUIRE_PTR(slot_map);
        REQUIRE_PTR(positions);
    }
    gdn::PlanArgs a;
    a.ctx_lens = ctx_lens;
    a.new_lens = new_lens;
    a.n = n;
    a.block_size = block_size;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.free_blocks = free_blocks;
    a.n_free = n_free;
    a.max_tokens = max_tokens;
    a.cu_seqlens = cu_seqlens;
    a.seq_lens = seq_lens;
    a.slot_map = slot_map;
    a.positions = positions;
    a.counts = counts;
    return launch_status(gdn::launch_paged_plan(a, static_cast<hipStream_t>(stream)),
                         "gdn_paged_plan");
}

int gdn_paged_append(int32_t dtype, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, const int64_t* slot_map, int32_t tokens,
                     int32_t kv_heads, int32_t d, void* k_cache, void* v_cache,
                     int32_t n_blocks, int32_t block_size, void* stream) {
    const char* what = "gdn_paged_append";
    int st = check_cache(dtype, kv_heads, n_blocks, block_size);
    if (st) return st;
    if (!paged_dim_ok(d)) return fail(GDN_ERR_UNSUPPORTED, "d must be 64, 128 or 256 (got %d)", d);
    st = check_rows(dtype, tokens, k_stride, (int64_t)kv_heads * d, "k");
    if (!st) st = check_rows(dtype, tokens, v_stride, (int64_t)kv_heads * d, "v");
    if (st || tokens == 0) return st ? st : ok();
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_LIST(slot_map);
    REQUIRE_PTR(k_cache);
    REQUIRE_PTR(v_cache);
    const int per = dtype == GDN_DTYPE_BF16 ? 8 : 4;
    gdn::AppendArgs a;
    a.a = k;
    a.b = v;
    a.a_stride = k_stride / per;
    a.b_stride = v_stride / per;
    a.slot_map = slot_map;
    a.tokens = tokens;
    a.heads = kv_heads;
    a.a_row = d / per;
    a.b_row = d / per;
    a.a_cache = k_cache;
    a.b_cache = v_cache;
    a.n_blocks = n_blocks;
    a.block_size = block_size;
    DEBUG_DISTINCT_CACHE_SLOTS(slot_map, tokens, (int64_t)n_blocks * block_size, what);
    return launch_status(gdn::launch_append(a, static_cast<hipStream_t>(stream)), what);
}

int gdn_latent_append(int32_t dtype, const void* c, int64_t c_stride, const void* k_pe,
                      int64_t pe_stride, const int64_t* slot_map, int32_t tokens, int32_t rank,
                      int32_t d_rope, void* cache, int32_t n_blocks, int32_t block_size,
                      void* stream) {
    const char* what = "gdn_latent_append";
    int st = check_cache(dtype, 1, n_blocks, block_size);
    if (st) return st;
    if (rank < 8 || rank % 8 != 0 || rank > 65536 || d_rope < 8 || d_rope % 8 != 0 ||
        d_rope > 65536)
        return fail(GDN_ERR_UNSUPPORTED, "rank and d_rope must be multiples of 8 in [8, 65536] "
                                         "(got %d, %d)", rank, d_rope);
    st = check_rows(dtype, tokens, c_stride, rank, "c");
    if (!st) st = check_rows(dtype, tokens, pe_stride, d_rope, "k_pe");
    if (st || tokens == 0) return st ? st : ok();
    REQUIRE_PTR(c);
    REQUIRE_PTR(k_pe);
    REQUIRE_LIST(slot_map);
    REQUIRE_PTR(cache);
    const int per = dtype == GDN_DTYPE_BF16 ? 8 : 4;
    gdn::AppendArgs a;
    a.a = c;
    a.b = k_pe;
    a.a_stride = c_stride / per;
    a.b_stride = pe_stride / per;
    a.slot_map = slot_map;
    a.tokens = tokens;
    a.heads = 1;
    a.a_row = rank / per;
    a.b_row = d_rope / per;
    a.a_cache = cache;
    a.b_cache = nullptr;
    a.n_blocks = n_blocks;
    a.block_size = block_size;
    DEBUG_DISTINCT_CACHE_SLOTS(slot_map, tokens, (int64_t)n_blocks * block_size, what);
    return launch_status(gdn::launch_append(a, static_cast<hipStream_t>(stream)), what);
}

int gdn_paged_decode_workspace_bytes(const gdn_paged_dims_t* dims, int32_t batch, int32_t n_pos,
                                     size_t* bytes) {
    int st = check_paged_dims(dims, batch, n_pos);
    if (st) return st;
    if (bytes == nullptr) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn::PagedDecodeArgs a = paged_args(dims, batch, n_pos);
    *bytes = batch == 0 ? 0 : gdn::paged_decode_layout(&a, nullptr);
    return ok();
}

int gdn_paged_decode(const gdn_paged_dims_t* dims, const void* q, const void* k_cache,
                     const void* v_cache, int32_t n_blocks, int32_t block_size,
                     const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                     int32_t batch, int32_t n_pos, void* o, void* workspace, size_t ws_bytes,
                     void* stream) {
    int st = check_paged_dims(dims, batch, n_pos);
    if (!st) st = check_cache(dims->dtype, dims->num_kv_heads, n_blocks, block_size);
    if (!st) st = check_table(max_blocks, block_size);
    if (!st) st = check_chunks(batch, dims->num_kv_heads, max_blocks, block_size);
    if (st) return st;
    if (batch == 0) return ok();
    REQUIRE_PTR(q);
    REQUIRE_PTR(k_cache);
    REQUIRE_PTR(v_cache);
    REQUIRE_PTR(block_table);
    REQUIRE_PTR(seq_lens);
    REQUIRE_PTR(o);
    REQUIRE_PTR(workspace);
    gdn::PagedDecodeArgs a = paged_args(dims, batch, n_pos);
    const size_t need = gdn::paged_decode_layout(&a, workspace);
    if (ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.n_blocks = n_blocks;
    a.block = gdn::FastDiv::of((uint32_t)block_size);
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.split.seq_lens = seq_lens;
    a.split.max_keys = max_blocks * block_size;
    a.o = o;
    return launch_status(gdn::launch_paged_decode(a, static_cast<hipStream_t>(stream)),
                         "gdn_paged_decode");
}

int gdn_latent_decode_workspace_bytes(const gdn_latent_dims_t* dims, int32_t batch,
                                      int32_t n_pos, size_t* bytes) {
    int st = check_latent_dims(dims);
    if (!st) st = check_latent_batch(dims, batch, n_pos);
    if (st) return st;
    if (bytes == nullptr) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn::LatentDecodeArgs a = latent_decode_args(dims, batch, n_pos);
    *bytes = batch == 0 ? 0 : gdn::latent_decode_layout(&a, nullptr);
    return ok();
}

int gdn_latent_decode(const gdn_latent_dims_t* dims, const void* q_nope, const void* q_pe,
                      const void* w_kv, const void* cache, int32_t n_blocks, int32_t block_size,
                      const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                      int32_t batch, int32_t n_pos, void* o, void* workspace, size_t ws_bytes,
                      void* stream) {
    int st = check_latent_dims(dims);
    if (!st) st = check_latent_batch(dims, batch, n_pos);
    if (!st) st = check_cache(dims->dtype, 1, n_blocks, block_size);
    if (!st) st = check_table(max_blocks, block_size);
    if (!st) st = check_chunks(batch, 1, max_blocks, block_size);
    if (st) return st;
    if (batch == 0) return ok();
    REQUIRE_PTR(q_nope);
    REQUIRE_PTR(q_pe);
    REQUIRE_PTR(w_kv);
    REQUIRE_PTR(cache);
    REQUIRE_PTR(block_table);
    REQUIRE_PTR(seq_lens);
    REQUIRE_PTR(o);
    REQUIRE_PTR(workspace);
    gdn::LatentDecodeArgs a = latent_decode_args(dims, batch, n_pos);
    const size_t need = gdn::latent_decode_layout(&a, workspace);
    if (ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    a.q_nope = q_nope;
    a.q_pe = q_pe;
    a.w_kv = w_kv;
    a.cache = cache;
    a.n_blocks = n_blocks;
    a.block = gdn::FastDiv::of((uint32_t)block_size);
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.split.seq_lens = seq_lens;
    a.split.max_keys = max_blocks * block_size;
    a.o = o;
    return launch_status(gdn::launch_latent_decode(a, static_cast<hipStream_t>(stream)),
                         "gdn_latent_decode");
}

int gdn_latent_prefill_workspace_bytes(const gdn_latent_dims_t* dims, int32_t n_seqs,
                                       int32_t total_tokens, int64_t total_keys, size_t* bytes) {
    int st = check_latent_prefill(dims, n_seqs, total_tokens, total_keys);
    if (st) return st;
    if (bytes == nullptr) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn::LatentPrefillArgs a = latent_prefill_args(dims, n_seqs, total_tokens);
    *bytes = n_seqs == 0 || total_tokens == 0
                 ? 0 : gdn::latent_prefill_layout(&a, total_keys, nullptr);
    return ok();
}

int gdn_latent_prefill(const gdn_latent_dims_t* dims, const void* q_nope, const void* q_pe,
                       const void* w_kv, const void* cache, int32_t n_blocks, int32_t block_size,
                       const int32_t* block_table, int32_t max_blocks, const int32_t* cu_seqlens,
                       const int32_t* seq_lens, int32_t n_seqs, int32_t total_tokens,
                       int64_t total_keys, void* o, void* workspace, size_t ws_bytes,
                       void* stream) {
    int st = check_latent_prefill(dims, n_seqs, total_tokens, total_keys);
    if (!st) st = check_cache(dims->dtype, 1, n_blocks, block_size);
    if (!st) st = check_table(max_blocks, block_size);
    if (st) return st;
    if (n_seqs == 0 || total_tokens == 0) return ok();
    REQUIRE_PTR(q_nope);
    REQUIRE_PTR(q_pe);
    REQUIRE_PTR(w_kv);
    REQUIRE_PTR(cache);
    REQUIRE_PTR(block_table);
    REQUIRE_PTR(cu_seqlens);
    REQUIRE_PTR(seq_lens);
    REQUIRE_PTR(o);
    REQUIRE_PTR(workspace);
    gdn::LatentPrefillArgs a = latent_prefill_args(dims, n_seqs, total_tokens);
    const size_t need = gdn::latent_prefill_layout(&a, total_keys, workspace);
    if (ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    a.q_nope = q_nope;
    a.q_pe = q_pe;
    a.w_kv = w_kv;
    a.cache = cache;
    a.n_blocks = n_blocks;
    a.block = gdn::FastDiv::of((uint32_t)block_size);
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.max_keys = max_blocks * block_size;
    a.cu_seqlens = cu_seqlens;
    a.seq_lens = seq_lens;
    a.o = o;
    return launch_status(gdn::launch_latent_prefill(a, static_cast<hipStream_t>(stream)),
                         "gdn_latent_prefill");
}

const char* gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_NULL: return "null pointer";
        case GDN_ERR_SHAPE: return "bad shape";
        case GDN_ERR_UNSUPPORTED: return "unsupported configuration";
        case GDN_ERR_ALIGN: return "misaligned pointer";
        case GDN_ERR_WORKSPACE: return "workspace too small";
        case GDN_ERR_LAUNCH: return "launch failure";
    }
    return "unknown status";
}

const char* gdn_last_error(void) { return g_err; }

int gdn_abi_version(void) { return GDN_ABI_VERSION; }

}  // extern "C"
