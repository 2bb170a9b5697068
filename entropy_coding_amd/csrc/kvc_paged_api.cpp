// C ABI of the paged cache's calls (declared in include/kvc.h): argument
// checks, workspace layout, launches, and the outcome read back from a
// workspace.  Host code only.
#include "kvc.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "kvc_paged.hpp"

namespace {

constexpr int64_t kInt31 = int64_t(1) << 31;
constexpr int64_t kMaxScalars = int64_t(1) << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

int value_bytes(int32_t dtype) { return dtype == KVC_BF16 ? 2 : 1; }

// The pools of a descriptor against one layer's rows of `channels` values.
bool pools_ok(const kvc_paged_kv* g, int64_t layer, int32_t kv_dtype, int64_t channels) {
    if (!g || !g->d_pools || !aligned(g->d_pools, 8) || (kv_dtype != KVC_BF16 && kv_dtype != KVC_E4M3)) return false;
    if (g->heads < 1 || g->heads > 1 << 16 || g->num_pages < 1 || g->num_pages >= kInt31 || g->page_tokens < 1 ||
        g->reserved != 0 || g->n_pools < 2 || g->n_pools % 2 || layer < 0 || layer >= g->n_pools / 2)
        return false;
    if (channels < 64 || channels % 64 || channels > 1 << 16) return false;
    const uint64_t row = uint64_t(g->heads) * uint64_t(channels) * uint64_t(value_bytes(kv_dtype));
    if (row >= uint64_t(kInt31) || g->page_tokens >= (uint64_t(1) << 32) / row) return false;
    return g->pool_bytes / (row * g->page_tokens) >= uint64_t(g->num_pages);
}

int outcome(uint32_t flags) {
    if (flags & kvc::kPagedInvalid) return KVC_ERR_INVALID;
    return flags & kvc::kPagedCapacity ? KVC_ERR_CAPACITY : KVC_OK;
}

// Copies `bytes` of a workspace to the host behind everything on `stream`.
bool read_back(void* h, const void* d, uint64_t bytes, hipStream_t s) {
    return hipMemcpyAsync(h, d, bytes, hipMemcpyDeviceToHost, s) == hipSuccess && hipStreamSynchronize(s) == hipSuccess;
}

// ---- attention

// The scale of the scores in units of log 2.
float score_scale(const kvc_attention* p) {
    return static_cast<float>(double(p->softmax_scale) * double(p->k_scale) * 1.4426950408889634);
}

// The sizes of a call (all that kvc_paged_attention_sizes looks at).
bool attention_sizes_ok(const kvc_paged_kv* g, const kvc_attention* p) {
    if (!p || !pools_ok(g, 0, p->kv_dtype, p->channels)) return false;
    // (every workgroup reads all lengths: a batch has a bound)
    if (p->channels > 256 || g->batch < 1 || g->batch > 1 << 14 || g->max_pages < 1 || g->max_pages >= kInt31) return false;
    if (uint64_t(g->num_pages) * g->page_tokens >= uint64_t(kInt31)) return false;
    if (p->rows < 0 || p->rows >= 1 << 24 || p->rows_per_sequence < 0 || p->max_tokens < 0) return false;
    if (p->q_heads < 1 || p->q_heads % g->heads || p->q_heads / g->heads > 1024) return false;
    if (p->rows * p->q_heads >= kInt31) return false;
    if (kvc::attend_items(g->batch, g->heads, p->q_heads / g->heads, p->rows, 16) >= kvc::kMaxItems) return false;
    return std::isfinite(score_scale(p)) && positive(p->k_scale) && positive(p->v_scale);
}

bool attention_ok(const kvc_paged_kv* g, const kvc_attention* p) {
    if (!attention_sizes_ok(g, p) || !g->d_block_table || !aligned(g->d_block_table, 4)) return false;
    if (p->rows > 0 && (!p->d_q || !p->d_out || !aligned(p->d_q, 16) || !aligned(p->d_out, 16))) return false;
    // (strides between one row, or one head, say nothing)
    const auto stride_ok = [](int64_t stride, int64_t least) {
        return stride >= least && stride <= kMaxScalars && stride % 8 == 0;
    };
    if (p->rows > 1 && (!stride_ok(p->q_row_stride, 0) || !stride_ok(p->out_row_stride, p->q_heads * p->channels)))
        return false;
    if (p->q_heads > 1 && !stride_ok(p->q_head_stride, 0)) return false;
    if (!p->d_row_starts || !aligned(p->d_row_starts, 4) || !aligned(p->d_context_lens, 4) || !aligned(p->d_lse, 4) ||
        !aligned(p->d_tree_mask, 8))
        return false;
    return p->d_tree_mask ? p->mask_words >= 1 && p->mask_words <= 1 << 20 : p->mask_words == 0;
}

// The tokens that a row of the table has room for, at most kMaxTokens.
int64_t widest_of(const kvc_paged_kv* g) {
    const int64_t room = g->max_pages * int64_t(g->page_tokens);
    return room < kvc::kMaxTokens ? room : kvc::kMaxTokens;
}

kvc::AttendShape shape_of(const kvc_paged_kv* g, const kvc_attention* p) {
    const int64_t widest = widest_of(g);
    const int64_t longest = p->max_tokens > 0 && p->max_tokens < widest ? p->max_tokens : widest;
    const int64_t usual = p->rows_per_sequence < 1 << 24 ? p->rows_per_sequence : 1 << 24;    // (more than any has)
    return kvc::attend_shape(g->batch, g->heads, p->q_heads / g->heads, p->channels, p->kv_dtype == KVC_E4M3, p->rows,
                             usual, longest, widest);
}

}  // namespace

extern "C" {

int kvc_build_block_table(const kvc_block_table* p, void* d_workspace, uint64_t workspace_bytes, void* stream,
                          int64_t* h_rows) {
    if (!p || !d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    if (p->batch < 1 || p->batch >= kInt31 || p->max_pages < 1 || p->max_pages >= kInt31 ||
        p->batch * p->max_pages >= kInt31 || p->num_pages < 1 || p->num_pages >= kInt31 || p->free_capacity < 0 ||
        p->free_capacity >= kInt31 || p->max_rows < 0 || p->max_rows >= kInt31 || p->page_tokens < 1 || p->trim > 1)
        return KVC_ERR_INVALID;
    if (!p->d_held_in || !p->d_held_out || !p->d_block_table || !p->d_free_in || !p->d_free_out || !p->d_row_starts ||
        (!p->d_free_pages && p->free_capacity > 0))
        return KVC_ERR_INVALID;
    if (!aligned(p->d_cached_lens, 4) || !aligned(p->d_new_lens, 4) || !aligned(p->d_held_in, 4) ||
        !aligned(p->d_held_out, 4) || !aligned(p->d_block_table, 4) || !aligned(p->d_free_pages, 4) ||
        !aligned(p->d_free_in, 4) || !aligned(p->d_free_out, 4) || !aligned(p->d_row_starts, 4) ||
        !aligned(p->d_slots, 8) || !aligned(p->d_positions, 4))
        return KVC_ERR_INVALID;
    if (workspace_bytes < KVC_BLOCK_TABLE_WORKSPACE_BYTES(p->batch)) return KVC_ERR_CAPACITY;
    kvc::TableArgs a;
    a.batch = p->batch;
    a.max_pages = p->max_pages;
    a.num_pages = p->num_pages;
    a.free_capacity = p->free_capacity;
    a.max_rows = p->max_rows;
    a.page_tokens = p->page_tokens;
    a.trim = p->trim;
    a.cached = p->d_cached_lens;
    a.fresh = p->d_new_lens;
    a.held_in = p->d_held_in;
    a.held_out = p->d_held_out;
    a.table = p->d_block_table;
    a.free_pages = p->d_free_pages;
    a.free_in = p->d_free_in;
    a.free_out = p->d_free_out;
    a.row_starts = p->d_row_starts;
    a.slots = p->d_slots;
    a.positions = p->d_positions;
    a.ctl = static_cast<kvc::TableControl*>(d_workspace);
    a.arrays = reinterpret_cast<int32_t*>(static_cast<char*>(d_workspace) + kvc::kTableArraysOffset);
    if (kvc::launch_block_table(a, static_cast<hipStream_t>(stream)) != hipSuccess) return KVC_ERR_DEVICE;
    return h_rows ? kvc_block_table_result(d_workspace, stream, h_rows) : KVC_OK;
}

int kvc_block_table_result(const void* d_workspace, void* stream, int64_t* h_rows) {
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    kvc::TableControl c;
    if (!read_back(&c, d_workspace, sizeof(c), static_cast<hipStream_t>(stream))) return KVC_ERR_DEVICE;
    if (c.magic != kvc::kPagedMagic) return KVC_ERR_INVALID;
    if (h_rows) *h_rows = c.rows;
    return outcome(c.flags);
}

int kvc_paged_append(const kvc_paged_kv* h_paged, int64_t layer, int32_t kv_dtype, int64_t channels, const void* d_k,
                     const void* d_v, int32_t src_dtype, int64_t rows, int64_t k_row_stride, int64_t v_row_stride,
                     const int64_t* d_slots, float k_scale, float v_scale, void* stream) {
    if (!pools_ok(h_paged, layer, kv_dtype, channels)) return KVC_ERR_INVALID;
    if (src_dtype != kv_dtype && (src_dtype != KVC_BF16 || kv_dtype != KVC_E4M3)) return KVC_ERR_INVALID;
    if (!positive(k_scale) || !positive(v_scale)) return KVC_ERR_INVALID;
    if (src_dtype == kv_dtype && (k_scale != 1.0f || v_scale != 1.0f)) return KVC_ERR_INVALID;
    if (rows < 0 || rows >= kInt31) return KVC_ERR_INVALID;
    if (rows == 0) return KVC_OK;
    const int size = value_bytes(src_dtype);
    const int64_t width = h_paged->heads * channels;
    if (!d_k || !d_v || !d_slots || !aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_slots, 8)) return KVC_ERR_INVALID;
    for (int64_t stride : {k_row_stride, v_row_stride})
        if (rows > 1 && (stride < width || stride > kMaxScalars || (stride * size) % 16)) return KVC_ERR_INVALID;
    kvc::AppendArgs a;
    a.pools = h_paged->d_pools + 2 * layer;
    a.k = d_k;
    a.v = d_v;
    a.slots = d_slots;
    a.rows = rows;
    a.n_slots = h_paged->num_pages * int64_t(h_paged->page_tokens);
    a.k_stride = rows > 1 ? k_row_stride * size : 0;
    a.v_stride = rows > 1 ? v_row_stride * size : 0;
    a.row_bytes = static_cast<uint32_t>(width * value_bytes(kv_dtype));
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return kvc::launch_append(a, src_dtype != kv_dtype, static_cast<hipStream_t>(stream)) == hipSuccess
               ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_paged_attention_sizes(const kvc_paged_kv* h_paged, const kvc_attention* p, uint64_t* h_workspace_bytes) {
    if (!h_workspace_bytes || !attention_sizes_ok(h_paged, p)) return KVC_ERR_INVALID;
    *h_workspace_bytes = shape_of(h_paged, p).total;
    return KVC_OK;
}

int kvc_paged_attention(const kvc_paged_kv* h_paged, int64_t layer, const kvc_attention* p, void* d_workspace,
                        uint64_t workspace_bytes, void* stream) {
    if (!attention_ok(h_paged, p) || layer < 0 || layer >= h_paged->n_pools / 2) return KVC_ERR_INVALID;
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    const kvc::AttendShape shape = shape_of(h_paged, p);
    if (workspace_bytes < shape.total) return KVC_ERR_CAPACITY;
    char* const ws = static_cast<char*>(d_workspace);
    kvc::AttendArgs a;
    a.pools = h_paged->d_pools + 2 * layer;
    a.block_table = h_paged->d_block_table;
    a.max_pages = h_paged->max_pages;
    a.num_pages = h_paged->num_pages;
    a.max_tokens = static_cast<int32_t>(widest_of(h_paged));
    a.tile_shift = shape.tile_shift;
    a.unit_shift = shape.unit_shift;
    a.page_tokens = h_paged->page_tokens;
    a.heads = static_cast<uint32_t>(h_paged->heads);
    a.batch = static_cast<uint32_t>(h_paged->batch);
    a.ratio = static_cast<uint32_t>(p->q_heads / h_paged->heads);
    a.q = static_cast<const uint16_t*>(p->d_q);
    a.q_row = p->rows > 1 ? p->q_row_stride : 0;
    a.q_head = p->q_heads > 1 ? p->q_head_stride : 0;
    a.out = static_cast<uint16_t*>(p->d_out);
    a.out_row = p->rows > 1 ? p->out_row_stride : 0;
    a.lse = p->d_lse;
    a.row_starts = p->d_row_starts;
    a.context = p->d_context_lens;
    a.mask = p->d_tree_mask;
    a.mask_words = static_cast<uint32_t>(p->mask_words);
    a.rows = static_cast<uint32_t>(p->rows);
    a.scale_log2 = score_scale(p);
    a.v_scale = p->v_scale;
    a.target = shape.grid;
    a.split = shape.split;
    a.ctl = static_cast<kvc::AttendControl*>(d_workspace);
    a.spans = reinterpret_cast<kvc::AttendSpan*>(ws + shape.spans);
    a.words = reinterpret_cast<uint32_t*>(ws + shape.words);
    a.partial = reinterpret_cast<float*>(ws + shape.partial);
    a.pairs = reinterpret_cast<float*>(ws + shape.pairs);
    return kvc::launch_attend(a, shape, p->channels, p->kv_dtype == KVC_E4M3, static_cast<hipStream_t>(stream)) ==
                   hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_paged_attention_result(const void* d_workspace, void* stream) {
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    kvc::AttendControl c;
    if (!read_back(&c, d_workspace, sizeof(c), s)) return KVC_ERR_DEVICE;
    if (c.magic != kvc::kPagedMagic) return KVC_ERR_INVALID;
    uint32_t flags = c.flags;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(static_cast<const char*>(d_workspace) + c.words_offset);
    uint32_t part[1024];
    for (uint32_t at = 0; at < c.grid; at += 1024) {
        const uint32_t n = c.grid - at < 1024 ? c.grid - at : 1024;
        if (!read_back(part, words + at, 4ull * n, s)) return KVC_ERR_DEVICE;
        for (uint32_t i = 0; i < n; ++i) flags |= part[i];
    }
    return outcome(flags);
}

}  // extern "C"
