// C ABI of the calls that a speculative step makes around the attention over
// pages (declared in include/kvc.h): argument checks, workspace layout,
// launches, and the outcome read back from a workspace.  Host code only.
#include "kvc.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "kvc_checks.hpp"
#include "kvc_step.hpp"

namespace {

using kvc::aligned;
using kvc::kInt31;
using kvc::kMaxScalars;
using kvc::outcome;
using kvc::pools_ok;
using kvc::positive;
using kvc::read_back;

// The flags that a call left for its sequences, `words` of them.
int outcome_of_words(const void* d_words, uint64_t words, hipStream_t s) {
    uint32_t flags = 0, part[1024];
    for (uint64_t at = 0; at < words; at += 1024) {
        const uint64_t n = words - at < 1024 ? words - at : 1024;
        if (!read_back(part, static_cast<const uint32_t*>(d_words) + at, 4 * n, s)) return KVC_ERR_DEVICE;
        for (uint64_t i = 0; i < n; ++i) flags |= part[i];
    }
    return outcome(flags);
}

// Rows of a projection; a stride between one row or one head is not looked at.
bool heads_ok(const void* d, int64_t row_stride, int64_t head_stride, int64_t rows, int64_t heads) {
    const auto stride_ok = [](int64_t s) { return s >= 0 && s <= kMaxScalars && s % 8 == 0; };
    return d && aligned(d, 16) && (rows < 2 || stride_ok(row_stride)) && (heads < 2 || stride_ok(head_stride));
}

kvc::HeadRows head_rows(const void* d, int64_t row_stride, int64_t head_stride, int64_t rows, int64_t heads) {
    return kvc::HeadRows{static_cast<const uint16_t*>(d), rows > 1 ? row_stride : 0, heads > 1 ? head_stride : 0};
}

bool verify_sizes_ok(const kvc_drafts* p) {
    if (!p || p->batch < 1 || p->batch > 1 << 20 || p->rows < 0 || p->rows >= kInt31) return false;
    if (p->vocab < 1 || p->vocab > kvc::kMaxVocab) return false;
    return p->batch * ((p->vocab + kvc::kVerifyChunk - 1) / kvc::kVerifyChunk) < 1 << 24;   // workgroups of a launch
}

// The pools and the table of a descriptor, for calls that go through all of
// them.
bool pages_ok(const kvc_paged_kv* g, int32_t kv_dtype, int64_t channels) {
    return pools_ok(g, 0, kv_dtype, channels) && g->n_pools <= 1 << 20 && g->batch >= 1 && g->batch < kInt31 &&
           g->max_pages >= 1 && g->max_pages < kInt31;
}

kvc::PagesOf pages_of(const kvc_paged_kv* g, int32_t kv_dtype, int64_t channels) {
    kvc::PagesOf p;
    p.pools = g->d_pools;
    p.n_pools = g->n_pools;
    p.batch = g->batch;
    p.max_pages = g->max_pages;
    p.num_pages = g->num_pages;
    p.page_tokens = g->page_tokens;
    p.pieces = static_cast<uint32_t>(g->heads * channels * kvc::value_bytes(kv_dtype) / 16);
    return p;
}

bool shared_ok(const kvc_paged_kv* g, int32_t kv_dtype, int64_t channels, const kvc_shared_pages* p, int64_t count) {
    if (!p || !pages_ok(g, kv_dtype, channels) || count < 0 || count > kvc::kMaxShared) return false;
    if (p->free_capacity < g->num_pages || p->free_capacity >= kInt31) return false;
    for (const void* d : {static_cast<const void*>(p->d_block_table), static_cast<const void*>(p->d_held_in),
                          static_cast<const void*>(p->d_held_out), static_cast<const void*>(p->d_free_pages),
                          static_cast<const void*>(p->d_free_in), static_cast<const void*>(p->d_free_out),
                          static_cast<const void*>(p->d_extra)})
        if (!d || !aligned(d, 4)) return false;
    return true;
}

kvc::SharedArgs shared_args(const kvc_paged_kv* g, int32_t kv_dtype, int64_t channels, const kvc_shared_pages* p,
                            int64_t count, void* d_workspace) {
    char* const ws = static_cast<char*>(d_workspace);
    kvc::SharedArgs a;
    a.g = pages_of(g, kv_dtype, channels);
    a.table = p->d_block_table;
    a.free_capacity = p->free_capacity;
    a.held_in = p->d_held_in;
    a.held_out = p->d_held_out;
    a.free_pages = p->d_free_pages;
    a.free_in = p->d_free_in;
    a.free_out = p->d_free_out;
    a.extra = p->d_extra;
    a.count = static_cast<int32_t>(count);
    a.parents = nullptr;
    a.children = nullptr;
    a.context = nullptr;
    a.ctl = static_cast<kvc::SharedControl*>(d_workspace);
    a.arrivals = reinterpret_cast<uint32_t*>(ws + 256);
    a.bits = reinterpret_cast<uint32_t*>(ws + kvc::kSharedBits);
    return a;
}

}  // namespace

extern "C" {

int kvc_paged_qkv(const kvc_paged_kv* h_paged, int64_t layer, const kvc_qkv* p, void* stream) {
    if (!p || !pools_ok(h_paged, layer, p->kv_dtype, p->channels) || p->channels > 256) return KVC_ERR_INVALID;
    if (p->rows < 0 || p->rows >= kInt31 || p->q_heads < 0 || p->q_heads > 1 << 16 || p->neighbours > 1)
        return KVC_ERR_INVALID;
    if (p->rotary < 0 || p->rotary > p->channels || p->rotary % 16) return KVC_ERR_INVALID;
    if (!positive(p->k_scale) || !positive(p->v_scale)) return KVC_ERR_INVALID;
    if (p->kv_dtype == KVC_BF16 && (p->k_scale != 1.0f || p->v_scale != 1.0f)) return KVC_ERR_INVALID;
    if (p->norm_dtype != KVC_BF16 && p->norm_dtype != KVC_F32) return KVC_ERR_INVALID;
    if (!aligned(p->d_q_norm, 16) || !aligned(p->d_k_norm, 16)) return KVC_ERR_INVALID;
    if ((p->d_q_norm || p->d_k_norm) && !(std::isfinite(p->eps) && p->eps >= 1e-30f)) return KVC_ERR_INVALID;
    if (p->rotary > 0 && !p->d_frequencies) return KVC_ERR_INVALID;
    if (!aligned(p->d_frequencies, 8) || !aligned(p->d_positions, 4)) return KVC_ERR_INVALID;
    if (p->rows == 0) return KVC_OK;
    if (p->rotary > 0 && !p->d_positions) return KVC_ERR_INVALID;
    const int64_t heads = h_paged->heads;
    if (p->q_heads > 0 && !heads_ok(p->d_q, p->q_row_stride, p->q_head_stride, p->rows, p->q_heads)) return KVC_ERR_INVALID;
    if (!heads_ok(p->d_k, p->k_row_stride, p->k_head_stride, p->rows, heads) ||
        !heads_ok(p->d_v, p->v_row_stride, p->v_head_stride, p->rows, heads))
        return KVC_ERR_INVALID;
    if (!p->d_slots || !aligned(p->d_slots, 8)) return KVC_ERR_INVALID;
    if (p->q_heads > 0 && (!p->d_q_out || !aligned(p->d_q_out, 16))) return KVC_ERR_INVALID;
    if (p->q_heads > 0 && p->rows > 1 &&
        (p->q_out_row_stride < p->q_heads * p->channels || p->q_out_row_stride > kMaxScalars || p->q_out_row_stride % 8))
        return KVC_ERR_INVALID;
    kvc::QkvArgs a;
    a.pools = h_paged->d_pools + 2 * layer;
    a.q = head_rows(p->d_q, p->q_row_stride, p->q_head_stride, p->rows, p->q_heads);
    a.k = head_rows(p->d_k, p->k_row_stride, p->k_head_stride, p->rows, heads);
    a.v = head_rows(p->d_v, p->v_row_stride, p->v_head_stride, p->rows, heads);
    a.out = static_cast<uint16_t*>(p->d_q_out);
    a.out_row = p->rows > 1 ? p->q_out_row_stride : 0;
    a.q_norm = p->d_q_norm;
    a.k_norm = p->d_k_norm;
    a.frequencies = p->d_frequencies;
    a.positions = p->d_positions;
    a.slots = p->d_slots;
    a.rows = p->rows;
    a.n_slots = h_paged->num_pages * int64_t(h_paged->page_tokens);
    a.q_heads = static_cast<uint32_t>(p->q_heads);
    a.heads = static_cast<uint32_t>(heads);
    a.rotary = static_cast<uint32_t>(p->rotary);
    a.norm_f32 = p->norm_dtype == KVC_F32;
    a.parts = 1;
    a.eps = p->eps;
    a.per_k_scale = 1.0 / double(p->k_scale);
    a.per_v_scale = 1.0 / double(p->v_scale);
    return kvc::launch_qkv(a, p->channels, p->kv_dtype == KVC_E4M3, p->neighbours != 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_verify_drafts_sizes(const kvc_drafts* p, uint64_t* h_workspace_bytes) {
    if (!h_workspace_bytes || !verify_sizes_ok(p)) return KVC_ERR_INVALID;
    *h_workspace_bytes = kvc::verify_layout(p->batch, p->vocab).total;
    return KVC_OK;
}

int kvc_verify_drafts(const kvc_drafts* p, void* d_workspace, uint64_t workspace_bytes, void* stream) {
    if (!verify_sizes_ok(p) || !d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    const auto stride_ok = [p](int64_t s) { return p->rows < 2 || (s >= p->vocab && s <= kMaxScalars); };
    if (!p->d_row_starts || !p->d_kept_lens || !p->d_sample) return KVC_ERR_INVALID;
    if (p->rows > 0 && (!p->d_tokens || !p->d_target || !p->d_accept || !p->d_kept || !p->d_out_tokens)) return KVC_ERR_INVALID;
    for (const void* d : {static_cast<const void*>(p->d_row_starts), static_cast<const void*>(p->d_tokens),
                          static_cast<const void*>(p->d_parents), static_cast<const void*>(p->d_target),
                          static_cast<const void*>(p->d_draft), static_cast<const void*>(p->d_accept),
                          static_cast<const void*>(p->d_sample), static_cast<const void*>(p->d_kept),
                          static_cast<const void*>(p->d_kept_lens), static_cast<const void*>(p->d_out_tokens)})
        if (!aligned(d, 4)) return KVC_ERR_INVALID;
    if (!stride_ok(p->target_row_stride) || (p->d_draft && !stride_ok(p->draft_row_stride))) return KVC_ERR_INVALID;
    const kvc::VerifyLayout l = kvc::verify_layout(p->batch, p->vocab);
    if (workspace_bytes < l.total) return KVC_ERR_CAPACITY;
    char* const ws = static_cast<char*>(d_workspace);
    kvc::VerifyArgs a;
    a.batch = p->batch;
    a.rows = p->rows;
    a.vocab = static_cast<uint32_t>(p->vocab);
    a.chunks = l.chunks;
    a.row_starts = p->d_row_starts;
    a.tokens = p->d_tokens;
    a.parents = p->d_parents;
    a.target = p->d_target;
    a.draft = p->d_draft;
    a.target_row = p->target_row_stride;
    a.draft_row = p->draft_row_stride;
    a.accept = p->d_accept;
    a.sample = p->d_sample;
    a.kept = p->d_kept;
    a.kept_lens = p->d_kept_lens;
    a.out_tokens = p->d_out_tokens;
    a.ctl = static_cast<kvc::VerifyControl*>(d_workspace);
    a.words = reinterpret_cast<uint32_t*>(ws + l.words);
    a.arrived = reinterpret_cast<uint32_t*>(ws + l.arrived);
    a.sums = reinterpret_cast<kvc::VerifySums*>(ws + l.sums);
    a.first_nodes = reinterpret_cast<int32_t*>(ws + l.first_nodes);
    a.first_sums = reinterpret_cast<uint64_t*>(ws + l.first_sums);
    a.first_parts = 0;
    return kvc::launch_verify(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_verify_drafts_result(const void* d_workspace, void* stream) {
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    kvc::VerifyControl c;
    if (!read_back(&c, d_workspace, sizeof(c), s)) return KVC_ERR_DEVICE;
    if (c.magic != kvc::kVerifyMagic) return KVC_ERR_INVALID;
    return outcome_of_words(static_cast<const char*>(d_workspace) + 256, 2 * uint64_t(c.batch), s);
}

int kvc_paged_compact(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels, int64_t rows,
                      const int32_t* d_row_starts, const int32_t* d_context_lens, const int32_t* d_kept,
                      const int32_t* d_kept_lens, void* d_workspace, uint64_t workspace_bytes, void* stream) {
    if (!pages_ok(h_paged, kv_dtype, channels) || h_paged->batch > 1 << 20 || rows < 0 || rows >= kInt31) return KVC_ERR_INVALID;
    if (!d_workspace || !aligned(d_workspace, 256) || !h_paged->d_block_table || !aligned(h_paged->d_block_table, 4))
        return KVC_ERR_INVALID;
    if (!d_row_starts || !d_kept_lens || (rows > 0 && !d_kept) || !aligned(d_row_starts, 4) || !aligned(d_context_lens, 4) ||
        !aligned(d_kept, 4) || !aligned(d_kept_lens, 4))
        return KVC_ERR_INVALID;
    if (workspace_bytes < KVC_COMPACT_WORKSPACE_BYTES(h_paged->batch)) return KVC_ERR_CAPACITY;
    kvc::CompactArgs a;
    a.g = pages_of(h_paged, kv_dtype, channels);
    a.table = h_paged->d_block_table;
    a.rows = rows;
    a.row_starts = d_row_starts;
    a.context = d_context_lens;
    a.kept = d_kept;
    a.kept_lens = d_kept_lens;
    a.ctl = static_cast<kvc::CompactControl*>(d_workspace);
    a.words = reinterpret_cast<uint32_t*>(static_cast<char*>(d_workspace) + 256);
    return kvc::launch_compact(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_paged_compact_result(const void* d_workspace, void* stream) {
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    kvc::CompactControl c;
    if (!read_back(&c, d_workspace, sizeof(c), s)) return KVC_ERR_DEVICE;
    if (c.magic != kvc::kCompactMagic) return KVC_ERR_INVALID;
    return outcome_of_words(static_cast<const char*>(d_workspace) + 256, c.batch, s);
}

int kvc_fork_pages(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels, const kvc_shared_pages* p, int64_t count,
                   const int32_t* d_parents, const int32_t* d_children, const int32_t* d_context_lens, void* d_workspace,
                   uint64_t workspace_bytes, void* stream) {
    if (!shared_ok(h_paged, kv_dtype, channels, p, count) || !d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    if ((count > 0 && (!d_parents || !d_children)) || !aligned(d_parents, 4) || !aligned(d_children, 4) ||
        !aligned(d_context_lens, 4))
        return KVC_ERR_INVALID;
    if (workspace_bytes < KVC_SHARED_PAGES_WORKSPACE_BYTES(h_paged->num_pages)) return KVC_ERR_CAPACITY;
    kvc::SharedArgs a = shared_args(h_paged, kv_dtype, channels, p, count, d_workspace);
    a.parents = d_parents;
    a.children = d_children;
    a.context = d_context_lens;
    return kvc::launch_fork(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_release_pages(const kvc_paged_kv* h_paged, int32_t kv_dtype, int64_t channels, const kvc_shared_pages* p,
                      int64_t count, const int32_t* d_requests, void* d_workspace, uint64_t workspace_bytes, void* stream) {
    if (!shared_ok(h_paged, kv_dtype, channels, p, count) || !d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    if ((count > 0 && !d_requests) || !aligned(d_requests, 4)) return KVC_ERR_INVALID;
    if (workspace_bytes < KVC_SHARED_PAGES_WORKSPACE_BYTES(h_paged->num_pages)) return KVC_ERR_CAPACITY;
    kvc::SharedArgs a = shared_args(h_paged, kv_dtype, channels, p, count, d_workspace);
    a.children = d_requests;
    return kvc::launch_release(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

int kvc_shared_pages_result(const void* d_workspace, void* stream) {
    if (!d_workspace || !aligned(d_workspace, 256)) return KVC_ERR_INVALID;
    kvc::SharedControl c;
    if (!read_back(&c, d_workspace, sizeof(c), static_cast<hipStream_t>(stream))) return KVC_ERR_DEVICE;
    return c.magic == kvc::kSharedMagic ? outcome(c.flags) : KVC_ERR_INVALID;
}

}  // extern "C"
