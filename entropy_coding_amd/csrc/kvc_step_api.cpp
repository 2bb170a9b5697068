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
using kvc::pools_ok;
using kvc::positive;

// Rows of a projection; a stride between one row or one head is not looked at.
bool heads_ok(const void* d, int64_t row_stride, int64_t head_stride, int64_t rows, int64_t heads) {
    const auto stride_ok = [](int64_t s) { return s >= 0 && s <= kMaxScalars && s % 8 == 0; };
    return d && aligned(d, 16) && (rows < 2 || stride_ok(row_stride)) && (heads < 2 || stride_ok(head_stride));
}

kvc::HeadRows head_rows(const void* d, int64_t row_stride, int64_t head_stride, int64_t rows, int64_t heads) {
    return kvc::HeadRows{static_cast<const uint16_t*>(d), rows > 1 ? row_stride : 0, heads > 1 ? head_stride : 0};
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
    a.k_scale = p->k_scale;
    a.v_scale = p->v_scale;
    return kvc::launch_qkv(a, p->channels, p->kv_dtype == KVC_E4M3, p->neighbours != 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess ? KVC_OK : KVC_ERR_DEVICE;
}

}  // extern "C"
