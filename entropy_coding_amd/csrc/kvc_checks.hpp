// Argument checks and outcomes that the C ABI's calls on pages share.  Host
// code only.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "kvc.h"
#include "kvc_paged.hpp"

namespace kvc {

constexpr int64_t kInt31 = int64_t(1) << 31;
constexpr int64_t kMaxScalars = int64_t(1) << 40;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

inline int value_bytes(int32_t dtype) { return dtype == KVC_BF16 ? 2 : 1; }

// The pools of a descriptor against one layer's rows of `channels` values.
inline bool pools_ok(const kvc_paged_kv* g, int64_t layer, int32_t kv_dtype, int64_t channels) {
    if (!g || !g->d_pools || !aligned(g->d_pools, 8) || (kv_dtype != KVC_BF16 && kv_dtype != KVC_E4M3)) return false;
    if (g->heads < 1 || g->heads > 1 << 16 || g->num_pages < 1 || g->num_pages >= kInt31 || g->page_tokens < 1 ||
        g->reserved != 0 || g->n_pools < 2 || g->n_pools % 2 || layer < 0 || layer >= g->n_pools / 2)
        return false;
    if (channels < 64 || channels % 64 || channels > 1 << 16) return false;
    const uint64_t row = uint64_t(g->heads) * uint64_t(channels) * uint64_t(value_bytes(kv_dtype));
    if (row >= uint64_t(kInt31) || g->page_tokens >= (uint64_t(1) << 32) / row) return false;
    return g->pool_bytes / (row * g->page_tokens) >= uint64_t(g->num_pages);
}

inline int outcome(uint32_t flags) {
    if (flags & kPagedInvalid) return KVC_ERR_INVALID;
    return flags & kPagedCapacity ? KVC_ERR_CAPACITY : KVC_OK;
}

// Copies `bytes` of a workspace to the host behind everything on `stream`.
inline bool read_back(void* h, const void* d, uint64_t bytes, hipStream_t s) {
    return hipMemcpyAsync(h, d, bytes, hipMemcpyDeviceToHost, s) == hipSuccess && hipStreamSynchronize(s) == hipSuccess;
}

}  // namespace kvc
