// Host-side interface between the C ABI (kvc_step_api.cpp) and the kernels of
// a speculative step around the attention over pages: norms, rotation and
// append (kvc_qkv.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace kvc {

// ---- norms, rotation, append

struct HeadRows {                       // [rows][heads][channels], strides in values
    const uint16_t* at;
    int64_t row, head;
};
struct QkvArgs {
    void* const* pools;                 // the layer's K pool, then its V pool
    HeadRows q, k, v;
    uint16_t* out;                      // the heads of a row `channels` values apart
    int64_t out_row;
    const void* q_norm;                 // null: no norm
    const void* k_norm;
    const double* frequencies;
    const int32_t* positions;           // null: every row is one (nothing is rotated)
    const int64_t* slots;
    int64_t rows, n_slots;
    uint32_t q_heads, heads, rotary;
    uint32_t norm_f32;                  // the norms' weights are float32 (bf16 otherwise)
    uint32_t parts;                     // that a row's heads are split into (the launch sets it)
    float eps, k_scale, v_scale;
};
hipError_t launch_qkv(const QkvArgs& args, int64_t channels, bool fp8, bool neighbours, hipStream_t s);

}  // namespace kvc
