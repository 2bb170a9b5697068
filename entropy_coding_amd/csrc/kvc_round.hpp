// Roundings of cache values that the paged kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvc {

// A NaN passes both comparisons and stays.
__device__ inline float clamp448(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

// Two values as e4m3 of x / scale: the quotient in float32, clamped to
// +-448, then rounded to nearest even by the conversion.
__device__ inline uint32_t round_two(float lo, float hi, float scale) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(lo / scale), clamp448(hi / scale), 0, false)) &
           0xFFFFu;
}
// ... of two bf16 values (low half first).
__device__ inline uint32_t round_pair(uint32_t two, float scale) {
    return round_two(__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u), scale);
}

}  // namespace kvc
