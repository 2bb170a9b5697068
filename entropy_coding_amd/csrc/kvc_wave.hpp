// Sums over a wave's lanes and searches that the paged cache's kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvc {

// Sums over a wave's lanes, without the trip through LDS that a shuffle
// takes: of the lanes up to this one, and of all.
template <int CTRL, int ROWS>
__device__ uint32_t add_moved(uint32_t x) {
    return x + static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xF, false));
}
__device__ inline uint32_t scan(uint32_t x) {
    x = add_moved<0x111, 0xF>(x);               // within rows of 16 lanes: from 1, 2, 4 and 8 lanes before
    x = add_moved<0x112, 0xF>(x);
    x = add_moved<0x114, 0xF>(x);
    x = add_moved<0x118, 0xF>(x);
    x = add_moved<0x142, 0xA>(x);               // the last lane of the row before, into rows 1 and 3
    return add_moved<0x143, 0xC>(x);            // lane 31 into rows 2 and 3
}
__device__ inline uint32_t of_lane(uint32_t x, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}

}  // namespace kvc
