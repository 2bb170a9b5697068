// Norms of queries and keys, their rotation by position, and the append of
// K and V to the pages, in one pass over a projection's rows (declared in
// include/kvc.h).
#include <hip/hip_runtime.h>

#include "kvc_round.hpp"
#include "kvc_step.hpp"

namespace kvc {
namespace {

constexpr int kQkvWaves = 4;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ uint32_t two_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

// A value of the lane that CTRL names within 16 lanes.
template <int CTRL>
__device__ float moved(float x) {
    return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(__float_as_uint(x)), CTRL, 0xF, 0xF, false)));
}
template <int CTRL>
__device__ double moved(double x) {
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xF, 0xF, false);
    return __longlong_as_double((uint64_t(hi) << 32) | lo);
}
// The sum over a group of 4, 8 or 16 lanes, in each of them.
template <int GROUP, class T>
__device__ T group_sum(T x) {
    x += moved<0xB1>(x);                        // lanes 1 0 3 2
    x += moved<0x4E>(x);                        // lanes 2 3 0 1
    if (GROUP > 4) x += moved<0x141>(x);        // the mirrored half row
    if (GROUP > 8) x += moved<0x140>(x);        // the mirrored row
    return x;
}

// Sixteen channels of a head in a lane: two pieces of eight.  Among the first
// `rotary` channels the second piece lies half of them behind the first, so
// that a lane has both values of every pair, whether pairs are such halves or
// neighbours; behind them the pieces follow each other.
struct Pieces {
    uint4 raw[2];
    __device__ void unpack(float (&x)[2][8]) const {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t w[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[p][2 * i] = __uint_as_float(w[i] << 16);
                x[p][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};

// One row's heads (queries, then keys, then values), as many at a time as a
// wave has groups of lanes.
template <int D, bool FP8, bool NEIGHBOURS>
__global__ __launch_bounds__(64 * kQkvWaves) void k_qkv(QkvArgs a) {
    constexpr int kUnits = D / 16;              // lanes that a head needs
    constexpr int kGroup = kUnits == 12 ? 16 : kUnits;
    constexpr int kHeads = 64 / kGroup;
    __shared__ float2 turns[kQkvWaves][D / 2];  // (cosine, sine) of the row's angles
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t u = lane % kGroup, group = lane / kGroup;
    const uint32_t half = a.rotary / 2, rotated = a.rotary / 16;
    const bool here = u < kUnits, turned = u < rotated;
    const uint32_t first = turned ? 8 * u : 16 * u, second = turned ? half + 8 * u : 16 * u + 8;
    const uint32_t all = a.q_heads + 2 * a.heads, steps = (all + kHeads - 1) / kHeads;
    const uint32_t per = (steps + a.parts - 1) / a.parts;
    const int64_t items = a.rows * a.parts;
    for (int64_t item = int64_t(blockIdx.x) * kQkvWaves + wave; item < items; item += int64_t(gridDim.x) * kQkvWaves) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const uint32_t part = static_cast<uint32_t>(item - row * a.parts);
        const int32_t position = a.positions ? a.positions[row] : 0;
        if (position < 0) continue;
        const int64_t slot = a.slots[row];
        float c[8], s[8];
        if (a.rotary) {
            // Whole turns are taken off in 64 bits, so that far positions are as exact as near ones.
            for (uint32_t i = lane; i < half; i += 64) {
                double t = double(position) * (a.frequencies[i] * 0.15915494309189535);
                t -= rint(t);
                float sine, cosine;
                sincospif(2.0f * static_cast<float>(t), &sine, &cosine);
                turns[wave][i] = float2{cosine, sine};
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = NEIGHBOURS ? (i < 4 ? 4 * u + i : half / 2 + 4 * u + i - 4) : 8 * u + i;
                const float2 t = turned ? turns[wave][at] : float2{1.0f, 0.0f};
                c[i] = t.x;
                s[i] = t.y;
            }
            __builtin_amdgcn_wave_barrier();
        }
        const uint32_t end = (part + 1) * per < steps ? (part + 1) * per : steps;
        for (uint32_t step = part * per; step < end; ++step) {
            const uint32_t index = step * kHeads + group;
            const int kind = index < a.q_heads ? 0 : index < a.q_heads + a.heads ? 1 : 2;
            const uint32_t head = kind == 0 ? index : kind == 1 ? index - a.q_heads : index - a.q_heads - a.heads;
            const bool real = here && index < all;
            const HeadRows from = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
            Pieces in{};
            if (real) {
                const uint16_t* const x = from.at + row * from.row + int64_t(head) * from.head;
                in.raw[0] = *reinterpret_cast<const uint4*>(x + first);
                in.raw[1] = *reinterpret_cast<const uint4*>(x + second);
            }
            float x[2][8];
            in.unpack(x);
            const void* const norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
            if (norm) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(x[i / 8][i % 8], x[i / 8][i % 8], sum);
                sum = group_sum<kGroup>(sum);
                float r = __builtin_amdgcn_rsqf(fmaf(sum, 1.0f / D, a.eps));
                if (__any(sum > 3.0e38f)) {     // squares beyond float32
                    double wide = 0.0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) wide = fma(double(x[i / 8][i % 8]), double(x[i / 8][i % 8]), wide);
                    wide = group_sum<kGroup>(wide);
                    if (sum > 3.0e38f) r = static_cast<float>(1.0 / sqrt(wide / D + double(a.eps)));
                }
                float w[2][8];
                if (a.norm_f32) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 y = here ? *reinterpret_cast<const float4*>(static_cast<const float*>(norm) + (p ? second : first) + 4 * i) : float4{};
                            w[p][4 * i] = y.x;
                            w[p][4 * i + 1] = y.y;
                            w[p][4 * i + 2] = y.z;
                            w[p][4 * i + 3] = y.w;
                        }
                } else {
                    Pieces y{};
                    if (here) {
                        y.raw[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(norm) + first);
                        y.raw[1] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(norm) + second);
                    }
                    y.unpack(w);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i / 8][i % 8] = x[i / 8][i % 8] * r * w[i / 8][i % 8];
            }
            if (turned && kind != 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float& left = NEIGHBOURS ? x[i / 4][2 * (i % 4)] : x[0][i];
                    float& right = NEIGHBOURS ? x[i / 4][2 * (i % 4) + 1] : x[1][i];
                    const float l = fmaf(left, c[i], -(right * s[i])), t = fmaf(left, s[i], right * c[i]);
                    left = l;
                    right = t;
                }
            }
            if (!real) continue;
            if (kind != 0 && (slot < 0 || slot >= a.n_slots)) continue;
            uint8_t* to = reinterpret_cast<uint8_t*>(a.out + row * a.out_row + int64_t(head) * D);
            if (kind != 0)
                to = static_cast<uint8_t*>(a.pools[kind - 1]) + (slot * a.heads + head) * int64_t(D) * (FP8 ? 1 : 2);
            if (FP8 && kind != 0) {
                const float scale = kind == 1 ? a.k_scale : a.v_scale;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[i] = round_two(x[p][4 * i], x[p][4 * i + 1], scale) |
                               (round_two(x[p][4 * i + 2], x[p][4 * i + 3], scale) << 16);
                    *reinterpret_cast<uint2*>(to + (p ? second : first)) = uint2{w[0], w[1]};
                }
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint4 y = in.raw[p];
                    if (kind != 2)
                        y = uint4{two_bf16(x[p][0], x[p][1]), two_bf16(x[p][2], x[p][3]),
                                  two_bf16(x[p][4], x[p][5]), two_bf16(x[p][6], x[p][7])};
                    *reinterpret_cast<uint4*>(to + 2 * (p ? second : first)) = y;
                }
            }
        }
    }
}

template <int D>
hipError_t launch(const QkvArgs& args, bool fp8, bool neighbours, hipStream_t s) {
    QkvArgs a = args;
    constexpr int kHeads = 64 / (D == 192 ? 16 : D / 16);
    const int64_t steps = (int64_t(a.q_heads) + 2 * int64_t(a.heads) + kHeads - 1) / kHeads;
    a.parts = a.rows * steps <= 4096 ? static_cast<uint32_t>(steps) : 1;
    int64_t blocks = (a.rows * a.parts + kQkvWaves - 1) / kQkvWaves;
    if (blocks > 1 << 16) blocks = 1 << 16;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(64 * kQkvWaves);
    if (fp8 && neighbours) k_qkv<D, true, true><<<grid, block, 0, s>>>(a);
    else if (fp8) k_qkv<D, true, false><<<grid, block, 0, s>>>(a);
    else if (neighbours) k_qkv<D, false, true><<<grid, block, 0, s>>>(a);
    else k_qkv<D, false, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qkv(const QkvArgs& a, int64_t channels, bool fp8, bool neighbours, hipStream_t s) {
    switch (channels) {
        case 64: return launch<64>(a, fp8, neighbours, s);
        case 128: return launch<128>(a, fp8, neighbours, s);
        case 192: return launch<192>(a, fp8, neighbours, s);
        default: return launch<256>(a, fp8, neighbours, s);
    }
}

}  // namespace kvc
