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

// Sixteen channels of a head in a lane: two pieces of eight, so that a lane
// has both values of every pair.  Where a channel's other one lies half of the
// `rotary` channels behind it, so does the second piece behind the first; else
// the pieces follow each other.
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

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class T>
using Global = __attribute__((address_space(1))) T;     // (a pool's pointer, read from memory, says nothing of it)

enum : uint32_t { kQuery, kKey, kValue };

// Two float32 values as e4m3 of x / scale, the scale given as its reciprocal
// in float64: the product rounded to float32 is the float32 quotient to the
// last bit (a quotient of two float32 values lies further from the middle of
// two neighbouring ones, 2^-49 of itself, than the product is off; what is
// subnormal in float32 is 0 in e4m3 either way), and takes a third of the
// instructions of a division.
__device__ uint32_t round_scaled(float lo, float hi, double per_scale) {
    const float x = static_cast<float>(double(lo) * per_scale), y = static_cast<float>(double(hi) * per_scale);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(x), clamp448(y), 0, false)) & 0xFFFFu;
}

// A row's heads (queries, then keys, then values), as many at a time as a wave
// has groups of lanes; UNIFORM: all of a step's heads are of one kind.  The
// next step's values are asked for before this one's are looked at, a row's
// first ones before its position.  An angle's sine and cosine are formed once
// a row, one in a lane, and read from LDS for every head (kept in registers
// they left four waves a SIMD instead of five: 82 -> 80 us and 29 -> 27 us for
// the calls named here).  Stores are not kept in the caches (80 -> 75 us, 27 ->
// 23 us; an attention behind them takes as long as before).  Bound by HBM where
// rows are many (16384 of 32 and 16 heads of 128 bf16 channels, 403 MB: 75 us,
// 5.4 TB/s; a copy of as many bytes 82; vector instructions 39% of the cycles),
// by a wave's trips to memory where they are few (4 rows: 4.0 us on the GPU),
// by a short launch's start and end between (5003 rows to e4m3, 101 MB: 23 us,
// a copy's rate gives 21; 28 where the last-level cache has none of the rows).
template <int D, bool FP8, bool NEIGHBOURS, bool UNIFORM>
__global__ __launch_bounds__(64 * kQkvWaves, 5) void k_qkv(QkvArgs a) {
    constexpr int kUnits = D / 16;              // lanes that a head needs
    constexpr int kGroup = kUnits == 12 ? 16 : kUnits;
    constexpr int kHeads = 64 / kGroup;
    __shared__ float2 turns[kQkvWaves][D / 2];  // (cosine, sine) of the row's angles
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t u = lane % kGroup, group = lane / kGroup;
    const uint32_t half = a.rotary / 2, rotated = a.rotary / 16;
    const bool here = u < kUnits, turned = u < rotated;
    const bool apart = turned && !NEIGHBOURS;
    const uint32_t first = apart ? 8 * u : 16 * u, second = apart ? half + 8 * u : 16 * u + 8;
    const uint32_t all = a.q_heads + 2 * a.heads, steps = (all + kHeads - 1) / kHeads;
    const int64_t items = a.rows * a.parts;

    struct Step {
        uint32_t kind, head;
        bool real;
    };
    const auto step_of = [&](uint32_t step) {
        const uint32_t begin = step * kHeads;
        Step r;
        const uint32_t index = UNIFORM ? begin : begin + group;
        r.kind = index < a.q_heads ? kQuery : index < a.q_heads + a.heads ? kKey : kValue;
        r.head = index - (r.kind == kQuery ? 0 : r.kind == kKey ? a.q_heads : a.q_heads + a.heads) + (UNIFORM ? group : 0);
        r.real = here && (UNIFORM || index < all);
        return r;
    };
    const auto fetch = [&](int64_t row, uint32_t step) {
        const Step t = step_of(step);
        const HeadRows from = t.kind == kQuery ? a.q : t.kind == kKey ? a.k : a.v;
        Pieces in{};
        if (t.real) {
            const uint16_t* const x = from.at + row * from.row + int64_t(t.head) * from.head;
            in.raw[0] = *reinterpret_cast<const uint4*>(x + first);
            in.raw[1] = *reinterpret_cast<const uint4*>(x + second);
        }
        return in;
    };

    for (int64_t item = int64_t(blockIdx.x) * kQkvWaves + wave; item < items; item += int64_t(gridDim.x) * kQkvWaves) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const uint32_t part = static_cast<uint32_t>(item - row * a.parts);
        const uint32_t begin = part * steps / a.parts, end = (part + 1) * steps / a.parts;
        Pieces next = fetch(row, begin);
        const int32_t position = a.positions ? a.positions[row] : 0;
        if (position < 0) continue;
        const int64_t slot = a.slots[row];
        if (a.rotary) {
            // Whole turns are taken off in 64 bits, so that far positions are as exact as near ones.
            __builtin_amdgcn_wave_barrier();    // (the last row's are read)
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
            __builtin_amdgcn_wave_barrier();
        }
        for (uint32_t step = begin; step < end; ++step) {
            const Pieces in = next;
            if (step + 1 < end) next = fetch(row, step + 1);
            const Step t = step_of(step);
            float x[2][8];
            in.unpack(x);
            const void* const norm = t.kind == kQuery ? a.q_norm : t.kind == kKey ? a.k_norm : nullptr;
            if (norm) {
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
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(x[i / 8][i % 8], x[i / 8][i % 8], sum);
                sum = group_sum<kGroup>(sum);
                float r = __builtin_amdgcn_rsqf(fmaf(sum, 1.0f / D, a.eps));
                if (__any(sum > 3.0e38f)) {     // squares beyond float32
                    double wide = 0.0;
#pragma nounroll
                    for (int i = 0; i < 8; ++i) {
                        float y[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k == i) {
                                y[0] = x[0][k];
                                y[1] = x[1][k];
                            }
                        wide = fma(double(y[1]), double(y[1]), fma(double(y[0]), double(y[0]), wide));
                    }
                    wide = group_sum<kGroup>(wide);
                    if (sum > 3.0e38f) r = static_cast<float>(1.0 / sqrt(wide / D + double(a.eps)));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i / 8][i % 8] = x[i / 8][i % 8] * r * w[i / 8][i % 8];
            }
            if (turned && t.kind != kValue) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float& left = NEIGHBOURS ? x[i / 4][2 * (i % 4)] : x[0][i];
                    float& right = NEIGHBOURS ? x[i / 4][2 * (i % 4) + 1] : x[1][i];
                    const float2 t = turns[wave][8 * u + i];
                    const float l = fmaf(left, t.x, -(right * t.y)), y = fmaf(left, t.y, right * t.x);
                    left = l;
                    right = y;
                }
            }
            if (!t.real) continue;
            if (t.kind != kQuery && (slot < 0 || slot >= a.n_slots)) continue;
            Global<uint8_t>* to;
            if (t.kind == kQuery)
                to = (Global<uint8_t>*)(a.out + row * a.out_row + int64_t(t.head) * D);
            else
                to = (Global<uint8_t>*)(a.pools[t.kind - kKey]) + (slot * a.heads + t.head) * int64_t(D) * (FP8 ? 1 : 2);
            if (FP8 && t.kind != kQuery) {
                const double per_scale = t.kind == kKey ? a.per_k_scale : a.per_v_scale;
                u32x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* const four = x[i / 2] + 4 * (i % 2);
                    y[i] = round_scaled(four[0], four[1], per_scale) | (round_scaled(four[2], four[3], per_scale) << 16);
                }
                if (apart) {
                    __builtin_nontemporal_store(u32x2{y[0], y[1]}, (Global<u32x2>*)(to + first));
                    __builtin_nontemporal_store(u32x2{y[2], y[3]}, (Global<u32x2>*)(to + second));
                } else {
                    __builtin_nontemporal_store(y, (Global<u32x4>*)(to + first));
                }
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    u32x4 y = {in.raw[p].x, in.raw[p].y, in.raw[p].z, in.raw[p].w};     // (values keep every bit)
                    if (t.kind != kValue)
                        y = u32x4{two_bf16(x[p][0], x[p][1]), two_bf16(x[p][2], x[p][3]),
                                  two_bf16(x[p][4], x[p][5]), two_bf16(x[p][6], x[p][7])};
                    __builtin_nontemporal_store(y, (Global<u32x4>*)(to + 2 * (p ? second : first)));
                }
            }
        }
    }
}

template <int D, bool FP8, bool NEIGHBOURS>
hipError_t launch(const QkvArgs& args, hipStream_t s) {
    QkvArgs a = args;
    constexpr int kHeads = 64 / (D == 192 ? 16 : D / 16);
    const int64_t steps = (int64_t(a.q_heads) + 2 * int64_t(a.heads) + kHeads - 1) / kHeads;
    // Few rows: a wave a step.  Else at most four steps a wave: whole rows leave the chip's waves unevenly filled where
    // they are long (6081 rows of 64 and 8 heads of 256 channels 94 us, with two waves a row 105; two or three steps a
    // wave take as long as four), and each part forms the row's angles.
    a.parts = static_cast<uint32_t>(a.rows * steps <= 4096 ? steps : (steps + 3) / 4);
    int64_t blocks = (a.rows * a.parts + kQkvWaves - 1) / kQkvWaves;
    if (blocks > 1 << 16) blocks = 1 << 16;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(64 * kQkvWaves);
    if (a.q_heads % kHeads == 0 && a.heads % kHeads == 0) k_qkv<D, FP8, NEIGHBOURS, true><<<grid, block, 0, s>>>(a);
    else k_qkv<D, FP8, NEIGHBOURS, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const QkvArgs& a, bool fp8, bool neighbours, hipStream_t s) {
    if (fp8) return neighbours ? launch<D, true, true>(a, s) : launch<D, true, false>(a, s);
    return neighbours ? launch<D, false, true>(a, s) : launch<D, false, false>(a, s);
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
