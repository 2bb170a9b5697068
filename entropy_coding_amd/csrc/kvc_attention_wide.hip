// Attention of drafted tokens over a paged cache for sequences with more than
// 16 query rows a KV head (trees, pieces of a prompt).  The mathematics and the
// operands' layouts are those of kvc_attention.hip; here the four waves of a
// workgroup hold different rows (RT groups of 16, dealt to the waves in turn, so
// that few rows keep four SIMDs busy) and walk the same tokens, tiles of
// 64 of which they stage in LDS together, so that K and V are read from memory,
// widened from e4m3 and transposed once for 64 RT rows.
//
// LDS holds a tile as the matrix instruction's operands, 1 KB each, lane after
// lane: K in 4 x D / 32 of them (16 tokens x 32 channels), V^T in 2 x D / 16
// (16 channels x 32 tokens).  Writes and reads are 16 bytes a lane in lane
// order, free of bank conflicts.  Waves 0 and 1 stage 32 tokens of K each,
// waves 2 and 3 of V.  The next tile is on its way from memory to registers
// while the current one is multiplied; it is then written beside it before
// the one barrier of a tile or, where LDS holds one tile only, between two.
//
// What bounds it: with 128 channels and RT = 2 a wave's tile takes 64 matrix
// instructions of 16 cycles and about as many cycles of vector instructions
// (32 exponentials at 16 cycles, 150 others at 4), and the two waves that a
// SIMD holds overlap them in part.  Two pieces of 1000 tokens behind 7001
// cached ones (8 KV heads, 4 query heads each, bf16: 246 GFLOP) take 263 to
// 277 us, 890 to 930 TFLOP/s, where a library's large matrix product reaches
// 1390 on the same card.  RT = 4 needs registers that a wave does not have, and 64 rows
// (RT = 1) read each operand from LDS for half as many products.  Tried and
// slower: the tile after the next on its way too (4 sequences of 16 drafted
// tokens over 4096: 30.2 us instead of 28.3).
//
// Registers are what there is least of: 250 of the 256 that two workgroups a
// CU leave a wave.  No variant keeps any in scratch memory: what only a tile
// that is masked or an item's end needs is formed there (`again`), not before
// the loop over tiles, and in the fullest variants a lane's place in a tile too.
#include "kvc_attend_device.hpp"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kWideTile = 64;

constexpr int kAhead = 4;
constexpr int kNoDs = 0x7F;                     // the scheduler may move all across but LDS instructions

// Workgroups (of a wave a SIMD) that a CU can hold at once: by the registers
// of a wave (sums, queries, scores, weights, the staged quarter of a tile and
// up to 80 for the rest, of 512: bf16 of 256 channels is counted as 264 and
// takes less than 256 in fact) and by the tiles in 160 KB of LDS.
constexpr int groups_of(int d, bool fp8, int rt, int bufs) {
    const int need = d * rt / 4 + d * rt / 8 + 16 * rt + 8 * rt + d * (fp8 ? 1 : 2) / 8 + 80;
    const int regs = need <= 168 ? 3 : need <= 264 ? 2 : 1;
    const int fit = 160 * 1024 / (bufs * kWideTile * d * 4 + 256);
    return regs < fit ? regs : fit;
}

template <int D, int BUFS>
struct WideLds {
    u32x4 k[BUFS][4 * (D / 32)][64];
    u32x4 v[BUFS][2 * (D / 16)][64];
    u32x4 said;                                 // a word a wave
};

// Whether any of the workgroup's waves has x (one value a wave).  The vote
// over all threads that the runtime offers keeps the packed thread numbers in
// a register over the whole kernel.
__device__ inline bool any_wave(bool x, u32x4& said, int wave) {
    if ((threadIdx.x & 63) == 0) reinterpret_cast<uint32_t*>(&said)[wave] = x;
    __syncthreads();
    const u32x4 all = said;
    __syncthreads();                            // (read before the next vote writes)
    return (all[0] | all[1] | all[2] | all[3]) != 0;
}

// PAGE: 16, 4 or 1, the largest that divides the tokens of a page: with 16 a
// half of a wave's 32 tokens lies in one page, its rows a constant stride
// apart; with 4 a lane's run of four V rows does.
// BUFS: tiles that LDS holds.
template <int D, bool FP8, int RT, int BUFS, int PAGE>
__global__ __launch_bounds__(64 * kWaves, groups_of(D, FP8, RT, BUFS)) void k_attend_wide(AttendArgs a) {
    constexpr int C = D / 16;                   // channels of V a lane stages
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int VW = C * ES / 4;              // words of them
    constexpr int KG = D * ES / 64;             // 16-byte pieces of K a lane stages of one token
    constexpr int KK = D / 32;                  // products over the channels
    constexpr int N4 = 2 * KG;                  // 16-byte registers a lane stages, of K or of V
    constexpr int VS = PAGE == 1 ? 8 : 2;
    // whether a lane's place in a tile keeps its registers: where there are none left it is formed for each tile
    constexpr bool KEEP = FP8 || !((D == 256 && BUFS == 1) || (D == 128 && RT == 2 && PAGE == 1));
    __shared__ WideLds<D, BUFS> lds;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool is_v = wave >= 2;
    const uint32_t place = place_of(blockIdx.x, gridDim.x);
    const Plan plan = plan_of(a, 1);
    const Scale sc(a);
    uint32_t bad_page = 0;
    const uint32_t from = place * plan.per, end = from + plan.per;
    uint32_t at = from;
    bool note = blockIdx.x == 0 && wave == 0;
    Share sh;
    while (at < end) {
        share_of(a, plan, at, &sh, note);
        note = false;
        if (!sh.any) break;
        const Part pt = part_of(a, sh, place, at, from, end, kWideTile);
        at = sh.first + sh.units;               // the next item's first unit
        const int length = pt.length, ctx = pt.context, ta = pt.ta, tb = pt.tb;
        const int row0 = pt.row0 + wave * 16;   // of this wave's first group; the others are 64 apart
        const int groups = row0 < pt.rows ? (pt.rows - row0 + 63) / 64 : 0;

        const uint32_t row_bytes = a.heads * D * ES;
        const GlobalBytes pool =
            reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[is_v])) + sh.head * (D * ES);
        const int32_t* const table = a.block_table + int64_t(sh.b) * a.max_pages;

        bf16x8 qf[RT][KK];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const Query query(a, sh, row0 + rt * 64 + (again(lane) & 15), pt.rows);
            const int part = (again(lane) >> 4);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                qf[rt][kk] = query.at(FP8 ? 64 * (kk / 2) + 16 * part + 8 * (kk & 1) : 32 * kk + 8 * part, sc.flip);
        }
        f32x4 o[RT][C];
        RowSum row[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int c = 0; c < C; ++c) o[rt][c] = f32x4{0, 0, 0, 0};

        // Staging.  A wave has 32 tokens of a tile: a lane of K token n of both halves, a lane of V a run of four of
        // each half.  Page numbers are read a tile ahead of the rows.
        const int half32 = (wave & 1) * 32;
        // This lane's place in that, kept or formed for each tile anew.
        const int kept_n = lane & 15, kept_q4 = lane >> 4;
        auto place_n = [&]() -> int { return KEEP ? kept_n : again(lane) & 15; };
        auto place_q4 = [&]() -> int { return KEEP ? kept_q4 : again(lane) >> 4; };
        auto stages_v = [&]() -> bool { return KEEP ? is_v : again_uniform(wave) >= 2; };
        auto token = [&](int t, int i, int n, int q4) -> uint32_t {
            const int x = t * kWideTile + half32 +
                          (PAGE == 16 ? 16 * i : is_v ? (VS == 2 ? 16 * i : (i < 4 ? 0 : 12) + i) + q4 * 4 : 16 * (i & 1) + n);
            return static_cast<uint32_t>(x < length ? x : PAGE == 16 ? (length - 1) & ~15
                                                          : PAGE == 4 && is_v ? (length - 1) & ~3 : length - 1);
        };
        int32_t page[VS];
        auto read_pages = [&](int t) {
            const int n = place_n(), q4 = place_q4();
#pragma unroll
            for (int i = 0; i < VS; ++i) {
                const int32_t* const at_page = table + page_index(a, token(t, i, n, q4));
                page[i] = PAGE == 16 ? uniform_word(at_page) : *at_page;
            }
        };
        u32x4 st[N4];
        auto load = [&](int t) {
            const int n = place_n(), q4 = place_q4();
            const bool is_v = stages_v();
            auto row_at = [&](int i) -> uint64_t {
                return uint64_t(slot_in(a, page[i], token(t, i, n, q4), &bad_page)) * row_bytes;
            };
            if (is_v) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const GlobalBytes p = pool + row_at(VS == 2 ? j / 4 : j) +
                                          ((PAGE == 16 ? q4 * 4 + (j & 3) : PAGE == 4 ? j & 3 : 0) * row_bytes +
                                           uint32_t(n) * (C * ES));
                    Words<VW> w;
                    w.load(p);
#pragma unroll
                    for (int x = 0; x < VW; ++x) st[(j * VW + x) / 4][(j * VW + x) % 4] = w[x];
                }
            } else {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const GlobalBytes p = pool + row_at(hf) + ((PAGE == 16 ? n * row_bytes : 0u) + 16u * q4);
#pragma unroll
                    for (int kg = 0; kg < KG; ++kg)
                        st[hf * KG + kg] = *reinterpret_cast<const KVC_GLOBAL u32x4*>(p + 64 * kg);
                }
            }
        };
        bool any_wild = false;
        auto write = [&](int t, int buf) {
            if (stages_v()) {
                const int t0 = t * kWideTile + half32;
                if (t0 + 32 > ctx) {
                    // tokens behind the last one are cleared, and infinities and NaN of drafted ones
                    uint32_t wild = 0;
                    const int first = (again(lane) >> 4) * 4;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int tok = t0 + (j < 4 ? 0 : 12) + first + j;
                        const uint32_t there = tok < length ? ~0u : 0u, drafted = tok >= ctx ? ~0u : 0u;
#pragma unroll
                        for (int x = 0; x < VW; ++x) {
                            uint32_t w = st[(j * VW + x) / 4][(j * VW + x) % 4] & there;
                            const uint32_t bits = wild_bits<FP8>(w) & drafted;
                            wild |= bits;
                            if (drafted) w = without_wild<FP8>(w);
                            st[(j * VW + x) / 4][(j * VW + x) % 4] = w;
                        }
                    }
                    any_wild = any_wild || __any(wild != 0);
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    u32x4 f;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int x = 2 * p * VW + c * ES / 4, y = x + VW;
                        f[p] = pair_of<FP8>(st[x / 4][x % 4], st[y / 4][y % 4], c);
                    }
                    lds.v[buf][(wave & 1) * C + c][lane] = f;
                }
            } else {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int kg = 0; kg < KG; ++kg) {
                        const u32x4 x = st[hf * KG + kg];
                        u32x4* const to = &lds.k[buf][((wave & 1) * 2 + hf) * KK + kg * (FP8 ? 2 : 1)][lane];
                        if constexpr (FP8) {
                            to[0] = u32x4{widen<false>(x[0]), widen<true>(x[0]), widen<false>(x[1]), widen<true>(x[1])};
                            to[64] = u32x4{widen<false>(x[2]), widen<true>(x[2]), widen<false>(x[3]), widen<true>(x[3])};
                        } else {
                            to[0] = x;
                        }
                    }
            }
        };

        auto compute = [&](int t, int buf, auto held) {
            constexpr int G = held;             // groups that have rows
            const int t0 = t * kWideTile;
            // (the waves that multiply go before those that form weights on the same SIMD: 3%)
            __builtin_amdgcn_s_setprio(1);
            // Operands are read from LDS kAhead before their products: one by one, each pair of products would wait for
            // a whole trip to LDS (the pieces of a prompt above 369 us and, so, 315 at the time).  The four sums of a group take
            // turns, so that no product waits for the one before it (0.7%).
            u32x4 ring[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ring[i] = lds.k[buf][(i & 3) * KK + (i >> 2)][lane];
            __builtin_amdgcn_sched_barrier(0);
            f32x4 s[G][4];
#pragma unroll
            for (int i = 0; i < 4 * KK; ++i) {
                const int hf = i & 3, kk = i >> 2;
                const bf16x8 kf = __builtin_bit_cast(bf16x8, ring[i % kAhead]);
#pragma unroll
                for (int rt = 0; rt < G; ++rt)
                    s[rt][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][kk], kk ? s[rt][hf] : f32x4{0, 0, 0, 0}, 0, 0, 0);
                if (i + kAhead < 4 * KK) ring[i % kAhead] = lds.k[buf][((i + kAhead) & 3) * KK + ((i + kAhead) >> 2)][lane];
                __builtin_amdgcn_sched_barrier(0);
            }
            if (t0 + kWideTile > pt.full) {
#pragma unroll
                for (int rt = 0; rt < G; ++rt) {
                    const int node = Query(a, sh, row0 + rt * 64 + (again(lane) & 15), pt.rows).node;
                    const uint64_t win = window_of(a, sh.seq.start, node, t0 - ctx, length - ctx) >> ((again(lane) >> 4) * 4);
#pragma unroll
                    for (int hf = 0; hf < 4; ++hf)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((win >> (hf * 16 + i)) & 1u)) s[rt][hf][i] = kNegInf;
                }
            }
            __builtin_amdgcn_s_setprio(0);
            float top[G];
            bool grows = false;
#pragma unroll
            for (int rt = 0; rt < G; ++rt) {
                top[rt] = kNegInf;
#pragma unroll
                for (int hf = 0; hf < 4; ++hf) top[rt] = larger(top[rt], s[rt][hf]);
                grows = grows || top[rt] > row[rt].limit;
            }
            if (__any(grows)) {
#pragma unroll
                for (int rt = 0; rt < G; ++rt) {
                    const float f = row[rt].raise(top[rt], sc.scale, sc.slack);
#pragma unroll
                    for (int c = 0; c < C; ++c) o[rt][c] *= f;
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ring[i] = lds.v[buf][i][lane];
            __builtin_amdgcn_sched_barrier(kNoDs);
            bf16x8 pf[G][2];
#pragma unroll
            for (int st2 = 0; st2 < 2; ++st2) {
#pragma unroll
                for (int rt = 0; rt < G; ++rt) {
                    float e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][2 * st2 + (j >> 2)][j & 3], sc.scale, row[rt].shift));
                    row[rt].sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    pf[rt][st2] = frag_of(two_bf16(e[0], e[1]), two_bf16(e[2], e[3]), two_bf16(e[4], e[5]), two_bf16(e[6], e[7]));
                }
            }
            // (Left to itself the scheduler draws the exponentials in among the products, and the reads back to one ahead of
            // theirs: the pieces above in pages of 12 tokens 298 us instead of 281, of 16 tokens 275 and 270.)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 2 * C; ++i) {
                const int st2 = i / C, c = i % C;
                const bf16x8 vf = __builtin_bit_cast(bf16x8, ring[i % kAhead]);
#pragma unroll
                for (int rt = 0; rt < G; ++rt)
                    o[rt][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt][st2], o[rt][c], 0, 0, 0);
                if (i + kAhead < 2 * C) ring[i % kAhead] = lds.v[buf][i + kAhead][lane];
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        if (ta < tb) {
            read_pages(ta);
            load(ta);
            read_pages(ta + 1);
            write(ta, 0);
            __syncthreads();
            for (int t = ta; t < tb; ++t) {
                const int buf = BUFS == 2 ? (t - ta) & 1 : 0;
                if (t + 1 < tb) {
                    load(t + 1);
                    read_pages(t + 2);
                }
                if (RT == 2 && groups > 1) compute(t, buf, std::integral_constant<int, RT>{});
                else if (groups) compute(t, buf, std::integral_constant<int, 1>{});
                if (BUFS == 1) __syncthreads();
                if (t + 1 < tb) write(t + 1, BUFS == 2 ? buf ^ 1 : 0);
                __syncthreads();
            }
        }
        any_wild = any_wave(any_wild, lds.said, wave);

        // each wave has its rows' sums: lane l those of row n, channels 4 q C .. 4 (q + 1) C - 1
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float sum = row[rt].sum;
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            const int m = row0 + rt * 64 + (again(lane) & 15), at_ch = (again(lane) >> 4) * 4 * C;
            if (m < pt.rows) {
                const int node = m / static_cast<int>(a.ratio);
                const float best = row[rt].top();
                if (pt.whole) {
                    const int64_t out_row = int64_t(sh.seq.start) + node;
                    const int64_t head = int64_t(sh.head) * a.ratio + (m - node * static_cast<int>(a.ratio));
                    const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
                    uint16_t* const out = a.out + out_row * a.out_row + head * D + at_ch;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < C; c += 4)
                            *reinterpret_cast<uint2*>(out + i * C + c) =
                                uint2{two_bf16(o[rt][c][i] * inv, o[rt][c + 1][i] * inv),
                                      two_bf16(o[rt][c + 2][i] * inv, o[rt][c + 3][i] * inv)};
                    if (a.lse && lane < 16)
                        a.lse[out_row * (int64_t(a.heads) * a.ratio) + head] =
                            sum == 0.0f ? kNegInf : (best + __builtin_amdgcn_logf(sum)) * kLn2;
                } else {
                    const uint64_t to = (uint64_t(pt.slot) << a.tile_shift) + (m - pt.row0);
                    float* const out = a.partial + to * D + at_ch;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < C; c += 4)
                            *reinterpret_cast<f32x4*>(out + i * C + c) =
                                f32x4{o[rt][c][i], o[rt][c + 1][i], o[rt][c + 2][i], o[rt][c + 3][i]};
                    if (lane < 16) *reinterpret_cast<float2*>(a.pairs + 2 * to) = float2{best, sum};
                }
            }
        }
        if (any_wild) {
            // Rare: added to what this lane has just written.
            const GlobalBytes vp =
                reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[1])) + sh.head * (D * ES);
            const int last = tb * kWideTile < length ? tb * kWideTile : length;
            const int at_ch = (again(lane) >> 4) * 4 * C;
            for (int m = row0 + (again(lane) & 15); m < pt.rows && m < row0 + 64 * RT; m += 64) {
                const int nd = m / static_cast<int>(a.ratio);
                const int64_t out_row = int64_t(sh.seq.start) + nd;
                const int64_t head = int64_t(sh.head) * a.ratio + (m - nd * static_cast<int>(a.ratio));
                uint16_t* const out = a.out + out_row * a.out_row + head * D + at_ch;
                float* const part = a.partial + ((uint64_t(pt.slot) << a.tile_shift) + (m - pt.row0)) * D + at_ch;
                for (int tok = ta * kWideTile > ctx ? ta * kWideTile : ctx; tok < last; ++tok) {
                    if (!sees(a, sh.seq.start, nd, static_cast<uint32_t>(tok - ctx))) continue;
                    uint32_t known = 0;
                    const GlobalBytes p =
                        vp + uint64_t(slot_in(a, table[page_index(a, tok)], tok, &known)) * row_bytes + at_ch * ES;
                    for (int c = 0; c < 4 * C; ++c) {
                        const uint32_t w = *reinterpret_cast<const KVC_GLOBAL uint32_t*>(p + 4 * (c * ES / 4));
                        const float x = wild_part<FP8>(w, c);
                        if (x == 0.0f) continue;
                        if (pt.whole) out[c] = static_cast<uint16_t>(two_bf16(__uint_as_float(uint32_t(out[c]) << 16) + x, 0.0f));
                        else part[c] += x;
                    }
                }
            }
        }
    }
    const bool any = any_wave(__any(bad_page != 0), lds.said, wave);
    if (wave == 0 && again(lane) == 0) a.words[blockIdx.x] = any ? kPagedInvalid : 0u;
}

template <int D, bool FP8, int RT, int BUFS, int PAGE>
hipError_t launch_one(const AttendArgs& a, const AttendShape& sh, hipStream_t s) {
    k_attend_wide<D, FP8, RT, BUFS, PAGE><<<sh.grid, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <int D, bool FP8, int PAGE>
hipError_t launch(const AttendArgs& a, const AttendShape& sh, hipStream_t s) {
    if constexpr (D <= 128) return sh.row_tiles == 1 ? launch_one<D, FP8, 1, 2, PAGE>(a, sh, s) : launch_one<D, FP8, 2, 2, PAGE>(a, sh, s);
    else if constexpr (FP8) return launch_one<D, FP8, 1, 1, PAGE>(a, sh, s);
    else return sh.lds_tiles == 1 ? launch_one<D, FP8, 1, 1, PAGE>(a, sh, s) : launch_one<D, FP8, 1, 2, PAGE>(a, sh, s);
}

template <int D>
hipError_t launch_channels(const AttendArgs& a, const AttendShape& sh, bool fp8, hipStream_t s) {
    if (a.page_tokens % 16 == 0) return fp8 ? launch<D, true, 16>(a, sh, s) : launch<D, false, 16>(a, sh, s);
    if (a.page_tokens % 4 == 0) return fp8 ? launch<D, true, 4>(a, sh, s) : launch<D, false, 4>(a, sh, s);
    return fp8 ? launch<D, true, 1>(a, sh, s) : launch<D, false, 1>(a, sh, s);
}

}  // namespace

int wide_groups(int64_t channels, bool fp8, int row_tiles, int lds_tiles) {
    return groups_of(static_cast<int>(channels), fp8, row_tiles, lds_tiles);
}

hipError_t launch_attend_wide(const AttendArgs& a, const AttendShape& sh, int64_t channels, bool fp8, hipStream_t s) {
    switch (channels) {
        case 64: return launch_channels<64>(a, sh, fp8, s);
        case 128: return launch_channels<128>(a, sh, fp8, s);
        case 192: return launch_channels<192>(a, sh, fp8, s);
        case 256: return launch_channels<256>(a, sh, fp8, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace kvc
