// Attention of drafted tokens over a paged cache (kvc_paged_attention in
// include/kvc.h), for sequences with up to 16 query rows a KV head: the next
// token of a sequence and small trees.  kvc_attention_wide.hip has the kernel
// for more rows; the choice between them and the join of split sequences are
// here.
//
// The query rows of one KV head of one sequence are its (drafted token, query
// head of the group) pairs: all read the same K and V.  One pass over the
// tokens keeps, for each row, the running maximum m of its scores (in units of
// log 2), the sum l of 2^(s - m) and the weighted sum o of V; parts of the
// tokens are joined by
//     m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),
// here first the four waves of a workgroup (which take tiles of 32 tokens in
// turn) through LDS, then the workgroups of a split sequence through a second,
// small kernel.
//
// Tiles never pass through LDS.  With S^T = K Q^T and O^T = V^T P^T on the
// 16 x 16 x 32 matrix instruction, lane l = 16 q + n holds
//   - of S^T column n (a query row) and, of the two 16-token halves of a tile,
//     tokens 4 q .. 4 q + 3 of each: eight scores, which rounded to bf16 are
//     the eight values that the second product wants from lane l for its
//     inner index, in an order of tokens that only V has to share;
//   - of K token n (of a half) and eight channels: sixteen bytes of its row;
//   - of V the same eight tokens and channels n C .. n C + C - 1 (C = D / 16),
//     whose transposes, 2 x 2 values at a time, are byte permutes within the
//     lane; row i of the c-th product is then channel i C + c.
// The weights' rounding to bf16 is what the matrix instruction takes; their
// sum l is of the unrounded ones, in float32.
//
// What bounds it: reading K and V once.  The next tokens of 64 sequences of
// 4000 (8 KV heads, 4 query heads each, 128 channels, bf16: 1.05 GB) take 196
// us, 5.3 TB/s (a copy of 2 GiB 4.9, read and written).  Those of 4 sequences
// of 4096 (67 MB) take 20.9 us, 16.4 of them here (4.1 TB/s), 4.4 in the join:
// a workgroup has nine tiles and a wave two or three, which is too few to hide
// the start (lengths, page numbers, the first K and V, each read waiting for
// the one before).  One token over 512 tokens: 10.6 us, a chain of such reads.
#include "kvc_attend_device.hpp"

#include <type_traits>

namespace kvc {
namespace {

constexpr int kTile = 32;                       // tokens a wave takes at a time

template <int D>
struct Lds {
    float o[kWaves][16][D + 4];
    float m[kWaves][16], l[kWaves][16];
};

// Waves that a SIMD can hold at once, from the registers that a wave needs:
// queries, a tile of K and of V, the sums, and about 80 for the rest, of 512
// (fewer waves rather than registers kept in memory).
constexpr int waves_of(int d, bool fp8) {
    const int need = d / 8 + 2 * (d * (fp8 ? 1 : 2) / 8) + d / 4 + 80;
    return need <= 128 ? 4 : need <= 168 ? 3 : need <= 232 ? 2 : 1;
}

// PAGE: 16, 4 or 1, the largest that divides the tokens of a page: with 16 a
// half of a tile lies in one page, its rows a constant stride apart; with 4 a
// lane's run of four V rows does.
template <int D, bool FP8, int PAGE>
__global__ __launch_bounds__(64 * kWaves, waves_of(D, FP8)) void k_attend(AttendArgs a) {
    constexpr int C = D / 16;                   // channels of V a lane holds
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int VW = C * ES / 4;              // words of them
    constexpr int KG = D * ES / 64;             // 16-byte pieces of K a lane holds of one token
    constexpr int KK = D / 32;                  // products over the channels
    __shared__ Lds<D> lds;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const uint32_t place = place_of(blockIdx.x, gridDim.x);
    const Plan plan = plan_of(a, kWaves);
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
        const Part pt = part_of(a, sh, place, at, from, end, kTile);
        at = sh.first + sh.units;               // the next item's first unit
        const int length = pt.length, ctx = pt.context, ta = pt.ta, tb = pt.tb;

        const uint32_t row_bytes = a.heads * D * ES;
        const GlobalBytes kp = reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[0])) + sh.head * (D * ES);
        const GlobalBytes vp = reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[1])) + sh.head * (D * ES);
        const int32_t* const table = a.block_table + int64_t(sh.b) * a.max_pages;

        // the query rows, as the second operand of K Q^T
        const Query query(a, sh, pt.row0 + n, pt.rows);
        bf16x8 qf[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            qf[kk] = query.at(FP8 ? 64 * (kk / 2) + 16 * q4 + 8 * (kk & 1) : 32 * kk + 8 * q4, sc.flip);

        f32x4 o[C];
        RowSum row;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = f32x4{0, 0, 0, 0};

        // Where a tile's tokens lie: with PAGE 16 the page numbers of its halves; with 4 the slots of this lane's K
        // tokens and of its two runs of V; with 1 of its V tokens.  Tokens behind the last one take a place before
        // it (a run of four its place in the last run).
        constexpr int VS = PAGE == 1 ? 8 : 2;
        struct Where {
            int32_t page[2];
            uint32_t k[2], v[VS];
        };
        auto find = [&](int t) -> Where {
            Where w;
            if constexpr (PAGE == 16) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int tok = t * kTile + hf * 16;
                    w.page[hf] = uniform_word(table + page_index(a, static_cast<uint32_t>(tok < length ? tok : length - 1)));
                }
            } else {
                auto slot = [&](int tok, int behind) {
                    const uint32_t x = static_cast<uint32_t>(tok < length ? tok : behind);
                    return slot_in(a, table[page_index(a, x)], x, &bad_page);
                };
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) w.k[hf] = slot(t * kTile + hf * 16 + n, length - 1);
#pragma unroll
                for (int j = 0; j < VS; ++j)
                    w.v[j] = PAGE == 4 ? slot(t * kTile + j * 16 + q4 * 4, (length - 1) & ~3)
                                       : slot(t * kTile + (j < 4 ? 0 : 12) + q4 * 4 + j, length - 1);
            }
            return w;
        };
        // byte offset of a half's first row in its pool
        auto half_at = [&](const Where& w, int t, int hf) -> uint64_t {
            const int tok = t * kTile + hf * 16;
            return uint64_t(slot_in(a, w.page[hf], static_cast<uint32_t>(tok < length ? tok : (length - 1) & ~15), &bad_page)) *
                   row_bytes;
        };

        // K: token n of each half; V: the eight tokens of this lane's scores
        Words<4> kw[2][KG];
        Words<VW> vw[8];
        auto load_k = [&](const Where& w, int t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const GlobalBytes p = PAGE == 16 ? kp + half_at(w, t, hf) + (uint32_t(n) * row_bytes + 16u * q4)
                                                 : kp + uint64_t(w.k[hf]) * row_bytes + 16 * q4;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) kw[hf][kg].load(p + 64 * kg);
            }
        };
        auto load_v = [&](const Where& w, int t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint64_t first = PAGE == 16 ? half_at(w, t, hf) : PAGE == 4 ? uint64_t(w.v[hf]) * row_bytes : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const GlobalBytes p = PAGE == 16 ? vp + first + (uint32_t(q4 * 4 + j) * row_bytes + uint32_t(n) * (C * ES))
                                          : PAGE == 4 ? vp + first + (uint32_t(j) * row_bytes + uint32_t(n) * (C * ES))
                                                      : vp + uint64_t(w.v[(hf * 4 + j) % VS]) * row_bytes + n * (C * ES);
                    vw[hf * 4 + j].load(p);
                }
            }
        };

        // A wave takes every fourth tile.  Its K registers are free once the scores are formed and its V registers
        // once they are summed, so the next tile's K is under way during the weights and the sum, and its V during
        // the next scores and weights.  That is the loop over tiles of context, which every row sees in full; the others
        // (and the last one) go through a second copy of the body, which knows of masks and prefetches nothing, so that the
        // first has no loads under a condition, which would be waited for with the count of the other path.
        bool any_wild = false;
        auto one_tile = [&](int t, auto inner) {
            const int t0 = t * kTile;
            Where w;
            if constexpr (inner) w = find(t + kWaves);

            // scores
            f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    bf16x8 kf;
                    if constexpr (FP8) {
                        const uint32_t lo = kw[hf][kk / 2][2 * (kk & 1)], hi = kw[hf][kk / 2][2 * (kk & 1) + 1];
                        kf = frag_of(widen<false>(lo), widen<true>(lo), widen<false>(hi), widen<true>(hi));
                    } else {
                        kf = __builtin_bit_cast(bf16x8, kw[hf][kk].v[0]);
                    }
                    s[hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[kk], s[hf], 0, 0, 0);
                }
            }
            // (held in place: started any earlier, the loads need registers of their own)
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (inner) load_k(w, t + kWaves);
            __builtin_amdgcn_sched_barrier(0);

            if (!inner && t0 + kTile > ctx) {
                const uint32_t win = static_cast<uint32_t>(window_of(a, sh.seq.start, query.node, t0 - ctx, length - ctx));
                uint32_t wild = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int x = (j < 4 ? 0 : 12) + q4 * 4 + j;
                    if (!((win >> x) & 1u)) s[j >> 2][j & 3] = kNegInf;
                    // tokens behind the last one are cleared
                    const uint32_t there = t0 + x < length ? ~0u : 0u, drafted = t0 + x >= ctx ? ~0u : 0u;
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        vw[j].set(i, vw[j][i] & there);
                        wild |= wild_bits<FP8>(vw[j][i]) & drafted;
                    }
                }
                if (__any(wild != 0)) {
                    // (of drafted tokens alone: every row sees those of the context)
                    any_wild = true;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (t0 + (j < 4 ? 0 : 12) + q4 * 4 + j < ctx) continue;
#pragma unroll
                        for (int i = 0; i < VW; ++i) vw[j].set(i, without_wild<FP8>(vw[j][i]));
                    }
                }
            }

            // weights (a NaN among the scores a row sees makes them and its sums NaN)
            const float top = larger(larger(kNegInf, s[0]), s[1]);
            if (__any(top > row.limit)) {
                const float f = row.raise(top, sc.scale, sc.slack);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] *= f;
            }
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j >> 2][j & 3], sc.scale, row.shift));
            row.sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            const bf16x8 pf = frag_of(two_bf16(e[0], e[1]), two_bf16(e[2], e[3]), two_bf16(e[4], e[5]), two_bf16(e[6], e[7]));

            // the weighted sum of V, one product for each of a lane's channels
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t f[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) f[p] = pair_of<FP8>(vw[2 * p][c * ES / 4], vw[2 * p + 1][c * ES / 4], c);
                o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag_of(f[0], f[1], f[2], f[3]), pf, o[c], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (inner) load_v(w, t + kWaves);
            __builtin_amdgcn_sched_barrier(0);
        };
        int t = ta + wave;
        if (t < tb) {
            const Where w = find(t);
            load_k(w, t);
            load_v(w, t);
            const int last = (tb - kWaves < ctx / kTile ? tb - kWaves : ctx / kTile) - 1;
            if (t <= last) {
                int left = (last - t) / kWaves + 1;
                do {
                    one_tile(t, std::true_type{});
                    t += kWaves;
                } while (--left);
            }
            for (;;) {
                one_tile(t, std::false_type{});
                t += kWaves;
                if (t >= tb) break;
                const Where v = find(t);
                load_k(v, t);
                load_v(v, t);
            }
        }

        // the four waves' sums, joined through LDS
        const float mx = row.top();
        float l = row.sum;
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (q4 == 0) {
            lds.m[wave][n] = mx;
            lds.l[wave][n] = l;
        }
        any_wild = __syncthreads_or(any_wild);
        float best = lds.m[0][n];
        for (int w = 1; w < kWaves; ++w) best = fmaxf(best, lds.m[w][n]);
        const float f = __builtin_amdgcn_exp2f(mx - (best == kNegInf ? 0.0f : best));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < C; c += 4)
                *reinterpret_cast<f32x4*>(&lds.o[wave][n][(q4 * 4 + i) * C + c]) =
                    f32x4{o[c][i], o[c + 1][i], o[c + 2][i], o[c + 3][i]} * f;
        __syncthreads();
        const int lr = threadIdx.x >> 4, part = threadIdx.x & 15;
        const int m = pt.row0 + lr;
        if (m < pt.rows) {
            best = lds.m[0][lr];
            for (int w = 1; w < kWaves; ++w) best = fmaxf(best, lds.m[w][lr]);
            const float zero = best == kNegInf ? 0.0f : best;
            float sum = 0.0f;
            for (int w = 0; w < kWaves; ++w)
                sum = __builtin_fmaf(lds.l[w][lr], __builtin_amdgcn_exp2f(lds.m[w][lr] - zero), sum);
            f32x4 acc[C / 4];
#pragma unroll
            for (int i = 0; i < C / 4; ++i) {
                acc[i] = *reinterpret_cast<const f32x4*>(&lds.o[0][lr][part * C + 4 * i]);
#pragma unroll
                for (int w = 1; w < kWaves; ++w) acc[i] += *reinterpret_cast<const f32x4*>(&lds.o[w][lr][part * C + 4 * i]);
            }
            const int node = m / static_cast<int>(a.ratio), g = m - node * static_cast<int>(a.ratio);
            if (any_wild) {
                const int last = tb * kTile < length ? tb * kTile : length;
                for (int tok = ta * kTile > ctx ? ta * kTile : ctx; tok < last; ++tok) {
                    if (!sees(a, sh.seq.start, node, static_cast<uint32_t>(tok - ctx))) continue;
                    uint32_t known = 0;
                    Words<VW> w;
                    w.load(vp + uint64_t(slot_in(a, table[page_index(a, tok)], tok, &known)) * row_bytes + part * (C * ES));
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[c / 4][c & 3] += wild_part<FP8>(w[c * ES / 4], c);
                }
            }
            if (pt.whole) {
                const int64_t out_row = int64_t(sh.seq.start) + node;
                const int64_t head = int64_t(sh.head) * a.ratio + g;
                const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
                uint16_t* const out = a.out + out_row * a.out_row + head * D + part * C;
#pragma unroll
                for (int i = 0; i < C / 4; ++i)
                    *reinterpret_cast<uint2*>(out + 4 * i) =
                        uint2{two_bf16(acc[i][0] * inv, acc[i][1] * inv), two_bf16(acc[i][2] * inv, acc[i][3] * inv)};
                if (a.lse && part == 0)
                    a.lse[out_row * (int64_t(a.heads) * a.ratio) + head] =
                        sum == 0.0f ? kNegInf : (best + __builtin_amdgcn_logf(sum)) * kLn2;
            } else {
                const uint64_t to = uint64_t(pt.slot) * 16 + lr;
#pragma unroll
                for (int i = 0; i < C / 4; ++i)
                    *reinterpret_cast<f32x4*>(a.partial + to * D + part * C + 4 * i) = acc[i];
                if (part == 0) *reinterpret_cast<float2*>(a.pairs + 2 * to) = float2{best, sum};
            }
        }
        __syncthreads();                        // the next item's sums go to the same place
    }
    const uint32_t any = __syncthreads_or(static_cast<int>(bad_page));
    if (threadIdx.x == 0) a.words[blockIdx.x] = any ? kPagedInvalid : 0u;
}

// ---------------------------------------------------------------- the join

// The last of `batch` sequences that starts at or before a row: 64 starts at
// a time, one load where the batch is no larger.
__device__ uint32_t sequence_of(const int32_t* starts, uint32_t batch, uint32_t row, uint32_t lane) {
    uint32_t lo = 0, n = batch;                 // it is among [lo, lo + n)
    for (;;) {
        const uint32_t step = (n + 63) / 64;
        const uint32_t i = lane * step;
        const uint64_t who = __ballot(i < n && starts[lo + i] <= static_cast<int32_t>(row));
        const uint32_t last = who ? 63 - __builtin_clzll(who) : 0;
        if (step == 1) return lo + last;
        lo += last * step;
        n = n - last * step < step ? n - last * step : step;
    }
}

// x w + y; an infinity stays one where its weight is too small for a float32,
// as the drafted tokens' do that a part had added to it.
__device__ inline float weighted(float x, float w, float y) {
    return __builtin_isinf(x) ? x + y : __builtin_fmaf(x, w, y);
}

// Joins the parts of split items, by the formula above: one wave a (row,
// query head).  N parts at a time, read before their weights are known, so
// that a row costs two trips to memory (its place, its parts), which is what
// bounds it: 4 to 11 us.
template <int D>
struct Joined {
    static constexpr int E = D / 64;
    float top = kNegInf, sum = 0.0f, o[E] = {};

    template <int N, typename Place>
    __device__ void add(const AttendArgs& a, uint32_t lane, uint32_t parts, const Place& place) {
        for (uint32_t s0 = 0; s0 < parts; s0 += N) {
            float v[N][E];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float* const p = a.partial + place(s0 + i < parts ? s0 + i : s0) * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = p[e];
            }
            float2 x{kNegInf, 0.0f};
            if (lane < N && s0 + lane < parts) x = *reinterpret_cast<const float2*>(a.pairs + 2 * place(s0 + lane));
            float best = x.x;
            for (int d = N / 2; d; d >>= 1) best = fmaxf(best, __shfl_xor(best, d));
            best = fmaxf(top, __shfl(best, 0));
            const float zero = best == kNegInf ? 0.0f : best;
            const float old = __builtin_amdgcn_exp2f(top - zero), f = __builtin_amdgcn_exp2f(x.x - zero);
            float l = x.y * f;
            for (int d = N / 2; d; d >>= 1) l += __shfl_xor(l, d);
            sum = __builtin_fmaf(sum, old, __shfl(l, 0));
            top = best;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = weighted(o[e], old, 0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (s0 + i < parts) {
                    const float w = __shfl(f, i);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = weighted(v[i][e], w, o[e]);
                }
            }
        }
    }
};

// each: (row, query head) pairs of a wave, one after the other.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a, uint32_t grid, uint32_t each) {
    constexpr int E = D / 64;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t heads = a.heads * a.ratio;
    const uint32_t first_id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6)) * each;
    const uint32_t per = a.ctl->per;
    const bool aligned = a.ctl->aligned;
    int32_t start = 0, next = 0;                // of the sequence that `span` is of
    AttendSpan span{};
    uint32_t row = first_id / heads, head = first_id - row * heads;
    for (uint32_t i = 0; i < each && row < a.rows; ++i, head = head + 1 < heads ? head + 1 : 0, row += head ? 0 : 1) {
        if (static_cast<int32_t>(row) >= next) {
            const uint32_t b = sequence_of(a.row_starts, a.batch, row, lane);
            start = a.row_starts[b];
            next = a.row_starts[b + 1];
            span = a.spans[b];
        }
        // (outside any sequence, or of one whose items nobody shares)
        if (static_cast<int32_t>(row) < start || static_cast<int32_t>(row) >= next || (aligned && span.units <= per)) continue;
        const uint32_t h = head / a.ratio, m = (row - static_cast<uint32_t>(start)) * a.ratio + (head - h * a.ratio);
        const uint32_t tile = m >> a.tile_shift;
        if (tile >= span.tiles) continue;
        const uint32_t first = span.base + (h * span.tiles + tile) * span.units;
        const Sharers who = sharers_of(first, span.units, per);
        if (who.first >= who.last || who.last >= grid) continue;
        const uint32_t parts = who.last - who.first + 1;
        const uint32_t lr = m - (tile << a.tile_shift);
        auto place = [&](uint32_t s) { return (uint64_t(who.slot(s)) << a.tile_shift) + lr; };
        Joined<D> j;
        if (parts <= 4) j.template add<4>(a, lane, parts, place);
        else j.template add<E <= 2 ? 16 : 8>(a, lane, parts, place);
        const float inv = j.sum == 0.0f ? 0.0f : a.v_scale / j.sum;
        uint16_t* const out = a.out + int64_t(row) * a.out_row + int64_t(head) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) out[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(j.o[e] * inv));
        if (a.lse && lane == 0)
            a.lse[int64_t(row) * heads + head] = j.sum == 0.0f ? kNegInf : (j.top + __builtin_amdgcn_logf(j.sum)) * kLn2;
    }
}

template <int D>
hipError_t launch_channels(const AttendArgs& a, const AttendShape& sh, bool fp8, hipStream_t s) {
    if (sh.wide) {
        const hipError_t e = launch_attend_wide(a, sh, D, fp8, s);
        if (e != hipSuccess) return e;
    } else if (a.page_tokens % 16 == 0) {
        if (fp8) k_attend<D, true, 16><<<sh.grid, 64 * kWaves, 0, s>>>(a);
        else k_attend<D, false, 16><<<sh.grid, 64 * kWaves, 0, s>>>(a);
    } else if (a.page_tokens % 4 == 0) {
        if (fp8) k_attend<D, true, 4><<<sh.grid, 64 * kWaves, 0, s>>>(a);
        else k_attend<D, false, 4><<<sh.grid, 64 * kWaves, 0, s>>>(a);
    } else {
        if (fp8) k_attend<D, true, 1><<<sh.grid, 64 * kWaves, 0, s>>>(a);
        else k_attend<D, false, 1><<<sh.grid, 64 * kWaves, 0, s>>>(a);
    }
    if (sh.split) {
        // at most as many waves as the chip holds at once: where nothing was split, more of them than that only to
        // find it out cost a prompt of 2000 rows 15 us
        const uint64_t pairs = uint64_t(a.rows) * a.heads * a.ratio;
        const uint64_t each = (pairs + 8191) / 8192, waves = (pairs + each - 1) / each;
        k_attend_join<D><<<static_cast<uint32_t>((waves + 3) / 4), 256, 0, s>>>(a, sh.grid, static_cast<uint32_t>(each));
    }
    return hipGetLastError();
}

}  // namespace

AttendShape attend_shape(int64_t batch, int64_t heads, int64_t ratio, int64_t channels, bool fp8, int64_t rows,
                         int64_t rows_per_sequence, int64_t max_tokens, int64_t widest) {
    AttendShape s;
    const int64_t usual = (rows_per_sequence > 0 ? rows_per_sequence : (rows + batch - 1) / batch) * ratio;
    s.wide = usual > 16;
    // Two groups of 16 rows a wave halve the reads of LDS for a product.  Beyond 128 channels their sums leave room for
    // one workgroup a CU, and two workgroups of one group a wave are faster, where LDS holds one tile each instead of
    // two (two pieces of 1000 tokens over 7001 with 192 channels: bf16 997 and 767 us, e4m3 781 and 620; with 256 and one
    // workgroup 1287, two 839).  In bf16 that second workgroup is paid for with registers, so that up to 64 rows, which
    // wait for K and V, keep one (two sequences of 32000 tokens, 192 channels: 56 and 62 us, 256: 67 and 80; but 32 of up
    // to 4096, 192 channels: 124 and 103); e4m3 gains there, or loses nothing (67 and 49; 52 and 53; 135 and 78).  A third
    // workgroup by the same means, e4m3 of 128 channels: 57 and 49 us, but with 4 sequences 26 and 29.
    s.row_tiles = !s.wide || usual <= 64 || channels > 128 ? 1 : 2;
    s.lds_tiles = channels > 128 && (fp8 || usual > 64) ? 1 : 2;
    s.tile_shift = !s.wide ? 4 : s.row_tiles == 1 ? 6 : 7;
    // Long sequences are split.  Of short ones each item gets a workgroup and no join is launched (one token over 512
    // tokens: 10.2 us instead of 12.4; 200 sequences of up to 500: 52 instead of 92); but each reads the lengths up to
    // its own, so that many sequences are dealt to fewer workgroups, which go on where they are (1000 sequences of up
    // to 300 tokens: 308 us and dealt 223, with six drafted tokens each 387 and 256; 4000 of up to 100: 2117 and 490,
    // with six 578).
    // (A launch has fewer than 2^32 threads.)
    const uint64_t tile_rows = uint64_t(1) << s.tile_shift;
    const uint64_t items = attend_items(batch, heads, ratio, rows, tile_rows);
    s.split = max_tokens > (s.wide ? 512 : 1024) || batch > 1024 || items >= uint64_t(1) << 24;
    // ends at 31 at the latest: items < kMaxItems, widest <= kMaxTokens
    s.unit_shift = s.wide ? 6 : 5;
    while (items * ((uint64_t(widest) >> s.unit_shift) + 1) >= kMaxItems) ++s.unit_shift;
    uint64_t grid = items;
    if (s.split) grid = 256u * (s.wide ? wide_groups(channels, fp8, s.row_tiles, s.lds_tiles) : waves_of(static_cast<int>(channels), fp8));
    if (grid < 1) grid = 1;
    s.grid = static_cast<uint32_t>(grid);
    const auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
    s.spans = 256;
    s.words = up(s.spans + uint64_t(batch) * sizeof(AttendSpan));
    s.pairs = up(s.words + 4 * grid);
    s.partial = up(s.pairs + (s.split ? 16 * grid * tile_rows : 0));
    s.total = up(s.partial + (s.split ? 8 * grid * tile_rows * channels : 0));
    return s;
}

hipError_t launch_attend(const AttendArgs& args, const AttendShape& sh, int64_t channels, bool fp8, hipStream_t s) {
    AttendArgs a = args;
    set_page_product(a.page_tokens, &a.page_mul, &a.page_shift);
    if (a.rows == 0) {                          // nothing to compute, but the outcome
        k_attend<64, false, 1><<<1, 64 * kWaves, 0, s>>>(a);
        return hipGetLastError();
    }
    switch (channels) {
        case 64: return launch_channels<64>(a, sh, fp8, s);
        case 128: return launch_channels<128>(a, sh, fp8, s);
        case 192: return launch_channels<192>(a, sh, fp8, s);
        case 256: return launch_channels<256>(a, sh, fp8, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace kvc
