// Attention of drafted tokens over a paged cache (kvc_paged_attention in
// include/kvc.h).
//
// A workgroup takes the query rows of one KV head of one sequence (its rows
// are (drafted token, query head of the group) pairs: all read the same K and
// V) and a range of the sequence's tokens.  One pass over the range keeps, for
// each row, the running maximum m of its scores (in units of log 2), the sum l
// of 2^(s - m) and the weighted sum o of V; ranges are joined by
//     m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),
// first the four waves of the workgroup (which take tiles of 32 tokens in
// turn) through LDS, then the workgroups of a sequence through a second,
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
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kvc_paged.hpp"

namespace kvc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kTile = 32;                       // tokens a wave takes at a time
constexpr float kNegInf = -__builtin_inff();

// ---------------------------------------------------------------- the split

struct Seq {
    int32_t start, rows, context;               // rows 0: nothing to compute
    bool bad;
};

__device__ Seq seq_of(const AttendArgs& a, uint32_t b) {
    Seq s;
    s.start = a.row_starts[b];
    const int64_t end = a.row_starts[b + 1];
    s.context = a.context ? a.context[b] : 0;
    const int64_t n = end - s.start;
    s.bad = s.start < 0 || n < 0 || end > int64_t(a.rows) || s.context < 0 ||
            s.context + n > a.max_pages * int64_t(a.page_tokens) || s.context + n > 0x7FFFFF00;
    s.rows = s.bad ? 0 : static_cast<int32_t>(n);
    return s;
}

template <typename T>
__device__ T wave_sum(T x) {
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// What workgroup `id` computes: rows [row0, row0 + 16 RT) of the M = n x ratio
// rows of KV head `head` of a sequence, over part `split` of `splits`.
struct Share {
    bool any;
    Seq seq;
    uint32_t b, head, tile, split, splits;
};

// Every wave finds its share from the lengths (no launch of its own for a
// plan, nothing kept between calls): sequence b has heads x tiles_b items of
// u_b token tiles, and each is split evenly into ceil(u_b / per) parts, where
// `per` is such that the parts of all items fill the chip's `target`
// workgroups about once; parts of one item are heads x tiles_b workgroups
// apart, and a KV head's row tiles `heads` apart, so that with eight heads
// those that read the same K and V run on one XCD.  Workgroup 0 writes the
// spans and the flags.
__device__ Share share_of(const AttendArgs& a, uint32_t id, uint32_t tile_rows, uint32_t grid) {
    const uint32_t lane = threadIdx.x & 63;
    uint64_t units = 0, items = 0;
    bool bad = false;
    uint32_t tiles0 = 0, u0 = 0;
    Seq seq0{};
    for (uint32_t b0 = 0; b0 < a.batch; b0 += 64) {
        const uint32_t b = b0 + lane;
        uint32_t tiles = 0, u = 0;
        Seq s{};
        if (b < a.batch) {
            s = seq_of(a, b);
            bad = bad || s.bad;
            tiles = (uint32_t(s.rows) * a.ratio + tile_rows - 1) / tile_rows;
            u = (uint32_t(s.context + s.rows) + kTile - 1) / kTile;
        }
        if (b0 == 0) {
            tiles0 = tiles;
            u0 = u;
            seq0 = s;
        }
        items += uint64_t(tiles) * a.heads;
        units += uint64_t(tiles) * a.heads * u;
    }
    items = wave_sum(items);
    units = wave_sum(units);
    uint32_t per = 0x7FFFFFFFu;
    if (a.split) {
        const uint32_t half = a.target / 2;
        const uint32_t parts = items < half ? a.target - static_cast<uint32_t>(items) : half;
        const float want = float(units) / float(parts) + 1.0f;
        // whole rounds of the four waves
        per = want > 2e9f ? 2000000000u : (static_cast<uint32_t>(want) + kWaves - 1) / kWaves * kWaves;
    }
    Share r{};
    uint64_t base = 0;
    for (uint32_t b0 = 0; b0 < a.batch; b0 += 64) {
        const uint32_t b = b0 + lane;
        uint32_t tiles = tiles0, u = u0;
        Seq s = seq0;
        if (b0) {
            tiles = u = 0;
            s = Seq{};
            if (b < a.batch) {
                s = seq_of(a, b);
                tiles = (uint32_t(s.rows) * a.ratio + tile_rows - 1) / tile_rows;
                u = (uint32_t(s.context + s.rows) + kTile - 1) / kTile;
            }
        }
        const uint32_t splits = tiles ? (u + per - 1) / per : 0u;
        const uint64_t count = uint64_t(splits) * tiles * a.heads;
        uint64_t end = count;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint64_t x = __shfl_up(end, d);
            if (lane >= d) end += x;
        }
        end += base;
        const bool over = end > grid;           // row starts that are no prefix sums
        if (id == 0 && threadIdx.x < 64 && b < a.batch) {
            bad = bad || (count && over);
            a.spans[b] = AttendSpan{static_cast<uint32_t>(end - count), over ? 0u : splits, tiles, 0u};
        }
        const bool mine = count && !over && id >= end - count && id < end;
        const uint64_t who = __ballot(mine);
        if (who) {
            const int l = __builtin_ctzll(who);
            r.any = true;
            r.b = b0 + l;
            r.seq.start = __shfl(s.start, l);
            r.seq.rows = __shfl(s.rows, l);
            r.seq.context = __shfl(s.context, l);
            const uint32_t t = __shfl(tiles, l);
            r.splits = __shfl(splits, l);
            uint32_t rest = id - static_cast<uint32_t>(__shfl(end - count, l));
            r.head = rest % a.heads;
            rest /= a.heads;
            r.tile = rest % t;
            r.split = rest / t;
            if (id) break;
        }
        base = __shfl(end, 63);
        if (id && base > id) break;
    }
    if (id == 0 && threadIdx.x < 64) {
        bad = __any(bad);
        if (lane == 0) {
            a.ctl->magic = kPagedMagic;
            a.ctl->flags = bad ? kPagedInvalid : 0u;
            a.ctl->grid = grid;
            a.ctl->words_offset =
                static_cast<uint32_t>(reinterpret_cast<char*>(a.words) - reinterpret_cast<char*>(a.ctl));
        }
    }
    r.b = __builtin_amdgcn_readfirstlane(r.b);
    r.seq.start = __builtin_amdgcn_readfirstlane(r.seq.start);
    r.seq.rows = __builtin_amdgcn_readfirstlane(r.seq.rows);
    r.seq.context = __builtin_amdgcn_readfirstlane(r.seq.context);
    r.head = __builtin_amdgcn_readfirstlane(r.head);
    r.tile = __builtin_amdgcn_readfirstlane(r.tile);
    r.split = __builtin_amdgcn_readfirstlane(r.split);
    r.splits = __builtin_amdgcn_readfirstlane(r.splits);
    return r;
}

// ---------------------------------------------------------------- fragments

__device__ bf16x8 frag_of(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Two of the four e4m3 values of a word (its low or high half) as bf16: exact.
template <bool HIGH>
__device__ uint32_t widen(uint32_t four) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, HIGH));
}

// The pools' addresses are read from memory: that they are global ones has
// to be said.
#define GLOBAL __attribute__((address_space(1)))
typedef const GLOBAL uint8_t* GlobalBytes;

// WORDS 32-bit words, in the vectors that they are loaded as: kept whole,
// they stay in the registers that the loads write.
template <int WORDS>
struct Words {
    static constexpr int W = WORDS % 4 == 0 ? 4 : WORDS % 2 == 0 ? 2 : 1;
    typedef uint32_t Vec __attribute__((ext_vector_type(W)));
    Vec v[WORDS / W];

    __device__ uint32_t operator[](int i) const { return v[i / W][i % W]; }
    __device__ void set(int i, uint32_t x) { v[i / W][i % W] = x; }
    __device__ void load(GlobalBytes p) {
#pragma unroll
        for (int i = 0; i < WORDS / W; ++i) v[i] = *reinterpret_cast<const GLOBAL Vec*>(p + 4 * W * i);
    }
};

__device__ uint32_t two_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

// Infinities and NaN among a word's values (two bf16; four e4m3, which has
// no infinity): the top bit of each value's place is set where it is one.
__device__ bool wild_half(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

template <bool FP8>
__device__ uint32_t wild_bits(uint32_t w) {
    return FP8 ? ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

template <bool FP8>
__device__ uint32_t without_wild(uint32_t w) {
    return w & ~(FP8 ? (wild_bits<true>(w) >> 7) * 0xFFu : (wild_bits<false>(w) >> 15) * 0xFFFFu);
}

// Value c of words (w is its word) if it is an infinity or a NaN, else zero.
template <bool FP8>
__device__ float wild_part(uint32_t w, int c) {
    if constexpr (FP8) return ((w >> (8 * (c & 3))) & 0x7Fu) == 0x7Fu ? __builtin_nanf("") : 0.0f;
    const uint32_t h = (c & 1) ? w >> 16 : w;
    return wild_half(h) ? __uint_as_float(h << 16) : 0.0f;
}

// ---------------------------------------------------------------- the kernel

template <int D, bool FP8, int RT>
struct Lds {
    float o[kWaves][16][D + 4];
    float m[kWaves][16 * RT], l[kWaves][16 * RT];
};

// Words read through the scalar cache: they are not written while the kernel
// runs, and every lane wants the same ones.
__device__ int32_t uniform_word(const int32_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p));
}

// The largest of the four lanes n, n + 16, n + 32, n + 48.
__device__ float top_of_column(float x) {
    u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Waves that a SIMD can hold at once, from the registers that a wave needs:
// queries, a tile of K and of V, the sums, scores and weights, and about 50
// for the rest, of 512.
constexpr int waves_of(int d, bool fp8, int rt) {
    const int need = d * rt / 8 + 2 * (d * (fp8 ? 1 : 2) / 8) + d * rt / 4 + 12 * rt + 44;
    return need <= 128 ? 4 : need <= 168 ? 3 : need <= 256 ? 2 : 1;
}

// PAGE16: pages are a multiple of 16 tokens, so that a half of a tile lies in
// one page and its rows are a constant stride apart.
template <int D, bool FP8, int RT, bool PAGE16>
__global__ __launch_bounds__(64 * kWaves, waves_of(D, FP8, RT)) void k_attend(AttendArgs a) {
    constexpr int C = D / 16;                   // channels of V a lane holds
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int VW = C * ES / 4;              // words of them
    constexpr int KG = D * ES / 64;             // 16-byte pieces of K a lane holds of one token
    constexpr int KK = D / 32;                  // products over the channels
    __shared__ Lds<D, FP8, RT> lds;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const Share sh = share_of(a, blockIdx.x, 16 * RT, gridDim.x);
    uint32_t bad_page = 0;
    if (sh.any) {
        const int rows = sh.seq.rows * static_cast<int>(a.ratio);    // M
        const int row0 = static_cast<int>(sh.tile) * 16 * RT;
        const int ctx = sh.seq.context;
        // a chain's rows see nothing behind their last token
        const int last_row = (row0 + 16 * RT < rows ? row0 + 16 * RT : rows) - 1;
        const int seen = a.mask ? sh.seq.rows : last_row / static_cast<int>(a.ratio) + 1;
        const int length = ctx + seen;
        const uint32_t tiles = (static_cast<uint32_t>(length) + kTile - 1) / kTile;
        const int ta = static_cast<int>(uint64_t(tiles) * sh.split / sh.splits);
        const int tb = static_cast<int>(uint64_t(tiles) * (sh.split + 1) / sh.splits);

        const uint32_t num_pages = static_cast<uint32_t>(a.num_pages);     // x page_tokens < 2^31
        const uint32_t row_bytes = a.heads * D * ES;
        const GlobalBytes kp = reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[0])) + sh.head * (D * ES);
        const GlobalBytes vp = reinterpret_cast<GlobalBytes>(reinterpret_cast<uintptr_t>(a.pools[1])) + sh.head * (D * ES);
        const int32_t* const table = a.block_table + int64_t(sh.b) * a.max_pages;

        // The query rows, as the second operand of K Q^T.  The scale is made positive by their sign, so that the
        // largest scaled score is the scaled largest score; a scale of zero becomes the smallest one.
        const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
        const float scale = fmaxf(fabsf(a.scale_log2), 0x1p-126f);
        bf16x8 qf[RT][KK];
        int node[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int m = row0 + rt * 16 + n;
            const bool real = m < rows;
            node[rt] = real ? m / static_cast<int>(a.ratio) : 0;
            const int g = real ? m - node[rt] * static_cast<int>(a.ratio) : 0;
            const uint16_t* const q =
                a.q + (int64_t(sh.seq.start) + node[rt]) * a.q_row + (int64_t(sh.head) * a.ratio + g) * a.q_head;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int ch = FP8 ? 64 * (kk / 2) + 16 * q4 + 8 * (kk & 1) : 32 * kk + 8 * q4;
                const uint4 x = real ? *reinterpret_cast<const uint4*>(q + ch) : uint4{0, 0, 0, 0};
                qf[rt][kk] = frag_of(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
            }
        }

        f32x4 o[RT][C];
        float mx[RT], l[RT];                    // mx: of the scores before their scale
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            mx[rt] = kNegInf;
            l[rt] = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[rt][c] = f32x4{0, 0, 0, 0};
        }

        // Where a tile's tokens lie: with PAGE16 the page numbers of its halves, otherwise this lane's slot (page x
        // page_tokens + row of token lane % 32).  Tokens behind the last one take its place.
        struct Where {
            int32_t page[2];
            uint32_t slot;
        };
        auto find = [&](int t) -> Where {
            Where w{};
            if constexpr (PAGE16) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int at = t * kTile + hf * 16;
                    const uint32_t tok = static_cast<uint32_t>(at < length ? at : length - 1);
                    w.page[hf] = uniform_word(table + ((uint64_t(tok) * a.page_mul) >> a.page_shift));
                }
            } else {
                const int at = t * kTile + (lane & 31);
                const uint32_t tok = static_cast<uint32_t>(at < length ? at : length - 1);
                const uint32_t j = static_cast<uint32_t>((uint64_t(tok) * a.page_mul) >> a.page_shift);
                uint32_t page = static_cast<uint32_t>(table[j]);
                if (page >= num_pages) {
                    bad_page = kPagedInvalid;
                    page = 0;
                }
                w.slot = page * a.page_tokens + (tok - j * a.page_tokens);
            }
            return w;
        };
        // byte offset of a half's first row in its pool
        auto half_at = [&](const Where& w, int t, int hf) -> uint64_t {
            const int at = t * kTile + hf * 16;
            const uint32_t tok = static_cast<uint32_t>(at < length ? at : (length - 1) & ~15);
            const uint32_t j = static_cast<uint32_t>((uint64_t(tok) * a.page_mul) >> a.page_shift);
            uint32_t page = static_cast<uint32_t>(w.page[hf]);
            if (page >= num_pages) {
                bad_page = kPagedInvalid;
                page = 0;
            }
            return uint64_t(page * a.page_tokens + (tok - j * a.page_tokens)) * row_bytes;
        };

        // K: token n of each half; V: the eight tokens of this lane's scores
        Words<4> kw[2][KG];
        Words<VW> vw[8];
        auto load_k = [&](const Where& w, int t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const GlobalBytes p = PAGE16
                    ? kp + half_at(w, t, hf) + (uint32_t(n) * row_bytes + 16u * q4)
                    : kp + uint64_t(__shfl(w.slot, hf * 16 + n)) * row_bytes + 16 * q4;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) kw[hf][kg].load(p + 64 * kg);
            }
        };
        auto load_v = [&](const Where& w, int t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint64_t at = PAGE16 ? half_at(w, t, hf) : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const GlobalBytes p = PAGE16
                        ? vp + at + (uint32_t(q4 * 4 + j) * row_bytes + uint32_t(n) * (C * ES))
                        : vp + uint64_t(__shfl(w.slot, hf * 16 + q4 * 4 + j)) * row_bytes + n * (C * ES);
                    vw[hf * 4 + j].load(p);
                }
            }
        };

        // A wave takes every fourth tile.  Its K registers are free once the scores are formed and its V registers
        // once they are summed, so the next tile's K is under way during the weights and the sum, and its V during
        // the next scores and weights.  That is the loop over tiles that every row sees in full; the others (and the
        // last one) go through a second copy of the body, which knows of masks and prefetches nothing, so that the
        // first has no loads under a condition, which would be waited for with the count of the other path.
        const int full = ctx + (a.mask ? 0 : row0 / static_cast<int>(a.ratio) + 1);
        bool any_wild = false;
        auto one_tile = [&](int t, auto inner) {
            const int t0 = t * kTile;
            const int next = t + kWaves;
            Where w{};
            if constexpr (inner) w = find(next);

            // scores
            f32x4 s[RT][2];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0, 0, 0, 0};
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
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        s[rt][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][kk], s[rt][hf], 0, 0, 0);
                }
            }
            // (held in place: started any earlier, the loads need registers of their own)
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (inner) load_k(w, next);
            __builtin_amdgcn_sched_barrier(0);

            // What a row sees of a tile is a window of 32 bits.  V values of unseen tokens meet weights of zero, which
            // an infinity or a NaN would turn into NaN: tokens behind the last are cleared, and so are such values of
            // drafted ones; they are added at the end to the rows that see them.
            if (!inner && t0 + kTile > full) {
                uint32_t wild = 0;
                const int j0 = t0 - ctx;                              // > -32
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    uint32_t w32;
                    if (a.mask) {
                        const uint64_t* const bits =
                            a.mask + (int64_t(sh.seq.start) + node[rt]) * a.mask_words;
                        if (j0 < 0) {
                            w32 = (static_cast<uint32_t>(bits[0]) << -j0) | ((1u << -j0) - 1u);
                        } else {
                            const uint32_t at = static_cast<uint32_t>(j0) >> 6, by = j0 & 63;
                            uint64_t x = at < a.mask_words ? bits[at] >> by : 0u;
                            if (by > 32 && at + 1 < a.mask_words) x |= bits[at + 1] << (64 - by);
                            w32 = static_cast<uint32_t>(x);
                        }
                        const int there = sh.seq.rows - j0;           // >= 1
                        if (there < 32) w32 &= (1u << there) - 1u;
                    } else {
                        const int see = node[rt] - j0 + 1;
                        w32 = see >= 32 ? 0xFFFFFFFFu : see <= 0 ? 0u : (1u << see) - 1u;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (!((w32 >> ((j < 4 ? 0 : 12) + q4 * 4 + j)) & 1u)) s[rt][j >> 2][j & 3] = kNegInf;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int tok = t0 + (j < 4 ? 0 : 12) + q4 * 4 + j;
                    const uint32_t there = tok < length ? ~0u : 0u, drafted = tok >= ctx ? ~0u : 0u;
#pragma unroll
                    for (int x = 0; x < VW; ++x) {
                        vw[j].set(x, vw[j][x] & there);
                        wild |= wild_bits<FP8>(vw[j][x]) & drafted;
                    }
                }
                if (__any(wild != 0)) {
                    any_wild = true;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int x = 0; x < VW; ++x) vw[j].set(x, without_wild<FP8>(vw[j][x]));
                }
            }

            // weights 2^(scale (s - max))
            bf16x8 pf[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 x = s[rt][0], y = s[rt][1];
                float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
                top = fmaxf(top_of_column(top), mx[rt]);
                const float zero = top == kNegInf ? 0.0f : top;
                if (__any(top > mx[rt])) {
                    const float f = __builtin_amdgcn_exp2f((mx[rt] - zero) * scale);
                    l[rt] *= f;
#pragma unroll
                    for (int c = 0; c < C; ++c) o[rt][c] *= f;
                    mx[rt] = top;
                }
                const float shift = -zero * scale;
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j >> 2][j & 3], scale, shift));
                l[rt] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                pf[rt] = frag_of(two_bf16(e[0], e[1]), two_bf16(e[2], e[3]), two_bf16(e[4], e[5]), two_bf16(e[6], e[7]));
            }

            // the weighted sum of V, one product for each of a lane's channels
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t f[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int x = c * ES / 4;
                    if constexpr (FP8) {
                        const uint32_t pair = (c & 2) ? __builtin_amdgcn_perm(vw[2 * p + 1][x], vw[2 * p][x], 0x07030602u)
                                                      : __builtin_amdgcn_perm(vw[2 * p + 1][x], vw[2 * p][x], 0x05010400u);
                        f[p] = (c & 1) ? widen<true>(pair) : widen<false>(pair);
                    } else {
                        f[p] = (c & 1) ? __builtin_amdgcn_perm(vw[2 * p + 1][x], vw[2 * p][x], 0x07060302u)
                                       : __builtin_amdgcn_perm(vw[2 * p + 1][x], vw[2 * p][x], 0x05040100u);
                    }
                }
                const bf16x8 vf = frag_of(f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    o[rt][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt], o[rt][c], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (inner) load_v(w, next);
            __builtin_amdgcn_sched_barrier(0);
        };
        int t = ta + wave;
        if (t < tb) {
            const Where w = find(t);
            load_k(w, t);
            load_v(w, t);
            const int last = (tb - kWaves < full / kTile ? tb - kWaves : full / kTile) - 1;
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

        // from here on the maxima are of the scaled scores
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) mx[rt] *= scale;

        // the four waves' sums, joined through LDS
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            l[rt] += __shfl_xor(l[rt], 16);
            l[rt] += __shfl_xor(l[rt], 32);
            if (q4 == 0) {
                lds.m[wave][rt * 16 + n] = mx[rt];
                lds.l[wave][rt * 16 + n] = l[rt];
            }
        }
        any_wild = __syncthreads_or(any_wild);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = lds.m[0][rt * 16 + n];
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds.m[w][rt * 16 + n]);
            const float f = __builtin_amdgcn_exp2f(mx[rt] - (top == kNegInf ? 0.0f : top));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < C; c += 4)
                    *reinterpret_cast<f32x4*>(&lds.o[wave][n][(q4 * 4 + i) * C + c]) =
                        f32x4{o[rt][c][i], o[rt][c + 1][i], o[rt][c + 2][i], o[rt][c + 3][i]} * f;
            __syncthreads();
            const int lr = threadIdx.x >> 4, part = threadIdx.x & 15;
            const int m = row0 + rt * 16 + lr;
            if (m < rows) {
                float best = lds.m[0][rt * 16 + lr];
                for (int w = 1; w < kWaves; ++w) best = fmaxf(best, lds.m[w][rt * 16 + lr]);
                const float zero = best == kNegInf ? 0.0f : best;
                float sum = 0.0f;
                for (int w = 0; w < kWaves; ++w)
                    sum = __builtin_fmaf(lds.l[w][rt * 16 + lr], __builtin_amdgcn_exp2f(lds.m[w][rt * 16 + lr] - zero), sum);
                f32x4 acc[C / 4];
#pragma unroll
                for (int i = 0; i < C / 4; ++i) {
                    acc[i] = *reinterpret_cast<const f32x4*>(&lds.o[0][lr][part * C + 4 * i]);
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        acc[i] += *reinterpret_cast<const f32x4*>(&lds.o[w][lr][part * C + 4 * i]);
                }
                if (any_wild) {
                    // an infinity or a NaN in V is what it makes of every row that sees its token
                    const int nd = m / static_cast<int>(a.ratio);
                    const int end = tb * kTile < length ? tb * kTile : length;
                    for (int tok = ta * kTile > ctx ? ta * kTile : ctx; tok < end; ++tok) {
                        const uint32_t j = static_cast<uint32_t>(tok - ctx);
                        const uint64_t* const bits = a.mask + (int64_t(sh.seq.start) + nd) * a.mask_words;
                        if (a.mask ? j / 64 >= a.mask_words || !((bits[j / 64] >> (j & 63)) & 1u)
                                   : static_cast<int>(j) > nd)
                            continue;
                        const uint32_t at = static_cast<uint32_t>((uint64_t(uint32_t(tok)) * a.page_mul) >> a.page_shift);
                        uint32_t page = static_cast<uint32_t>(table[at]);
                        if (page >= num_pages) page = 0;
                        const uint64_t slot = page * a.page_tokens + (uint32_t(tok) - at * a.page_tokens);
                        Words<VW> w;
                        w.load(vp + slot * row_bytes + part * (C * ES));
#pragma unroll
                        for (int c = 0; c < C; ++c) acc[c / 4][c & 3] += wild_part<FP8>(w[c * ES / 4], c);
                    }
                }
                if (sh.splits == 1) {
                    const int nd = m / static_cast<int>(a.ratio), g = m - nd * static_cast<int>(a.ratio);
                    const int64_t row = int64_t(sh.seq.start) + nd;
                    const int64_t head = int64_t(sh.head) * a.ratio + g;
                    const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
                    uint16_t* const out = a.out + row * a.out_row + head * D + part * C;
#pragma unroll
                    for (int i = 0; i < C / 4; ++i)
                        *reinterpret_cast<uint2*>(out + 4 * i) = uint2{two_bf16(acc[i][0] * inv, acc[i][1] * inv),
                                                                       two_bf16(acc[i][2] * inv, acc[i][3] * inv)};
                    if (a.lse && part == 0)
                        a.lse[row * (int64_t(a.heads) * a.ratio) + head] =
                            sum == 0.0f ? kNegInf : (best + __builtin_amdgcn_logf(sum)) * 0.69314718056f;
                } else {
                    const int64_t at = int64_t(blockIdx.x) * (16 * RT) + rt * 16 + lr;
#pragma unroll
                    for (int i = 0; i < C / 4; ++i)
                        *reinterpret_cast<f32x4*>(a.partial + at * D + part * C + 4 * i) = acc[i];
                    if (part == 0) *reinterpret_cast<float2*>(a.pairs + 2 * at) = float2{best, sum};
                }
            }
            if (rt + 1 < RT) __syncthreads();
        }
    }
    const uint32_t any = __syncthreads_or(static_cast<int>(bad_page));
    if (threadIdx.x == 0) a.words[blockIdx.x] = any ? kPagedInvalid : 0u;
}

// Joins the parts of split sequences: one wave a (row, query head).
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a, uint32_t tile_rows) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const uint32_t heads = a.heads * a.ratio;
    const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const uint32_t row = id / heads, head = id - row * heads;
    if (row >= a.rows) return;
    uint32_t lo = 0, hi = a.batch - 1;          // the last sequence that starts at or before the row
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (a.row_starts[mid] <= static_cast<int32_t>(row)) lo = mid;
        else hi = mid - 1;
    }
    const int32_t start = a.row_starts[lo];
    const AttendSpan span = a.spans[lo];
    if (span.splits < 2 || static_cast<int32_t>(row) < start || static_cast<int32_t>(row) >= a.row_starts[lo + 1]) return;
    const uint32_t h = head / a.ratio, m = (row - static_cast<uint32_t>(start)) * a.ratio + (head - h * a.ratio);
    const uint32_t tile = m / tile_rows;
    if (tile >= span.tiles) return;
    const uint64_t step = uint64_t(span.tiles) * a.heads * tile_rows;
    const uint64_t first = (uint64_t(span.base) + tile * a.heads + h) * tile_rows + (m - tile * tile_rows);

    float top = kNegInf;
    for (uint32_t s = lane; s < span.splits; s += 64) top = fmaxf(top, a.pairs[2 * (first + s * step)]);
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float zero = top == kNegInf ? 0.0f : top;
    float sum = 0.0f, o[E] = {};
    for (uint32_t s0 = 0; s0 < span.splits; s0 += 64) {
        float f = 0.0f;
        if (s0 + lane < span.splits) {
            const float2 x = *reinterpret_cast<const float2*>(a.pairs + 2 * (first + (s0 + lane) * step));
            f = __builtin_amdgcn_exp2f(x.x - zero);
            sum = __builtin_fmaf(x.y, f, sum);
        }
        const uint32_t n = span.splits - s0 < 64 ? span.splits - s0 : 64;
        for (uint32_t s = 0; s < n; ++s) {
            const float w = __shfl(f, s);
            const float* const p = a.partial + (first + (s0 + s) * step) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(p[e], w, o[e]);
        }
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
    uint16_t* const out = a.out + int64_t(row) * a.out_row + int64_t(head) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[e] * inv));
    if (a.lse && lane == 0)
        a.lse[int64_t(row) * heads + head] =
            sum == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(sum)) * 0.69314718056f;
}

int row_tiles_of(int64_t rows, int64_t channels) {
    const int most = channels <= 128 ? 4 : 2;
    return rows <= 16 ? 1 : rows <= 32 || most == 2 ? 2 : 4;
}

template <int D, bool FP8, bool PAGE16>
hipError_t launch(const AttendArgs& a, const AttendShape& sh, hipStream_t s) {
    switch (sh.row_tiles) {
        case 1: k_attend<D, FP8, 1, PAGE16><<<sh.grid, 64 * kWaves, 0, s>>>(a); break;
        case 2: k_attend<D, FP8, 2, PAGE16><<<sh.grid, 64 * kWaves, 0, s>>>(a); break;
        default:
            if constexpr (D <= 128) k_attend<D, FP8, 4, PAGE16><<<sh.grid, 64 * kWaves, 0, s>>>(a);
            else return hipErrorInvalidValue;
    }
    if (sh.split) {
        const uint64_t waves = uint64_t(a.rows) * a.heads * a.ratio;
        k_attend_join<D><<<static_cast<uint32_t>((waves + 3) / 4), 256, 0, s>>>(a, 16u * sh.row_tiles);
    }
    return hipGetLastError();
}

}  // namespace

AttendShape attend_shape(int64_t batch, int64_t heads, int64_t ratio, int64_t channels, bool fp8, int64_t rows,
                         int64_t rows_per_sequence, int64_t max_tokens) {
    AttendShape s;
    const int64_t usual = rows_per_sequence > 0 ? rows_per_sequence : (rows + batch - 1) / batch;
    s.row_tiles = row_tiles_of(usual * ratio, channels);
    const int64_t tile_rows = 16 * s.row_tiles;
    s.target = 256u * waves_of(static_cast<int>(channels), fp8, s.row_tiles);
    s.split = (max_tokens + kTile - 1) / kTile > kWaves;
    // every sequence's rows fill whole tiles but the last one
    const uint64_t items = uint64_t(heads) * (uint64_t(rows) * ratio / tile_rows + (rows < batch ? rows : batch));
    uint64_t grid = s.split ? (items + s.target / 2 > s.target ? items + s.target / 2 : s.target) : items;
    if (grid < 1) grid = 1;
    s.grid = static_cast<uint32_t>(grid);
    const auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
    s.spans = 256;
    s.words = up(s.spans + uint64_t(batch) * sizeof(AttendSpan));
    s.pairs = up(s.words + 4 * grid);
    s.partial = up(s.pairs + (s.split ? 8 * grid * tile_rows : 0));
    s.total = up(s.partial + (s.split ? 4 * grid * tile_rows * channels : 0));
    return s;
}

template <int D>
hipError_t launch_channels(const AttendArgs& a, const AttendShape& sh, bool fp8, hipStream_t s) {
    if (a.page_tokens % 16 == 0) return fp8 ? launch<D, true, true>(a, sh, s) : launch<D, false, true>(a, sh, s);
    return fp8 ? launch<D, true, false>(a, sh, s) : launch<D, false, false>(a, sh, s);
}

hipError_t launch_attend(const AttendArgs& args, const AttendShape& sh, int64_t channels, bool fp8, hipStream_t s) {
    AttendArgs a = args;
    // t / page_tokens = t page_mul >> page_shift for t < 2^31: page_mul = ceil(2^(31 + e) / page_tokens) with
    // 2^e >= page_tokens exceeds the quotient by less than 2^e / 2^(31 + e) parts of a page a token
    uint32_t e = 0;
    while ((uint64_t(1) << e) < a.page_tokens) ++e;
    a.page_shift = 31 + e;
    a.page_mul = static_cast<uint32_t>(((uint64_t(1) << a.page_shift) + a.page_tokens - 1) / a.page_tokens);
    if (a.rows == 0) {                          // nothing to compute, but the outcome
        k_attend<64, false, 1, false><<<1, 64 * kWaves, 0, s>>>(a);
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
