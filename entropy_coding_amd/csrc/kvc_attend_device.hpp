// What the attention kernels share: how work is dealt to workgroups, operand
// fragments, infinities and NaN, and the query rows.
#pragma once

#include <hip/hip_runtime.h>

#include "kvc_paged.hpp"
#include "kvc_split.hpp"
#include "kvc_wave.hpp"

namespace kvc {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr float kNegInf = -__builtin_inff();

// The same number, for the compiler another one: what is computed from it is
// computed where it is used, not kept in registers over the loop.
__device__ inline int again(int x) {
    asm volatile("" : "+v"(x));
    return x;
}
__device__ inline uint32_t again_uniform(uint32_t x) {
    x = __builtin_amdgcn_readfirstlane(x);
    asm volatile("" : "+s"(x));
    return x;
}

// ---------------------------------------------------------------- the split

struct Seq {
    int32_t start, rows, context;               // rows 0: nothing to compute
    bool bad;
};

__device__ inline Seq seq_of(const AttendArgs& a, uint32_t b) {
    Seq s;
    s.start = a.row_starts[b];
    const int32_t end = a.row_starts[b + 1];
    s.context = a.context ? a.context[b] : 0;
    // max_tokens < 2^31 - 255: no difference or sum below passes 32 bits where the terms before it hold
    s.bad = s.start < 0 || end < s.start || end > static_cast<int32_t>(a.rows) || s.context < 0 ||
            s.context > a.max_tokens || end - s.start > a.max_tokens - s.context;
    s.rows = s.bad ? 0 : end - s.start;
    return s;
}

// The work of a call as a line of units.  Sequence b has heads x tiles_b
// items (a KV head and a tile of its rows, the tile changing fastest), each of
// one unit for 2^unit_shift tokens; workgroup w of the launch takes units
// [w per, (w + 1) per), wherever items begin and end in it.  So every
// workgroup has the same number of units, whatever the lengths, and leaves at
// most two parts of items that others share: the end of one that began before
// its range (part 2 w) and the beginning of one that ends behind it (2 w + 1).
// Where the units of each item can be rounded up to a multiple of `per`, or
// of an eighth more, and still fit the workgroups, they are: then none works
// on two items (few long ones, or many of one length).  Every wave finds its
// place from the lengths (no launch of its own for a plan, nothing
// kept between calls).  unit_shift is such that the units of a call whose row
// starts are prefix sums stay below 2^31; where they are not, sums may wrap,
// and what a workgroup takes for its share still lies within one sequence.
__device__ inline uint32_t tiles_of(const AttendArgs& a, const Seq& s) { return row_tiles(s.rows, a.ratio, a.tile_shift); }
__device__ inline uint32_t real_of(const AttendArgs& a, const Seq& s) {
    return !a.split ? 1u : units_in(uint32_t(s.context) + uint32_t(s.rows), a.unit_shift);
}

__device__ inline Plan split_plan(const AttendArgs& a, uint32_t least) {
    Plan p;
    p.aligned = 0;
    const uint32_t lane = threadIdx.x & 63;
    // the first 64 sequences' items and units, kept for all sums
    uint32_t items0 = 0, real0 = 0;
    if (lane < a.batch) {
        const Seq s = seq_of(a, lane);
        items0 = tiles_of(a, s) * a.heads;
        real0 = real_of(a, s);
    }
    auto each = [&](auto add) {                 // the items and units of this lane's sequences
        add(items0, real0);
        for (uint32_t b = 64 + lane; b < a.batch; b += 64) {
            const Seq s = seq_of(a, b);
            add(tiles_of(a, s) * a.heads, real_of(a, s));
        }
    };
    uint32_t units = 0, all = 0;
    each([&](uint32_t items, uint32_t real) {
        units += items * real;
        all += items;
    });
    units = of_lane(scan(units), 63);
    uint32_t per = first_per(units, a.target, least);
    p.per = per;
    const bool fits = of_lane(scan(all), 63) <= a.target;
    for (int i = 0; fits && i < 2 && !p.aligned; ++i, per = next_per(per)) {
        uint32_t groups = 0;
        each([&](uint32_t items, uint32_t real) { groups += items * groups_in(real, per); });
        if (of_lane(scan(groups), 63) > a.target) continue;
        p.aligned = 1;
        p.per = per;
    }
    return p;
}

__device__ inline Plan plan_of(const AttendArgs& a, uint32_t least) {
    Plan p{1, 0};                               // an item a workgroup
    if (a.split) p = split_plan(a, least);
    return Plan{uint32_t(__builtin_amdgcn_readfirstlane(p.per)), uint32_t(__builtin_amdgcn_readfirstlane(p.aligned))};
}

// The item that holds a unit, and where it lies.
struct Share {
    bool any = false;
    Seq seq;
    uint32_t b, head, tile;
    uint32_t units, real;                       // rounded up to what workgroups take, and not
    uint32_t first;                             // its first unit
    uint32_t tiles, begin, past;                // its sequence's: row tiles, first unit, the unit behind the last
    uint32_t b0 = 0, base = 0;                  // the 64 sequences that the sequence is among, the units before them
};

__device__ inline void item_of(Share* r, uint32_t at) {
    const Item i = item_at(r->begin, r->units, r->tiles, at);
    r->head = __builtin_amdgcn_readfirstlane(i.head);
    r->tile = __builtin_amdgcn_readfirstlane(i.tile);
    r->first = __builtin_amdgcn_readfirstlane(i.first);
}

// Finds the item that holds unit `at`, not before what *r holds: it is looked
// for from there on.  note: workgroup 0 writes the spans that the join reads,
// and the flags.
__device__ inline void share_of(const AttendArgs& a, const Plan& p, uint32_t at, Share* r, bool note) {
    if (r->any && at < r->past) return item_of(r, at);
    const uint32_t lane = again(threadIdx.x & 63);
    uint32_t base = r->base;
    bool bad = false;
    r->any = false;
    for (uint32_t b0 = r->b0; b0 < a.batch; b0 += 64) {
        const uint32_t b = b0 + lane;
        uint32_t tiles = 0, real = 0;
        Seq s{};
        if (b < a.batch) {
            s = seq_of(a, b);
            bad = bad || s.bad;
            tiles = tiles_of(a, s);
            real = real_of(a, s);
        }
        const uint32_t u = p.units(real);
        const uint32_t count = tiles * a.heads * u;
        const uint32_t end = scan(count) + base;
        if (note && b < a.batch) a.spans[b] = AttendSpan{end - count, u, tiles, 0};
        const uint64_t who = __ballot(count && at >= end - count && at < end);
        if (who) {
            const int l = __builtin_ctzll(who);
            r->any = true;
            r->b = b0 + l;
            r->b0 = b0;
            r->base = base;
            r->seq.start = static_cast<int32_t>(of_lane(s.start, l));
            r->seq.rows = static_cast<int32_t>(of_lane(s.rows, l));
            r->seq.context = static_cast<int32_t>(of_lane(s.context, l));
            r->units = of_lane(u, l);
            r->real = of_lane(real, l);
            r->tiles = of_lane(tiles, l);
            r->begin = of_lane(end - count, l);
            r->past = of_lane(end, l);
            item_of(r, at);
            if (!note) break;
        }
        base = of_lane(end, 63);
    }
    if (note) {
        bad = __any(bad);
        if (lane == 0) {
            a.ctl->magic = again_uniform(kPagedMagic);
            a.ctl->flags = bad ? kPagedInvalid : 0u;
            a.ctl->grid = gridDim.x;
            a.ctl->words_offset =
                static_cast<uint32_t>(reinterpret_cast<char*>(a.words) - reinterpret_cast<char*>(a.ctl));
            a.ctl->per = again_uniform(p.per);
            a.ctl->aligned = again_uniform(p.aligned);
        }
    }
}

// Workgroups are dealt to the eight XCDs in turn; this numbers them so that
// one XCD has neighbours on the line, whose row tiles read the same K and V.
__device__ inline uint32_t place_of(uint32_t id, uint32_t grid) {
    const uint32_t eighth = grid / 8;
    return id < 8 * eighth ? (id & 7) * eighth + (id >> 3) : id;
}

// ---------------------------------------------------------------- fragments

__device__ inline bf16x8 frag_of(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Two of the four e4m3 values of a word (its low or high half) as bf16: exact.
template <bool HIGH>
__device__ uint32_t widen(uint32_t four) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, HIGH));
}

// Values c of two tokens (x the first's word, y the second's, that holds
// value c) as a pair of bf16.
template <bool FP8>
__device__ uint32_t pair_of(uint32_t x, uint32_t y, int c) {
    if constexpr (FP8) {
        const uint32_t two = (c & 2) ? __builtin_amdgcn_perm(y, x, 0x07030602u) : __builtin_amdgcn_perm(y, x, 0x05010400u);
        return (c & 1) ? widen<true>(two) : widen<false>(two);
    }
    return (c & 1) ? __builtin_amdgcn_perm(y, x, 0x07060302u) : __builtin_amdgcn_perm(y, x, 0x05040100u);
}

// The pools' addresses are read from memory: that they are global ones has
// to be said.
#define KVC_GLOBAL __attribute__((address_space(1)))
typedef const KVC_GLOBAL uint8_t* GlobalBytes;

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
        for (int i = 0; i < WORDS / W; ++i) v[i] = *reinterpret_cast<const KVC_GLOBAL Vec*>(p + 4 * W * i);
    }
};

__device__ inline uint32_t two_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

// The larger one, NaN if one is: three at a time are one instruction, while
// the maximum that prefers numbers needs its arguments quieted first.
__device__ inline float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }
__device__ inline float larger(float top, f32x4 x) { return larger(larger(larger(larger(top, x[0]), x[1]), x[2]), x[3]); }

// A row's weights are 2^(scale s - m) with m the largest scaled score when it
// was last set: it is set anew only when a score passes it by kSlack, so that
// the sums are rarely rescaled (with every new largest score, some row of a
// wave would be at every other tile of a long sequence).  Weights up to
// 2^kSlack lose nothing in floating point.
constexpr float kSlack = 8.0f;

// The largest of the four lanes n, n + 16, n + 32, n + 48.
__device__ inline float top_of_column(float x) {
    u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = larger(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return larger(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// A row's reference m (as -m, what a weight's exponent adds to the scaled
// score), the score that sets it anew, and the sum of its weights.
struct RowSum {
    float shift = 0.0f, limit = kNegInf, sum = 0.0f;

    __device__ float top() const { return limit == kNegInf ? kNegInf : -shift; }

    // Sets m to the largest of the column where that passes the limit; returns what the sums are multiplied with.
    __device__ float raise(float top, float scale, float slack) {
        top = top_of_column(top);
        if (!(top > limit)) return 1.0f;
        const float now = -top * scale;
        const float f = limit == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(now - shift);
        shift = now;
        limit = top + slack;
        sum *= f;
        return f;
    }
};

// The scale of the scores as a positive number, the same for all lanes (a
// scale of zero becomes the smallest one), and the bits that the queries'
// values take for its sign: so the largest scaled score is the scaled largest.
struct Scale {
    float scale, slack;
    uint32_t flip;

    __device__ explicit Scale(const AttendArgs& a) {
        const uint32_t bits = __builtin_amdgcn_readfirstlane(__float_as_uint(a.scale_log2));
        flip = (bits >> 31) ? 0x80008000u : 0u;
        const uint32_t size = bits & 0x7FFFFFFFu;
        scale = __uint_as_float(size < 0x00800000u ? 0x00800000u : size);
        slack = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(kSlack / scale)));
    }
};

// Words read through the scalar cache: they are not written while the kernel
// runs, and every lane wants the same ones.
__device__ inline int32_t uniform_word(const int32_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p));
}

// ---------------------------------------------------------------- infinities and NaN

// V values of unseen tokens meet weights of zero, which an infinity or a NaN
// would turn into NaN.  So such values of drafted tokens are cleared on their
// way into the sum and added at the end to the rows that see them (what a row
// sees of an infinity is an infinity, whatever its weight).

// Among a word's values (two bf16; four e4m3, which has no infinity): the top
// bit of each value's place is set where it is one.
template <bool FP8>
__device__ uint32_t wild_bits(uint32_t w) {
    return FP8 ? ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

template <bool FP8>
__device__ uint32_t without_wild(uint32_t w) {
    return w & ~(FP8 ? (wild_bits<true>(w) >> 7) * 0xFFu : (wild_bits<false>(w) >> 15) * 0xFFFFu);
}

// Value c (w is its word) if it is an infinity or a NaN, else zero.
template <bool FP8>
__device__ float wild_part(uint32_t w, int c) {
    if constexpr (FP8) return ((w >> (8 * (c & 3))) & 0x7Fu) == 0x7Fu ? __builtin_nanf("") : 0.0f;
    const uint32_t h = (c & 1) ? w >> 16 : w << 16 >> 16;
    return (h & 0x7F80u) == 0x7F80u ? __uint_as_float(h << 16) : 0.0f;
}

// ---------------------------------------------------------------- a workgroup's part of an item

struct Part {
    int rows;                                   // M = drafted tokens x ratio
    int row0;                                   // the first row of the tile
    int context, length;                        // length: of what its rows see at all
    int full;                                   // tokens before this one are seen by every row
    int ta, tb;                                 // tiles of `unit` tokens
    bool whole;                                 // nobody else works on the item
    uint32_t slot;                              // else: where the part goes
};

__device__ inline Part part_of(const AttendArgs& a, const Share& sh, uint32_t place, uint32_t at, uint32_t from,
                               uint32_t end, uint32_t unit) {
    Part r;
    r.rows = sh.seq.rows * static_cast<int>(a.ratio);
    r.row0 = static_cast<int>(sh.tile << a.tile_shift);
    r.context = sh.seq.context;
    const Extent e = extent_of(!a.mask, r.context, sh.seq.rows, r.rows, r.row0, 1 << a.tile_shift, static_cast<int>(a.ratio));
    r.length = e.length;
    r.full = e.full;
    const Range g = range_of(sh.first, sh.units, sh.real, (static_cast<uint32_t>(r.length) + unit - 1) / unit, place, at,
                             from, end);
    r.whole = g.whole;
    r.slot = g.slot;
    r.ta = g.ta;
    r.tb = g.tb;
    return r;
}

// The drafted token of row m, and the row's queries: channels ch .. ch + 7.
struct Query {
    int node;
    const uint16_t* q;

    __device__ Query(const AttendArgs& a, const Share& sh, int m, int rows) {
        node = m < rows ? m / static_cast<int>(a.ratio) : 0;
        const int g = m - node * static_cast<int>(a.ratio);
        q = m < rows ? a.q + (int64_t(sh.seq.start) + node) * a.q_row + (int64_t(sh.head) * a.ratio + g) * a.q_head
                     : nullptr;
    }
    __device__ bf16x8 at(int ch, uint32_t flip) const {
        const uint4 x = q ? *reinterpret_cast<const uint4*>(q + ch) : uint4{0, 0, 0, 0};
        return frag_of(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
    }
};

// What the row of drafted token `node` sees of the 64 tokens that begin with
// drafted token j0 (negative: context, > -64); `seen`: drafted tokens there
// are (> j0).
__device__ inline uint64_t window_of(const AttendArgs& a, int32_t start, int node, int j0, int seen) {
    if (!a.mask) {
        const int see = node - j0 + 1;
        return see >= 64 ? ~0ull : see <= 0 ? 0ull : (1ull << see) - 1;
    }
    const uint64_t* const bits = a.mask + (int64_t(start) + node) * a.mask_words;
    uint64_t w;
    if (j0 < 0) {
        w = (bits[0] << -j0) | ((1ull << -j0) - 1);
    } else {
        const uint32_t at = static_cast<uint32_t>(j0) >> 6, by = j0 & 63;
        w = at < a.mask_words ? bits[at] >> by : 0ull;
        if (by && at + 1 < a.mask_words) w |= bits[at + 1] << (64 - by);
    }
    return seen - j0 < 64 ? w & ((1ull << (seen - j0)) - 1) : w;
}

// Whether that row sees drafted token j < seen.
__device__ inline bool sees(const AttendArgs& a, int32_t start, int node, uint32_t j) {
    if (!a.mask) return static_cast<int>(j) <= node;
    return j / 64 < a.mask_words &&
           ((a.mask[(int64_t(start) + node) * a.mask_words + j / 64] >> (j & 63)) & 1u);
}

// Slot (page x page_tokens + row) of a token of a sequence; a page number
// outside the pools gives page 0 and raises *bad.
__device__ inline uint32_t page_index(const AttendArgs& a, uint32_t t) {
    return static_cast<uint32_t>((uint64_t(t) * a.page_mul) >> a.page_shift);
}
__device__ inline uint32_t slot_in(const AttendArgs& a, int32_t page, uint32_t t, uint32_t* bad) {
    uint32_t p = static_cast<uint32_t>(page);
    if (p >= static_cast<uint32_t>(a.num_pages)) {
        *bad = kPagedInvalid;
        p = 0;
    }
    return p * a.page_tokens + (t - page_index(a, t) * a.page_tokens);     // < 2^31
}

constexpr float kLn2 = 0.69314718056f;

}  // namespace kvc
