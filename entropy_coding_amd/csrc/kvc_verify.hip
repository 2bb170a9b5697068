// Verification of drafted tokens against the target's probabilities (declared
// in include/kvc.h).
#include <hip/hip_runtime.h>

#include "kvc_paged.hpp"
#include "kvc_step.hpp"
#include "kvc_wave.hpp"

namespace kvc {
namespace {

// Probabilities are summed in whole units of 2^-42, so that every sum is
// exact in whatever order it is formed, and a token drawn from a sum does not
// depend on how the vocabulary is split.  A value's units are two halves of
// 21 bits, each summed in 32: y 2^21 is exact in float32, and so is what its
// whole part leaves.
struct Units {
    uint32_t high, low;
    __device__ void add(Units o) {
        high += o.high;
        low += o.low;
    }
    __device__ uint64_t all() const { return (uint64_t(high) << 21) + low; }
};
__device__ Units units_of(float y) {
    const float x = y * 0x1p21f;
    const uint32_t high = static_cast<uint32_t>(x);
    return Units{high, static_cast<uint32_t>((x - static_cast<float>(high)) * 0x1p21f)};
}

// What is no number between 0 and 1 counts as the nearer of them, NaN as 0.
__device__ float clean(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }

// What is left of probabilities after `rejected` siblings drawn with
// probabilities q were rejected: each rejection takes q off, and the next
// sibling meets the rest scaled to a sum of 1 (scales[k], k > 0).  All of them
// are taken again from the row every time, so that a node's time grows with the
// square of its rejected siblings.
template <int N>
__device__ void reject(float (&y)[N], const float (&q)[N], const float* scales, int rejected) {
    for (int k = 0; k < rejected; ++k) {
        const float s = k ? scales[k] : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = fmaxf(y[i] * s - q[i], 0.0f);
    }
}

typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));     // (a row may begin at any value)

// Four values of a row from `at` on, 0 behind its end.
__device__ void load4(const float* row, uint32_t at, uint32_t vocab, float* x) {
    if (at + 4 <= vocab) {
        const float4u y = *reinterpret_cast<const float4u*>(row + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = clean(y[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = at + i < vocab ? clean(row[at + i]) : 0.0f;
    }
}

// The sum over a workgroup, in every thread.  A thread's halves are of at most
// 1024 values: a value is at most 1, up to what the scale after a rejection is
// off by where next to nothing was left; together they are less than 2 each,
// so that 1024 of them pass no 32 bits, and a wave's threads are summed by
// halves.
template <int THREADS>
__device__ uint64_t block_sum(Units x, uint64_t* of_wave) {
    const uint32_t parts[3] = {x.high >> 16, x.high & 0xFFFFu, x.low >> 16};
    uint32_t halves[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) halves[i] = of_lane(scan(parts[i]), 63);
    uint64_t all = ((uint64_t(halves[0]) << 16) + halves[1]) << 21;
    all += (uint64_t(halves[2]) << 16) + of_lane(scan(x.low & 0xFFFFu), 63);
    if ((threadIdx.x & 63) == 63) of_wave[threadIdx.x >> 6] = all;
    __syncthreads();
    uint64_t sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) sum += of_wave[w];
    __syncthreads();
    return sum;
}

// ---- the walk

// One sequence's tree.
struct Tree {
    int64_t start;
    int n;                                      // 0: nothing to walk
    bool bad;
};
__device__ Tree tree_of(const VerifyArgs& a, int64_t b) {
    const int64_t start = a.row_starts[b], end = a.row_starts[b + 1];
    Tree t;
    t.bad = start < 0 || end < start || end > a.rows || end - start > kMaxNodes;
    t.start = start;
    t.n = t.bad ? 0 : static_cast<int>(end - start);
    return t;
}

// Node i as a lane has it.
struct Node {
    int parent, token;                          // -1: none that can be reached, none of the vocabulary
    float u, p, q;
    bool wrong;
};
__device__ Node node_of(const VerifyArgs& a, const Tree& t, int i) {
    Node x{-1, -1, 0.0f, 0.0f, 0.0f, false};
    if (i < 1 || i >= t.n) return x;            // (of the first nothing is looked at)
    const int64_t r = t.start + i;
    const int parent = a.parents ? a.parents[r] : i - 1, token = a.tokens[r];
    x.u = a.accept[r];
    if (parent >= 0 && parent < i) x.parent = parent;
    else x.wrong = true;
    if (token >= 0 && token < static_cast<int64_t>(a.vocab)) x.token = token;
    else x.wrong = true;
    if (x.wrong) return x;
    x.p = clean(a.target[(t.start + parent) * a.target_row + token]);
    if (a.draft) x.q = clean(a.draft[(t.start + parent) * a.draft_row + token]);
    return x;
}

__device__ float value_of_lane(float x, int lane) { return __uint_as_float(of_lane(__float_as_uint(x), lane)); }

// Where a walk is, and what it leaves.
struct Walk {
    int32_t path[kMaxNodes], tokens[kMaxNodes]; // kept nodes and theirs
    int32_t rejects[kMaxNodes];                 // tokens that are out at the current node, each once
    float scales[kMaxNodes];                    // between its rejections, the second and on
    int32_t current, kept, rejected, listed;
    uint32_t wrong;
};

// The walk down a tree, by whole waves that all take it alike: nodes are
// looked at in order, 64 at a time in a wave's lanes; those whose parent is
// the current node are tested, an accepted one becomes the current one.
// scale(current, rejected) gives what is left after so many rejections its
// scale, where nodes were drawn from the draft's probabilities and a node has
// several children; `writes`: whether this thread writes the lists.
template <class Scale, class Sync>
__device__ void walk(const VerifyArgs& a, const Tree& t, Walk& w, bool writes, Scale scale, Sync sync) {
    const int lane = threadIdx.x & 63;
    int current = 0, kept = 1, rejected = 0, listed = 0;
    uint64_t mass = uint64_t(1) << 42;          // without probabilities: of tokens that are not out
    bool wrong = false;
    if (writes) w.path[0] = 0;
    for (int base = 0; base < t.n; base += 64) {
        const Node x = node_of(a, t, base + lane);
        wrong = wrong || x.wrong;
        uint64_t ahead = ~uint64_t(0);          // nodes behind the last one tested
        for (;;) {
            const uint64_t next = __ballot(x.parent == current) & ahead;
            if (!next) break;
            const int bit = __builtin_ctzll(next);
            ahead = bit == 63 ? 0 : ~uint64_t(0) << (bit + 1);
            const double u = value_of_lane(x.u, bit);
            const float p = value_of_lane(x.p, bit), q = value_of_lane(x.q, bit);
            const int token = __builtin_amdgcn_readlane(x.token, bit);
            bool ok, again = false;
            if (a.draft) {
                float y = p;
                if (rejected) {
                    const float s = scale(current, rejected), one[1] = {q};
                    float rest[1] = {p};
                    reject(rest, one, w.scales, rejected);
                    y = rest[0] * s;
                }
                ok = u * double(q) < double(y);
            } else {
                for (int k = lane; k < listed; k += 64) again = again || w.rejects[k] == token;
                again = __any(again);
                const float y = again ? 0.0f : p;
                ok = u * static_cast<double>(mass) < double(y) * 0x1p42;
            }
            if (ok) {
                current = base + bit;
                if (writes) {
                    w.path[kept] = current;
                    w.tokens[kept] = token;
                }
                ++kept;
                rejected = listed = 0;
                mass = uint64_t(1) << 42;
            } else {
                ++rejected;
                if (!a.draft && !again && token >= 0) {
                    if (writes) w.rejects[listed] = token;
                    sync();                     // (the next test reads the list)
                    ++listed;
                    const uint64_t out = units_of(p).all();
                    mass = mass > out ? mass - out : 0;
                }
            }
        }
    }
    const bool any = __any(wrong);
    if (writes) {
        w.current = current;
        w.kept = kept;
        w.rejected = rejected;
        w.listed = listed;
        w.wrong = any ? kPagedInvalid : 0u;
    }
}

// What the walk left, for the caller: by a whole workgroup.
template <int THREADS>
__device__ void write_walk(const VerifyArgs& a, const Tree& t, const Walk& w, int64_t b) {
    for (int j = threadIdx.x; j < t.n; j += THREADS) {
        a.kept[t.start + j] = j < w.kept ? w.path[j] : -1;
        if (j != w.kept - 1)                    // (there the drawn token goes)
            a.out_tokens[t.start + j] = j + 1 < w.kept ? w.tokens[j + 1] : -1;
    }
    if (threadIdx.x == 0) {
        a.kept_lens[b] = t.n ? w.kept : 0;
        a.words[2 * b] = t.n ? w.wrong : t.bad ? kPagedInvalid : 0u;
    }
}

// ---- the draw


// The distribution that a sequence draws from.
struct Draw {
    int64_t stop;                               // row of the node
    int rejected;                               // entries of its list
    const float* scales;
    const int32_t* rejects;
};

// N values of a row from `base` on, in fours at place(0), place(1), ..., 0 from
// `end` on; and what the rejections left of them.
template <int THREADS, int N, class Place>
__device__ void values_of(const VerifyArgs& a, const Draw& d, uint32_t base, uint32_t end, Place place, float (&x)[N],
                          float (&left)[N]) {
    const float* const target = a.target + d.stop * a.target_row;
    const bool both = a.draft && d.rejected > 0;
    float q[N];
#pragma unroll
    for (int g = 0; g < N / 4; ++g) load4(target, base + place(g), end, x + 4 * g);
    if (both) {
        const float* const draft = a.draft + d.stop * a.draft_row;
#pragma unroll
        for (int g = 0; g < N / 4; ++g) load4(draft, base + place(g), end, q + 4 * g);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) left[i] = x[i];
    if (both) reject(left, q, d.scales, d.rejected);
    if (a.draft) return;
    for (int k = 0; k < d.rejected; ++k) {      // tokens that are out
        const uint32_t at = static_cast<uint32_t>(d.rejects[k]) - base;
        if (at >= uint32_t(N) * THREADS) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) left[i] = at == place(i / 4) + i % 4 ? 0.0f : left[i];
    }
}

// The sum of the lanes up to this one, of values below 2^62.
__device__ uint64_t scan_wide(uint64_t x) {
    constexpr uint32_t kLow = (1u << 21) - 1;
    const uint32_t low = scan(static_cast<uint32_t>(x) & kLow), mid = scan(static_cast<uint32_t>(x >> 21) & kLow),
                   high = scan(static_cast<uint32_t>(x >> 42));
    return (uint64_t(high) << 42) + (uint64_t(mid) << 21) + low;
}

// ---- first rejections

// A drawn tree's nodes whose first child would be rejected and that have
// another: what that rejection leaves is needed there, should the walk come by,
// and depends on no other node.  (Of a node whose first child is accepted, only
// that one can be reached.)  All of them are summed over the vocabulary by as
// many workgroups as the chip takes, so that the walk, which has one CU, need
// not: 8 trees of 12 nodes over 131072 tokens 59 -> 40 us.  Nodes behind
// the 64th and more than kFirsts of them are left to the walk.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_verify_first(VerifyArgs a, uint32_t parts, uint32_t per) {
    constexpr int kValues = 16;
    __shared__ int32_t firsts[kFirsts];
    __shared__ int32_t found;
    __shared__ uint64_t of_wave[THREADS / 64];
    const uint32_t b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const Tree t = tree_of(a, b);
    if (tid < 64) {
        int count = 0;
        if (t.n) {
            const Node x = node_of(a, t, lane);
            const uint64_t accepted = __ballot(double(x.u) * double(x.q) < double(x.p));
            uint64_t reached = 1, done = 0;
            while (const uint64_t left = reached & ~done) {
                const int v = __builtin_ctzll(left);
                done |= uint64_t(1) << v;
                const uint64_t children = __ballot(x.parent == v), first = children & -children;
                if (!children) continue;
                if (first & accepted) {
                    reached |= first;
                } else if (children != first) {
                    reached |= children ^ first;
                    if (count < kFirsts && lane == 0) firsts[count] = v;
                    count += count < kFirsts;
                }
            }
        }
        if (lane == 0) found = count;
    }
    __syncthreads();
    const int count = found;
    if (part == 0 && tid < uint32_t(kFirsts)) a.first_nodes[b * kFirsts + tid] = int(tid) < count ? firsts[tid] : -1;
    const uint32_t begin = part * per * kVerifyChunk, past = begin + per * kVerifyChunk;
    const uint32_t end = past < a.vocab ? past : a.vocab;
    const auto in_turn = [&](int g) { return 4 * (THREADS * g + tid); };
    for (int k = 0; k < count; ++k) {
        const Draw here{t.start + firsts[k], 1, nullptr, nullptr};
        Units sum{0, 0};
        for (uint32_t base = begin; base < end; base += kValues * THREADS) {
            float x[kValues], left[kValues];
            values_of<THREADS>(a, here, base, end, in_turn, x, left);
#pragma unroll
            for (int i = 0; i < kValues; ++i) sum.add(units_of(left[i]));
        }
        const uint64_t z = block_sum<THREADS>(sum, of_wave);
        if (tid == 0) a.first_sums[(uint64_t(b) * kFirsts + k) * parts + part] = z;
    }
}

// ---- walk, sums and draw

// Chunks of one sequence's distribution, `per` at a time, are summed by a
// workgroup; the last workgroup of a sequence to be done draws the token.
// Every workgroup walks the tree for itself: chains, and trees without
// probabilities, by its first wave, a chain of trips to memory as long as a
// kernel of its own would take, and a launch less.  Of trees whose nodes were
// drawn from the draft's probabilities (DRAWN) the sum of what the rejections
// left is needed before a sibling of a rejected node is tested: a first
// rejection's may be there (k_verify_first), others are formed by the whole
// workgroup, bound by what one CU reads (4.6 us for 32000 tokens) and, beyond a
// few siblings, by what it computes: 4 stars of 8, 32 and 64 rejected siblings
// take 56, 381 and 1244 us over 32000 tokens, 147, 1285 and 4396 over 131072.
template <int THREADS, bool DRAWN>
__global__ __launch_bounds__(THREADS) void k_verify(VerifyArgs a, uint32_t parts, uint32_t per) {
    constexpr int kWaves = THREADS / 64, kValues = 16;      // of a thread, asked for together
    constexpr int kChunksAtOnce = kValues * THREADS / kVerifyChunk;
    __shared__ Walk w;
    __shared__ uint64_t of_wave[2][kWaves], of_value[kWaves];
    __shared__ uint64_t of_chunk[2][kMostChunks][kWaves];
    __shared__ uint32_t place;
    __shared__ uint64_t place_before;
    const uint32_t b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x == 0 && tid == 0) *a.ctl = VerifyControl{kVerifyMagic, static_cast<uint32_t>(a.batch)};
    const float u = a.sample[b];                // (asked for now: a trip less behind the sums)
    const Tree t = tree_of(a, b);
    if (t.n == 0) {
        if (part == 0) write_walk<THREADS>(a, t, w, b);
        if (part == 0 && tid == 0) a.words[2 * b + 1] = 0u;
        return;
    }
    const auto in_turn = [&](int g) { return 4 * (THREADS * g + tid); };
    if (DRAWN) {
        const auto known_scale = [&](uint64_t z, int rejected) {
            const float s = z ? static_cast<float>(0x1p42 / static_cast<double>(z)) : 0.0f;
            if (tid == 0) w.scales[rejected] = s;
            __syncthreads();
            return s;
        };
        const auto scale = [&](int current, int rejected) {
            uint64_t z = 0;
            int known = -1;
            if (rejected == 1 && a.first_parts)
                for (int k = 0; k < kFirsts; ++k)
                    if (a.first_nodes[b * kFirsts + k] == current) known = k;
            if (known >= 0) {
                const uint64_t* const from = a.first_sums + (uint64_t(b) * kFirsts + known) * a.first_parts;
                const uint64_t sum = scan_wide(tid < a.first_parts ? from[tid] : 0);
                if (lane == 63) of_wave[0][wave] = sum;
                __syncthreads();
                for (int k = 0; k < kWaves; ++k) z += of_wave[0][k];
                __syncthreads();
                return known_scale(z, rejected);
            }
            const Draw here{t.start + current, rejected, w.scales, nullptr};
            Units sum{0, 0};
            for (uint32_t base = 0; base < a.vocab; base += kValues * THREADS) {
                float x[kValues], left[kValues];
                values_of<THREADS>(a, here, base, a.vocab, in_turn, x, left);
#pragma unroll
                for (int i = 0; i < kValues; ++i) sum.add(units_of(left[i]));
            }
            return known_scale(block_sum<THREADS>(sum, of_wave[0]), rejected);
        };
        walk(a, t, w, tid == 0, scale, [] { __syncthreads(); });
    } else if (wave == 0) {
        walk(a, t, w, tid == 0, [](int, int) { return 0.0f; }, [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); });
    }
    __syncthreads();
    const Draw d{t.start + w.current, a.draft ? w.rejected : w.listed, w.scales, w.rejects};
    const int64_t last = t.start + w.kept - 1;  // of the sequence's new tokens
    const uint32_t first_chunk = part * per;
    const uint32_t count = first_chunk + per <= a.chunks ? per : a.chunks - first_chunk;
    const uint32_t here = (first_chunk + count) * kVerifyChunk, end = here < a.vocab ? here : a.vocab;
    for (uint32_t c = 0; c < count; c += kChunksAtOnce) {
        float x[kValues], left[kValues];
        values_of<THREADS>(a, d, (first_chunk + c) * kVerifyChunk, end, in_turn, x, left);
#pragma unroll
        for (int k = 0; k < kChunksAtOnce; ++k) {
            constexpr int kOfChunk = kValues / kChunksAtOnce;
            Units before{0, 0}, after{0, 0};
#pragma unroll
            for (int i = k * kOfChunk; i < (k + 1) * kOfChunk; ++i) {
                before.add(units_of(x[i]));
                after.add(units_of(left[i]));
            }
            // (a wave's 1024 values pass no 32 bits: see block_sum)
            const uint64_t sum[2] = {Units{scan(after.high), scan(after.low)}.all(), Units{scan(before.high), scan(before.low)}.all()};
            if (lane == 63 && c + k < count) {
                of_chunk[0][c + k][wave] = sum[0];
                of_chunk[1][c + k][wave] = sum[1];
            }
        }
    }
    __syncthreads();
    VerifySums* const sums = a.sums + uint64_t(b) * a.chunks;
    uint64_t mine[2] = {0, 0};
    if (tid < count) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < kWaves; ++k) mine[i] += of_chunk[i][tid][k];
    }
    if (parts > 1) {
        // The sums first, as exchanges: what they return says that they are done where all dies see them, with no
        // cache to write back (with a release and an acquire of every workgroup 64 sequences took 73 us in place of 24).
        if (wave == 0) {
            if (lane < count) {
                VerifySums* const to = sums + first_chunk + lane;
                const uint64_t done[2] = {
                    __hip_atomic_exchange(&to->left, mine[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                    __hip_atomic_exchange(&to->whole, mine[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
                asm volatile("" ::"v"(done[0]), "v"(done[1]) : "memory");
            }
            if (lane == 0) {
                place = __hip_atomic_fetch_add(&a.arrived[uint64_t(b) * kArrivedStride], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (place == parts - 1) __hip_atomic_store(&a.arrived[uint64_t(b) * kArrivedStride], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        __syncthreads();
        if (place != parts - 1) return;
        mine[0] = mine[1] = 0;
        if (tid < a.chunks) {
            mine[0] = __hip_atomic_load(&sums[tid].left, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            mine[1] = __hip_atomic_load(&sums[tid].whole, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    // the chunk that the drawn point lies in: a thread a chunk
    uint64_t upto[2], total[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        upto[i] = scan_wide(mine[i]);
        if (lane == 63) of_wave[i][wave] = upto[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        total[i] = 0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            if (k == int(wave)) upto[i] += total[i];
            total[i] += of_wave[i][k];
        }
    }
    const int which = total[0] == 0;            // nothing is left: the target's own probabilities
    const uint64_t all = which ? total[1] : total[0];
    if (all == 0) {
        if (tid == 0) {
            a.out_tokens[last] = -1;
            a.words[2 * b + 1] = kPagedInvalid;
        }
        write_walk<THREADS>(a, t, w, b);
        return;
    }
    uint64_t point = u > 0.0f ? static_cast<uint64_t>(fmin(double(u), 1.0) * static_cast<double>(all)) : 0;
    if (point >= all) point = all - 1;
    const uint64_t past = which ? upto[1] : upto[0], first = past - (which ? mine[1] : mine[0]);
    if (first <= point && point < past) {
        place = tid;
        place_before = first;
    }
    __syncthreads();
    // ... and there the value, a thread's values one after the other
    constexpr int kOwn = kVerifyChunk / THREADS;
    const uint32_t base = place * kVerifyChunk;
    float x[kOwn], left[kOwn];
    values_of<THREADS>(a, d, base, a.vocab, [&](int g) { return kOwn * tid + 4 * g; }, x, left);
    Units own{0, 0};
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        if (which) left[i] = x[i];
        own.add(units_of(left[i]));
    }
    uint64_t sum = Units{scan(own.high), scan(own.low)}.all();
    if (lane == 63) of_value[wave] = sum;
    __syncthreads();
    sum += place_before - own.all();
#pragma unroll
    for (int k = 0; k < kWaves - 1; ++k)
        if (k < int(wave)) sum += of_value[k];
    if (sum <= point && point < sum + own.all()) {
        int at = 0;
#pragma unroll
        for (int i = 0; i < kOwn - 1; ++i) {
            sum += units_of(left[i]).all();
            if (sum <= point) at = i + 1;
        }
        a.out_tokens[last] = static_cast<int32_t>(base + kOwn * tid + at);
        a.words[2 * b + 1] = 0u;
    }
    write_walk<THREADS>(a, t, w, b);
}

// Workgroups of 1024 threads for drawn trees, each of which may read a whole
// vocabulary for its walk: fewer than the chip holds, and fewest where that is
// short (16 trees over 32000 tokens: 21 us, with 16 or 256 of them 24 and 23).
constexpr uint32_t kDrawnGroups = 64, kDrawnGroupsWide = 256;
// From this many chunks on, first rejections are summed ahead: another launch
// that saves a CU's pass over a wide vocabulary.  Without it and with it, us:
//               1 tree of 8    8 trees of 12    64 of 8
//    32000 tokens  11.0  13.4     18.9  20.0    29.2  31.2
//    49152         12.8  14.5     22.3  21.3    37.6  32.7
//    61441         11.1  13.4     28.4  23.3    51.6  42.8
//    98304         11.2  13.4     41.7  32.3    70.4  57.7
//   131072         15.8  14.6     58.8  39.8    95.7  63.8
constexpr uint32_t kFirstChunks = 16;

}  // namespace

hipError_t launch_verify(const VerifyArgs& args, hipStream_t s) {
    VerifyArgs a = args;
    const uint32_t batch = static_cast<uint32_t>(a.batch);
    uint32_t per, parts = verify_parts(kDrawGroups, batch, a.chunks, &per);
    if (!a.draft || !a.parents) {
        k_verify<256, false><<<batch * parts, 256, 0, s>>>(a, parts, per);
        return hipGetLastError();
    }
    const bool wide = a.chunks >= kFirstChunks;
    a.first_parts = wide ? parts : 0;
    if (wide) k_verify_first<256><<<batch * parts, 256, 0, s>>>(a, parts, per);
    parts = verify_parts(wide ? kDrawnGroupsWide : kDrawnGroups, batch, a.chunks, &per);
    k_verify<1024, true><<<batch * parts, 1024, 0, s>>>(a, parts, per);
    return hipGetLastError();
}

}  // namespace kvc
