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

// What is left of a probability p after `rejected` siblings drawn with
// probability q were rejected: each rejection takes q off and the next
// sibling meets the rest scaled to a sum of 1.
__device__ float left_of(float p, float q, const float* scales, int rejected) {
    float y = p;
    for (int k = 0; k < rejected; ++k) {
        if (k) y *= scales[k];
        y = fmaxf(y - q, 0.0f);
    }
    return y;
}

typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));     // (a row may begin at any value)

// Four values of a row from `at` on, 0 behind its end.
__device__ void load4(const float* row, uint32_t at, uint32_t vocab, float (&x)[4]) {
    if (at + 4 <= vocab) {
        const float4u y = *reinterpret_cast<const float4u*>(row + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = clean(y[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = at + i < vocab ? clean(row[at + i]) : 0.0f;
    }
}

// The sum over a workgroup, in every thread; a thread's halves are of at most
// VALUES values.  (A value is at most 1, up to what the scale after a
// rejection is off by where next to nothing was left; together they are less
// than 2 each, so that 1024 of them pass no 32 bits.)
template <int THREADS, int VALUES>
__device__ uint64_t block_sum(Units x, uint64_t* of_wave) {
    uint64_t all;
    if (VALUES * 64 <= 1024) {
        all = Units{of_lane(scan(x.high), 63), of_lane(scan(x.low), 63)}.all();
    } else {
        const uint32_t parts[3] = {x.high >> 16, x.high & 0xFFFFu, x.low >> 16};
        uint32_t sum[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) sum[i] = of_lane(scan(parts[i]), 63);
        all = ((uint64_t(sum[0]) << 16) + sum[1]) << 21;
        all += (uint64_t(sum[2]) << 16) + of_lane(scan(x.low & 0xFFFFu), 63);
    }
    if ((threadIdx.x & 63) == 63) of_wave[threadIdx.x >> 6] = all;
    __syncthreads();
    uint64_t sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) sum += of_wave[w];
    __syncthreads();
    return sum;
}

// ---- the walk

struct Nodes {
    int32_t parent[kMaxNodes];                  // -1: of none that can be reached
    int32_t token[kMaxNodes];                   // -1: none of the vocabulary
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];
    int32_t path[kMaxNodes];
};

constexpr int kWalkThreads = 1024;

// A sequence's walk down its tree: nodes are looked at in order, those whose
// parent is the current node are tested, an accepted one becomes the current
// one.  Every wave takes it alike, so that all of them meet where a sum over
// the vocabulary is needed: before a sibling of a rejected node, where nodes
// were drawn from the draft's probabilities.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_verify_walk(VerifyArgs a) {
    __shared__ Nodes nodes;
    __shared__ float scales[kMaxNodes];
    __shared__ int32_t rejects[kMaxNodes];
    __shared__ uint64_t of_wave[THREADS / 64];
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    if (b == 0 && tid == 0) *a.ctl = VerifyControl{kPagedMagic, static_cast<uint32_t>(a.batch)};
    const int64_t start = a.row_starts[b], end = a.row_starts[b + 1];
    const bool bad = start < 0 || end < start || end > a.rows || end - start > kMaxNodes;
    const int n = bad ? 0 : static_cast<int>(end - start);
    if (n == 0) {
        if (tid == 0) {
            a.kept_lens[b] = 0;
            a.words[2 * b] = bad ? kPagedInvalid : 0u;
            a.states[b] = VerifyState{0, 0, 0, 0, 0, {0, 0, 0}};
        }
        return;
    }
    bool wrong = false;
    for (int i = tid; i < n; i += THREADS) {
        const int64_t r = start + i;
        int parent = a.parents ? a.parents[r] : i - 1;
        int token = a.tokens[r];
        if (i > 0 && (parent < 0 || parent >= i)) wrong = true;
        if (i > 0 && (token < 0 || token >= static_cast<int64_t>(a.vocab))) {
            wrong = true;
            token = -1;
        }
        if (i == 0 || parent < 0 || parent >= i) parent = -1;
        const bool there = parent >= 0 && token >= 0;
        nodes.parent[i] = parent;
        nodes.token[i] = token;
        nodes.u[i] = a.accept[r];
        nodes.p[i] = there ? clean(a.target[(start + parent) * a.target_row + token]) : 0.0f;
        nodes.q[i] = there && a.draft ? clean(a.draft[(start + parent) * a.draft_row + token]) : 0.0f;
    }
    wrong = __syncthreads_or(wrong);
    int current = 0, kept = 1, rejected = 0, listed = 0;
    uint64_t mass = uint64_t(1) << 42;          // without probabilities: of tokens that were not rejected
    if (tid == 0) nodes.path[0] = 0;
    for (int base = 0; base < n; base += 64) {
        const int i = base + lane;
        const int parent = i < n ? nodes.parent[i] : -1;
        uint64_t ahead = ~uint64_t(0);          // nodes behind the last one tested
        for (;;) {
            const uint64_t next = __ballot(parent == current) & ahead;
            if (!next) break;
            const int bit = __builtin_ctzll(next), j = base + bit;
            ahead = bit == 63 ? 0 : ~uint64_t(0) << (bit + 1);
            const double u = nodes.u[j];
            const float p = nodes.p[j], q = nodes.q[j];
            const int token = nodes.token[j];
            bool ok, again = false;
            if (a.draft) {
                if (rejected > 0) {
                    // what the rejections left, over the whole vocabulary
                    const float* const target = a.target + (start + current) * a.target_row;
                    const float* const draft = a.draft + (start + current) * a.draft_row;
                    Units sum{0, 0};
                    for (uint32_t at = 4 * tid; at < a.vocab; at += 4 * THREADS) {
                        float x[4], y[4];
                        load4(target, at, a.vocab, x);
                        load4(draft, at, a.vocab, y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum.add(units_of(left_of(x[e], y[e], scales, rejected)));
                    }
                    const uint64_t z = block_sum<THREADS, kMaxVocab / THREADS>(sum, of_wave);
                    if (tid == 0) scales[rejected] = z ? static_cast<float>(0x1p42 / static_cast<double>(z)) : 0.0f;
                    __syncthreads();
                }
                float y = left_of(p, q, scales, rejected);
                if (rejected) y *= scales[rejected];
                ok = u * double(q) < double(y);
            } else {
                for (int k = lane; k < listed; k += 64) again = again || rejects[k] == token;
                again = __any(again);
                const float y = again ? 0.0f : p;
                ok = u * static_cast<double>(mass) < double(y) * 0x1p42;
            }
            if (ok) {
                current = j;
                if (tid == 0) nodes.path[kept] = j;
                ++kept;
                rejected = listed = 0;
                mass = uint64_t(1) << 42;
            } else {
                ++rejected;
                if (!a.draft && !again && token >= 0) {
                    __syncthreads();            // (every wave has read the list)
                    if (tid == 0) rejects[listed] = token;
                    __syncthreads();
                    ++listed;
                    const uint64_t w = units_of(p).all();
                    mass = mass > w ? mass - w : 0;
                }
            }
        }
    }
    __syncthreads();
    const int entries = a.draft ? rejected : listed;
    for (int k = tid; k < entries; k += THREADS) {
        if (a.draft) a.scales[start + k] = k ? scales[k] : 0.0f;
        else a.rejects[start + k] = rejects[k];
    }
    for (int j = tid; j < n; j += THREADS) {
        a.kept[start + j] = j < kept ? nodes.path[j] : -1;
        a.out_tokens[start + j] = j + 1 < kept ? nodes.token[nodes.path[j + 1]] : -1;
    }
    if (tid == 0) {
        a.kept_lens[b] = kept;
        a.words[2 * b] = wrong ? kPagedInvalid : 0u;
        a.states[b] = VerifyState{static_cast<int32_t>(start), n, static_cast<int32_t>(start) + current,
                                  static_cast<int32_t>(start) + kept - 1, entries, {0, 0, 0}};
    }
}

// ---- the draw

constexpr int kSumThreads = 256;
constexpr int kGroups = kVerifyChunk / (4 * kSumThreads);

// The units of a chunk of the distribution that a sequence draws from.
__global__ __launch_bounds__(kSumThreads) void k_verify_sums(VerifyArgs a) {
    __shared__ uint64_t of_wave[kSumThreads / 64];
    const uint32_t b = blockIdx.x / a.chunks, chunk = blockIdx.x - b * a.chunks;
    const VerifyState s = a.states[b];
    if (s.rows == 0) return;
    const float* const target = a.target + s.stop * a.target_row;
    const float* const draft = a.draft + s.stop * a.draft_row;
    const float* const scales = a.scales + s.start;
    const bool both = a.draft && s.rejected > 0;
    const uint32_t base = chunk * kVerifyChunk, tid = threadIdx.x;
    float x[kGroups][4], y[kGroups][4];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) load4(target, base + 4 * (g * kSumThreads + tid), a.vocab, x[g]);
    Units whole{0, 0}, left{0, 0};
    if (both) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) load4(draft, base + 4 * (g * kSumThreads + tid), a.vocab, y[g]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) left.add(units_of(left_of(x[g][e], y[g][e], scales, s.rejected)));
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) whole.add(units_of(x[g][e]));
    if (!both) {
        left = whole;
        // tokens that were rejected are taken out by the thread that has their values
        for (int k = 0; k < s.rejected; ++k) {
            const uint32_t token = static_cast<uint32_t>(a.rejects[s.start + k]), at = token - base;
            if (at >= uint32_t(kVerifyChunk) || (at >> 2) % kSumThreads != tid) continue;
            const Units w = units_of(clean(target[token]));
            left.high -= w.high;
            left.low -= w.low;
        }
    }
    const uint64_t l = block_sum<kSumThreads, 4 * kGroups>(left, of_wave),
                   w = block_sum<kSumThreads, 4 * kGroups>(whole, of_wave);
    if (tid == 0) a.sums[blockIdx.x] = VerifySums{l, w};
}

constexpr int kPickThreads = kVerifyChunk / 4;

// The token at which the sum in the vocabulary's order passes the drawn point.
__global__ __launch_bounds__(kPickThreads) void k_verify_pick(VerifyArgs a) {
    __shared__ uint64_t of_wave[kPickThreads / 64];
    const uint32_t b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const VerifyState s = a.states[b];
    if (s.rows == 0) {
        if (tid == 0) a.words[2 * b + 1] = 0u;
        return;
    }
    const VerifySums* const sums = a.sums + uint64_t(b) * a.chunks;
    uint64_t left = 0, whole = 0;
    for (uint32_t c = 0; c < a.chunks; ++c) {
        left += sums[c].left;
        whole += sums[c].whole;
    }
    const bool nothing = left == 0;             // the target's own probabilities then
    const uint64_t total = nothing ? whole : left;
    if (total == 0) {
        if (tid == 0) a.words[2 * b + 1] = kPagedInvalid;
        return;
    }
    const float u = a.sample[b];
    uint64_t point = u > 0.0f ? static_cast<uint64_t>(fmin(double(u), 1.0) * static_cast<double>(total)) : 0;
    if (point >= total) point = total - 1;
    uint64_t before = 0;
    uint32_t chunk = 0;
    for (; chunk + 1 < a.chunks; ++chunk) {
        const uint64_t here = nothing ? sums[chunk].whole : sums[chunk].left;
        if (before + here > point) break;
        before += here;
    }
    const float* const target = a.target + s.stop * a.target_row;
    const uint32_t at = chunk * kVerifyChunk + 4 * tid;
    float x[4];
    load4(target, at, a.vocab, x);
    if (!nothing && a.draft && s.rejected > 0) {
        float y[4];
        load4(a.draft + s.stop * a.draft_row, at, a.vocab, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = left_of(x[e], y[e], a.scales + s.start, s.rejected);
    } else if (!nothing && !a.draft) {
        for (int k = 0; k < s.rejected; ++k) {
            const uint32_t token = static_cast<uint32_t>(a.rejects[s.start + k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = token == at + e ? 0.0f : x[e];
        }
    }
    Units w[4], mine{0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[e] = units_of(x[e]);
        mine.add(w[e]);
    }
    const uint64_t upto = Units{scan(mine.high), scan(mine.low)}.all();     // within the wave
    if (lane == 63) of_wave[tid >> 6] = upto;
    __syncthreads();
    uint64_t sum = before + upto - mine.all();
    for (uint32_t k = 0; k < tid >> 6; ++k) sum += of_wave[k];
    if (sum <= point && point < sum + mine.all()) {
        int e = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            sum += w[i].all();
            if (sum <= point) e = i + 1;
        }
        a.out_tokens[s.last] = static_cast<int32_t>(at + e);
        a.words[2 * b + 1] = 0u;
    }
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
    if (a.draft && a.parents) k_verify_walk<kWalkThreads><<<static_cast<uint32_t>(a.batch), kWalkThreads, 0, s>>>(a);
    else k_verify_walk<64><<<static_cast<uint32_t>(a.batch), 64, 0, s>>>(a);
    k_verify_sums<<<static_cast<uint32_t>(a.batch * a.chunks), kSumThreads, 0, s>>>(a);
    k_verify_pick<<<static_cast<uint32_t>(a.batch), kPickThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace kvc
