// Rows moved together in the pages, pages shared by several requests and
// given back (declared in include/kvc.h).
#include <hip/hip_runtime.h>

#include "kvc_paged.hpp"
#include "kvc_step.hpp"
#include "kvc_wave.hpp"

namespace kvc {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- compaction

constexpr int kCompactThreads = 256;
constexpr int kAtOnce = 8;                      // rows that a thread reads before it writes any

// A thread has 16 bytes of a sequence's rows in one pool and moves them row
// after row: row j goes to place j from a place at or behind it, and places
// rise, so that what is written was read before by the same thread.
__global__ __launch_bounds__(kCompactThreads) void k_compact(CompactArgs a, uint32_t blocks) {
    __shared__ int64_t from[64], to[64];        // slots; from -1: stays
    __shared__ uint32_t moves;
    const int64_t b = blockIdx.x / blocks;
    const uint32_t block = blockIdx.x - static_cast<uint32_t>(b) * blocks;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t start = a.row_starts[b], n = a.row_starts[b + 1] - start;
    const int64_t context = a.context ? a.context[b] : 0, kept = a.kept_lens[b];
    bool bad = start < 0 || n < 0 || start + n > a.rows || context < 0 || kept < 0 || kept > n ||
               context + n > a.g.max_pages * int64_t(a.g.page_tokens) || context + n > 0x7FFFFFFF;
    if (!bad) {
        bool wrong = false;
        for (int64_t j = tid; j < kept; j += kCompactThreads) {
            const int32_t at = a.kept[start + j], before = j ? a.kept[start + j - 1] : -1;
            wrong = wrong || at <= before || at < 0 || at >= n;
        }
        bad = __syncthreads_or(wrong);
    }
    if (block == 0 && tid == 0) {
        if (b == 0) *a.ctl = CompactControl{kPagedMagic, static_cast<uint32_t>(a.g.batch)};
        a.words[b] = bad ? kPagedInvalid : 0u;
    }
    if (bad) return;
    const uint64_t all = uint64_t(a.g.n_pools) * a.g.pieces;
    const int32_t* const table = a.table + b * a.g.max_pages;
    for (int64_t j0 = 0; j0 < kept; j0 += 64) {
        if (tid < 64) {
            const int64_t j = j0 + lane;
            int64_t x = -1, y = -1;
            bool unsound = false;
            if (j < kept) {
                const int32_t node = a.kept[start + j];
                if (node != j) {
                    const uint32_t s = static_cast<uint32_t>(context + node), d = static_cast<uint32_t>(context + j);
                    const uint32_t sp = s / a.g.page_tokens, dp = d / a.g.page_tokens;
                    const int64_t source = table[sp], target = table[dp];
                    unsound = source < 0 || source >= a.g.num_pages || target < 0 || target >= a.g.num_pages;
                    if (!unsound) {
                        x = source * a.g.page_tokens + (s - sp * a.g.page_tokens);
                        y = target * a.g.page_tokens + (d - dp * a.g.page_tokens);
                    }
                }
            }
            // the moves, one after the other
            const uint64_t move = __ballot(x >= 0);
            const int at = __builtin_popcountll(move & ((uint64_t(1) << lane) - 1));
            if (x >= 0) {
                from[at] = x;
                to[at] = y;
            }
            if (lane == 0) moves = __builtin_popcountll(move);
            if (block == 0 && __any(unsound) && lane == 0) a.words[b] = kPagedInvalid;
        }
        __syncthreads();
        const uint32_t count = moves;
        for (uint64_t i = uint64_t(block) * kCompactThreads + tid; i < all; i += uint64_t(blocks) * kCompactThreads) {
            const uint32_t pool = static_cast<uint32_t>(i / a.g.pieces), piece = static_cast<uint32_t>(i - uint64_t(pool) * a.g.pieces);
            u32x4* const base = static_cast<u32x4*>(a.g.pools[pool]) + piece;
            for (uint32_t m = 0; m < count; m += kAtOnce) {
                u32x4 x[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) x[k] = base[from[m + k < count ? m + k : m] * a.g.pieces];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (m + k < count) base[to[m + k] * a.g.pieces] = x[k];
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- forks

constexpr int kForkThreads = 1024;

// Whether all of a fork can be done, and its entries: one workgroup.
__global__ __launch_bounds__(kForkThreads) void k_fork_plan(SharedArgs a) {
    __shared__ int32_t children[kMaxShared];
    __shared__ uint32_t of_wave[kForkThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t count = *a.free_in;
    ForkEntry e{-1, -1, 0, 0, -1, -1};
    bool wrong = count < 0 || count > a.free_capacity;
    if (tid < a.count) {
        e.child = a.children[tid];
        e.parent = a.parents[tid];
    }
    children[tid] = e.child;
    __syncthreads();
    uint32_t need = 0;
    if (e.child != -1) {
        const bool in = e.child >= 0 && e.child < a.g.batch && e.parent >= 0 && e.parent < a.g.batch && e.parent != e.child;
        wrong = wrong || !in;
        if (in) {
            const int64_t tokens = a.context ? a.context[e.parent] : 0, held = a.held_in[e.parent];
            const int64_t pages = tokens > 0 ? (tokens + a.g.page_tokens - 1) / a.g.page_tokens : 0;
            if (tokens < 0 || held > a.g.max_pages || pages > held || a.held_in[e.child] != 0) {
                wrong = true;
            } else {
                e.whole = static_cast<int32_t>(tokens / a.g.page_tokens);
                e.rest = static_cast<int32_t>(tokens - int64_t(e.whole) * a.g.page_tokens);
                need = e.rest > 0;
                if (need) e.from = a.table[int64_t(e.parent) * a.g.max_pages + e.whole];
            }
        }
        for (int k = 0; k < tid; ++k) wrong = wrong || children[k] == e.child;
    }
    const uint32_t upto = scan(need);
    if (lane == 63) of_wave[wave] = upto;
    wrong = __syncthreads_or(wrong);
    uint32_t before = 0, all = 0;
    for (int w = 0; w < kForkThreads / 64; ++w) {
        if (w < wave) before += of_wave[w];
        all += of_wave[w];
    }
    const bool room = int64_t(all) <= count;
    bool unsound = false;
    if (!wrong && room && need) {
        e.page = a.free_pages[count - 1 - (before + upto - 1)];
        unsound = e.page < 0 || e.page >= a.g.num_pages || e.from < 0 || e.from >= a.g.num_pages;
    }
    wrong = __syncthreads_or(wrong || unsound);
    const bool go = !wrong && room;
    for (int64_t b = tid; b < a.g.batch; b += kForkThreads) a.held_out[b] = a.held_in[b];
    __syncthreads();
    if (go && e.child >= 0) a.held_out[e.child] = e.whole + static_cast<int32_t>(need);
    if (tid < a.count) a.entries[tid] = e;
    if (tid == 0) {
        *a.free_out = static_cast<int32_t>(go ? count - all : count);
        a.ctl->magic = kPagedMagic;
        a.ctl->flags = wrong ? kPagedInvalid : room ? 0u : kPagedCapacity;
        a.ctl->entries = go ? a.count : 0;
    }
}

constexpr int kFillThreads = 256;

// The children's rows of the table and the counts of holders (the first
// `tables` workgroups of an entry), and the tokens of unfilled pages.
__global__ __launch_bounds__(kFillThreads) void k_fork_fill(SharedArgs a, uint32_t tables, uint32_t copies) {
    const uint32_t k = blockIdx.x / (tables + copies), block = blockIdx.x - k * (tables + copies);
    if (static_cast<int32_t>(k) >= a.ctl->entries) return;
    const ForkEntry e = a.entries[k];
    if (e.child < 0) return;
    if (block < tables) {
        const int32_t* const from = a.table + int64_t(e.parent) * a.g.max_pages;
        int32_t* const to = a.table + int64_t(e.child) * a.g.max_pages;
        bool unsound = false;
        for (int64_t j = int64_t(block) * kFillThreads + threadIdx.x; j < e.whole; j += int64_t(tables) * kFillThreads) {
            const int32_t page = from[j];
            to[j] = page;
            if (page >= 0 && page < a.g.num_pages) atomicAdd(&a.extra[page], 1);
            else unsound = true;
        }
        if (block == 0 && threadIdx.x == 0 && e.page >= 0) to[e.whole] = e.page;
        if (unsound) atomicOr(&a.ctl->flags, kPagedInvalid);
        return;
    }
    if (e.page < 0) return;
    const uint64_t each = uint64_t(e.rest) * a.g.pieces, page = uint64_t(a.g.page_tokens) * a.g.pieces;
    const uint64_t all = each * a.g.n_pools;
    for (uint64_t i = uint64_t(block - tables) * kFillThreads + threadIdx.x; i < all; i += uint64_t(copies) * kFillThreads) {
        const uint64_t pool = i / each, piece = i - pool * each;
        u32x4* const base = static_cast<u32x4*>(a.g.pools[pool]) + piece;
        base[e.page * page] = base[e.from * page];
    }
}

// ---------------------------------------------------------------- releases

// Every page of the requests loses a holder; those that had one only are
// marked.  (Their counts are then -1, and set to 0 again when they are given
// back.)
__global__ __launch_bounds__(kFillThreads) void k_release_mark(SharedArgs a, uint32_t blocks) {
    const uint32_t k = blockIdx.x / blocks, block = blockIdx.x - k * blocks;
    const int32_t count = *a.free_in;
    if (count < 0 || count > a.free_capacity) return;           // (reported behind)
    const int32_t row = a.children[k];
    if (row == -1) return;
    bool wrong = false;
    for (uint32_t i = threadIdx.x; i < k; i += kFillThreads) wrong = wrong || a.children[i] == row;
    wrong = __syncthreads_or(wrong || row < 0 || row >= a.g.batch);
    const int64_t held = wrong ? 0 : a.held_in[row];
    if (held < 0 || held > a.g.max_pages) wrong = true;
    if (!wrong) {
        const int32_t* const table = a.table + int64_t(row) * a.g.max_pages;
        for (int64_t j = int64_t(block) * kFillThreads + threadIdx.x; j < held; j += int64_t(blocks) * kFillThreads) {
            const int32_t page = table[j];
            if (page < 0 || page >= a.g.num_pages) {
                wrong = true;
                continue;
            }
            const int32_t others = atomicSub(&a.extra[page], 1);
            if (others == 0) atomicOr(&a.bits[page >> 5], 1u << (page & 31));
            else if (others < 0) wrong = true;
        }
    }
    if (wrong) atomicOr(&a.ctl->pending, kPagedInvalid);
}

// The marked pages go to the stack, the highest on top: one workgroup.
__global__ __launch_bounds__(kForkThreads) void k_release_push(SharedArgs a) {
    __shared__ uint32_t of_wave[kForkThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t count = *a.free_in;
    const bool sound = count >= 0 && count <= a.free_capacity;
    for (int64_t b = tid; b < a.g.batch; b += kForkThreads) a.held_out[b] = a.held_in[b];
    __syncthreads();
    if (sound && tid < a.count) {
        const int32_t row = a.children[tid];
        if (row >= 0 && row < a.g.batch && a.held_out[row] >= 0 && a.held_out[row] <= a.g.max_pages) a.held_out[row] = 0;
    }
    int64_t at = count;
    const int64_t words = (a.g.num_pages + 31) / 32;
    bool full = false;
    for (int64_t w0 = 0; sound && w0 < words; w0 += kForkThreads) {
        const int64_t w = w0 + tid;
        uint32_t bits = w < words ? a.bits[w] : 0u;
        const uint32_t mine = __builtin_popcount(bits), upto = scan(mine);
        if (lane == 63) of_wave[wave] = upto;
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int i = 0; i < kForkThreads / 64; ++i) {
            if (i < wave) before += of_wave[i];
            all += of_wave[i];
        }
        __syncthreads();
        if (bits) a.bits[w] = 0u;
        int64_t place = at + before + upto - mine;
        for (; bits; bits &= bits - 1, ++place) {
            const int32_t page = static_cast<int32_t>(w * 32 + __builtin_ctz(bits));
            a.extra[page] = 0;
            if (place < a.free_capacity) a.free_pages[place] = page;
            else full = true;
        }
        at += all;
    }
    full = __syncthreads_or(full);
    if (tid == 0) {
        *a.free_out = static_cast<int32_t>(at < a.free_capacity || !sound ? at : a.free_capacity);
        a.ctl->magic = kPagedMagic;
        a.ctl->flags = (sound ? 0u : kPagedInvalid) | a.ctl->pending | (full ? kPagedCapacity : 0u);
        a.ctl->pending = 0u;
    }
}

}  // namespace

hipError_t launch_compact(const CompactArgs& a, hipStream_t s) {
    const uint64_t all = uint64_t(a.g.n_pools) * a.g.pieces;
    uint64_t blocks = (all + kCompactThreads - 1) / kCompactThreads;
    const uint64_t most = (uint64_t(1) << 23) / uint64_t(a.g.batch);
    if (blocks > most) blocks = most;
    if (blocks > 1024) blocks = 1024;
    k_compact<<<static_cast<uint32_t>(a.g.batch * blocks), kCompactThreads, 0, s>>>(a, static_cast<uint32_t>(blocks));
    return hipGetLastError();
}

hipError_t launch_fork(const SharedArgs& a, hipStream_t s) {
    k_fork_plan<<<1, kForkThreads, 0, s>>>(a);
    if (a.count == 0) return hipGetLastError();
    int64_t tables = (a.g.max_pages + 4 * kFillThreads - 1) / (4 * kFillThreads);
    if (tables > 64) tables = 64;
    const uint64_t most = uint64_t(a.g.n_pools) * (a.g.page_tokens - 1) * a.g.pieces;
    uint64_t copies = (most + 4 * kFillThreads - 1) / (4 * kFillThreads);
    if (copies > 1024) copies = 1024;
    k_fork_fill<<<static_cast<uint32_t>(a.count * (tables + copies)), kFillThreads, 0, s>>>(
        a, static_cast<uint32_t>(tables), static_cast<uint32_t>(copies));
    return hipGetLastError();
}

hipError_t launch_release(const SharedArgs& a, hipStream_t s) {
    if (a.count) {
        int64_t blocks = (a.g.max_pages + 4 * kFillThreads - 1) / (4 * kFillThreads);
        if (blocks > 64) blocks = 64;
        k_release_mark<<<static_cast<uint32_t>(a.count * blocks), kFillThreads, 0, s>>>(a, static_cast<uint32_t>(blocks));
    }
    k_release_push<<<1, kForkThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace kvc
