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
// rise, so that what is written was read before by the same thread.  Every
// workgroup checks its sequence and finds its moves for itself, 64 at a time.
// Bound by memory (128 trees, 36 layers, 114 MB: 23.0 us, 4.9 TB/s, 24.9 us with
// stores that stay in the caches; 31 us where the last-level cache has none of the
// rows), for small batches by five trips to memory (4.1 us on the GPU).
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
        if (b == 0) *a.ctl = CompactControl{kCompactMagic, static_cast<uint32_t>(a.g.batch)};
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
            const uint32_t pool = static_cast<uint32_t>(all >> 32 ? i / a.g.pieces : static_cast<uint32_t>(i) / a.g.pieces);
            const uint32_t piece = static_cast<uint32_t>(i - uint64_t(pool) * a.g.pieces);
            u32x4* const base = static_cast<u32x4*>(a.g.pools[pool]) + piece;
            for (uint32_t m = 0; m < count; m += kAtOnce) {
                u32x4 x[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) x[k] = base[from[m + k < count ? m + k : m] * a.g.pieces];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (m + k < count) __builtin_nontemporal_store(x[k], base + to[m + k] * a.g.pieces);
            }
        }
        __syncthreads();
    }
}

// Whether this workgroup is the last of the launch to arrive, for all of its
// threads.  What the others read they have read by then, and what they did
// with atomics is done: every wave waits for its own.  Workgroups count in 16
// places first (one place takes 13 ns each, 544 of them 7 us), whose last ones
// count once more; all counts are 0 again behind the last.
__device__ uint32_t count_in(uint32_t* at, uint32_t all) {
    const uint32_t n = __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (n != all - 1) return 0;
    __hip_atomic_store(at, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return 1;
}
__device__ bool last_to_arrive(const SharedArgs& a, uint32_t* lds) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t place = blockIdx.x % kArrivals, here = (gridDim.x - place + kArrivals - 1) / kArrivals;
        if (gridDim.x <= 4 * kArrivals) *lds = count_in(&a.ctl->arrived, gridDim.x);
        else *lds = count_in(a.arrivals + place * kArrivalStride, here) ? count_in(&a.ctl->arrived, kArrivals) : 0u;
    }
    __syncthreads();
    return *lds;
}

// ---------------------------------------------------------------- forks

constexpr int kForkThreads = 256;
constexpr int kForkSlice = 4 * kForkThreads;                // pages, or pieces of 16 bytes, of a work item

struct ForkEntry {
    int32_t parent, child;              // -1: none
    int32_t whole, rest;                // the parent's full pages; tokens of its last one
    int32_t page;                       // the page that these are copied to; -1: none
    int32_t from;                       // ... and from
    int32_t holders;                    // that the full pages get, for all children of the parent: one entry has them
};
struct ForkPlan {
    ForkEntry entries[kMaxShared];
    int32_t seen[2][2 * kMaxShared];    // children and parents, by their hash; -1: none
    int32_t sharing[2 * kMaxShared];    // children of such a parent
    uint32_t of_wave[kForkThreads / 64];
    uint32_t all;                       // pages taken from the stack
    int32_t count;                      // its height before
};

// The place of a number in a table of 2 kMaxShared, of which at most half are
// taken; first: it was not there before.
__device__ int enter(int32_t* table, int32_t x, bool& first) {
    uint32_t at = (static_cast<uint32_t>(x) * 2654435761u) >> 21;
    static_assert(2 * kMaxShared == 1 << 11, "the hash's bits");
    for (;;) {
        const int32_t other = atomicCAS(&table[at], -1, x);
        first = other == -1;
        if (first || other == x) return static_cast<int>(at);
        at = (at + 1) % (2 * kMaxShared);
    }
}

// Whether all of a fork can be done (a status), and its entries, kForkThreads
// at a time.
__device__ uint32_t plan_fork(const SharedArgs& a, ForkPlan& p) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t count = *a.free_in;
    for (int i = tid; i < 2 * kMaxShared; i += kForkThreads) {
        p.seen[0][i] = p.seen[1][i] = -1;
        p.sharing[i] = 0;
    }
    bool wrong = count < 0 || count > a.free_capacity;
    uint32_t taken = 0;                         // pages, by the entries of the rounds before
    for (int k0 = 0; k0 < a.count; k0 += kForkThreads) {
        const int k = k0 + tid;
        ForkEntry e{-1, -1, 0, 0, -1, -1, -1};
        if (k < a.count) {
            e.child = a.children[k];
            e.parent = a.parents[k];
        }
        __syncthreads();                        // (the tables are empty; the last round's counts are read)
        uint32_t need = 0;
        const bool in = e.child >= 0 && e.child < a.g.batch && e.parent >= 0 && e.parent < a.g.batch && e.parent != e.child;
        if (in) {
            const int32_t tokens = a.context ? a.context[e.parent] : 0;
            const int32_t held = a.held_in[e.parent], mine = a.held_in[e.child];
            bool first;
            enter(p.seen[0], e.child, first);
            wrong = wrong || !first;
            e.holders = enter(p.seen[1], e.parent, first);      // (its place, for now)
            atomicAdd(&p.sharing[e.holders], 1);
            e.whole = tokens > 0 ? static_cast<int32_t>(static_cast<uint32_t>(tokens) / a.g.page_tokens) : 0;
            e.rest = tokens - e.whole * static_cast<int32_t>(a.g.page_tokens);
            need = e.rest > 0;
            if (tokens < 0 || held > a.g.max_pages || e.whole + int64_t(need) > held || mine != 0) {
                wrong = true;
                need = 0;
            }
            if (need) e.from = a.table[int64_t(e.parent) * a.g.max_pages + e.whole];
        } else if (e.child != -1) {
            wrong = true;
        }
        const uint32_t upto = scan(need);
        if (lane == 63) p.of_wave[wave] = upto;
        __syncthreads();
        uint32_t before = taken + upto - need;
        for (int w = 0; w < kForkThreads / 64; ++w) {
            if (w < wave) before += p.of_wave[w];
            taken += p.of_wave[w];
        }
        if (need && before < count && count <= a.free_capacity) {
            e.page = a.free_pages[count - 1 - before];
            wrong = wrong || e.page < 0 || e.page >= a.g.num_pages || e.from < 0 || e.from >= a.g.num_pages;
        }
        if (k < a.count) p.entries[k] = e;
    }
    // a parent's new holders are one entry's, the first's (the same in every workgroup)
    __syncthreads();
    for (int k = tid; k < a.count; k += kForkThreads)
        if (p.entries[k].holders >= 0) p.seen[1][p.entries[k].holders] = kMaxShared;
    __syncthreads();
    for (int k = tid; k < a.count; k += kForkThreads)
        if (p.entries[k].holders >= 0) atomicMin(&p.seen[1][p.entries[k].holders], k);
    __syncthreads();
    for (int k = tid; k < a.count; k += kForkThreads) {
        const int32_t at = p.entries[k].holders;
        p.entries[k].holders = at >= 0 && p.seen[1][at] == k ? p.sharing[at] : 0;
    }
    if (tid == 0) {
        p.all = taken;
        p.count = static_cast<int32_t>(count);
    }
    wrong = __syncthreads_or(wrong);
    return wrong ? kPagedInvalid : int64_t(taken) <= count ? 0u : kPagedCapacity;
}

// Every workgroup plans the fork for itself (a chain of four trips to memory,
// as long as a kernel of its own would take) and takes work items in turn:
// for each child `tables` slices of its row of the table (a parent's pages get
// all their new holders at once, from one of its children: 256 children of 32
// prompts 15.7 -> 11.2 us) and `copies` of the tokens of its unfilled page.
// The last workgroup to be done enters the new state, which the others may
// still have to read.
__global__ __launch_bounds__(kForkThreads) void k_fork(SharedArgs a, uint32_t tables, uint32_t copies) {
    __shared__ ForkPlan p;
    __shared__ uint32_t order;
    const int tid = threadIdx.x;
    const uint32_t status = plan_fork(a, p);
    const uint32_t slices = tables + copies, items = status ? 0u : static_cast<uint32_t>(a.count) * slices;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t k = item / slices, slice = item - k * slices;
        const ForkEntry e = p.entries[k];
        if (e.child < 0) continue;
        if (slice < tables) {
            const int32_t* const from = a.table + int64_t(e.parent) * a.g.max_pages;
            int32_t* const to = a.table + int64_t(e.child) * a.g.max_pages;
            bool unsound = false;
            for (int64_t j0 = int64_t(slice) * kForkSlice; j0 < e.whole; j0 += int64_t(tables) * kForkSlice) {
                int32_t page[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t j = j0 + i * kForkThreads + tid;
                    page[i] = j < e.whole ? from[j] : -1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t j = j0 + i * kForkThreads + tid;
                    if (j >= e.whole) continue;
                    to[j] = page[i];
                    if (page[i] < 0 || page[i] >= a.g.num_pages) unsound = true;
                    else if (e.holders) atomicAdd(&a.extra[page[i]], e.holders);
                }
            }
            if (slice == 0 && tid == 0 && e.page >= 0) to[e.whole] = e.page;
            if (unsound) atomicOr(&a.ctl->pending, kPagedInvalid);
            continue;
        }
        if (e.page < 0) continue;
        const uint64_t each = uint64_t(e.rest) * a.g.pieces, page = uint64_t(a.g.page_tokens) * a.g.pieces;
        const uint64_t all = each * a.g.n_pools;
        for (uint64_t i0 = uint64_t(slice - tables) * kForkSlice; i0 < all; i0 += uint64_t(copies) * kForkSlice) {
            u32x4 x[4];
            u32x4* at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t piece = i0 + i * kForkThreads + tid < all ? i0 + i * kForkThreads + tid : all - 1;
                const uint64_t pool = all >> 32 ? piece / each : static_cast<uint32_t>(piece) / static_cast<uint32_t>(each);
                at[i] = static_cast<u32x4*>(a.g.pools[pool]) + (piece - pool * each);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = at[i][e.from * page];
#pragma unroll
            for (int i = 0; i < 4; ++i) __builtin_nontemporal_store(x[i], at[i] + e.page * page);
        }
    }
    if (!last_to_arrive(a, &order)) return;
    uint32_t pending = 0;                       // (asked for now, needed at the end)
    if (tid == 0) pending = __hip_atomic_exchange(&a.ctl->pending, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (a.held_out != a.held_in) {
        for (int64_t b = tid; b < a.g.batch; b += kForkThreads) a.held_out[b] = a.held_in[b];
        __syncthreads();
    }
    if (!status)
        for (int k = tid; k < a.count; k += kForkThreads)
            if (p.entries[k].child >= 0) a.held_out[p.entries[k].child] = p.entries[k].whole + (p.entries[k].rest > 0);
    if (tid == 0) {
        *a.free_out = status ? p.count : p.count - static_cast<int32_t>(p.all);
        a.ctl->magic = kSharedMagic;
        a.ctl->flags = status | pending;
    }
}

// ---------------------------------------------------------------- releases

constexpr int kReleaseThreads = 1024;
constexpr int kColumns = 4;                                 // of the table, of a work item
constexpr int kRowsAtOnce = kReleaseThreads / kColumns;
constexpr int kMerged = 2048;

// Every page of the requests loses a holder; those that have none left (their
// count passes 0) are marked, a bit a page.  A workgroup takes a few columns of
// all the requests' rows (four: 256 requests on 8 prompts 15.5 us, sixteen 16.8,
// both before the marks lay apart), where those that share a prompt have the
// same pages, and takes a page's holders off at once: they are counted in LDS,
// in a place by the page's hash (a page whose place is another's is counted
// down by itself).  The last workgroup to be done pushes the marked pages in the
// order of their numbers, clears marks and counts and enters the new state.
// Bound by its chain of trips to memory: requests, held counts, table, counts,
// marks, two arrivals, marks (10.5 us, 6.8 for four requests); in large pools by
// the last workgroup's way through all the marks, 64 bytes for 32 pages, 1024
// of them a turn, whatever was released (calls for 4 requests of 63 pages: 7.4 us
// of 4000 pages, 11.2 of 32768, 21 of 120000, 119 of a million).
__global__ __launch_bounds__(kReleaseThreads) void k_release(SharedArgs a) {
    __shared__ int32_t requests[kMaxShared], held_by[kMaxShared];
    __shared__ int32_t pages[kMerged], holders[kMerged];
    __shared__ uint32_t of_wave[kReleaseThreads / 64], order;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t count = *a.free_in;
    const bool sound = count >= 0 && count <= a.free_capacity;
    bool wrong = false;
    int32_t row = -1, held = 0;
    if (tid < a.count) row = a.children[tid];
    requests[tid] = row;
    if (row >= 0 && row < a.g.batch) held = a.held_in[row];
    else if (row != -1) wrong = true;
    const bool clears = row >= 0 && row < a.g.batch && held >= 0 && held <= a.g.max_pages;
    if (held < 0 || held > a.g.max_pages) {
        wrong = true;
        held = 0;
    }
    for (int i = tid; i < kMerged; i += kReleaseThreads) {
        pages[i] = -1;
        holders[i] = 0;
    }
    __syncthreads();
    if (row >= 0 && row < a.g.batch) {
        bool first;
        enter(pages, row, first);
        if (!first) {                           // it stands twice
            wrong = true;
            held = 0;
        }
    }
    __syncthreads();
    static_assert(kMerged == 2 * kMaxShared, "one table for both");
    for (int i = tid; i < kMerged; i += kReleaseThreads) pages[i] = -1;
    held_by[tid] = held;
    int64_t widest = 0;
    for (int w = 32; w; w >>= 1) {
        const int32_t other = __shfl_xor(held, w);
        held = held > other ? held : other;
    }
    if (lane == 0) of_wave[wave] = held;
    __syncthreads();
    for (int w = 0; w < kReleaseThreads / 64; ++w) widest = widest > of_wave[w] ? widest : of_wave[w];
    // what a page's count is behind the holders that leave
    const auto left_by = [&](int32_t page, int32_t left) {
        if (left < 0) atomicOr(&a.bits[(page >> 5) * kMarkStride], 1u << (page & 31));
        if (left < -1) wrong = true;
    };
    constexpr int kEach = kMerged / kReleaseThreads, kRounds = 4;
    for (int64_t j0 = int64_t(blockIdx.x) * kColumns; sound && j0 < widest; j0 += int64_t(gridDim.x) * kColumns) {
        const int64_t j = j0 + tid % kColumns;
        for (int k0 = 0; k0 < a.count; k0 += kRounds * kRowsAtOnce) {
            int32_t page[kRounds];
            bool there[kRounds];
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int k = k0 + i * kRowsAtOnce + tid / kColumns;
                there[i] = k < a.count && j < held_by[k];
                page[i] = there[i] ? a.table[int64_t(requests[k]) * a.g.max_pages + j] : -1;
            }
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                if (!there[i]) continue;
                if (page[i] < 0 || page[i] >= a.g.num_pages) {
                    wrong = true;
                    there[i] = false;
                    continue;
                }
                const uint32_t at = (static_cast<uint32_t>(page[i]) * 2654435761u) >> 21;
                static_assert(kMerged == 1 << 11, "the hash's bits");
                const int32_t other = atomicCAS(&pages[at], -1, page[i]);
                if (other == -1 || other == page[i]) {
                    atomicAdd(&holders[at], 1);
                    there[i] = false;
                }
            }
            int32_t left[kRounds];
#pragma unroll
            for (int i = 0; i < kRounds; ++i) left[i] = there[i] ? atomicSub(&a.extra[page[i]], 1) - 1 : 0;
#pragma unroll
            for (int i = 0; i < kRounds; ++i) left_by(page[i], left[i]);
        }
        __syncthreads();
        int32_t page[kEach], left[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * kReleaseThreads + tid;
            page[i] = pages[at];
            left[i] = page[i] >= 0 ? atomicSub(&a.extra[page[i]], holders[at]) - holders[at] : 0;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * kReleaseThreads + tid;
            left_by(page[i], left[i]);
            pages[at] = -1;
            holders[at] = 0;
        }
        __syncthreads();
    }
    if (wrong) atomicOr(&a.ctl->pending, kPagedInvalid);
    if (!last_to_arrive(a, &order)) return;
    uint32_t pending = 0;                       // (asked for now, needed at the end)
    if (tid == 0) pending = __hip_atomic_exchange(&a.ctl->pending, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (a.held_out != a.held_in) {
        for (int64_t b = tid; b < a.g.batch; b += kReleaseThreads) a.held_out[b] = a.held_in[b];
        __syncthreads();
    }
    if (sound && clears) a.held_out[row] = 0;
    // 1024 words of marks at a time: their places on the stack first, then a lane a page
    int64_t at = count;
    const int64_t words = (a.g.num_pages + 31) / 32;
    uint32_t* const marks = reinterpret_cast<uint32_t*>(pages);
    int32_t* const places = holders;
    for (int64_t w0 = 0; sound && w0 < words; w0 += kReleaseThreads) {
        const int64_t w = w0 + tid;
        const uint32_t bits = w < words ? __hip_atomic_load(&a.bits[w * kMarkStride], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
        const uint32_t mine = __builtin_popcount(bits), upto = scan(mine);
        if (w0) __syncthreads();                // (the last words' are read)
        if (lane == 63) of_wave[wave] = upto;
        marks[tid] = bits;
        places[tid] = static_cast<int32_t>(upto - mine);    // within the wave's 64 words
        __syncthreads();
        uint32_t before[kReleaseThreads / 64], all = 0;
        for (int i = 0; i < kReleaseThreads / 64; ++i) {
            before[i] = all;
            all += of_wave[i];
        }
        const int pairs = !all ? 0 : words - w0 < kReleaseThreads ? static_cast<int>(words - w0 + 1) / 2 : kReleaseThreads / 2;
        constexpr int kPairs = 4;               // of a wave, looked up together
        for (int pair0 = kPairs * wave; pair0 < pairs; pair0 += kPairs * (kReleaseThreads / 64)) {
            uint32_t word[kPairs], from[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                word[i] = marks[2 * (pair0 + i) + (lane >> 5)];
                from[i] = places[2 * (pair0 + i) + (lane >> 5)];
            }
            uint32_t base = 0;                  // of the wave that had these words
#pragma unroll
            for (int i = 0; i < kReleaseThreads / 64; ++i) base = pair0 / 32 == i ? before[i] : base;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const uint32_t bit = lane & 31;
                if (!(word[i] >> bit & 1u)) continue;
                const int64_t place = at + base + from[i] + __builtin_popcount(word[i] & ((1u << bit) - 1));
                const int32_t page = static_cast<int32_t>(w0 * 32 + 64 * (pair0 + i) + lane);
                a.extra[page] = 0;
                if (place < a.free_capacity) a.free_pages[place] = page;
            }
        }
        if (bits) __hip_atomic_store(&a.bits[w * kMarkStride], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        at += all;
    }
    if (tid == 0) {
        const bool full = sound && at > a.free_capacity;
        *a.free_out = static_cast<int32_t>(full ? a.free_capacity : at);
        a.ctl->magic = kSharedMagic;
        a.ctl->flags = (sound ? 0u : kPagedInvalid) | pending | (full ? kPagedCapacity : 0u);
    }
}

// Workgroups of a launch that stay: as many as the chip holds at once (those
// of a fork have 53 KB of LDS each, those of a release 1024 threads), so that
// each makes its plan once.
constexpr uint64_t kForkGroups = 768, kReleaseGroups = 512;

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
    int64_t tables = (a.g.max_pages + kForkSlice - 1) / kForkSlice;
    if (tables > 64) tables = 64;
    const uint64_t most = uint64_t(a.g.n_pools) * (a.g.page_tokens - 1) * a.g.pieces;
    uint64_t copies = (most + kForkSlice - 1) / kForkSlice;
    if (copies > 4096) copies = 4096;
    uint64_t groups = a.count * (tables + copies);
    if (groups > kForkGroups) groups = kForkGroups;
    if (groups == 0) groups = 1;
    k_fork<<<static_cast<uint32_t>(groups), kForkThreads, 0, s>>>(a, static_cast<uint32_t>(tables), static_cast<uint32_t>(copies));
    return hipGetLastError();
}

hipError_t launch_release(const SharedArgs& a, hipStream_t s) {
    uint64_t groups = (a.g.max_pages + kColumns - 1) / kColumns;
    if (groups > kReleaseGroups) groups = kReleaseGroups;
    if (a.count == 0) groups = 1;
    k_release<<<static_cast<uint32_t>(groups), kReleaseThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace kvc
