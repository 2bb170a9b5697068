// Block tables and slot maps from request lengths, and the append of new
// K/V rows to the pages (declared in include/kvc.h).
#include <hip/hip_runtime.h>

#include "kvc_paged.hpp"
#include "kvc_wave.hpp"

namespace kvc {
namespace {

// ---------------------------------------------------------------- block tables

// Prefix sums over the requests say where each one's rows, pages to take and
// pages to give back lie; from them every row finds its request by bisection,
// and every slot, table entry and push follows by itself (Stack below).  A
// small step is bound by a chain of reads and barriers in one workgroup: 8
// requests 6.5 us (the launch alone 3.3), where two launches took 8.2; the
// sums and the rows of 256 requests with trees 12.8 us in two launches; 64
// prompts of up to 32768 tokens (1.3 million slots and positions, 16 MB)
// 12.0 us, 3.1 of them the sums.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// What one request asks for.  ok: its numbers are sound; fits: its tokens
// fit its row of the table.
struct Ask {
    int32_t cached, rows, held, need, taken, given;
    bool ok, fits;
};

// t / page_tokens for t < 2^31, as a product.
__device__ uint32_t page_of(const TableArgs& a, uint32_t t) {
    return static_cast<uint32_t>((uint64_t(t) * a.page_mul) >> a.page_shift);
}

__device__ Ask ask_of(const TableArgs& a, int64_t b) {
    const int64_t cached = a.cached ? a.cached[b] : 0, fresh = a.fresh ? a.fresh[b] : 0;
    Ask r;
    r.cached = static_cast<int32_t>(cached);
    r.held = a.held_in[b];
    r.ok = cached >= 0 && fresh >= 0 && r.held >= 0 && r.held <= a.max_pages;
    const int64_t total = cached + fresh;
    r.fits = total <= a.max_pages * int64_t(a.page_tokens) && total <= 0x7FFFFFFF;
    r.rows = r.need = r.taken = r.given = 0;
    if (!r.ok || !r.fits) return r;
    r.rows = static_cast<int32_t>(fresh);
    r.need = total ? static_cast<int32_t>(page_of(a, static_cast<uint32_t>(total - 1)) + 1) : 0;
    r.taken = r.need > r.held ? r.need - r.held : 0;
    r.given = a.trim && r.held > r.need ? r.held - r.need : 0;
    return r;
}

// The prefix sums of the step: rows, pages taken, pages given back, and the
// held counts before; one entry a request and the totals behind.  They stand
// in LDS where a step has at most kPlanThreads requests.
struct Sums {
    int32_t* rows;
    int32_t* taken;
    int32_t* given;
    int32_t* held;
    const int32_t* cached;                      // (and the lengths; null: all zero)
};
struct LdsSums {
    int32_t v[5][kPlanThreads + 1];
    __device__ Sums sums() { return Sums{v[0], v[1], v[2], v[3], v[4]}; }
};
__device__ Sums global_sums(const TableArgs& a) {
    const int64_t step = table_array(a.batch);
    return Sums{a.row_starts, a.arrays, a.arrays + step, a.arrays + 2 * step, a.cached};
}

// Height of the stack before, and the step's pages and rows (0 where it fails).
struct Totals {
    int32_t count, taken, given, rows;
};

// The prefix sums and checks of all requests, and the new counts: one
// workgroup, 1024 requests at a time.  Rows are summed in 32 bits, which hold
// them where the step can be done, and in two halves for the check.
template <bool KEEP>                            // in LDS, for this workgroup
__device__ Totals plan(const TableArgs& a, LdsSums* lds) {
    __shared__ uint32_t of_wave[6][kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Sums to = KEEP ? lds->sums() : global_sums(a);
    const int64_t count = *a.free_in;
    uint32_t base[3] = {0, 0, 0};
    uint64_t rows = 0;
    uint32_t wrong = 0;                         // 1: not sound, 2: does not fit
    Ask k{};
    for (int64_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int64_t b = b0 + tid;
        k = Ask{};
        bool ok = true, fits = true;
        if (b < a.batch) {
            k = ask_of(a, b);
            ok = k.ok;
            fits = k.fits;
        }
        const uint32_t mine[3] = {uint32_t(k.rows), uint32_t(k.taken), uint32_t(k.given)};
        uint32_t sum[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            sum[i] = scan(mine[i]);
            if (lane == 63) of_wave[i][wave] = sum[i];
        }
        const uint32_t low = scan(mine[0] & 0xFFFFu), high = scan(mine[0] >> 16);
        const uint32_t bad = (__any(!ok) ? 1u : 0u) | (__any(!fits) ? 2u : 0u);
        if (lane == 63) {
            of_wave[3][wave] = low;
            of_wave[4][wave] = high;
            of_wave[5][wave] = bad;
        }
        __syncthreads();
        uint32_t all[6];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const uint32_t upto = scan(lane < kPlanWaves ? of_wave[i][lane] : 0u);
            all[i] = of_lane(upto, 63);
            if (i < 3) sum[i] += base[i] + (wave ? of_lane(upto, wave - 1) : 0u);
        }
        const uint32_t b_wave = lane < kPlanWaves ? of_wave[5][lane] : 0u;
        wrong |= (__any(b_wave & 1u) ? 1u : 0u) | (__any(b_wave & 2u) ? 2u : 0u);
        if (b < a.batch) {
            to.rows[b] = static_cast<int32_t>(sum[0] - mine[0]);
            to.taken[b] = static_cast<int32_t>(sum[1] - mine[1]);
            to.given[b] = static_cast<int32_t>(sum[2] - mine[2]);
            to.held[b] = k.held;
            if (KEEP) lds->v[4][b] = k.cached;
        }
        rows += (uint64_t(all[4]) << 16) + all[3];
        for (int i = 0; i < 3; ++i) base[i] += all[i];
        __syncthreads();                        // (behind it, every read of free_in and held_in is done)
    }
    const int64_t taken = base[1], given = base[2], left = count + given - taken;
    // (places on the stack are 32 bits)
    if (count < 0 || count > a.free_capacity || count + given > 0x7FFFFFFF) wrong |= 1u;
    if (left < 0 || left > a.free_capacity || rows > static_cast<uint64_t>(a.max_rows)) wrong |= 2u;
    const bool go = !wrong;
    for (int64_t b = tid; b < a.batch; b += kPlanThreads) {
        // the outputs may be the inputs' own arrays: what is needed of them was kept
        const int32_t held = to.held[b];
        int32_t need = k.need;
        if (a.batch > kPlanThreads && go) need = ask_of(a, b).need;
        a.held_out[b] = go && (a.trim || need > held) ? need : held;
        if (KEEP || !go) a.row_starts[b] = go ? to.rows[b] : 0;
    }
    const Totals t{static_cast<int32_t>(count), static_cast<int32_t>(go ? taken : 0),
                   static_cast<int32_t>(go ? given : 0), static_cast<int32_t>(go ? rows : 0)};
    if (tid == 0) {
        a.row_starts[a.batch] = t.rows;
        to.rows[a.batch] = t.rows;
        to.taken[a.batch] = t.taken;
        to.given[a.batch] = t.given;
        *a.free_out = static_cast<int32_t>(go ? left : count);
        *a.ctl = TableControl{kPagedMagic, (wrong & 1u) ? kPagedInvalid : wrong ? kPagedCapacity : 0u, t.rows,
                              t.count, t.taken, t.given, 0u};
    }
    return t;
}

// The last i in [lo, hi] with at[i] <= x (at rises; at[lo] <= x).
__device__ int32_t last_not_above(const int32_t* at, int32_t lo, int32_t hi, int32_t x) {
    while (lo < hi) {
        const int32_t mid = lo + ((hi - lo + 1) >> 1);
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The stack after the surplus pages were pushed has `count` old entries and
// above them the s-th surplus page at place count + given - 1 - s; pages are
// popped from the top.  Nothing is pushed in fact but what stays: a pop finds
// its page where it stood, so every page, slot and push below is independent
// of the others (what is read of the table, entries below the held counts,
// and of the stack, places below `count`, is not written).
struct Stack {
    const TableArgs& a;
    const Sums& s;
    const Totals& t;

    // where the page at a place stands
    __device__ const int32_t* at(int32_t place) const {
        if (place < t.count) return a.free_pages + place;
        const int32_t x = t.given - 1 - (place - t.count);
        const int32_t b = last_not_above(s.given, 0, static_cast<int32_t>(a.batch) - 1, x);
        return a.table + b * a.max_pages + s.held[b] - (s.given[b + 1] - x);
    }
    __device__ const int32_t* popped(int32_t k) const { return at(t.count + t.given - 1 - k); }
    __device__ const int32_t* page(int32_t b, int32_t j) const {
        const int32_t held = s.held[b];
        return j < held ? a.table + b * a.max_pages + j : popped(s.taken[b] + j - held);
    }
};

// Rows, pages and pushes, dealt to `blocks` workgroups of THREADS threads of
// which this is the block-th; rows U x THREADS at a time (U to a thread, so
// that as many reads of page numbers are under way).
template <int THREADS, int U>
__device__ void fill(const TableArgs& a, const Sums& s, const Totals& t, int64_t block, int64_t blocks) {
    const Stack st{a, s, t};
    const int32_t last_b = static_cast<int32_t>(a.batch) - 1;
    const int64_t limit = a.slots || a.positions ? a.max_rows : t.rows;
    bool bad = false;
    for (int64_t r0 = block * (THREADS * U); r0 < limit; r0 += blocks * (THREADS * U)) {
        // the requests of these rows: most often one
        int32_t lo = 0, hi = 0;
        if (r0 < t.rows) {
            const int64_t end = r0 + THREADS * U < t.rows ? r0 + THREADS * U : t.rows;
            lo = last_not_above(s.rows, 0, last_b, static_cast<int32_t>(r0));
            hi = last_not_above(s.rows, lo, last_b, static_cast<int32_t>(end - 1));
        }
        const int32_t* from[U];
        int32_t* to[U];
        int32_t pos[U];
        uint32_t rest[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * THREADS + threadIdx.x;
            from[u] = nullptr;
            to[u] = nullptr;
            pos[u] = -1;
            rest[u] = 0;
            if (r < t.rows) {
                const int32_t b = last_not_above(s.rows, lo, hi, static_cast<int32_t>(r));
                const int32_t i = static_cast<int32_t>(r) - s.rows[b];
                pos[u] = (s.cached ? s.cached[b] : 0) + i;
                const uint32_t j = page_of(a, static_cast<uint32_t>(pos[u]));
                rest[u] = uint32_t(pos[u]) - j * a.page_tokens;
                from[u] = st.page(b, static_cast<int32_t>(j));
                // the first new token of a page that was taken enters the page in the table
                if (static_cast<int32_t>(j) >= s.held[b] && (i == 0 || rest[u] == 0)) to[u] = a.table + b * a.max_pages + j;
            }
        }
        int32_t page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) page[u] = from[u] ? *from[u] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * THREADS + threadIdx.x;
            if (r >= limit) continue;
            const bool in = page[u] >= 0 && page[u] < a.num_pages;
            bad = bad || (from[u] && !in);
            if (to[u]) *to[u] = page[u];
            if (a.slots) a.slots[r] = in ? int64_t(page[u]) * a.page_tokens + rest[u] : -1;
            if (a.positions) a.positions[r] = pos[u];
        }
    }
    // what is left goes to the workgroups from the last on, which have rows last
    const int64_t n = blocks * THREADS, first = (blocks - 1 - block) * THREADS + threadIdx.x;
    // pages taken for cached tokens alone (a request that comes with tokens and no pages): a wave a request
    if (t.taken) {
        for (int64_t b = first >> 6; b < a.batch; b += blocks * (THREADS / 64)) {
            const int32_t taken = s.taken[b + 1] - s.taken[b], held = s.held[b];
            const int32_t cached = s.cached ? s.cached[b] : 0;
            const int32_t fresh = s.rows[b + 1] - s.rows[b];
            // without new tokens the last, unfilled page is among them
            const int32_t end = fresh ? static_cast<int32_t>(page_of(a, static_cast<uint32_t>(cached))) : held + taken;
            for (int32_t j = held + (threadIdx.x & 63); j < end && j < held + taken; j += 64) {
                const int32_t page = *st.popped(s.taken[b] + j - held);
                bad = bad || page < 0 || page >= a.num_pages;
                a.table[b * a.max_pages + j] = page;
            }
        }
    }
    for (int64_t p = first; p < int64_t(t.given) - t.taken; p += n) {
        const int32_t page = *st.at(static_cast<int32_t>(t.count + p));
        bad = bad || page < 0 || page >= a.num_pages;
        a.free_pages[t.count + p] = page;
    }
    if (bad) atomicOr(&a.ctl->flags, kPagedInvalid);
}

__global__ __launch_bounds__(kPlanThreads) void k_table_plan(TableArgs a) { plan<false>(a, nullptr); }

constexpr int kFillThreads = 256;
constexpr int kFillRows = 4;                    // a thread

// LDS: the sums are copied there first.
template <bool LDS>
__global__ __launch_bounds__(kFillThreads) void k_table_fill(TableArgs a) {
    const Totals t{a.ctl->count, a.ctl->taken, a.ctl->given, static_cast<int32_t>(a.ctl->rows)};
    const Sums global = global_sums(a);
    if constexpr (LDS) {
        __shared__ LdsSums lds;
#pragma unroll
        for (int u = 0; u <= kPlanThreads / kFillThreads; ++u) {
            const int i = u * kFillThreads + threadIdx.x;
            if (i > a.batch) continue;
            lds.v[0][i] = global.rows[i];
            lds.v[1][i] = global.taken[i];
            lds.v[2][i] = global.given[i];
            if (i == a.batch) continue;
            lds.v[3][i] = global.held[i];
            lds.v[4][i] = global.cached ? global.cached[i] : 0;
        }
        __syncthreads();
        fill<kFillThreads, kFillRows>(a, lds.sums(), t, blockIdx.x, gridDim.x);
    } else {
        fill<kFillThreads, kFillRows>(a, global, t, blockIdx.x, gridDim.x);
    }
}

__global__ __launch_bounds__(kPlanThreads) void k_table_one(TableArgs a) {
    __shared__ LdsSums lds;
    const Totals t = plan<true>(a, &lds);
    __syncthreads();
    fill<kPlanThreads, 2>(a, lds.sums(), t, 0, 1);
}

// One workgroup plans and fills a step of up to kPlanThreads requests and
// this many rows, two a thread; more go to a second launch (8700 rows of 256
// requests take one workgroup 20 us).
constexpr int64_t kOneGroupRows = 2048;

}  // namespace

hipError_t launch_block_table(const TableArgs& args, hipStream_t s) {
    TableArgs a = args;
    set_page_product(a.page_tokens, &a.page_mul, &a.page_shift);
    if (a.batch <= kPlanThreads && a.max_rows <= kOneGroupRows) {
        k_table_one<<<1, kPlanThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    k_table_plan<<<1, kPlanThreads, 0, s>>>(a);
    int64_t blocks = (a.max_rows + kFillThreads * kFillRows - 1) / (kFillThreads * kFillRows);
    if (blocks > 2048) blocks = 2048;
    if (blocks < 64) blocks = 64;
    if (a.batch <= kPlanThreads) k_table_fill<true><<<static_cast<uint32_t>(blocks), kFillThreads, 0, s>>>(a);
    else k_table_fill<false><<<static_cast<uint32_t>(blocks), kFillThreads, 0, s>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- append

namespace {

// Two bf16 values (low half first) as the e4m3 of x / scale: the quotient in
// float32, clamped to +-448 (a NaN passes both comparisons and stays), then
// rounded to nearest even by the conversion.
__device__ float clamp448(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

__device__ uint32_t round_pair(uint32_t two, float scale) {
    const float lo = clamp448(__uint_as_float(two << 16) / scale);
    const float hi = clamp448(__uint_as_float(two & 0xFFFF0000u) / scale);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, 0, false)) & 0xFFFFu;
}

// One piece of a row a thread, 16 bytes as it is written, in workgroups of
// 256 pieces; blockIdx.y: K or V.  A prompt of 16384 rows of 1024 bf16 values
// takes 28 us, as many bytes of a copy 27; four pieces a thread, all read
// before the first is written, took 37 us, and four one after the other 30.
template <bool ROUND>
__global__ __launch_bounds__(256) void k_append(AppendArgs a, uint32_t pieces) {
    const bool is_v = blockIdx.y != 0;
    uint8_t* const pool = static_cast<uint8_t*>(a.pools[is_v]);
    const uint8_t* const src = static_cast<const uint8_t*>(is_v ? a.v : a.k);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const float scale = is_v ? a.v_scale : a.k_scale;
    const uint64_t n = uint64_t(a.rows) * pieces;
    for (uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += uint64_t(gridDim.x) * 256) {
        const uint64_t r = n >> 32 ? i / pieces : static_cast<uint32_t>(i) / pieces;
        const uint32_t c = static_cast<uint32_t>(i - r * pieces);
        const int64_t slot = a.slots[r];
        const uint4* const from = reinterpret_cast<const uint4*>(src + int64_t(r) * stride) + c * (ROUND ? 2 : 1);
        uint4 x = from[0];
        if (ROUND) {
            const uint4 y = from[1];
            x = uint4{round_pair(x.x, scale) | (round_pair(x.y, scale) << 16),
                      round_pair(x.z, scale) | (round_pair(x.w, scale) << 16),
                      round_pair(y.x, scale) | (round_pair(y.y, scale) << 16),
                      round_pair(y.z, scale) | (round_pair(y.w, scale) << 16)};
        }
        if (slot >= 0 && slot < a.n_slots)
            *reinterpret_cast<uint4*>(pool + uint64_t(slot) * a.row_bytes + 16u * c) = x;
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, bool rounds, hipStream_t s) {
    const uint32_t pieces = a.row_bytes / 16;
    uint64_t blocks = (uint64_t(a.rows) * pieces + 255) / 256;
    if (blocks > (1u << 22)) blocks = 1u << 22;
    const dim3 grid(static_cast<uint32_t>(blocks), 2);
    if (rounds) k_append<true><<<grid, 256, 0, s>>>(a, pieces);
    else k_append<false><<<grid, 256, 0, s>>>(a, pieces);
    return hipGetLastError();
}

}  // namespace kvc
