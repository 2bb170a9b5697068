// Block tables and slot maps from request lengths, and the append of new
// K/V rows to the pages (declared in include/kvc.h).
#include <hip/hip_runtime.h>

#include "kvc_paged.hpp"

namespace kvc {
namespace {

// ---------------------------------------------------------------- block tables

constexpr int kPlanThreads = 1024;

// What one request asks for.  ok: its numbers are sound; fits: its tokens
// fit its row of the table.
struct Ask {
    int64_t rows;
    int32_t held, need, taken, given;
    bool ok, fits;
};

__device__ Ask ask_of(const TableArgs& a, int64_t b) {
    const int64_t cached = a.cached ? a.cached[b] : 0, fresh = a.fresh ? a.fresh[b] : 0;
    Ask r;
    r.held = a.held_in[b];
    r.ok = cached >= 0 && fresh >= 0 && r.held >= 0 && r.held <= a.max_pages;
    const int64_t total = cached + fresh;
    r.fits = total <= a.max_pages * int64_t(a.page_tokens) && total <= 0x7FFFFFFF;
    r.rows = 0;
    r.need = r.taken = r.given = 0;
    if (!r.ok || !r.fits) return r;
    r.rows = fresh;
    r.need = static_cast<int32_t>((total + a.page_tokens - 1) / a.page_tokens);
    r.taken = r.need > r.held ? r.need - r.held : 0;
    r.given = a.trim && r.held > r.need ? r.held - r.need : 0;
    return r;
}

// The prefix sums of the rows and pages of all requests, the checks, and the
// new counts: one workgroup, 1024 requests at a time.  The pages taken and
// given back are summed in the two halves of one 64-bit word (each at most
// batch x max_pages < 2^31).  Returns whether the step can be done; the
// results stand in ctl, arrays and row_starts for the same workgroup and for
// later kernels.
__device__ bool plan(const TableArgs& a) {
    __shared__ uint64_t rows_of_wave[kPlanThreads / 64], pages_of_wave[kPlanThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t step = table_array(a.batch);
    int32_t* const taken_at = a.arrays;
    int32_t* const given_at = a.arrays + step;
    int32_t* const held_old = a.arrays + 2 * step;
    uint64_t rows = 0, pages = 0;
    bool ok = true, fits = true;
    for (int64_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int64_t b = b0 + tid;
        uint64_t r = 0, p = 0;
        if (b < a.batch) {
            const Ask k = ask_of(a, b);
            ok = ok && k.ok;
            fits = fits && k.fits;
            r = static_cast<uint64_t>(k.rows);
            p = (uint64_t(uint32_t(k.given)) << 32) | uint32_t(k.taken);
            held_old[b] = k.held;
        }
        uint64_t r_sum = r, p_sum = p;
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t x = __shfl_up(r_sum, d), y = __shfl_up(p_sum, d);
            if (lane >= d) {
                r_sum += x;
                p_sum += y;
            }
        }
        if (lane == 63) {
            rows_of_wave[wave] = r_sum;
            pages_of_wave[wave] = p_sum;
        }
        __syncthreads();
        uint64_t r_all = 0, p_all = 0;
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w == wave) {
                r_sum += r_all;
                p_sum += p_all;
            }
            r_all += rows_of_wave[w];
            p_all += pages_of_wave[w];
        }
        if (b < a.batch) {
            const uint64_t at = rows + r_sum - r, pg = pages + p_sum - p;
            a.row_starts[b] = static_cast<int32_t>(at < 0x7FFFFFFF ? at : 0x7FFFFFFF);
            taken_at[b] = static_cast<int32_t>(pg & 0xFFFFFFFFu);
            given_at[b] = static_cast<int32_t>(pg >> 32);
        }
        rows += r_all;
        pages += p_all;
        __syncthreads();
    }
    ok = __syncthreads_and(ok);
    fits = __syncthreads_and(fits);
    const int64_t taken = static_cast<int64_t>(pages & 0xFFFFFFFFu), given = static_cast<int64_t>(pages >> 32);
    const int64_t count = *a.free_in, left = count + given - taken;
    ok = ok && count >= 0 && count <= a.free_capacity;
    fits = fits && left >= 0 && left <= a.free_capacity && rows <= static_cast<uint64_t>(a.max_rows);
    const bool go = ok && fits;
    // every read of free_in and held_in is done: the outputs may be the same arrays
    __syncthreads();
    for (int64_t b = tid; b < a.batch; b += kPlanThreads) {
        const int32_t held = held_old[b];
        if (go) {
            const Ask k = ask_of(a, b);
            a.held_out[b] = a.trim || k.need > held ? k.need : held;
        } else {
            a.held_out[b] = held;
            a.row_starts[b] = 0;
        }
    }
    if (tid == 0) {
        a.row_starts[a.batch] = go ? static_cast<int32_t>(rows) : 0;
        taken_at[a.batch] = static_cast<int32_t>(taken);
        given_at[a.batch] = static_cast<int32_t>(given);
        *a.free_out = static_cast<int32_t>(go ? left : count);
        a.ctl->magic = kPagedMagic;
        a.ctl->flags = !ok ? kPagedInvalid : !fits ? kPagedCapacity : 0u;
        a.ctl->rows = go ? static_cast<int64_t>(rows) : 0;
        a.ctl->count = static_cast<int32_t>(count);
        a.ctl->taken = static_cast<int32_t>(go ? taken : 0);
        a.ctl->given = static_cast<int32_t>(go ? given : 0);
    }
    return go;
}

// The last i in [lo, hi] with at[i] <= x (at rises; at[lo] <= x).
__device__ int64_t last_not_above(const int32_t* at, int64_t lo, int64_t hi, int32_t x) {
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
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
    const int32_t* taken_at;
    const int32_t* given_at;
    const int32_t* held_old;
    int64_t count, taken, given;

    __device__ explicit Stack(const TableArgs& args)
        : a(args), taken_at(args.arrays), given_at(args.arrays + table_array(args.batch)),
          held_old(args.arrays + 2 * table_array(args.batch)), count(args.ctl->count), taken(args.ctl->taken),
          given(args.ctl->given) {}

    __device__ int32_t at(int64_t place) const {
        if (place < count) return a.free_pages[place];
        const int32_t s = static_cast<int32_t>(given - 1 - (place - count));
        const int64_t b = last_not_above(given_at, 0, a.batch - 1, s);
        return a.table[b * a.max_pages + held_old[b] - (given_at[b + 1] - s)];
    }
    __device__ int32_t pop(int64_t k) const { return at(count + given - 1 - k); }
    __device__ int32_t page(int64_t b, int32_t j) const {
        const int32_t held = held_old[b];
        return j < held ? a.table[b * a.max_pages + j] : pop(taken_at[b] + j - held);
    }
};

// Pages, pushes and rows, dealt to `n` threads of which this is the t-th;
// rows in blocks of kFillRows for each workgroup, whose requests are found
// once.
constexpr int kFillRows = 2048;

__device__ void fill(const TableArgs& a, int64_t block, int64_t blocks, int threads) {
    const Stack st(a);
    const int64_t t = block * threads + threadIdx.x, n = blocks * threads;
    bool bad = false;
    for (int64_t k = t; k < st.taken; k += n) {
        const int64_t b = last_not_above(st.taken_at, 0, a.batch - 1, static_cast<int32_t>(k));
        const int32_t page = st.pop(k);
        bad = bad || page < 0 || page >= a.num_pages;
        a.table[b * a.max_pages + st.held_old[b] + (k - st.taken_at[b])] = page;
    }
    for (int64_t p = t; p < st.given - st.taken; p += n) {
        const int32_t page = st.at(st.count + p);
        bad = bad || page < 0 || page >= a.num_pages;
        a.free_pages[st.count + p] = page;
    }
    if (a.slots || a.positions) {
        const int64_t rows = a.ctl->rows;
        for (int64_t r0 = block * kFillRows; r0 < a.max_rows; r0 += blocks * kFillRows) {
            const int64_t last = r0 + kFillRows < a.max_rows ? r0 + kFillRows : a.max_rows;
            int64_t lo = 0, hi = 0;
            if (r0 < rows) {
                const int64_t real = last < rows ? last : rows;
                lo = last_not_above(a.row_starts, 0, a.batch - 1, static_cast<int32_t>(r0));
                hi = last_not_above(a.row_starts, lo, a.batch - 1, static_cast<int32_t>(real - 1));
            }
            for (int64_t r = r0 + threadIdx.x; r < last; r += threads) {
                int64_t slot = -1;
                int32_t pos = -1;
                if (r < rows) {
                    const int64_t b = last_not_above(a.row_starts, lo, hi, static_cast<int32_t>(r));
                    pos = static_cast<int32_t>((a.cached ? a.cached[b] : 0) + (r - a.row_starts[b]));
                    const uint32_t j = uint32_t(pos) / a.page_tokens;
                    const int32_t page = st.page(b, static_cast<int32_t>(j));
                    if (page < 0 || page >= a.num_pages) bad = true;
                    else slot = int64_t(page) * a.page_tokens + (uint32_t(pos) - j * a.page_tokens);
                }
                if (a.slots) a.slots[r] = slot;
                if (a.positions) a.positions[r] = pos;
            }
        }
    }
    if (bad) atomicOr(&a.ctl->flags, kPagedInvalid);
}

__global__ __launch_bounds__(kPlanThreads) void k_table_plan(TableArgs a) { plan(a); }

__global__ __launch_bounds__(256) void k_table_fill(TableArgs a) { fill(a, blockIdx.x, gridDim.x, 256); }

__global__ __launch_bounds__(kPlanThreads) void k_table_one(TableArgs a) {
    plan(a);
    __syncthreads();                    // ctl, arrays and row_starts are written
    fill(a, 0, 1, kPlanThreads);
}

// Steps with at most this many rows are planned and filled by one workgroup.
constexpr int64_t kOneGroupRows = 8192;

}  // namespace

hipError_t launch_block_table(const TableArgs& a, hipStream_t s) {
    if (a.max_rows <= kOneGroupRows) {
        k_table_one<<<1, kPlanThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    k_table_plan<<<1, kPlanThreads, 0, s>>>(a);
    int64_t blocks = (a.max_rows + kFillRows - 1) / kFillRows;
    if (blocks > 2048) blocks = 2048;
    k_table_fill<<<static_cast<uint32_t>(blocks), 256, 0, s>>>(a);
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

// One 16-byte piece of a source row a thread; blockIdx.y: K or V.
template <bool ROUND>
__global__ __launch_bounds__(256) void k_append(AppendArgs a, uint32_t pieces) {
    const bool is_v = blockIdx.y != 0;
    uint8_t* const pool = static_cast<uint8_t*>(a.pools[is_v]);
    const uint8_t* const src = static_cast<const uint8_t*>(is_v ? a.v : a.k);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const float scale = is_v ? a.v_scale : a.k_scale;
    const uint64_t n = uint64_t(a.rows) * pieces;
    for (uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += uint64_t(gridDim.x) * 256) {
        const uint64_t r = i / pieces;
        const uint32_t c = static_cast<uint32_t>(i - r * pieces);
        const int64_t slot = a.slots[r];
        if (slot < 0 || slot >= a.n_slots) continue;
        const uint4 x = *reinterpret_cast<const uint4*>(src + int64_t(r) * stride + 16u * c);
        uint8_t* const row = pool + uint64_t(slot) * a.row_bytes;
        if (ROUND) {
            uint2 y;
            y.x = round_pair(x.x, scale) | (round_pair(x.y, scale) << 16);
            y.y = round_pair(x.z, scale) | (round_pair(x.w, scale) << 16);
            *reinterpret_cast<uint2*>(row + 8u * c) = y;
        } else {
            *reinterpret_cast<uint4*>(row + 16u * c) = x;
        }
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, bool rounds, hipStream_t s) {
    const uint32_t pieces = rounds ? a.row_bytes / 8 : a.row_bytes / 16;
    const uint64_t n = uint64_t(a.rows) * pieces;
    uint64_t blocks = (n + 255) / 256;
    if (blocks > (1u << 20)) blocks = 1u << 20;
    const dim3 grid(static_cast<uint32_t>(blocks), 2);
    if (rounds) k_append<true><<<grid, 256, 0, s>>>(a, pieces);
    else k_append<false><<<grid, 256, 0, s>>>(a, pieces);
    return hipGetLastError();
}

}  // namespace kvc
