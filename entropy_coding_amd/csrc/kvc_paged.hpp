// Host-side interface between the C ABI (kvc_paged_api.cpp) and the kernels
// of the paged cache: block tables and appends (kvc_paged.hip), attention
// (kvc_attention.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace kvc {

constexpr uint32_t kPagedMagic = 0x6b766361u;      // a workspace that a call has written
enum : uint32_t {
    kPagedInvalid = 1u,
    kPagedCapacity = 2u,
};

// t / page_tokens = t mul >> shift for t < 2^31: mul = ceil(2^(31 + e) /
// page_tokens) with 2^e >= page_tokens exceeds the quotient by less than
// 2^e / 2^(31 + e) parts of a page a token.
inline void set_page_product(uint32_t page_tokens, uint32_t* mul, uint32_t* shift) {
    uint32_t e = 0;
    while ((uint64_t(1) << e) < page_tokens) ++e;
    *shift = 31 + e;
    *mul = static_cast<uint32_t>(((uint64_t(1) << *shift) + page_tokens - 1) / page_tokens);
}

// ---- block tables

// Head of the workspace; behind it (at kTableArraysOffset) three int32
// arrays of batch + 1 entries, table_array(batch) apart: the prefix sums of
// the pages taken, of the pages given back, and the held counts before.
struct TableControl {
    uint32_t magic;
    uint32_t flags;
    int64_t rows;
    int32_t count;                      // height of the stack before
    int32_t taken, given;               // pages
    uint32_t pad;
};
constexpr uint64_t kTableArraysOffset = 256;
inline __host__ __device__ int64_t table_array(int64_t batch) { return (batch + 64) & ~int64_t(15); }

struct TableArgs {
    int64_t batch, max_pages, num_pages, free_capacity, max_rows;
    uint32_t page_tokens, trim;
    uint32_t page_mul, page_shift;      // t / page_tokens as a product (the launch sets them)
    const int32_t* cached;
    const int32_t* fresh;
    const int32_t* held_in;
    int32_t* held_out;
    int32_t* table;
    int32_t* free_pages;
    const int32_t* free_in;
    int32_t* free_out;
    int32_t* row_starts;
    int64_t* slots;
    int32_t* positions;
    TableControl* ctl;
    int32_t* arrays;
};
hipError_t launch_block_table(const TableArgs& args, hipStream_t s);

// ---- append

struct AppendArgs {
    void* const* pools;                 // the layer's K pool, then its V pool
    const void* k;
    const void* v;
    const int64_t* slots;
    int64_t rows, n_slots;              // n_slots: num_pages x page_tokens
    int64_t k_stride, v_stride;         // bytes
    uint32_t row_bytes;                 // of a pool's row (heads x channels)
    float k_scale, v_scale;
};
hipError_t launch_append(const AppendArgs& a, bool rounds, hipStream_t s);

// ---- attention

// Head of the workspace; behind it one AttendSpan a sequence, then a word a
// workgroup (not 0: it met a page number outside the pool), then the (maximum,
// sum) pairs and the sums of V of the parts, two parts a workgroup, each
// region 256-byte aligned.
struct AttendControl {
    uint32_t magic;
    uint32_t flags;                     // kPagedInvalid: a sequence that does not fit
    uint32_t grid;
    uint32_t words_offset;
    uint32_t per;                       // units a workgroup takes
    uint32_t aligned;                   // items begin at multiples of it
};
struct AttendSpan {                     // a sequence on the line of units
    uint32_t base;                      // its first unit
    uint32_t units;                     // of each of its items
    uint32_t tiles;                     // row tiles; 0: none of its rows is computed
    uint32_t pad;
};

struct AttendShape {                    // what the launch is made for
    bool wide;                          // rows over the waves (kvc_attention_wide.hip), not tokens
    int row_tiles;                      // 16-row tiles a wave holds
    int lds_tiles;                      // tiles of tokens that LDS holds (wide)
    uint32_t tile_shift;                // 2^tile_shift rows of a workgroup
    uint32_t unit_shift;                // 2^unit_shift tokens of a unit of work
    uint32_t grid;                      // workgroups; where items may be split: that fill the chip
    bool split;                         // whether a sequence may be split
    uint64_t spans, words, partial, pairs, total;   // workspace offsets and size
};

struct AttendArgs {
    void* const* pools;                 // the layer's K pool, then its V pool
    const int32_t* block_table;
    int64_t max_pages, num_pages;
    int32_t max_tokens;                 // that the table has room for, < 2^31 - 255
    uint32_t page_tokens, heads, batch, ratio;
    uint32_t tile_shift, unit_shift;    // of the shape
    uint32_t page_mul, page_shift;      // t / page_tokens as a product (the launch sets them)
    const uint16_t* q;
    int64_t q_row, q_head;
    uint16_t* out;
    int64_t out_row;
    float* lse;
    const int32_t* row_starts;
    const int32_t* context;
    const uint64_t* mask;
    uint32_t mask_words, rows;
    float scale_log2, v_scale;
    uint32_t target, split;             // workgroups to deal units to; 0: an item a workgroup
    AttendControl* ctl;
    AttendSpan* spans;
    uint32_t* words;
    float* partial;
    float* pairs;                       // (maximum, sum) each
};
// At most as many items (KV heads x tiles of rows) as a call has: every
// sequence's rows fill whole tiles but the last one.
inline uint64_t attend_items(int64_t batch, int64_t heads, int64_t ratio, int64_t rows, int64_t tile_rows) {
    return uint64_t(heads) * (uint64_t(rows) * ratio / tile_rows + (rows < batch ? rows : batch));
}
constexpr uint64_t kMaxItems = uint64_t(1) << 30;       // of tiles of 16 rows
constexpr int64_t kMaxTokens = 0x7FFFFF00;              // of a sequence

AttendShape attend_shape(int64_t batch, int64_t heads, int64_t ratio, int64_t channels, bool fp8, int64_t rows,
                         int64_t rows_per_sequence, int64_t max_tokens, int64_t widest);
hipError_t launch_attend(const AttendArgs& args, const AttendShape& shape, int64_t channels, bool fp8, hipStream_t s);
hipError_t launch_attend_wide(const AttendArgs& a, const AttendShape& shape, int64_t channels, bool fp8, hipStream_t s);
int wide_groups(int64_t channels, bool fp8, int row_tiles, int lds_tiles);     // workgroups of it that a CU holds

}  // namespace kvc
