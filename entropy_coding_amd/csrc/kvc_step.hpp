// Host-side interface between the C ABI (kvc_step_api.cpp) and the kernels of
// a speculative step around the attention over pages: norms, rotation and
// append (kvc_qkv.hip), verification of drafted tokens (kvc_verify.hip), rows
// and pages moved, shared and given back (kvc_pages.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace kvc {

// Workspaces that a call of the kind has written.
constexpr uint32_t kVerifyMagic = 0x6b766376u, kCompactMagic = 0x6b76636du, kSharedMagic = 0x6b766373u;

// ---- norms, rotation, append

struct HeadRows {                       // [rows][heads][channels], strides in values
    const uint16_t* at;
    int64_t row, head;
};
struct QkvArgs {
    void* const* pools;                 // the layer's K pool, then its V pool
    HeadRows q, k, v;
    uint16_t* out;                      // the heads of a row `channels` values apart
    int64_t out_row;
    const void* q_norm;                 // null: no norm
    const void* k_norm;
    const double* frequencies;
    const int32_t* positions;           // null: every row is one (nothing is rotated)
    const int64_t* slots;
    int64_t rows, n_slots;
    uint32_t q_heads, heads, rotary;
    uint32_t norm_f32;                  // the norms' weights are float32 (bf16 otherwise)
    uint32_t parts;                     // that a row's heads are split into (the launch sets it)
    float eps;
    double per_k_scale, per_v_scale;    // 1 / scale
};
hipError_t launch_qkv(const QkvArgs& args, int64_t channels, bool fp8, bool neighbours, hipStream_t s);

// ---- verification

constexpr int kMaxNodes = 1024;         // of a sequence's tree
constexpr int kMaxVocab = 1 << 20;
constexpr int kVerifyChunk = 4096;      // values of a distribution that a workgroup sums

// Head of the workspace; behind it two words a sequence (what the walk and
// the draw found wrong), the workgroups of a sequence that are done (0 before
// the first call and between calls), the chunks' sums, and of drawn trees the
// nodes whose first rejections are summed ahead and these sums, a workgroup's
// each.
struct VerifyControl {
    uint32_t magic;
    uint32_t batch;
};
struct VerifySums {                     // units of 2^-42
    uint64_t left, whole;               // after the rejections, and before
};
struct VerifyLayout {
    uint64_t words, arrived, sums, first_nodes, first_sums, total;
    uint32_t chunks;
};
// Words between the sequences' counts, 64 bytes: counts side by side are added
// to in turn (64 sequences of 131072 tokens: 20.4 us, side by side 22.3).
constexpr int kArrivedStride = 16;
constexpr int kFirsts = 8;              // nodes of a sequence that are summed ahead
constexpr uint32_t kMostChunks = 64;    // of a workgroup
// Workgroups of a launch, where it has as many chunks: four a CU (64 sequences
// of 131072 tokens: 20.6 us, with 512 or 2048 of them 24.8 and 26.3).
constexpr uint32_t kDrawGroups = 1024;
// The workgroups of a sequence, and the chunks of each.
inline uint32_t verify_parts(uint32_t groups, uint32_t batch, uint32_t chunks, uint32_t* per) {
    const uint32_t least = (chunks + kMostChunks - 1) / kMostChunks;
    uint32_t parts = groups / batch;
    if (parts < least) parts = least;
    if (parts > chunks) parts = chunks;
    *per = (chunks + parts - 1) / parts;
    return (chunks + *per - 1) / *per;
}
inline VerifyLayout verify_layout(int64_t batch, int64_t vocab) {
    const auto up = [](uint64_t x) { return (x + 255) & ~uint64_t(255); };
    VerifyLayout l;
    l.chunks = static_cast<uint32_t>((vocab + kVerifyChunk - 1) / kVerifyChunk);
    l.words = 256;
    l.arrived = l.words + up(8 * uint64_t(batch));
    l.sums = l.arrived + up(4 * kArrivedStride * uint64_t(batch));
    l.first_nodes = l.sums + up(sizeof(VerifySums) * uint64_t(batch) * l.chunks);
    l.first_sums = l.first_nodes + up(4 * kFirsts * uint64_t(batch));
    uint32_t per;
    l.total = l.first_sums + up(8 * kFirsts * uint64_t(batch) * verify_parts(kDrawGroups, static_cast<uint32_t>(batch), l.chunks, &per));
    return l;
}
struct VerifyArgs {
    int64_t batch, rows;
    uint32_t vocab, chunks;
    const int32_t* row_starts;
    const int32_t* tokens;
    const int32_t* parents;             // null: chains
    const float* target;
    const float* draft;                 // null: drafted without probabilities
    int64_t target_row, draft_row;
    const float* accept;
    const float* sample;
    int32_t* kept;
    int32_t* kept_lens;
    int32_t* out_tokens;
    VerifyControl* ctl;
    uint32_t* words;
    uint32_t* arrived;
    VerifySums* sums;
    int32_t* first_nodes;
    uint64_t* first_sums;
    uint32_t first_parts;               // sums of a node, 0: none (the launch sets it)
};
hipError_t launch_verify(const VerifyArgs& args, hipStream_t s);

// ---- pages

struct PagesOf {                        // the pools and the table
    void* const* pools;
    int64_t n_pools;
    int64_t batch, max_pages, num_pages;
    uint32_t page_tokens;
    uint32_t pieces;                    // of 16 bytes in a row of a pool
};

// Head of a compaction's workspace; a word a sequence behind it (at 256).
struct CompactControl {
    uint32_t magic;
    uint32_t batch;
};
struct CompactArgs {
    PagesOf g;
    const int32_t* table;
    int64_t rows;
    const int32_t* row_starts;
    const int32_t* context;             // null: none has any
    const int32_t* kept;
    const int32_t* kept_lens;
    CompactControl* ctl;
    uint32_t* words;
};
hipError_t launch_compact(const CompactArgs& a, hipStream_t s);

constexpr int kMaxShared = 1024;        // requests of a fork or release

// Head of the workspace of forks and releases (zero before the first); behind
// it the places that workgroups count in, 256 bytes apart, 0 between calls,
// and a bit a page, zero between releases, 32 of them every kMarkStride words,
// 64 bytes: marks side by side wait for each other (8000 of 11000 pages given
// back at once: 15.3 us with the words side by side, 10.6 with 64 bytes each).
// What is read of a pool's marks grows with it: see k_release.
constexpr int kArrivals = 16, kArrivalStride = 64, kMarkStride = 16;
constexpr uint64_t kSharedBits = 256 + 4 * kArrivals * kArrivalStride;
struct SharedControl {
    uint32_t magic;
    uint32_t flags;                     // of the last call
    uint32_t pending;                   // of a call under way, 0 between
    uint32_t arrived;                   // places whose workgroups are all done, 0 between
};
struct SharedArgs {
    PagesOf g;
    int32_t* table;
    int64_t free_capacity;
    const int32_t* held_in;
    int32_t* held_out;
    int32_t* free_pages;
    const int32_t* free_in;
    int32_t* free_out;
    int32_t* extra;
    int32_t count;
    const int32_t* parents;             // forks
    const int32_t* children;            // ... or the requests released
    const int32_t* context;             // forks; null: none has any
    SharedControl* ctl;
    uint32_t* arrivals;
    uint32_t* bits;
};
hipError_t launch_fork(const SharedArgs& a, hipStream_t s);
hipError_t launch_release(const SharedArgs& a, hipStream_t s);

}  // namespace kvc
