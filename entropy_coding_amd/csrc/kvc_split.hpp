// How attention deals its work to workgroups: the integer arithmetic that the
// kernels share, as plain functions that a host compiler takes too.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KVC_BOTH __host__ __device__ inline
#else
#define KVC_BOTH inline
#endif

namespace kvc {

// The same for all lanes of a wave, where that has to be said.
KVC_BOTH int uniform(int x) {
#ifdef __HIP_DEVICE_COMPILE__
    return __builtin_amdgcn_readfirstlane(x);
#else
    return x;
#endif
}

// Row tiles of a sequence, and its units of work.
KVC_BOTH uint32_t row_tiles(uint32_t rows, uint32_t ratio, uint32_t tile_shift) {
    return (rows * ratio + (1u << tile_shift) - 1) >> tile_shift;
}
KVC_BOTH uint32_t units_in(uint32_t tokens, uint32_t unit_shift) {
    return (tokens + (1u << unit_shift) - 1) >> unit_shift;
}

// Units that a workgroup takes, at least `least`; the next number tried where
// items rounded up to it do not fit the workgroups.
KVC_BOTH uint32_t first_per(uint32_t units, uint32_t target, uint32_t least) {
    const uint32_t per = (units + target - 1) / target;
    return per < least ? least : per;
}
KVC_BOTH uint32_t next_per(uint32_t per) { return per + (per + 7) / 8; }
KVC_BOTH uint32_t groups_in(uint32_t real, uint32_t per) { return (real + per - 1) / per; }

struct Plan {
    uint32_t per;
    uint32_t aligned;                           // 0 or 1

    KVC_BOTH uint32_t units(uint32_t real) const { return aligned ? groups_in(real, per) * per : real; }
};

// The item that holds unit `at` of a sequence's, which begin with unit
// `begin`: a KV head and a row tile (the tile changing fastest).
struct Item {
    uint32_t head, tile;
    uint32_t first;                             // its first unit
};
KVC_BOTH Item item_at(uint32_t begin, uint32_t units, uint32_t tiles, uint32_t at) {
    const uint32_t item = (at - begin) / units, head = item / tiles;
    return Item{head, item - head * tiles, begin + item * units};
}

// Of an item's `tiles` tiles, those before its unit `done`.  As a rule a unit
// is a tile; where they differ (a chain's rows that see less than the whole
// sequence, units of many tiles) the tiles are spread over the units, exact
// at both ends: products stay below 2^53.
KVC_BOTH int tiles_before(uint32_t tiles, uint32_t done, uint32_t units) {
    if (done >= units) return static_cast<int>(tiles);
    if (tiles == units) return static_cast<int>(done);
    return uniform(static_cast<int>(double(tiles) * double(done) / double(units)));
}

// What a row tile sees: `length` tokens at all (a chain's rows nothing behind
// their last one), and those before `full` by every row of it.
struct Extent {
    int length, full;
};
KVC_BOTH Extent extent_of(bool chain, int context, int nodes, int rows, int row0, int tile_rows, int ratio) {
    const int last = (row0 + tile_rows < rows ? row0 + tile_rows : rows) - 1;
    return Extent{context + (chain ? last / ratio + 1 : nodes), context + (chain ? row0 / ratio + 1 : 0)};
}

// A workgroup's part of the item that begins with unit `first`, from unit
// `at` on: its tiles [ta, tb), whether it is the whole item, and where the
// part goes if not.  The workgroup's units are [from, end).
struct Range {
    int ta, tb;
    bool whole;
    uint32_t slot;
};
KVC_BOTH Range range_of(uint32_t first, uint32_t units, uint32_t real, uint32_t tiles, uint32_t place, uint32_t at,
                        uint32_t from, uint32_t end) {
    const uint32_t past = first + units;
    Range r;
    r.whole = first >= from && past <= end;
    r.slot = 2 * place + (first >= from ? 1u : 0u);
    r.ta = tiles_before(tiles, at - first, real);
    r.tb = tiles_before(tiles, (past < end ? past : end) - first, real);
    return r;
}

// The workgroups that share an item, and where the s-th of them left its part.
struct Sharers {
    uint32_t first, last;

    KVC_BOTH uint32_t slot(uint32_t s) const { return 2 * (first + s) + (s ? 0u : 1u); }
};
KVC_BOTH Sharers sharers_of(uint32_t first, uint32_t units, uint32_t per) {
    return Sharers{first / per, (first + units - 1) / per};
}

}  // namespace kvc
