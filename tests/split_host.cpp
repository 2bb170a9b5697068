// The kernels' own arithmetic of how attention deals its work
// (csrc/kvc_split.hpp), walked through on the host: what the waves find by
// sums over their lanes is summed here one sequence after the other.
#include <cstddef>
#include <vector>

#include "kvc_split.hpp"

using namespace kvc;

struct SplitPart {
    int32_t workgroup, sequence, head, tile, ta, tb, whole, slot, length;
};
struct SplitItem {
    int32_t sequence, head, tile, first_sharer, last_sharer, length;
};

extern "C" int split_parts(int batch, const int32_t* rows, const int32_t* contexts, int heads, int ratio, int chain,
                           int tile_shift, int unit_shift, int unit_tokens, int target, int least, uint32_t* per,
                           SplitPart* parts, int max_parts, SplitItem* items, int max_items, int* n_items) {
    std::vector<uint32_t> tiles(batch), real(batch), begin(batch + 1);
    uint32_t units = 0, all = 0;
    for (int b = 0; b < batch; ++b) {
        tiles[b] = row_tiles(rows[b], ratio, tile_shift);
        real[b] = units_in(uint32_t(contexts[b]) + uint32_t(rows[b]), unit_shift);
        units += tiles[b] * heads * real[b];
        all += tiles[b] * heads;
    }
    Plan plan{first_per(units, target, least), 0};
    uint32_t tried = plan.per;
    for (int i = 0; all <= uint32_t(target) && i < 2 && !plan.aligned; ++i, tried = next_per(tried)) {
        uint32_t groups = 0;
        for (int b = 0; b < batch; ++b) groups += tiles[b] * heads * groups_in(real[b], tried);
        if (groups <= uint32_t(target)) plan = Plan{tried, 1};
    }
    *per = plan.per;
    for (int b = 0; b < batch; ++b) begin[b + 1] = begin[b] + tiles[b] * heads * plan.units(real[b]);
    const auto extent = [&](int b, uint32_t tile) {
        return extent_of(chain, contexts[b], rows[b], rows[b] * ratio, int(tile << tile_shift), 1 << tile_shift, ratio);
    };
    *n_items = 0;
    for (int b = 0; b < batch; ++b)
        for (int h = 0; h < heads; ++h)
            for (uint32_t t = 0; t < tiles[b]; ++t) {
                const Sharers who = sharers_of(begin[b] + (h * tiles[b] + t) * plan.units(real[b]), plan.units(real[b]), plan.per);
                if (*n_items == max_items) return -1;
                items[(*n_items)++] = SplitItem{b, h, int32_t(t), int32_t(who.first), int32_t(who.last), extent(b, t).length};
            }
    int n = 0;
    for (int w = 0; w < target; ++w) {
        const uint32_t from = w * plan.per, end = from + plan.per;
        for (uint32_t at = from; at < end;) {
            int b = 0;
            while (b < batch && !(at >= begin[b] && at < begin[b + 1])) ++b;
            if (b == batch) break;
            const Item i = item_at(begin[b], plan.units(real[b]), tiles[b], at);
            const int length = extent(b, i.tile).length;
            const Range r = range_of(i.first, plan.units(real[b]), real[b], (uint32_t(length) + unit_tokens - 1) / unit_tokens,
                                     w, at, from, end);
            if (n == max_parts) return -1;
            parts[n++] = SplitPart{w, b, int32_t(i.head), int32_t(i.tile), r.ta, r.tb, r.whole, int32_t(r.slot), length};
            at = i.first + plan.units(real[b]);
        }
    }
    return n;
}

extern "C" uint32_t sharer_slot(uint32_t first, uint32_t last, uint32_t s) { return Sharers{first, last}.slot(s); }
extern "C" int tile_full(int chain, int context, int nodes, int row0, int tile_rows, int ratio) {
    return extent_of(chain, context, nodes, nodes * ratio, row0, tile_rows, ratio).full;
}
