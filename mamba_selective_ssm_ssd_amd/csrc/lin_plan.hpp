// lin_plan.hpp -- which heads' workgroups of a scan of k_linear.hpp stay
// together on one XCD.  Host code alone.
#pragma once

#include <stdint.h>

namespace m3 {

constexpr int64_t kLinXcds = 8, kLinXcdUnits = 32; // XCDs of the card, compute units of each

// Workgroups of the XCD that has the most of them, where `segments` x heads / hg
// groups of hg heads go round the XCDs and a group, `tiles` workgroups a head,
// stays on its own.
inline int64_t lin_busiest(int64_t segments, int32_t heads, int32_t hg, int32_t tiles) {
    return (segments * (heads / hg) + kLinXcds - 1) / kLinXcds * hg * tiles;
}

// Whether groups of hg heads leave no XCD much more work than its share: no
// more than its compute units take at once, or an eighth above the mean.
inline bool lin_spread(int64_t segments, int32_t heads, int32_t hg, int32_t tiles) {
    const int64_t most = lin_busiest(segments, heads, hg, tiles);
    return most <= kLinXcdUnits || 8 * kLinXcds * most <= 9 * segments * heads * tiles;
}

// Heads of a group, a divisor of `heads`, for `scans` scans over `columns`
// column tiles of `segments` segments, where up to `share` heads have a row in
// common.
//
// Heads that share rows, and more neighbours of them: their rows lie side by
// side in memory.  Up to 16 where that leaves 32 groups an XCD to spread: 65536
// x 64 x 64 takes 706 us, 769 with one; 16 ragged sequences of 32 heads of 128
// 224 us with 16, 205 with one.  Several scans of whole sequences, which are of
// like lengths, up to eight and two groups an XCD: gradients of 4 x 2048 x 64 x
// 64 148 us, 165 with one; of cut ones, 4999 x 32 (8) x 128, 225, 211 with no
// more than share rows.
// Fewer than share rows where groups of all of them would leave XCDs idle: 200
// tokens of 64 heads of 128 that share one row of k and of v 13.9 us, 58 as one
// group, its gradients 44 and 88; gradients of 1000 such tokens 89 and 282, of
// 256 tokens of 32 heads that share four 22.5 and 27.
inline int32_t lin_head_group(int32_t share, int32_t heads, int64_t segments, int32_t columns, int32_t scans, bool cut) {
    const int32_t tiles = columns * scans;
    int32_t hg = share;
    while (hg > 1 && !lin_spread(segments, heads, hg, tiles)) {
        int32_t f = 2;
        while (hg % f) ++f;
        hg /= f;
    }
    const int32_t widest = scans == 1 ? 16 : cut ? 1 : 8;
    const int64_t least = kLinXcds * (scans == 1 ? 32 : 2);
    while (hg < widest && heads % (2 * hg) == 0 && segments * (heads / (2 * hg)) >= least &&
           lin_spread(segments, heads, 2 * hg, tiles))
        hg *= 2;
    return hg;
}

} // namespace m3
