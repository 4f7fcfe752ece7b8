// paged_splits.h -- how far the key axis of a chunk of new tokens is cut.  Host only.
#pragma once

#include <cstdint>

namespace dit {

// Splits of the key axis for the tensor-memory kernel, whose blocks run one per SM
// in rounds of 148.  Of the splits that fill 1 to 8 rounds the one that is done
// first, by a block's start and end (9 us), its steps (1.8 us each) and the write
// and read of the parts (part_bytes per split) with their join (5 us); none unless
// a seventh is gained, and no run below 512 keys (a chunk of 1,000 rows of 40 heads
// over itself: 59 us whole, 185 in 4 splits).
// Measured (heads of 128, 30,000 keys): 256 rows of 16 heads, 16 tiles, 130 us in
// 10 splits (two rounds) and 85 in 9, as chosen; 300 rows of 75 heads, 150 tiles,
// 812 us whole, 609 in 2 and 526 as chosen.
// Never fewer splits for more keys: the time is keys * a(splits) + b(splits) and
// b only grows, so more keys can only turn the choice to smaller a, that is more
// splits.
inline int64_t tc_splits(int64_t blocks, int64_t keys, int64_t part_bytes)
{
    constexpr int64_t kSms = 148, kRounds = 8;
    const double steps_us = (double)keys / 128 * 1.8, part_us = (double)part_bytes * 2 / 6.4e6;
    int64_t best = 1;
    double best_us = 0.86 * (double)((blocks + kSms - 1) / kSms) * (steps_us + 9.0);
    for (int64_t rounds = 1; rounds <= kRounds; ++rounds) {
        int64_t s = kSms * rounds / blocks;
        s = s < keys / 512 ? s : keys / 512;
        const double us = (double)rounds * (steps_us / (double)s + 9.0) + 5.0 + part_us * (double)s;
        if (s > 1 && us < best_us) {
            best = s;
            best_us = us;
        }
    }
    return best;
}

}  // namespace dit
