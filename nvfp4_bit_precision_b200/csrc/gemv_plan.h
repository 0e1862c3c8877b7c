// gemv_plan.h -- how the few-token products cut their work: what the host decides from
// sizes alone.  Plain C++, without CUDA.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace nvfp4 {

// One matrix: even segments of at most `fit` rows, each with as many CTAs.  Bringing a
// row of x costs a CTA about as much as a tile, so a CTA has tiles of one segment
// alone, and `cost`, its tiles and rows over the waves of CTAs, is what a form's time
// goes by.  5120 x 20480 at 17 rows: 59 us so, 100 us with the tiles of all segments in
// equal runs; 512 x 20480 at 8 rows, 4 segments: 13 us, 27 us with a CTA for each tile
// of one segment.  Up to four waves are tried, and as many as there are where every
// multiprocessor has more segments than that.
struct Plan {
    int seg_rows = 1, ctas = 1;
    int64_t cost = INT64_MAX;
    Plan() = default;
    Plan(int64_t rows, int64_t tiles, int64_t fit, int sms)
    {
        const int64_t segments = (rows + fit - 1) / fit;
        seg_rows = static_cast<int>((rows + segments - 1) / segments);
        const int64_t fewest = (segments + sms - 1) / sms;
        for (int64_t wave = fewest; wave <= std::max<int64_t>(fewest, 4); ++wave) {
            const int64_t n = std::min(tiles, wave * sms / segments);
            const int64_t c = wave * ((tiles + n - 1) / n + seg_rows);
            if (c < cost) cost = c, ctas = static_cast<int>(n);
        }
    }
};

struct Form {
    int columns;  // of x a matrix instruction takes: 8 or 16
    bool panels;
    Plan plan;
};

// The form that costs least; a tile or a row costs a twentieth more with panels, where
// loads wait at each panel's start, and a fifth more with 16 columns of x.  (5120 x
// 20480: 4 rows 31 us, with panels 34; 16 rows 85 and 57, with 16 columns 109.  2048 x
// 24576, 8 rows: 36 us with 16 columns, 45 with panels, 47 without either.)  fit8,
// fit16: the whole rows of x that fit at once with 8 and with 16 columns.
inline Form cheapest_form(int64_t rows, int64_t tiles, int64_t fit8, int64_t fit16, int sms)
{
    const Form one{8, false, Plan(rows, tiles, fit8, sms)}, two{16, false, Plan(rows, tiles, fit16, sms)};
    const Form panels{8, true, Plan(rows, tiles, 8, sms)};
    if (20 * one.plan.cost <= std::min(24 * two.plan.cost, 21 * panels.plan.cost)) return one;
    return 24 * two.plan.cost <= 21 * panels.plan.cost ? two : panels;
}

}  // namespace nvfp4
