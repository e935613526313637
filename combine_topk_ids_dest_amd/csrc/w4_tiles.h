// Which tiles the products with 4-bit weights take: the cut of few-row tiles, and
// few-row or big ones by what they are estimated to take. Compiled for the host as
// well.
#pragma once

#include "tiles.h"

namespace moe_ep {

// How tiles of up to 16 rows are cut: 2^lw runs of 16 rows of w each, but in the
// grid's last, partial round 2^last, so that it is shorter where CUs would be
// idle.
struct FewCut {
    int lw, last;
    int nt;                      // tiles of a run, over all columns
    int whole, total;            // tiles before the last round, and of all rounds
};

// A cut's rounds times a tile's time, in columns of 16 rows of w: a tile's own and
// about 2048 for its start and end.
MOE_EP_TILES float few_columns(const FewCut& c, int H) {
    return (float)(c.whole / kGrid) * (float)((H << c.lw) + 2048) +
           (c.total > c.whole ? (float)((H << c.last) + 2048) : 0.f);
}

// The cut of `runs` runs of up to 16 rows that takes least. least: lw for runs
// of more than 8 rows (a step of 2048 columns of 16 rows is no segment).
MOE_EP_TILES FewCut few_cut(int runs, int N, int H, int bo, int least) {
    FewCut best = {};
    float best_cost = 0.f;
#ifdef __HIPCC__
#pragma unroll
#endif
    for (int lw = 3; lw >= 0; --lw) {
        if (lw < least) break;
        const int nt = (N + (bo << lw) - 1) / (bo << lw);
        const int tiles = runs * nt;
        const int whole = tiles / kGrid * kGrid, rest = tiles - whole;
        int split = rest * 8 <= kGrid ? 3 : rest * 4 <= kGrid ? 2 : rest * 2 <= kGrid ? 1 : 0;
        if (split > lw - least) split = lw - least;
        const FewCut c = {lw, lw - split, nt, whole, whole + (rest << split)};
        const float cost = few_columns(c, H);
        if (lw == 3 || cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

// What a product takes with tiles of a few rows, in us, and with big ones (`turns`
// whole rounds of the grid of `rows` rows each, then one of `last`; 0: none), from
// measured times. Both sides where the choice turns, in us, few and big: 7168 ->
// 2 x 2048, E4M3, 64 rows 23 and 57, 256 rows 65 and 73, 512 rows 125 and 73;
// 2048 -> 7168, 96 rows 22 and 22, 128 rows 26 and 22.
MOE_EP_TILES float few_time(const FewCut& c, int H, int group) {
    return 6.f + few_columns(c, H) * (group == 16 ? 16.f / 29300.f : 16.f / 39000.f);
}

MOE_EP_TILES float big_time(int turns, int rows, int last, int H, int group) {
    const float pairs = (float)((H + 127) / 128);
    const float start = group == 16 ? 0.55f : 0.4f, row = group == 16 ? 0.0135f : 0.0125f;
    return 8.f + (float)turns * pairs * (start + row * (float)rows) +
           (last ? pairs * (start + row * (float)last) : 0.f);
}

// Over all tokens: whether few-row tiles, cut so, take less than big ones.
MOE_EP_TILES bool few_over_all(const FewCut& few, int rows, int N, int H, int cols, int group) {
    const Cut c = cut_rows(rows, 0);
    const int tiles = c.runs * ((N + cols - 1) / cols);
    const int rest = tiles % kGrid, parts = last_parts(tiles);
    return few_time(few, H, group) <
           big_time(tiles / kGrid, c.kind * 32, rest ? (c.kind + parts - 1) / parts * 32 : 0, H,
                    group);
}

// By expert, with room for `rows` rows each: whether few-row tiles take less than
// big ones even where every group is full, so that no counts need looking at. (8
// experts of 17 to 32 rows, 512 -> 1024, powers of two: 9.1 us, beside the code of
// 32-row tiles 11.8; 32 of 32 rows, 7168 -> 2 x 2048, E4M3, 281 and 129.)
MOE_EP_TILES bool few_if_full(int groups, int rows, int N, int H, int bo, int cols, int group) {
    if (rows <= kSmall) return true;
    const Cut c = cut_rows(rows, 0);
    const int tiles = groups * c.runs * ((N + cols - 1) / cols);
    const int runs = groups * ((rows + kSmall - 1) / kSmall);
    return few_time(few_cut(runs, N, H, bo, 1), H, group) <
           big_time(tiles / kGrid, c.kind * 32, tiles % kGrid ? c.kind * 32 : 0, H, group);
}

// By expert, where groups of more than kSmall rows are `total` big tiles, one round
// of the grid at most, of up to 32 * most rows, with `low` runs of 16 rows of other
// groups behind them: whether few-row tiles for all `runs` runs take less. (Each
// block has its share of the runs behind its big tile.)
MOE_EP_TILES bool few_instead(int total, int most, int runs, int low, int N, int H, int bo,
                              int group) {
    const int cut = total < kGrid ? last_parts(total) : 1;
    float big = big_time(0, 0, (most + cut - 1) / cut * 32, H, group);
    if (low) big += few_time(few_cut(low, N, H, bo, 0), H, group) - 6.f;
    return few_time(few_cut(runs, N, H, bo, 1), H, group) < big;
}

}  // namespace moe_ep
