// Which rows and columns a block of the products works on: integer arithmetic
// only, compiled for the host as well, where every piece of a layout can be
// counted.
#pragma once

#ifdef __HIPCC__
#define MOE_EP_TILES __host__ __device__ __forceinline__
#else
#define MOE_EP_TILES inline
#endif

namespace moe_ep {

constexpr int kGrid = 256;                       // blocks of the products
constexpr int kGroup = 8;                        // runs of rows side by side
constexpr int kSmall = 16;                       // rows of a small tile
constexpr int kKinds = 9;                        // runs of 32 k rows, k = 1..8; small: 0

// Tile of block b in a round of `left` tiles over the grid, -1 for none.
// Blocks go to the eight XCDs in turn, so each XCD (with an L2 of its own)
// gets a run of neighbouring tiles, which share rows of x and w.
MOE_EP_TILES int tile_of(int b, int grid, int left) {
    const int r = left < grid ? left : grid;
    const int per = (r + 7) / 8;
    const int slot = b >> 3;
    const int t = (b & 7) * per + slot;
    return slot < per && t < r ? t : -1;
}

// A group's rows in equal runs of at most 256, or in small tiles.
struct Cut {
    int runs, kind;
};

MOE_EP_TILES Cut cut_rows(int rows, int small_to) {
    Cut c;
    if (rows <= small_to) {
        c.kind = 0;
        c.runs = (rows + kSmall - 1) / kSmall;
        return c;
    }
    c.runs = (rows + 255) / 256;
    c.kind = ((rows + c.runs - 1) / c.runs + 31) / 32;
    return c;
}

// The last, partial round of `total` tiles over the grid: with at most half (a
// quarter) as many tiles as blocks, each tile is cut in two (four) by its rows.
// 3.5 rounds then take 3.5 tiles' time and not 4, and a few rows an expert,
// bound by the weights' bytes, are read by all CUs.
MOE_EP_TILES int last_parts(int total) {
    const int rest = total - total / kGrid * kGrid;
    return rest * 4 <= kGrid ? 4 : rest * 2 <= kGrid ? 2 : 1;
}

// A block's tile in the round that starts at tile t0 (t < 0: none), and which
// part of how many it is.
struct Turn {
    int t, sub, cut;
};

MOE_EP_TILES Turn turn_of(int block, int t0, int total, int parts) {
    const int whole = total / kGrid * kGrid;
    if (t0 < whole) return Turn{t0 + (block & 7) * (kGrid / 8) + (block >> 3), 0, 1};
    const int u = tile_of(block, kGrid, (total - whole) * parts);
    if (u < 0) return Turn{-1, 0, 1};
    return Turn{whole + u / parts, u % parts, parts};
}

// Rows [m0, end) of a group (none if m0 >= end) by the columns of tile `col`,
// in fragments of 32 rows.
struct Piece {
    int m0, end, col, fragments;
};

// Part `sub` of `cut` of tile l of a group whose rows go in `runs` runs of
// 32 * kind rows, kGroup runs at a time over all `ntb` column tiles. A part ends
// where the next begins: its tile may be higher (tile_rows), and rows that two
// blocks store are wrong where the residual is the output.
MOE_EP_TILES Piece piece_of(int l, int rows, int runs, int kind, int ntb, int sub, int cut) {
    const int m8 = l / (kGroup * ntb) * kGroup;
    const int wide = runs - m8 < kGroup ? runs - m8 : kGroup;
    const int in = l - m8 * ntb;
    const int from = (m8 + in % wide) * kind * 32;
    const int run_end = from + kind * 32 < rows ? from + kind * 32 : rows;
    Piece p;
    p.fragments = (kind + cut - 1) / cut;
    p.m0 = from + sub * p.fragments * 32;
    p.end = p.m0 + p.fragments * 32 < run_end ? p.m0 + p.fragments * 32 : run_end;
    p.col = in / wide;
    return p;
}

// Rows of the tile that multiplies so many fragments (there is none of 96 and
// none below 64).
MOE_EP_TILES int tile_rows(int fragments) {
    return fragments > 4 ? fragments * 32 : fragments > 2 ? 128 : 64;
}

}  // namespace moe_ep
