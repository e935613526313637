// Deals out the products' big and narrow tiles as the kernel does, for every
// block of the grid, and counts the blocks that store each row of each column
// tile: it has to be one. Prints the layouts where it is not.
#include <cstdio>
#include <random>
#include <vector>

#include "tiles.h"

using namespace moe_ep;

struct Store {
    int from, to;
};

static int check(const std::vector<int>& counts, int ntb, int small_to) {
    int n[kKinds] = {};
    for (int rows : counts) {
        const Cut c = cut_rows(rows, small_to);
        n[c.kind] += c.runs * (c.kind ? ntb : 1);
    }
    int total = 0;
    for (int k = 1; k < kKinds; ++k) total += n[k];
    std::vector<std::vector<Store>> stores(counts.size() * ntb);
    const int parts = last_parts(total);
    for (int block = 0; block < kGrid; ++block)
        for (int t0 = 0; t0 < total; t0 += kGrid) {
            const Turn turn = turn_of(block, t0, total, parts);
            if (turn.t < 0) break;
            int t = turn.t, kind = kKinds - 1;
            while (kind > 1 && t >= n[kind]) t -= n[kind--];
            size_t g = 0;                        // the group of tile t of this kind
            for (;; ++g) {
                const Cut c = cut_rows(counts[g], small_to);
                const int tiles = c.kind == kind ? c.runs * ntb : 0;
                if (t < tiles) break;
                t -= tiles;
            }
            const Piece p = piece_of(t, counts[g], cut_rows(counts[g], small_to).runs, kind, ntb,
                                     turn.sub, turn.cut);
            if (p.m0 >= p.end) continue;
            // a tile stores the rows it has, up to its own height
            const int rows = tile_rows(p.fragments);
            stores[g * ntb + p.col].push_back({p.m0, p.end - p.m0 < rows ? p.end : p.m0 + rows});
        }
    for (size_t g = 0; g < counts.size(); ++g) {
        const int rows = cut_rows(counts[g], small_to).kind ? counts[g] : 0;
        for (int c = 0; c < ntb; ++c) {
            std::vector<int> by(rows, 0);
            for (const Store& s : stores[g * ntb + c])
                for (int r = s.from; r < s.to; ++r)
                    if (r >= rows || ++by[r] > 1) {
                        std::printf("group %zu of %zu, %d rows, column tile %d of %d: row %d twice\n",
                                    g, counts.size(), rows, c, ntb, r);
                        return 1;
                    }
            for (int r = 0; r < rows; ++r)
                if (!by[r]) {
                    std::printf("group %zu of %zu, %d rows, column tile %d of %d: row %d never\n",
                                g, counts.size(), rows, c, ntb, r);
                    return 1;
                }
        }
    }
    return 0;
}

int main() {
    int bad = 0, layouts = 0;
    // one group: the product over all tokens
    for (int ntb : {1, 2, 3, 5, 8, 16, 24, 28, 32, 40, 48, 56, 64, 100, 129, 256})
        for (int rows = 1; rows <= 1100; rows += rows < 600 ? 7 : 13) {
            bad += check({rows}, ntb, 0);
            ++layouts;
        }
    for (int rows : {513, 544, 576, 577, 4096, 8191}) bad += check({rows}, 28, 0), ++layouts;
    // experts
    std::mt19937 rng(5);
    for (int i = 0; i < 3000; ++i) {
        std::vector<int> counts(1 + rng() % 40);
        const int top = 1 + rng() % 700;
        for (int& c : counts) c = rng() % 4 ? rng() % (top + 1) : 0;
        bad += check(counts, 1 + rng() % 30, rng() % 2 ? kSmall : 0);
        ++layouts;
    }
    std::printf("%d of %d layouts wrong\n", bad, layouts);
    return bad ? 1 : 0;
}
