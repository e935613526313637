// Which tiles the products with 4-bit weights take, on the host: for each line
//   dense T H N gated group
//   experts rows H N gated group count...
// of the input prints the kernel and the heights of the tiles in use (few: tiles of
// up to 16 rows), as the kernels choose them from the same functions.
#include <climits>
#include <cstdio>
#include <iostream>
#include <set>
#include <sstream>
#include <string>
#include <vector>

#include "w4_tiles.h"

using namespace moe_ep;

constexpr int kCols = 256;                       // rows of w of a big tile

static int height(int fragments) {
    return fragments > 4 ? fragments * 32 : fragments > 2 ? 128 : fragments * 32;
}

static void big(const std::vector<int>& rows, int small_to, int ntb, std::set<int>& heights) {
    int n[kKinds] = {}, total = 0;
    for (int r : rows) {
        const Cut c = cut_rows(r, small_to);
        n[c.kind] += c.runs * (c.kind ? ntb : 1);
    }
    for (int k = 1; k < kKinds; ++k) total += n[k];
    const int parts = last_parts(total);
    for (int block = 0; block < kGrid; ++block)
        for (int t0 = 0; t0 < total; t0 += kGrid) {
            const Turn turn = turn_of(block, t0, total, parts);
            if (turn.t < 0) break;
            int t = turn.t, kind = kKinds - 1;
            while (kind > 1 && t >= n[kind]) t -= n[kind--];
            size_t g = 0;
            for (;; ++g) {
                const Cut c = cut_rows(rows[g], small_to);
                const int tiles = c.kind == kind ? c.runs * ntb : 0;
                if (t < tiles) break;
                t -= tiles;
            }
            const Piece p = piece_of(t, rows[g], cut_rows(rows[g], small_to).runs, kind, ntb,
                                     turn.sub, turn.cut);
            if (p.m0 < p.end) heights.insert(height(p.fragments));
        }
    if (n[0]) heights.insert(0);
}

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string what;
        int room, H, N, gated, group;
        in >> what >> room >> H >> N >> gated >> group;
        const int bo = gated ? kSmall / 2 : kSmall, cols = gated ? kCols / 2 : kCols;
        const int ntb = (N + cols - 1) / cols;
        std::set<int> heights;
        std::string kernel = "big";
        if (what == "dense") {
            const FewCut c = few_cut((room + kSmall - 1) / kSmall, N, H, bo, room > 8 ? 1 : 0);
            if (few_over_all(c, room, N, H, cols, group)) {
                kernel = "few";
                heights.insert(0);
            } else {
                big({room}, 0, ntb, heights);
            }
        } else {
            std::vector<int> rows;
            for (int c; in >> c;) rows.push_back(c < 0 ? 0 : c > room ? room : c);
            int low = 0, over = 0, all = 0, total = 0, most = 0;
            for (int r : rows) {
                all += (r + kSmall - 1) / kSmall;
                const Cut c = cut_rows(r, kSmall);
                (c.kind ? over : low) += c.runs;
                if (c.kind > most) most = c.kind;
            }
            total = over * ntb;
            int small_to = kSmall;
            if (room <= 2 * kSmall) {
                const bool few = few_if_full((int)rows.size(), room, N, H, bo, cols, group);
                kernel = few ? "few" : "low";
                if (few) small_to = INT_MAX;
            }
            if (small_to == kSmall && total > kGrid) small_to = 0;
            else if (small_to == kSmall && total &&
                     few_instead(total, most, all, low, N, H, bo, group))
                small_to = INT_MAX;
            big(rows, small_to, ntb, heights);
        }
        std::cout << kernel;
        for (int h : heights) std::cout << " " << (h ? std::to_string(h) : "few");
        std::cout << "\n";
    }
}
