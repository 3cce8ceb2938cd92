// cross_entropy_plan.cuh -- how cross_entropy.cu cuts its products into tiles,
// pieces and parts, deals them out, and what workspace that takes (host
// arithmetic; common.cuh's align256).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace moe {
namespace ce {

constexpr int ROWS = 128, BN = 256, BK = 64;  // a CTA's rows of a tile, its most columns, K of a step
constexpr size_t PIECE_BYTES = 256u << 20;

inline int tiles(int n, int b) { return (n + b - 1) / b; }

// Columns of a piece: what 256 MiB hold, in whole tiles, and pieces of nearly equal size, `more` of them than that takes.
inline int piece_columns(int T, int V, int more)
{
    const int64_t most = std::max<int64_t>(BN, (int64_t)(PIECE_BYTES / 2 / std::max(T, 1)) / BN * BN);
    const int64_t pieces = (V + most - 1) / most + more;
    return (int)((V + pieces - 1) / pieces + BN - 1) / BN * BN;
}

inline int round_up(int n, int b) { return tiles(n, b) * b; }

// Rows of a box of tokens: a single CTA's first tile has them all, where there are few.
inline int box_rows(int T, int C) { return C == 1 && T < ROWS ? round_up(T, 8) : ROWS; }

// Columns of a tile: equal ones over all n.
inline int tile_columns(int n) { return round_up(tiles(n, tiles(n, BN)), 32); }

// Measured time of a step (K = 64) of 256 columns in us: pairs read and store less through shared memory per product and
// have two more steps on their way.  Forward pass by single CTAs and by pairs, us: 4,096 x 65,536 and H = 2,048 557 and
// 523, 2,048 x 32,768 176 and 144, 512 x 32,000 49 and 42, 2,500 x 20,000 with H = 4,096 241 and 227.  The rule holds
// where a tile's steps cover its way out: with H = 512 and below pairs are taken too often (4,096 x 16,384 48 and 60,
// 1,500 x 30,000 with H = 256 25 and 32).
inline double step_us(int C) { return C == 1 ? 0.325 : 0.298; }

// Tiles of the logits: by single CTAs or pairs, as wide as they go unless narrower ones fill the last round better
// (100,003 columns for one row tile on 152 SMs: three rounds of 224 instead of 256).  A tile costs its steps and some 16
// columns' worth besides.
struct Cut {
    int C, bn;
};

// Tokens up to which narrower tiles are looked at.  Each tile leaves 16 bytes a token: behind 64 rounds of tiles of a
// large vocabulary, where they gain 1.6% at most (by these costs), the workspace stays that of the widest.
inline int64_t narrow_rows(int V, int sms) { return V <= 16384 ? INT32_MAX : (int64_t)ROWS * (64 * sms / tiles(V, BN)); }

// Bytes of the tiles' maxima and sums: enough for any number of tokens up to T, whichever tiles they get.
inline size_t stats_bytes(int T, int V, int sms)
{
    const int64_t narrow = std::min<int64_t>(T, narrow_rows(V, sms));
    return align256(16 * (size_t)std::max<int64_t>((int64_t)T * tiles(V, BN), narrow * tiles(V, BN / 2)));
}

inline Cut cut_logits(int rows, int V, int sms)
{
    Cut best = {1, BN};
    double least = 1e300;
    for (int C = 1; C <= 2; C++)
        for (int bn = BN; bn >= (rows <= narrow_rows(V, sms) ? BN / 2 : BN); bn -= 32) {
            const int64_t items = (int64_t)tiles(rows, ROWS * C) * tiles(V, bn), at_once = sms / C;
            const double cost = (double)((items + at_once - 1) / at_once) * (bn + 16) * step_us(C);
            if (cost < least) least = cost, best = {C, bn};
        }
    return best;
}

// What a CTA of the gradients takes, in steps of BK: dh's items (nk0 each) dealt out first, dW's (nk1 each) so that the
// longest CTA is as short as it gets.
struct Deal {
    int longer, long_items, short_items;
    int64_t steps;
};

inline Deal deal(int64_t items0, int64_t nk0, int64_t items1, int64_t nk1, int64_t G)
{
    // a tile's way out takes as long as some six steps, under the next tile's steps where those are more
    nk0 = std::max<int64_t>(nk0, 6);
    nk1 = std::max<int64_t>(nk1, 6);
    Deal best = {0, 0, 0, INT64_MAX};
    const int64_t q = items0 / G, r = items0 % G;
    auto with = [&](int64_t s) {  // s items of the second job for a CTA without an extra one of the first
        const int64_t rest = std::max<int64_t>(0, items1 - (G - r) * s);
        if (s < 0 || (r == 0 && rest > 0)) return;
        const int64_t l = r ? (rest + r - 1) / r : s;
        const int64_t steps = std::max(r ? (q + 1) * nk0 + l * nk1 : 0, q * nk0 + s * nk1);
        if (steps < best.steps) best = {(int)r, (int)l, (int)s, steps};
    };
    with((items1 + G - r - 1) / (G - r));
    if (items1 > 0) {  // about where all have the same
        const int64_t s = ((items0 * nk0 + items1 * nk1) / G - q * nk0) / nk1;
        for (int64_t i = s - 1; i <= s + 2; i++) with(i);
    }
    return best;
}

struct Layout {
    int columns, pieces, parts, C;  // dh's sums over a piece are split into parts; by CTAs or pairs
    int64_t part_rows;
    size_t d, sums, total;  // bytes: d after the top value, fp32 sums of dh when there are several pieces or parts
};

constexpr int MOST_PARTS = 32;
constexpr size_t SPLIT_BYTES = 64u << 20, ROOM_BYTES = 512u << 10;

// Bytes of one part's sums, by the longer of the rounded rows.
inline size_t one_part(int T, int H) { return (size_t)round_up(T, 2 * ROWS) * H * 4; }

// What a split into several parts may take: 64 MiB, and with d little more than what pieces without a split take.
inline bool split_fits(int T, int H, int columns, size_t sums)
{
    return sums <= SPLIT_BYTES && (size_t)T * columns * 2 + sums <= PIECE_BYTES + ROOM_BYTES + one_part(T, H);
}

// The workspace of T tokens: enough for any number up to T (every term grows with it), whichever pieces and parts they get.
inline size_t layout_bytes(int T, int H, int V)
{
    const size_t d = align256(std::max((size_t)T * BN * 2, std::min(PIECE_BYTES, (size_t)T * round_up(V, BN) * 2))), one = one_part(T, H);
    const size_t whole = piece_columns(T, V, 0) < V ? one : 0;
    const size_t parts = std::min(MOST_PARTS, tiles(V, BK));
    const size_t split = parts > 1 ? std::min(PIECE_BYTES + ROOM_BYTES + one, d + std::min(SPLIT_BYTES, parts * one)) : 0;
    return 256 + std::max(d + align256(whole), align256(split) + 512);  // (512: d and the sums begin at multiples of 256)
}

// Splitting dh's sums pays where its few, long items would leave the other CTAs waiting: the steps' time is weighed
// against a part's sums, written and read (8 bytes a value at 6 TB/s), and a launch for them.  Where the best split does
// not fit, splits with one more piece (two launches, some 16 us) are weighed as well.
inline Layout layout(int T, int H, int V, int sms)
{
    Layout l;
    const int nk1 = tiles(T, BK), nt = tiles(H, BN);
    double least = 1e300, any = 1e300;  // of what fits, of all
    bool limited = false;
    for (int more = 0; more == 0 || (more == 1 && limited); more++) {
        const int columns = piece_columns(T, V, more), pieces = tiles(V, columns);
        const int n = std::min(V, columns), nk0 = tiles(n, BK);
        for (int C = 1; C <= 2; C++) {
            const int64_t items0 = (int64_t)tiles(T, ROWS * C) * nt, items1 = (int64_t)tiles(n, ROWS * C) * nt;
            for (int s = 1 + more; s <= MOST_PARTS && s <= nk0; s++) {
                const bool fits = s == 1 || split_fits(T, H, columns, (size_t)s * round_up(T, ROWS * C) * H * 4);
                const Deal d = deal(items0 * s, tiles(nk0, s), items1, nk1, std::min<int64_t>(items0 * s + items1, sms / C));
                const double us = (step_us(C) * tile_columns(H) / BN * d.steps +
                                   (s > 1 || pieces > 1 ? 3.0 / pieces + 1.3e-6 * s * T * H * (pieces > 1 ? 2 : 1) : 0) + 16) * pieces;
                if (more == 0 && us < any) any = us, limited = !fits;
                if (fits && us < least) least = us, l.parts = s, l.C = C, l.columns = columns, l.pieces = pieces;
            }
        }
    }
    l.part_rows = round_up(T, ROWS * l.C);
    l.d = 256;
    l.sums = l.d + align256((size_t)T * l.columns * 2);
    l.total = layout_bytes(T, H, V);
    return l;
}

}  // namespace ce
}  // namespace moe
