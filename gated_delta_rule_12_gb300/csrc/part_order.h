// part_order.h -- which part of a row's statistics a tile of words belongs to where the tensor cores make the logits, and
// where in memory it goes.  Plain C++ on the host, so that a test can walk through it.
//
// The row tiles are taken in groups of up to 32 (rows whose h stays in L2; more where words are few), a group's words in
// windows; a window's tiles, row tile by row tile, are cut into runs of `each` for the pairs of CTAs.  So a pair meets the same
// rows for several tiles, and their statistics and best words stay in its registers: one part a run, or two where the run
// passes from one row tile to the next.
//
// The last group may have fewer row tiles than the others, down to one.  Its windows are wider then and its rows' runs are of
// more pairs, so each of the two kinds has its own number of parts a row (32 row tiles and 32768 words: 28), those of the last
// group's rows behind the others'.  One number for all rows, the most windows times the most slots, took 455 for 8193 tokens,
// 16 times the memory of 8192, and calls 5 to 26 % longer.  A row has at most one part more than there are tiles of words.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDN_BOTH __host__ __device__ __forceinline__
#else
#define GDN_BOTH inline
#endif

namespace gdn {

struct PartOrder {
    static constexpr int kRows = 256;   // of a row tile
    struct Group {
        int rows, window, each, windows, last_window, last_each;
        int rounds;   // tiles of a pair over the whole group
        int slots;    // parts a row may have in a window
        int parts;    // and in all
    } full, last;
    int pairs, size, groups;  // a group's row tiles; groups in front of the last one
    int split;                // rows of those

    static Group group(int rows, int nt, int pairs)
    {
        Group g = {};
        g.rows = rows;
        const int64_t tiles = (int64_t)rows * nt;
        g.window = tiles <= 8 * (int64_t)pairs ? nt : 8 * pairs / rows > 0 ? 8 * pairs / rows : 1;
        g.windows = (nt + g.window - 1) / g.window;
        g.last_window = nt - (g.windows - 1) * g.window;
        g.each = (rows * g.window + pairs - 1) / pairs;
        g.last_each = (rows * g.last_window + pairs - 1) / pairs;
        g.rounds = (g.windows - 1) * g.each + g.last_each;
        const int a = (g.window + g.each - 1) / g.each, b = (g.last_window + g.last_each - 1) / g.last_each;
        g.slots = (g.windows > 1 && a > b ? a : b) + 1;
        g.parts = g.windows * g.slots;
        return g;
    }
    // mt x nt tiles for `pairs` pairs of CTAs
    static PartOrder make(int mt, int nt, int pairs)
    {
        PartOrder o = {};
        o.pairs = pairs;
        o.size = nt >= 19 ? 32 : (8 * pairs + nt - 1) / nt;
        if (o.size < 32) o.size = 32;
        o.groups = (mt - 1) / o.size;
        o.full = group(o.size, nt, pairs);
        o.last = group(mt - o.size * o.groups, nt, pairs);
        o.split = o.groups * o.size * kRows;
        return o;
    }
    int rounds() const { return groups * full.rounds + last.rounds; }
    // Parts of N rows.
    int64_t total(int N) const { return (int64_t)full.parts * split + (int64_t)last.parts * (N - split); }

    // Tile `round` of a pair: its row tile, word tile and part; false where it has none.
    GDN_BOTH bool at(int pair, int round, int &m, int &n, int &part) const
    {
        const int k = round / full.rounds, g = k < groups ? k : groups;
        const Group &q = g < groups ? full : last;
        const int j = round - g * full.rounds, w = j / q.each, x = w < q.windows - 1 ? w : q.windows - 1;
        const int wide = x == q.windows - 1 ? q.last_window : q.window, each = x == q.windows - 1 ? q.last_each : q.each;
        const int i = pair * each + (j - x * q.each), row = i / wide;
        m = size * g + row;
        n = x * q.window + i % wide;
        part = x * q.slots + pair - row * wide / each;
        return i < q.rows * wide;
    }
    // The group that a row tile belongs to.
    GDN_BOTH const Group &of(int m) const { return m < size * groups ? full : last; }
    // Whether a row tile has this part.
    GDN_BOTH bool has(int m, int part) const
    {
        const Group &q = of(m);
        const int row = m < size * groups ? m % size : m - size * groups, x = part / q.slots;
        const int wide = x == q.windows - 1 ? q.last_window : q.window, each = x == q.windows - 1 ? q.last_each : q.each;
        return (row * wide / each + part % q.slots) * each < (row + 1) * wide;
    }
    // Where a row's part 0 lies among the N rows' parts, and how far apart its parts are.
    GDN_BOTH int64_t first(int row) const { return row < split ? row : (int64_t)full.parts * split + (row - split); }
    GDN_BOTH int64_t step(int row, int N) const { return row < split ? split : N - split; }
};

}  // namespace gdn
