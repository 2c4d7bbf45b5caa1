// How the attention kernels' work is cut, and how the SMs are shared out between the two parts of
// hs_latent_attend_shared.  Host code, without CUDA's headers.
#pragma once

#include <stdint.h>

#include "hs.h"

namespace hs_attn {

constexpr int kTile = 64;      // rows a tile of the own rows' kernels
constexpr int kMaxPairs = 76;  // pairs of SMs
constexpr int kMaxCtas = 2 * kMaxPairs;

// The own rows' kernels: a pair of SMs for up to 128 heads; and one SM for up to 32 heads and 8-bit
// rows, whose conversion, done twice by a pair, bounds them there (256 requests x 2048
// rows: 102 against 204 us with 16 heads, 128 against 206 with 32; a form for 48 heads took
// 262 where the pair takes 209, one for 16-bit rows 154 where it takes 140 with 16).
constexpr int kNarrowHeads = 32;

// Tiles' time that a unit's queries, first scores and output take.  Without it pieces of several short
// units end last: contexts of 32768, 1, 20001 and 777 rows 43 -> 34 us, 24 ragged ones of up to 16,384
// rows 56 -> 35, 90 requests x 2048 rows x 128 heads 91 -> 86 (4: 35, 38, 87; 12: 34, 35, 83, but 8-bit
// rows of 24 ragged contexts 43 -> 45).  On one SM: 24 ragged contexts of up to 16,384 rows 47 -> 35 us,
// 200 requests x 1000 rows x 32 heads 76 -> 72, 256 x 2048 x 16 102 (7: 34, 73, 105).
constexpr int kPairUnitCost = 7, kNarrowUnitCost = 3;
// Pieces also write and join up to two partial results a pair: about 10 us, 10 tiles' time; an SM: 8 us, 6 tiles'.
constexpr int kPairJoin = 10, kNarrowJoin = 6;
// The kernel over a shared prefix: tiles' time that a unit's queries and output take.  With the own rows' part first, 2
// instead of 4 cost 3 us (16 requests x 3 x 32 heads, 4096 rows: 42 against 39.5; 64 x 32 heads, 16,384 rows: 70 against
// 68), 7 changed nothing.
constexpr int kSharedUnitCost = 4;

// A unit is a request, a position and a block of heads; its rows come in tiles, one at
// least.  The tiles of all units form one line, which the workers (an SM, or a pair of
// SMs) cut into equal pieces (flat), or whole units go to each.  A unit's own time (its
// queries, its sums' way out) counts as `cost` tiles before its first one, but for the
// line's first unit: every piece has that once.  A cut inside it is a cut at the unit's
// start, so a worker may get no piece; the one before a piece that starts inside a unit
// always has one.
struct Cut {
    int flat;
    int units;         // at most HS_MAX_BATCH x HS_MAX_POSITIONS x HS_MAX_HEADS / 128, below 2^31
    int unit_tiles;    // tiles of a unit; with lengths, the most that one has
    int workers;
    int cost;
    int64_t share;     // slots: tiles (and cost) a worker, and how many workers have one more
    int extra;
    int unit_share, unit_extra;  // units a worker, likewise

    static int64_t tiles_of(int64_t rows, int tile) { return rows <= tile ? 1 : (rows + tile - 1) / tile; }
    // Pieces, where those are `join` tiles' time shorter than whole units.
    static bool in_pieces(int64_t units, int64_t tiles, int64_t workers, int join)
    {
        return (units + workers - 1) / workers * tiles > (units * tiles + workers - 1) / workers + join;
    }
    // Fill in the cut.
    void cut(int most, int64_t rows, int join, int unit_cost, int tile = kTile)
    {
        cost = unit_cost;
        unit_tiles = (int)tiles_of(rows, tile);
        const int64_t total = (int64_t)units * unit_tiles;
        workers = (int)(total < most ? total : most);
        flat = in_pieces(units, unit_tiles, workers, join);
        if (!flat && workers > units) workers = units;
        const int64_t line = (int64_t)units * (unit_tiles + cost) - cost;
        share = line / workers;
        extra = (int)(line % workers);
        unit_share = units / workers;
        unit_extra = units % workers;
    }
};

// Pairs of SMs for the own rows' part of hs_latent_attend_shared: all, so that the prefix's kernel follows it, or some,
// beside which that runs.  units, tiles: the prefix's, `ragged` with lengths.
// By an estimate in ns, fitted to both kernels' times over 1 to 128 heads, 1 to 32 tiles a unit and 6 to 60 pairs; 5 %
// less are asked for.  (64 requests x 16 heads, 16,384 shared rows, 1 to 512 own: 50.9 us one after the other, 44.7 with
// 26 pairs, 54.9 with 18, 56.6 with 44; 128 x 8 heads, 1000 shared rows, 64 own: 31.4, and 25.5 with 52; but 64 x 128
// heads, 16,384 shared 8-bit rows, 256 own: 206.3, and 207.3 with 6, 242 with 18; 64 x 16 heads, 2048 shared rows, 1 to
// 512 own: 31.9, and 33.4 with the 32 that the estimate takes.)  Contexts of more than 512 rows may be far shorter than
// that, so they are taken one after the other.
// Some pairs take whole units only: the join of units in pieces would stand between the own rows' kernel and the
// prefix's, which then begins behind both, on a part of the SMs.  And all pairs take pieces where those are shorter, so
// that few requests with long lists leave them all to the own rows first.  (Lists of 2048 entries: 5 requests x 3 x 20
// heads, 3001 8-bit rows 60 us, and 79 with 8 pairs in whole units; 1 x 128 heads, likewise, 51, and 75 with one; but
// 8 x 128 heads, 16,384 16-bit rows 71, and 55 with 8.  Over 120 cases of 1 to 256 requests, 2 to 32 tiles and both
// forms the choice was within 11 % of the best of 20 numbers of pairs, and 2 % off it at the mean.)
inline int pairs_beside(const hs_attend_t& a, bool ragged, int units, int tiles, int all)
{
    const int64_t own_tiles = Cut::tiles_of(a.slots ? a.entries : a.n_rows, kTile);
    if (!a.slots && own_tiles > 8) return all;
    const bool e4m3 = a.row_format == HS_ROWS_E4M3, narrow = e4m3 && a.heads <= kNarrowHeads;  // narrow: an SM a unit
    const int heads = a.heads < 128 ? a.heads : 128;
    const int64_t own_units = (int64_t)a.batch * a.positions * ((a.heads + 127) / 128);
    const int64_t own_begin = narrow ? 1200 + 200 * heads : 4200 + 30 * heads, own_tile = narrow ? 1350 : e4m3 ? 1700 : 1050;
    const int own_cost = narrow ? kNarrowUnitCost : kPairUnitCost, join = narrow ? kNarrowJoin : kPairJoin, join_time = narrow ? 8000 : 10000;
    const int64_t unit = (ragged ? (3 * (int64_t)tiles + 3) / 4 : tiles) + kSharedUnitCost;
    auto own_workers = [&](int64_t n) {
        const int64_t most = narrow ? 2 * n : n, total = own_units * own_tiles;
        return total < most ? total : most;
    };
    auto own_whole = [&](int64_t workers) { return 7000 + (own_units + workers - 1) / workers * (own_begin + own_tile * own_tiles); };
    auto prefix = [&](int64_t n) {
        const int64_t whole = (units + n - 1) / n * unit, pieces = (units * unit + n - 1) / n + 2;
        return 13000 + (e4m3 ? 1600 : 1450) * (whole < pieces ? whole : pieces);
    };
    const int64_t every = own_workers(all);
    const int64_t own_all = Cut::in_pieces(own_units, own_tiles, every, join)
                                ? 7000 + own_begin + ((own_units * (own_tiles + own_cost) - own_cost) / every + 1) * own_tile + join_time
                                : own_whole(every);
    int best = all;
    int64_t time = (own_all + prefix(all) - 2000) * 95 / 100 * 17;
    for (int n = 1; n < all; ++n) {
        const int64_t workers = own_workers(n);
        if (Cut::in_pieces(own_units, own_tiles, workers, join)) continue;
        const int64_t x = own_whole(workers), y = prefix(all - n), t = 16 * (x > y ? x : y) + (x < y ? x : y);  // the longer of both counts
        if (t < time) time = t, best = n;
    }
    return best;
}

}  // namespace hs_attn
