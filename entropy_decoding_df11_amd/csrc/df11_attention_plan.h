// How the attention over a paged cache is cut into work (df11_attention.hip).
// Plain constexpr C++ (no HIP), so that the gfx950 kernels call it and a CPU
// test builds it on its own.
//
// A unit is one tile of a sequence's query rows (row = token * group + head
// within the group of query heads that share a key head) against one step of
// places.  Sequence by sequence, key head by key head, tile by tile,
// step by step the units are numbered, and the workgroups take equal runs of
// them, whatever the lengths are: a run may begin and end inside a tile, whose
// parts the second kernel joins.  With a mask every tile has all of a sequence's
// steps; without one the later tiles see more, and a tile's steps are a bound
// whose sums have a closed form: at most one step too many, and for a sequence's last
// tile, which may not be full, as many more as a full one has of its own.  (With the
// tiles that add a step rounded down to whole ones, groups of 3 counted 7021 steps for
// 4720 in 10000 tokens: 4000 after 4000, three to a key head, 402 us against 355; 8000
// after 100, five to a key head, 294 against 257.)  A tile counts some units more,
// before its steps, for what it takes beside them (its queries, the first loads that
// nothing hides, the end of its sums): a run that has only those leaves the tile to
// the next one.
#ifndef DF11_ATTENTION_PLAN_H
#define DF11_ATTENTION_PLAN_H

#include <stdint.h>

namespace df11 {

// (A step is a block of 32 places for each wave of a workgroup that has few rows,
// and short enough to be cut evenly for many.)
constexpr uint32_t kFewStep = 256, kManyStep = 128;

// Places of a sequence's pages up to which tiles are never cut: then a unit is a
// whole tile, and no second kernel joins parts.  It is the number of tiles, which fill
// the chip or not, that decides: 64 sequences of one token over 960 places 61.0 us
// whole and 64.2 cut, 16 trees of 16 tokens 27.6 and 31.3 at 960, 45.9 and 41.4 at 1500; a
// tree of 32 of one sequence 28.5 and 22.3 at 500.  Few tiles of few rows, by the time
// that a place takes: one token of one sequence in a graph (from Python whole saves
// about half a microsecond more), heads of 128 whole 13.8 us and cut 15.3 at 608 places,
// 15.4 and 15.4 at 736, 15.7 and 15.7 at 800, 16.4 and 15.7 at 864; of 64 12.4 and 13.8 at
// 1024; of 256 15.5 and 17.9 at 320, 18.7 and 18.7 at 480, 20.4 and 18.5 at 544.
constexpr uint32_t kMostWhole = 1024, kManyWhole = 128;
constexpr uint32_t few_whole(uint32_t dim) { return dim > 128u ? 448u : dim > 64u ? 768u : kMostWhole; }
constexpr uint32_t whole_places(bool few, uint64_t tiles, uint32_t workgroups, uint32_t dim) {
    return tiles >= workgroups ? kMostWhole : few ? few_whole(dim) : kManyWhole;
}

// Places of a unit, for pages of `capacity` places of which `whole` are never cut.
constexpr uint32_t unit_places(uint64_t capacity, bool few, uint32_t whole) {
    return capacity <= whole ? whole : few ? kFewStep : kManyStep;
}

// A sequence as the kernels see it, after the checks of what the device holds.
struct SeqShape {
    int32_t begin;    // its first token
    uint32_t tokens;  // new tokens, 0: nothing to compute
    uint32_t rows;    // of them, those that the call's arrays have
    uint32_t length;  // places cached before them
    uint32_t places;  // places in its pages, length + tokens at most
    uint32_t tiles;
    uint32_t first;   // steps of a tile before what the tiles add
    uint32_t each;    // tiles that add `more` steps together: up to tile t
    uint32_t more;    // (t + 1) more / each, rounded up; 0: none
    uint32_t extra;   // units of a tile before its steps
};

// (tile_rows is a power of two.)
constexpr SeqShape seq_shape(int32_t begin, int32_t end, int32_t length, uint32_t n_tokens, uint64_t capacity,
                             uint32_t group, uint32_t tile_rows, uint32_t step, uint32_t extra, bool masked) {
    SeqShape s{begin, 0, 0, 0, 0, 0, 0, 1, 0, extra};
    if (begin < 0 || end <= begin || length < 0 || static_cast<uint32_t>(begin) >= n_tokens) return s;
    const uint32_t last = static_cast<uint32_t>(end) < n_tokens ? static_cast<uint32_t>(end) : n_tokens;
    s.tokens = static_cast<uint32_t>(end - begin);
    s.rows = last - static_cast<uint32_t>(begin);
    s.length = static_cast<uint32_t>(length);
    const uint64_t all = static_cast<uint64_t>(s.length) + s.tokens;
    s.places = static_cast<uint32_t>(all < capacity ? all : capacity);
    s.tiles = static_cast<uint32_t>((static_cast<uint64_t>(s.rows) * group + tile_rows - 1) / tile_rows);
    if (masked || capacity <= step || s.tiles <= 1u || all > capacity) {
        // (all > capacity: tokens that have no place, which no closed form is worth)
        s.first = (s.places + step - 1) / step;
        if (!s.first) s.first = 1;  // (no pages: its rows are still written)
    } else {
        // Tile t ends with token (t + 1) tile_rows / group, rounded up, and has that
        // many places more than are held: so many over `step` steps, rounded up.
        const uint32_t tokens = step * group;  // rows of a step's tokens
        const uint32_t lowest = tokens & (0u - tokens), common = lowest < tile_rows ? lowest : tile_rows;
        s.first = (s.length + step - 1) / step;
        s.each = tokens / common;
        s.more = tile_rows / common;
    }
    return s;
}

// Units of the tiles before tile t of one key head, and of tile t.
constexpr uint64_t units_before(const SeqShape &s, uint32_t t) {
    const uint64_t all = static_cast<uint64_t>(t) * (s.first + s.extra);
    // Of each round of tiles' steps the i-th is one that all have from i each / more
    // on: 1 + 1 + .. (each times) + 2 + 2 + .. from there.
    uint64_t steps = 0;
    for (uint32_t i = 0; i < s.more; ++i) {
        const uint32_t skip = i ? i * s.each / s.more : 0u;
        if (t <= skip) break;
        const uint64_t whole = (t - skip) / s.each, rest = (t - skip) % s.each;
        steps += s.each * (whole * (whole + 1) / 2) + rest * (whole + 1);
    }
    return all + steps;
}
constexpr uint32_t tile_units(const SeqShape &s, uint32_t t) {
    return s.extra + s.first +
           (s.more ? static_cast<uint32_t>(((static_cast<uint64_t>(t) + 1) * s.more + s.each - 1) / s.each) : 0u);
}

// Steps of a tile before its unit i.
constexpr uint32_t steps_before(const SeqShape &s, uint32_t i) { return i > s.extra ? i - s.extra : 0u; }

// The tile of unit u < units_before(tiles) of a key head.
constexpr uint32_t tile_of(const SeqShape &s, uint32_t u) {
    if (!s.more) return u / (s.first + s.extra);
    uint32_t lo = 0, hi = s.tiles;  // the last tile that begins at u or before is in [lo, hi)
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (units_before(s, mid) <= u) {
            lo = mid;
        } else {
            hi = mid;
        }
    }
    return lo;
}

constexpr uint64_t seq_units(const SeqShape &s, uint32_t kv_heads) {
    return s.tiles ? kv_heads * units_before(s, s.tiles) : 0;
}

// Units that a tile counts beside its steps, measured: a tile of many rows takes 12
// us and a step of it 5.5 (2.5 for heads up to 64, 10 beyond 128), one of few rows 8
// and 6.5.  (A batch of 24 trees over up to 4096 places, some over a few dozen: 50
// us without them, when a workgroup had several short tiles.)
constexpr uint32_t extra_units(uint64_t capacity, bool few, uint32_t whole, uint32_t dim) {
    return capacity <= whole ? 0u : few || dim > 128u ? 1u : dim > 64u ? 2u : 4u;
}

// The units of a call; more (of starts that decrease) are none at all.
constexpr uint64_t kMaxUnits = 1ull << 31;

// Workgroups that get a run: as many as there are units for.
constexpr uint32_t runs_of(uint32_t units, uint32_t workgroups) { return units < workgroups ? units : workgroups; }

// First unit of run w: the first units % runs of them have one unit more.  And the
// run of a unit.
constexpr uint32_t run_begin(uint32_t w, uint32_t units, uint32_t runs) {
    return w * (units / runs) + (w < units % runs ? w : units % runs);
}
constexpr uint32_t run_of(uint32_t u, uint32_t units, uint32_t runs) {
    const uint32_t each = units / runs, more = units % runs, longer = more * (each + 1u);
    return u < longer ? u / (each + 1u) : more + (u - longer) / each;
}

// The run of workgroup i: neighbouring runs, which share a sequence's places, on
// one XCD (workgroup i runs on XCD i mod 8).
constexpr uint32_t run_of_workgroup(uint32_t i, uint32_t runs) {
    const uint32_t xcd = i % 8u, each = runs / 8u, rest = runs % 8u;
    return xcd * each + (xcd < rest ? xcd : rest) + i / 8u;
}

// place / page_size for places below 2^31 and pages up to 2^20: with 2^s the
// power of two from page_size on, magic = floor(2^(31 + s) / page_size) + 1 is
// off by at most 1, and place / 2^(31 + s) stays below 1 / page_size.
constexpr uint32_t page_shift(uint32_t page_size) {
    uint32_t s = 0;
    while ((1u << s) < page_size) ++s;
    return s;
}
constexpr uint32_t page_magic(uint32_t page_size, uint32_t shift) {
    return static_cast<uint32_t>((1ull << (31u + shift)) / page_size + 1u);
}
constexpr uint32_t page_of(uint32_t place, uint32_t magic, uint32_t shift) {
    return static_cast<uint32_t>((static_cast<uint64_t>(place) * magic) >> (31u + shift));
}

// Places that every row of a tile sees, as far as they exist.
constexpr uint32_t tile_plain(const SeqShape &s, uint32_t tile, uint32_t tile_rows, uint32_t group, bool masked) {
    const uint64_t sees = masked ? s.length : s.length + static_cast<uint64_t>(tile) * tile_rows / group + 1;
    return static_cast<uint32_t>(sees < s.places ? sees : s.places);
}

// Places that some row of a tile may see.
constexpr uint32_t tile_places(const SeqShape &s, uint32_t tile, uint32_t tile_rows, uint32_t group, bool masked) {
    if (masked) return s.places;
    const uint64_t last_row = (static_cast<uint64_t>(tile) + 1) * tile_rows - 1;
    const uint64_t last = last_row / group < s.rows ? last_row / group : s.rows - 1;
    const uint64_t sees = s.length + last + 1;
    return static_cast<uint32_t>(sees < s.places ? sees : s.places);
}

}  // namespace df11

#endif  // DF11_ATTENTION_PLAN_H
