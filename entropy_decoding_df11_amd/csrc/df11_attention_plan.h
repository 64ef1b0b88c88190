// How the attention over a paged cache is cut into work (df11_attention.hip).
// Plain constexpr C++ (no HIP), so that the gfx950 kernels call it and a CPU
// test builds it on its own.
//
// A unit is one tile of a sequence's query rows (row = token * group + head
// within the group of query heads that share a key head) against one step of
// kStepPlaces places.  Sequence by sequence, key head by key head, tile by tile,
// step by step the units are numbered, and the workgroups take equal runs of
// them, whatever the lengths are: a run may begin and end inside a tile, whose
// parts the second kernel joins.
#ifndef DF11_ATTENTION_PLAN_H
#define DF11_ATTENTION_PLAN_H

#include <stdint.h>

namespace df11 {

constexpr uint32_t kStepPlaces = 128;

// A sequence as the kernels see it, after the checks of what the device holds.
struct SeqShape {
    int32_t begin;    // its first token
    uint32_t tokens;  // new tokens, 0: nothing to compute
    uint32_t rows;    // of them, those that the call's arrays have
    uint32_t length;  // places cached before them
    uint32_t places;  // places in its pages, length + tokens at most
    uint32_t tiles, steps;
};

constexpr SeqShape seq_shape(int32_t begin, int32_t end, int32_t length, uint32_t n_tokens, uint64_t capacity,
                             uint32_t group, uint32_t tile_rows) {
    SeqShape s{begin, 0, 0, 0, 0, 0, 0};
    if (begin < 0 || end <= begin || length < 0 || static_cast<uint32_t>(begin) >= n_tokens) return s;
    const uint32_t last = static_cast<uint32_t>(end) < n_tokens ? static_cast<uint32_t>(end) : n_tokens;
    s.tokens = static_cast<uint32_t>(end - begin);
    s.rows = last - static_cast<uint32_t>(begin);
    s.length = static_cast<uint32_t>(length);
    const uint64_t all = static_cast<uint64_t>(s.length) + s.tokens;
    s.places = static_cast<uint32_t>(all < capacity ? all : capacity);
    s.tiles = static_cast<uint32_t>((static_cast<uint64_t>(s.rows) * group + tile_rows - 1) / tile_rows);
    s.steps = (s.places + kStepPlaces - 1) / kStepPlaces;
    if (!s.steps) s.steps = 1;  // (no pages: its rows are still written)
    return s;
}

constexpr uint64_t seq_units(const SeqShape &s, uint32_t kv_heads) {
    return static_cast<uint64_t>(kv_heads) * s.tiles * s.steps;
}

// Workgroups that get a run: as many as there are, but no fewer than kMinUnits
// units each.
constexpr uint64_t kMinUnits = 1;
constexpr uint32_t runs_of(uint64_t units, uint32_t workgroups) {
    const uint64_t most = units / kMinUnits;
    return most >= workgroups ? workgroups : most ? static_cast<uint32_t>(most) : 1u;
}

// First unit of run w, and the run of a unit u < units (units < 2^40).
constexpr uint64_t run_begin(uint64_t w, uint64_t units, uint32_t runs) { return w * units / runs; }
constexpr uint32_t run_of(uint64_t u, uint64_t units, uint32_t runs) {
    return static_cast<uint32_t>(((u + 1) * runs + units - 1) / units - 1);
}

// The run of workgroup i: neighbouring runs, which share a sequence's places, on
// one XCD (workgroup i runs on XCD i mod 8).
constexpr uint32_t run_of_workgroup(uint32_t i, uint32_t runs) {
    const uint32_t xcd = i % 8u, each = runs / 8u, rest = runs % 8u;
    return xcd * each + (xcd < rest ? xcd : rest) + i / 8u;
}

// Tile of the t-th place in the order of work: without a mask later tiles see
// more, so that light and heavy ones take turns.
constexpr uint32_t tile_in_turn(uint32_t t, uint32_t tiles, bool masked) {
    return masked ? t : t % 2u ? tiles - 1u - t / 2u : t / 2u;
}

constexpr uint32_t turn_of_tile(uint32_t tile, uint32_t tiles, bool masked) {
    return masked ? tile : tile < (tiles + 1u) / 2u ? 2u * tile : 2u * (tiles - 1u - tile) + 1u;
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
