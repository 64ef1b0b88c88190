// The work plan of the attention over a paged cache (csrc/df11_attention_plan.h)
// for tests/test_attention_plan.py.
//   "P place page_size"            -> place / page_size by the kernels' multiplication
//   "R units workgroups"           -> "runs", then "begin" of every run and of the end
//   "W unit units workgroups"      -> the run of a unit
//   "X runs"                       -> the run of every workgroup
//   "T tiles masked"               -> "tile turn" for every place in the order of work
//   "S begin end length n_tokens capacity group tile_rows kv_heads masked"
//                                  -> "tokens rows length places tiles steps units", then the places of every tile
#include <stdint.h>
#include <stdio.h>

#include "df11_attention_plan.h"

int main() {
    char kind;
    while (scanf(" %c", &kind) == 1) {
        long long v[9];
        const int n = kind == 'S' ? 9 : kind == 'W' ? 3 : kind == 'X' ? 1 : 2;
        for (int i = 0; i < n; ++i)
            if (scanf("%lld", &v[i]) != 1) return 1;
        if (kind == 'P') {
            const uint32_t s = df11::page_shift(static_cast<uint32_t>(v[1]));
            printf("%u\n", df11::page_of(static_cast<uint32_t>(v[0]), df11::page_magic(static_cast<uint32_t>(v[1]), s), s));
        } else if (kind == 'R') {
            const uint64_t units = static_cast<uint64_t>(v[0]);
            const uint32_t runs = df11::runs_of(units, static_cast<uint32_t>(v[1]));
            printf("%u", runs);
            for (uint32_t w = 0; w <= runs; ++w) printf(" %llu", static_cast<unsigned long long>(df11::run_begin(w, units, runs)));
            printf("\n");
        } else if (kind == 'W') {
            const uint64_t units = static_cast<uint64_t>(v[1]);
            printf("%u\n", df11::run_of(static_cast<uint64_t>(v[0]), units, df11::runs_of(units, static_cast<uint32_t>(v[2]))));
        } else if (kind == 'X') {
            for (uint32_t i = 0; i < static_cast<uint32_t>(v[0]); ++i)
                printf("%u ", df11::run_of_workgroup(i, static_cast<uint32_t>(v[0])));
            printf("\n");
        } else if (kind == 'T') {
            for (uint32_t t = 0; t < static_cast<uint32_t>(v[0]); ++t) {
                const uint32_t tile = df11::tile_in_turn(t, static_cast<uint32_t>(v[0]), v[1] != 0);
                printf("%u %u ", tile, df11::turn_of_tile(tile, static_cast<uint32_t>(v[0]), v[1] != 0));
            }
            printf("\n");
        } else if (kind == 'S') {
            const df11::SeqShape s = df11::seq_shape(static_cast<int32_t>(v[0]), static_cast<int32_t>(v[1]),
                                                     static_cast<int32_t>(v[2]), static_cast<uint32_t>(v[3]),
                                                     static_cast<uint64_t>(v[4]), static_cast<uint32_t>(v[5]),
                                                     static_cast<uint32_t>(v[6]));
            printf("%u %u %u %u %u %u %llu", s.tokens, s.rows, s.length, s.places, s.tiles, s.steps,
                   static_cast<unsigned long long>(df11::seq_units(s, static_cast<uint32_t>(v[7]))));
            for (uint32_t t = 0; t < s.tiles; ++t)
                printf(" %u", df11::tile_places(s, t, static_cast<uint32_t>(v[6]), static_cast<uint32_t>(v[5]), v[8] != 0));
            printf("\n");
        } else {
            return 1;
        }
    }
    return 0;
}
