// The work plan of the attention over a paged cache (csrc/df11_attention_plan.h)
// for tests/test_attention_plan.py.
//   "P place page_size"            -> place / page_size by the kernels' multiplication
//   "R units workgroups"           -> "runs", then "begin" of every run and of the end
//   "W unit units workgroups"      -> the run of a unit
//   "X runs"                       -> the run of every workgroup
//   "S begin end length n_tokens capacity group tile_rows step kv_heads masked extra"
//                                  -> "tokens rows length places tiles units", then of every tile the places that all
//                                     of it sees, that some of it may see, its units, the units before it, and its number by its first and last unit
#include <stdint.h>
#include <stdio.h>

#include "df11_attention_plan.h"

int main() {
    char kind;
    while (scanf(" %c", &kind) == 1) {
        long long v[11];
        const int n = kind == 'S' ? 11 : kind == 'W' ? 3 : kind == 'X' ? 1 : 2;
        for (int i = 0; i < n; ++i)
            if (scanf("%lld", &v[i]) != 1) return 1;
        if (kind == 'P') {
            const uint32_t s = df11::page_shift(static_cast<uint32_t>(v[1]));
            printf("%u\n", df11::page_of(static_cast<uint32_t>(v[0]), df11::page_magic(static_cast<uint32_t>(v[1]), s), s));
        } else if (kind == 'R') {
            const uint32_t units = static_cast<uint32_t>(v[0]), runs = df11::runs_of(units, static_cast<uint32_t>(v[1]));
            printf("%u", runs);
            for (uint32_t w = 0; w <= runs; ++w) printf(" %u", df11::run_begin(w, units, runs));
            printf("\n");
        } else if (kind == 'W') {
            const uint32_t units = static_cast<uint32_t>(v[1]);
            printf("%u\n", df11::run_of(static_cast<uint32_t>(v[0]), units, df11::runs_of(units, static_cast<uint32_t>(v[2]))));
        } else if (kind == 'X') {
            for (uint32_t i = 0; i < static_cast<uint32_t>(v[0]); ++i)
                printf("%u ", df11::run_of_workgroup(i, static_cast<uint32_t>(v[0])));
            printf("\n");
        } else if (kind == 'S') {
            const auto u = [&](int i) { return static_cast<uint32_t>(v[i]); };
            const df11::SeqShape s = df11::seq_shape(static_cast<int32_t>(v[0]), static_cast<int32_t>(v[1]),
                                                     static_cast<int32_t>(v[2]), u(3), static_cast<uint64_t>(v[4]), u(5),
                                                     u(6), u(7), u(10), v[9] != 0);
            printf("%u %u %u %u %u %llu", s.tokens, s.rows, s.length, s.places, s.tiles,
                   static_cast<unsigned long long>(df11::seq_units(s, u(8))));
            for (uint32_t t = 0; t < s.tiles; ++t) {
                const uint32_t before = static_cast<uint32_t>(df11::units_before(s, t));
                printf(" %u %u %u %u %u %u", df11::tile_plain(s, t, u(6), u(5), v[9] != 0), df11::tile_places(s, t, u(6), u(5), v[9] != 0), df11::tile_units(s, t),
                       before, df11::tile_of(s, before),
                       df11::tile_of(s, before + df11::tile_units(s, t) - 1));
            }
            printf("\n");
        } else {
            return 1;
        }
    }
    return 0;
}
