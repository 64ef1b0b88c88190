// Prints what the dense products' loads (csrc/df11_dense_tiles.h, composed as
// df11_dense_kernel's `issue` composes them) read, for tests/test_dense_tiles.py.
//   "T mode edge tokens rows cols stride"   mode 0 plain, 1 gated, 2 backward;
//                                           edge 128 or 256; rows and cols of W
// -> for each tile and step, one line per 16 bytes that lie in the window,
//      "L tile step lds at"      left operand: byte in its LDS part, byte of x or dz
//      "R tile step lds at m"    W (m: which of a gated product's two)
//    "P ..." for a lane's 16 bytes that lie partly in a window, then "E".
// "O lane group stride" / "B r16 half panel_bytes"  ->  an offset.
#include <algorithm>

#include <stdint.h>
#include <stdio.h>

#include "df11_dense_tiles.h"

static void show(char kind, unsigned tile, unsigned step, unsigned lds, df11::DenseWindow w, uint32_t offset, int m) {
    if (offset >= w.bytes) return;
    if (offset + 16ull > w.bytes) kind = 'P';
    printf("%c %u %u %u %llu %d\n", kind, tile, step, lds, static_cast<unsigned long long>(w.at + offset), m);
}

static void tiles(unsigned mode, unsigned edge, unsigned tokens, unsigned rows, unsigned cols, unsigned stride) {
    const unsigned TN = 4;  // output blocks of a wave
    const unsigned outs = mode == 1 ? edge / 2 : edge, n_out = mode == 2 ? cols : rows;
    const unsigned n_tiles = (n_out + outs - 1) / outs, m_tiles = (tokens + edge - 1) / edge;
    const unsigned steps = mode == 2 ? rows / 64 : (cols + 63) / 64, k_len = mode == 2 ? rows : cols;
    const uint64_t panel_bytes = cols / 32 * 4096ull;
    static_assert(df11::kDenseStep == 64, "steps of 64");
    for (unsigned t = 0; t < m_tiles * n_tiles; ++t) {
        const unsigned m0 = t / n_tiles * edge, n0 = t % n_tiles * outs;
        const unsigned here = std::min(edge, tokens - m0);
        for (unsigned ks = 0; ks < steps; ++ks)
            for (unsigned g = 0; g < edge / 8; ++g)
                for (unsigned lane = 0; lane < 64; ++lane) {
                    const unsigned lds = 1024 * g + 16 * lane;
                    show('L', t, ks, lds, df11::dense_left_window(m0, here, stride, k_len, ks),
                         df11::dense_left_lane(lane, stride) + df11::dense_left_group(g, stride), 0);
                    if (mode == 2) {
                        show('R', t, ks, lds, df11::dense_back_window(n0, ks, panel_bytes),
                             16 * lane + df11::dense_back_block(g), 0);
                        continue;
                    }
                    const unsigned half = g / (edge / 16), nb = g % (edge / 16);
                    const bool second = mode == 1 && nb % TN >= TN / 2;
                    const unsigned r16 =
                        mode == 1 ? (n0 & 63) / 16 + nb / TN * (TN / 2) + nb % (TN / 2) : nb;
                    show('R', t, ks, lds, df11::dense_right_window(n0, ks, rows / 64, panel_bytes),
                         16 * lane + df11::dense_right_block(r16, half, static_cast<uint32_t>(panel_bytes)), second);
                }
    }
    printf("E\n");
}

int main() {
    char kind;
    while (scanf(" %c", &kind) == 1) {
        unsigned v[6];
        if (kind == 'T') {
            for (unsigned &x : v)
                if (scanf("%u", &x) != 1) return 1;
            tiles(v[0], v[1], v[2], v[3], v[4], v[5]);
        } else {
            for (int i = 0; i < 3; ++i)
                if (scanf("%u", &v[i]) != 1) return 1;
            printf("%u\n", kind == 'O' ? df11::dense_left_lane(v[0], v[2]) + df11::dense_left_group(v[1], v[2])
                                       : df11::dense_right_block(v[0], v[1], v[2]));
        }
    }
    return 0;
}
