// Index arithmetic of the dense products' loads into LDS (df11_dense.hip).
// Plain constexpr C++ (no HIP), so that the gfx950 kernel calls it and a CPU
// test builds it on its own and checks it against the operands' definition.
//
// A load reads 16 bytes a lane through a buffer resource, a window of the
// operand.  What the hardware compares with the window's size is the lane's
// own offset; whether the scalar offset counts too is told differently in
// different places, and the scalar offset is zero here.  So the window begins
// at the step's first byte, ends with the operand, and all that differs
// between a tile's rows, panels and blocks is in the lane's offset: what lies
// past the operand's end is past the window's end, and is not read.
#ifndef DF11_DENSE_TILES_H
#define DF11_DENSE_TILES_H

#include <stdint.h>

namespace df11 {

constexpr uint32_t kDenseStep = 64;  // K elements of one step

// Bytes of an operand that a step's loads may reach: `bytes` from `at` on.
struct DenseWindow {
    uint64_t at, bytes;
};

// Left operand: the rows of a tile from m0 on, `rows` of them before the last
// token, k_len elements each, `stride` elements apart; from step ks on.
constexpr DenseWindow dense_left_window(uint32_t m0, uint32_t rows, uint64_t stride, uint32_t k_len, uint32_t ks) {
    return {2u * (m0 * stride + static_cast<uint64_t>(kDenseStep) * ks),
            2u * ((rows - 1u) * stride + k_len - static_cast<uint64_t>(kDenseStep) * ks)};
}

// Eight rows of 128 bytes a load: of the group-th eight, lane l takes row l / 8
// and, to spread an operand's rows over the LDS banks, chunk (l mod 8) ^ (l / 8).
constexpr uint32_t dense_left_lane(uint32_t lane, uint32_t stride) {
    return (lane >> 3) * stride * 2u + 16u * ((lane & 7u) ^ (lane >> 3));
}
constexpr uint32_t dense_left_group(uint32_t group, uint32_t stride) { return 16u * group * stride; }

// W forward: the panels (64 rows of W, panel_bytes each) from output n0's on,
// from step ks on (two k-steps of 4 KB).
constexpr DenseWindow dense_right_window(uint32_t n0, uint32_t ks, uint32_t panels, uint64_t panel_bytes) {
    const uint64_t at = (n0 / 64u) * panel_bytes + 8192ull * ks;
    return {at, panels * panel_bytes - at};
}

// The 1 KB block of rows 16 r16 .. + 15, counted from the window's panel, of
// the step's k-step `half`.
constexpr uint32_t dense_right_block(uint32_t r16, uint32_t half, uint32_t panel_bytes) {
    return (r16 / 4u) * panel_bytes + half * 4096u + (r16 & 3u) * 1024u;
}

// W backward: of panel ks, the k-steps from output n0's on, four 1 KB blocks
// each.
constexpr DenseWindow dense_back_window(uint32_t n0, uint32_t ks, uint64_t panel_bytes) {
    const uint64_t at = (n0 / 32u) * 4096ull;
    return {ks * panel_bytes + at, panel_bytes - at};
}
constexpr uint32_t dense_back_block(uint32_t b) { return 1024u * b; }

}  // namespace df11

#endif  // DF11_DENSE_TILES_H
