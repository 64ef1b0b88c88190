// Products of a compressed matrix into slots of partial sums, and what the
// kernel that adds the slots needs to find them.
//
// A stream's super-groups (kPartialGroups consecutive groups, one per group
// slot of a workgroup) are split into contiguous ranges, one per workgroup.
// Workgroup w's group slot h holds wg_panels slots, one for each 64-row panel
// from the first to the last that w's range touches, at float
//     base + ((w * kPartialGroups + h) * wg_panels + panel - first) * 64 n_tokens
// A slot is n_tokens x 64 floats.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11.h"

namespace df11 {

constexpr uint32_t kPartialGroups = 2;
// Most tokens of a product into slots: one sweep with two token tiles.  Four
// tiles leave the decoder half its waves, and decoding once and multiplying
// the tiles (df11_dense.h) is faster: 14336 -> 4096 at 33 tokens 69 against
// 154 us, 4096 -> 4096 36 against 56; at 32 tokens two tiles take 60 and 29.
constexpr uint32_t kPartialTokens = DF11_EPILOGUE_FUSED_TOKENS;

// g / d for a global k-step g < 2^21 (2^32 elements of 2048 each) and the d =
// C / 32 k-steps of a panel, d <= 2^21, with magic = floor(2^42 / d) + 1: the
// quotient's error g / 2^42 stays below 1 / d.
__host__ __device__ inline uint32_t panel_of_step(uint32_t g, uint64_t magic) {
    return static_cast<uint32_t>(g * magic >> 42);
}

struct PartialStream {
    const uint32_t *out_pos;
    uint64_t tile_magic;  // floor(2^42 / (C / 32)) + 1 (panel_of_step)
    uint64_t base;        // floats into the slots
    uint32_t n_elements, n_groups, n_super, n_wg, wg_panels;
};

struct Partials {
    PartialStream s[2];
    uint64_t slot_bytes;
    uint32_t max_group[2];
};

int check_stream(const df11_device_stream *s);
bool stream_overlaps(const df11_device_stream *s, const void *p, uint64_t bytes);
bool same_table_bits(const df11_device_stream *a, const df11_device_stream *b);

// x W_i^T of n (1 or 2) checked, non-empty, tile-ordered streams of the same
// shape and table width into slots (capacity bytes; DF11_E_BUFFER_TOO_SMALL
// if they take more), for at most kPartialTokens tokens.  With slots null
// nothing is launched and p.slot_bytes says what they take on the current
// device.
int partial_products(const df11_device_stream *const *ws, uint32_t n, const uint16_t *x, uint64_t x_stride,
                     uint32_t n_tokens, float *slots, uint64_t capacity, hipStream_t stream, Partials &p);

}  // namespace df11
