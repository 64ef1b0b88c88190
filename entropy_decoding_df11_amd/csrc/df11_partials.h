// Products of a compressed matrix into slots of partial sums, and what the
// kernel that adds the slots needs to find them.
//
// A stream's super-groups (kPartialGroups consecutive groups, one per group
// slot of a workgroup) are split into contiguous ranges, one per workgroup;
// up to 8 tokens, a long enough stream deals the last few percent of its
// groups out at run time instead.  Workgroup w's group slot h holds
// wg_panels slots, one for each 64-row panel from the first to the last that
// w's range touches, at float
//     base + ((w * kPartialGroups + h) * wg_panels + panel - first) * 64 n_tokens
// and group g of the dealt tail group_panels slots likewise at
//     tail + ((g - tail_group0) * group_panels + panel - first) * 64 n_tokens
// A slot is n_tokens x 64 floats.  Which workgroup took a dealt group does
// not show in the slots, so the sums do not depend on the schedule.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11.h"

namespace df11 {

constexpr uint32_t kPartialGroups = 2;
// Most tokens of one product into slots (one sweep of the stream).
constexpr uint32_t kPartialTokens = 64;

struct PartialStream {
    const uint32_t *out_pos;
    uint64_t tile_magic;  // panel of k-step i: umulhi64(i, tile_magic), or i itself with 0 (C = 32)
    uint64_t base, tail;  // floats into the slots
    uint32_t n_elements, n_groups, n_super, n_wg;
    uint32_t fixed_len;   // 0: ranges over all super-groups; else the length of each, the rest dealt
    uint32_t wg_panels, group_panels, tail_group0;
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
// shape and table width into slots, for at most kPartialTokens tokens.  With
// slots null nothing is launched and p.slot_bytes says what they take on the
// current device.
int partial_products(const df11_device_stream *const *ws, uint32_t n, const uint16_t *x, uint64_t x_stride,
                     uint32_t n_tokens, float *slots, hipStream_t stream, Partials &p);

}  // namespace df11
