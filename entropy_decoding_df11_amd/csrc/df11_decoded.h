// Compressed weights decoded whole into a call's workspace, for products of more
// tokens than one sweep of the fused product takes, and for gradients.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11.h"
#include "df11_device.h"

namespace {

// Work counters of a decode.  Those of a weight are left alone: nothing orders
// this call after launches of the same weight by other threads, or a graph's
// replays after anything.  Two streams of kCounted weights or more decode by
// the dynamic schedule with counters of the workspace, zeroed first; shorter
// ones, and one alone, by the static schedule.  Gate and up of 64 tokens,
// counters against static: 14336 x 4096 each 131 against 136 us, 8192 x 4096
// 85 against 83, 4096 x 4096 56.0 against 54.4.
constexpr uint64_t kCounted = 3ull << 24;
constexpr uint32_t kCounterWords = 2 * DF11_SCHEDULE_WORDS;

[[maybe_unused]] __global__ void df11_zero_counters_kernel(uint32_t *p) {
    for (uint32_t i = threadIdx.x; i < kCounterWords; i += blockDim.x) p[i] = 0;
}

// Whether there are two different streams.  (Streams may share a buffer: those
// of a matrix and of its negative have the same exponents.)
[[maybe_unused]] bool two_streams(const df11_device_stream *const *ws, uint32_t n) {
    return n == 2 && (ws[1]->enc != ws[0]->enc || ws[1]->sm != ws[0]->sm);
}

// Bytes of the decoded weights (one copy of a stream given twice) and of the
// counters of their decode.
[[maybe_unused]] uint64_t decoded_bytes(const df11_device_stream *const *ws, uint32_t n) {
    const uint64_t one = round_up(2 * ws[0]->h.n_elements, 256);
    if (!two_streams(ws, n)) return one;
    return 2 * one + (ws[0]->h.n_elements >= kCounted ? round_up(4 * kCounterWords, 256) : 0);
}

// Decodes the streams into the workspace in tile order, as they are stored;
// out[i] receives where.
[[maybe_unused]] int decode_weights(const df11_device_stream *const *ws, uint32_t n, void *workspace, const uint16_t **out,
                   hipStream_t stream) {
    const uint64_t one = round_up(2 * ws[0]->h.n_elements, 256);
    df11_device_stream flat[2];
    uint16_t *to[2];
    const bool both = two_streams(ws, n);
    // (streams without counters of their own ask for the static schedule)
    const bool counted = both && ws[0]->h.n_elements >= kCounted && ws[0]->schedule && ws[1]->schedule;
    uint32_t *counters = counted ? reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + 2 * one) : nullptr;
    for (uint32_t i = 0; i < n; ++i) {
        flat[i] = *ws[i];
        flat[i].tile_cols = 0;
        flat[i].schedule = counted ? counters + i * DF11_SCHEDULE_WORDS : nullptr;
        to[i] = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) + (both ? i * one : 0));
        out[i] = to[i];
    }
    if (counted) {
        void *params[] = {&counters};
        const int rc = launch_kernel(reinterpret_cast<const void *>(&df11_zero_counters_kernel), dim3(1), dim3(256),
                                     params, 0, stream, nullptr, nullptr);
        if (rc) return rc;
    }
    if (both && flat[0].groups_per_workgroup == flat[1].groups_per_workgroup)
        return df11_decompress_batch(flat, 2, to, stream);
    int rc = df11_decompress(&flat[0], to[0], stream);
    if (!rc && both) rc = df11_decompress(&flat[1], to[1], stream);
    return rc;
}

}  // namespace
