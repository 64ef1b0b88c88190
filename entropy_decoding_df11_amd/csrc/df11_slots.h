// Sums of a panel's slots (df11_partials.h): what the kernels that end a product
// of few tokens begin with.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11_device.h"
#include "df11_partials.h"

namespace {

constexpr uint32_t kPanelRows = 64;  // output features of one panel

// Panel of element e of a tile-ordered stream.
__device__ __forceinline__ uint32_t panel_of(const df11::PartialStream &s, uint32_t e) {
    return df11::panel_of_step(min(e, s.n_elements - 1u) >> 11, s.tile_magic);
}

__device__ __forceinline__ uint32_t out_pos_of(const df11::PartialStream &s, uint32_t g) {
    return s.out_pos[min(g, s.n_groups)];
}

// First super-group of workgroup w's range: floor(w n_super / n_wg), as
// w * (n_super / n_wg) + floor(w * (n_super % n_wg) / n_wg) in 32 bits
// (n_wg is a grid size, far below 2^16).
__device__ __forceinline__ uint32_t range_begin(const df11::PartialStream &s, uint32_t w) {
    return w * (s.n_super / s.n_wg) + w * (s.n_super % s.n_wg) / s.n_wg;
}

// The workgroups [lo, hi) whose ranges touch a panel, and the panels that
// the first of them holds before it.  Ranges follow the stream, so those of
// a panel are consecutive, and every one but the first begins with it.
struct Found {
    uint32_t lo, hi, skip;
};

// Finds them with all threads at once: a search would wait for one load
// after the other.
__device__ __forceinline__ void find_ranges(const df11::PartialStream &s, uint32_t p, Found *f) {
    for (uint32_t w = threadIdx.x; w < s.n_wg; w += blockDim.x) {
        const uint32_t a = panel_of(s, out_pos_of(s, range_begin(s, w) * df11::kPartialGroups));
        const uint32_t b = panel_of(s, max(out_pos_of(s, range_begin(s, w + 1u) * df11::kPartialGroups), 1u) - 1u);
        if (a <= p && p <= b) {
            atomicMin(&f->lo, w);
            atomicMax(&f->hi, w + 1u);
            atomicMax(&f->skip, p - a);
        }
    }
}

// Adds the slots of panel p for up to TOKENS tokens from t0 on, by a workgroup
// of four waves: a lane per output feature, the slots split between the waves,
// whose sums are left in s_sum, to be added in wave order.  A wave takes
// several slots at once, so that more loads than one slot's are in flight.
template <int kStreams, int TOKENS>
__device__ __forceinline__ void panel_sums(const df11::PartialStream *streams, const float *all, uint32_t n_tokens,
                                           uint32_t p, uint32_t t0, uint32_t tokens, Found *s_found,
                                           float (*s_sum)[4][TOKENS][kWaveSize]) {
    constexpr int kAtOnce = TOKENS >= 4 ? 4 : 8;  // slots
    constexpr uint32_t kPartialGroups = df11::kPartialGroups;
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint64_t slot = static_cast<uint64_t>(kPanelRows) * n_tokens;
    if (threadIdx.x < kStreams) s_found[threadIdx.x] = Found{~0u, 0u, 0u};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStreams; ++i) find_ranges(streams[i], p, &s_found[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
        const df11::PartialStream &s = streams[i];
        const Found f = s_found[i];
        const uint32_t n = f.lo < f.hi ? (f.hi - f.lo) * kPartialGroups : 0u, each = (n + 3u) / 4u;
        const uint32_t begin = wave * each, end = min(n, begin + each);
        const uint32_t skip = min(f.skip, s.wg_panels - 1u);
        // Float offset of the c-th group slot's slot.
        auto at = [&](uint32_t c) {
            return s.base + (static_cast<uint64_t>(f.lo * kPartialGroups + c) * s.wg_panels +
                             (c < kPartialGroups ? skip : 0u)) * slot;
        };
        float sum[TOKENS];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) sum[t] = 0.0f;
        const float *slots = all + static_cast<uint64_t>(t0) * kPanelRows + lane;
        for (uint32_t c = begin; c < end; c += kAtOnce) {
            // (past the end the last slot again, not added; past the last
            // token the first one, not written)
            float v[kAtOnce][TOKENS];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float *q = slots + at(min(c + k, end - 1u));
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) v[k][t] = q[t < static_cast<int>(tokens) ? t * kPanelRows : 0u];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (c + k < end)
#pragma unroll
                    for (int t = 0; t < TOKENS; ++t) sum[t] += v[k][t];
        }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) s_sum[i][wave][t][lane] = sum[t];
    }
    __syncthreads();
}

}  // namespace
