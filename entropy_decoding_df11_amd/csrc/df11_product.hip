// Products of compressed weights with an epilogue (gfx950):
//
//   y = act(x W^T + bias) + residual                        df11_matmul_epilogue
//   y = act(x Wg^T + bias0) * (x Wu^T + bias1) + residual   df11_gated_matmul
//
// The weights are DF11 streams in MFMA tile order.  Up to kPartialTokens
// tokens at a time the decode is fused into the product
// (df11::partial_products): partial sums go to slots, and one kernel adds a
// panel's slots in the order of the stream, applies the epilogue and rounds
// once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include <stdint.h>

#include "df11.h"
#include "df11_device.h"
#include "df11_epilogue.h"
#include "df11_partials.h"

namespace {

using df11::kPartialGroups;
using df11::kPartialTokens;
using df11::Partials;
using df11::PartialStream;

constexpr uint32_t kPanelRows = 64;  // output features of one panel
constexpr int kSumTokens = 16;       // tokens of one workgroup of the slots' kernel

struct SumArgs {
    PartialStream s[2];
    const float *slots;
    Epilogue e;
    uint32_t n_tokens, features;
};

// Panel of element e of a tile-ordered stream.
__device__ __forceinline__ uint32_t panel_of(const PartialStream &s, uint32_t e) {
    const uint32_t step = min(e, s.n_elements - 1u) >> 11;
    return s.tile_magic ? static_cast<uint32_t>(__umul64hi(step, s.tile_magic)) : step;
}

__device__ __forceinline__ uint32_t out_pos_of(const PartialStream &s, uint32_t g) {
    return s.out_pos[min(g, s.n_groups)];
}

// First super-group of workgroup w's fixed range.
__device__ __forceinline__ uint32_t range_begin(const PartialStream &s, uint32_t w) {
    return s.fixed_len ? w * s.fixed_len
                       : static_cast<uint32_t>(static_cast<uint64_t>(w) * s.n_super / s.n_wg);
}

// Panels of the stream's regions that hold slots of panel p: ranges
// [wg_lo, wg_hi) and dealt groups [g_lo, g_hi), found by all threads at once
// (a search would wait for one load after the other).  Regions follow the
// stream, so those of a panel are consecutive.
struct Found {
    uint32_t wg_lo, wg_hi, g_lo, g_hi;
};

__device__ void find_regions(const PartialStream &s, uint32_t p, Found *f) {
    if (threadIdx.x == 0) *f = Found{~0u, 0u, ~0u, 0u};
    __syncthreads();
    for (uint32_t w = threadIdx.x; w < s.n_wg; w += blockDim.x) {
        const uint32_t a = panel_of(s, out_pos_of(s, range_begin(s, w) * kPartialGroups));
        const uint32_t b = panel_of(s, max(out_pos_of(s, range_begin(s, w + 1u) * kPartialGroups), 1u) - 1u);
        if (a <= p && p <= b) {
            atomicMin(&f->wg_lo, w);
            atomicMax(&f->wg_hi, w + 1u);
        }
    }
    for (uint32_t g = s.tail_group0 + threadIdx.x; g < s.n_groups; g += blockDim.x) {
        const uint32_t a = panel_of(s, out_pos_of(s, g)), b = panel_of(s, max(out_pos_of(s, g + 1u), 1u) - 1u);
        if (a <= p && p <= b) {
            atomicMin(&f->g_lo, g);
            atomicMax(&f->g_hi, g + 1u);
        }
    }
    __syncthreads();
}

// One workgroup adds the slots of one panel for up to kSumTokens tokens: a
// lane per output feature, the slots split between the four waves, whose
// sums meet in LDS in wave order.
template <bool kGated>
__global__ __launch_bounds__(256) void df11_sum_slots_kernel(SumArgs a) {
    __shared__ Found s_found[2];
    __shared__ float s_sum[2][4][kSumTokens][kWaveSize];
    const uint32_t p = blockIdx.x, t0 = blockIdx.y * kSumTokens;
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t tokens = min(static_cast<uint32_t>(kSumTokens), a.n_tokens - t0);
    const uint64_t slot = static_cast<uint64_t>(kPanelRows) * a.n_tokens;
    constexpr int kStreams = kGated ? 2 : 1;
    for (int i = 0; i < kStreams; ++i) find_regions(a.s[i], p, &s_found[i]);
    for (int i = 0; i < kStreams; ++i) {
        const PartialStream &s = a.s[i];
        const Found f = s_found[i];
        const uint32_t n_fixed = f.wg_lo < f.wg_hi ? (f.wg_hi - f.wg_lo) * kPartialGroups : 0u;
        const uint32_t n_dealt = f.g_lo < f.g_hi ? f.g_hi - f.g_lo : 0u;
        float sum[kSumTokens];
#pragma unroll
        for (int t = 0; t < kSumTokens; ++t) sum[t] = 0.0f;
        const uint32_t n = n_fixed + n_dealt, each = (n + 3u) / 4u;
        const uint32_t end = min(n, (wave + 1u) * each);
        for (uint32_t c = wave * each; c < end; ++c) {
            uint64_t at;
            if (c < n_fixed) {
                const uint32_t w = f.wg_lo + c / kPartialGroups, h = c % kPartialGroups;
                const uint32_t first = panel_of(s, out_pos_of(s, range_begin(s, w) * kPartialGroups));
                at = s.base + (static_cast<uint64_t>(w * kPartialGroups + h) * s.wg_panels +
                               min(p - first, s.wg_panels - 1u)) * slot;
            } else {
                const uint32_t g = f.g_lo + c - n_fixed;
                const uint32_t first = panel_of(s, out_pos_of(s, g));
                at = s.tail + (static_cast<uint64_t>(g - s.tail_group0) * s.group_panels +
                               min(p - first, s.group_panels - 1u)) * slot;
            }
            const float *q = a.slots + at + static_cast<uint64_t>(t0) * kPanelRows + lane;
#pragma unroll
            for (int t = 0; t < kSumTokens; ++t)
                if (t < static_cast<int>(tokens)) sum[t] += q[t * kPanelRows];
        }
#pragma unroll
        for (int t = 0; t < kSumTokens; ++t)
            if (t < static_cast<int>(tokens)) s_sum[i][wave][t][lane] = sum[t];
    }
    __syncthreads();
    for (uint32_t t = wave; t < tokens; t += 4u) {
        float z[2] = {};
        for (int i = 0; i < kStreams; ++i)
            z[i] = (s_sum[i][0][t][lane] + s_sum[i][1][t][lane]) + (s_sum[i][2][t][lane] + s_sum[i][3][t][lane]);
        finish<kGated>(a.e, t0 + t, kPanelRows * p + lane, a.features, z[0], z[1]);
    }
}

// ---------------------------------------------------------------------------
// Host.

// One call's checked arguments.
struct Call {
    const df11_device_stream *w[2];
    uint32_t n;  // streams: 1, or 2 for a gated product
    const uint16_t *x;
    uint64_t x_stride;
    uint32_t n_tokens, in_features, out_features;
    Epilogue e;
};

uint64_t rows_span(uint32_t rows, uint32_t cols, uint64_t stride, uint32_t bytes) {
    return rows && cols ? ((rows - 1ull) * stride + cols) * bytes : 0;
}

constexpr uint64_t kMaxStride = 1ull << 31;

// Checks of the streams and the sizes that every entry point shares.
int check_streams(const df11_device_stream *const *ws, uint32_t n, uint32_t n_tokens, uint32_t in_features,
                  uint32_t out_features) {
    for (uint32_t i = 0; i < n; ++i) {
        if (!ws[i]) return DF11_E_INVALID_ARG;
        const int rc = df11::check_stream(ws[i]);
        if (rc) return rc;
        if (in_features < 32 || in_features % 32 || out_features % kPanelRows ||
            static_cast<uint64_t>(in_features) * out_features != ws[i]->h.n_elements ||
            (ws[i]->h.n_elements && ws[i]->tile_cols != in_features))
            return DF11_E_INVALID_ARG;
    }
    if (n == 2 && out_features && !df11::same_table_bits(ws[0], ws[1])) return DF11_E_INVALID_ARG;
    if (static_cast<uint64_t>(n_tokens) * std::max(in_features, out_features) >= (1ull << 32)) return DF11_E_TOO_LARGE;
    return DF11_OK;
}

// Checks one forward call (no launch); *empty is set when there is nothing to compute.
int check_call(Call &c, const df11_epilogue *e, void *workspace, bool &empty) {
    int rc = check_streams(c.w, c.n, c.n_tokens, c.in_features, c.out_features);
    if (rc) return rc;
    if (!e || e->activation > DF11_ACT_GELU_TANH) return DF11_E_INVALID_ARG;
    const uint32_t out_bytes = e->out_dtype == DF11_FP16 ? 0 : dtype_bytes(e->out_dtype);
    const uint32_t res_bytes = e->residual_dtype == DF11_FP16 ? 0 : dtype_bytes(e->residual_dtype);
    const uint32_t bias_bytes = e->bias_dtype == DF11_FP16 ? 0 : dtype_bytes(e->bias_dtype);
    if (!out_bytes || (e->residual && !res_bytes) || ((e->bias[0] || e->bias[1]) && !bias_bytes))
        return DF11_E_INVALID_ARG;
    if (c.n == 1 && (e->bias[1] || e->pre[1])) return DF11_E_INVALID_ARG;
    if (c.n == 2 && !e->pre[0] != !e->pre[1]) return DF11_E_INVALID_ARG;
    empty = c.n_tokens == 0 || c.out_features == 0;
    if (empty) return DF11_OK;
    if (!c.x || !aligned(c.x, 16) || c.x_stride % 8 || c.x_stride > kMaxStride || !e->out ||
        !aligned(e->out, out_bytes) || e->out_stride > kMaxStride ||
        (c.n_tokens > 1 && e->out_stride < c.out_features))
        return DF11_E_INVALID_ARG;
    if (e->residual && (!aligned(e->residual, res_bytes) || e->residual_stride > kMaxStride)) return DF11_E_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        if ((e->bias[i] && !aligned(e->bias[i], bias_bytes)) || (e->pre[i] && !aligned(e->pre[i], 4)))
            return DF11_E_INVALID_ARG;
    // Every buffer written stays clear of everything else, but the output
    // may lie exactly on the residual (same address, stride and type).
    const uint64_t elems = static_cast<uint64_t>(c.n_tokens) * c.out_features;
    const void *outs[] = {e->out, e->pre[0], e->pre[1]};
    const uint64_t spans[] = {rows_span(c.n_tokens, c.out_features, e->out_stride, out_bytes),
                              e->pre[0] ? 4 * elems : 0, e->pre[1] ? 4 * elems : 0};
    const uint64_t res_span = e->residual ? rows_span(c.n_tokens, c.out_features, e->residual_stride, res_bytes) : 0;
    for (int i = 0; i < 3; ++i) {
        const bool on_residual = i == 0 && e->residual == e->out && e->residual_stride == e->out_stride &&
                                 e->residual_dtype == e->out_dtype;
        if (overlaps(outs[i], spans[i], c.x, rows_span(c.n_tokens, c.in_features, c.x_stride, 2)) ||
            (!on_residual && overlaps(outs[i], spans[i], e->residual, res_span)))
            return DF11_E_INVALID_ARG;
        for (int j = 0; j < 2; ++j)
            if (overlaps(outs[i], spans[i], e->bias[j], e->bias[j] ? static_cast<uint64_t>(bias_bytes) * c.out_features : 0))
                return DF11_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], spans[i], outs[j], spans[j])) return DF11_E_INVALID_ARG;
        for (uint32_t j = 0; j < c.n; ++j)
            if (df11::stream_overlaps(c.w[j], outs[i], spans[i])) return DF11_E_INVALID_ARG;
    }
    if (workspace && !aligned(workspace, 256)) return DF11_E_INVALID_ARG;
    c.e = Epilogue{{e->bias[0], e->bias[1]}, e->residual, e->out, {e->pre[0], e->pre[1]}, e->residual_stride,
                   e->out_stride, e->bias_dtype, e->residual_dtype, e->out_dtype, e->activation};
    return DF11_OK;
}

// The workspace stays clear of everything the call reads or writes.
bool workspace_clear(const Call &c, const void *ws, uint64_t bytes) {
    const uint64_t elems = static_cast<uint64_t>(c.n_tokens) * c.out_features;
    const Epilogue &e = c.e;
    bool bad = overlaps(ws, bytes, c.x, rows_span(c.n_tokens, c.in_features, c.x_stride, 2)) ||
               overlaps(ws, bytes, e.out, rows_span(c.n_tokens, c.out_features, e.out_stride, dtype_bytes(e.out_dtype))) ||
               overlaps(ws, bytes, e.residual, e.residual ? rows_span(c.n_tokens, c.out_features, e.residual_stride,
                                                                      dtype_bytes(e.residual_dtype)) : 0);
    for (int i = 0; i < 2; ++i)
        bad = bad || overlaps(ws, bytes, e.bias[i], e.bias[i] ? static_cast<uint64_t>(dtype_bytes(e.bias_dtype)) * c.out_features : 0) ||
              overlaps(ws, bytes, e.pre[i], e.pre[i] ? 4 * elems : 0);
    for (uint32_t i = 0; i < c.n; ++i) bad = bad || df11::stream_overlaps(c.w[i], ws, bytes);
    return !bad;
}

int slots_impl(const Call &c, uint32_t t0, uint32_t tokens, void *workspace, hipStream_t stream) {
    SumArgs a{};
    Partials p{};
    float *slots = static_cast<float *>(workspace);
    int rc = df11::partial_products(c.w, c.n, c.x + t0 * c.x_stride, c.x_stride, tokens, slots, stream, p);
    if (rc) return rc;
    a.s[0] = p.s[0];
    a.s[1] = p.s[1];
    a.slots = slots;
    a.e = c.e;
    const uint64_t done = static_cast<uint64_t>(t0) * c.out_features;
    a.e.out = static_cast<uint8_t *>(a.e.out) + t0 * a.e.out_stride * dtype_bytes(a.e.out_dtype);
    if (a.e.residual)
        a.e.residual = static_cast<const uint8_t *>(a.e.residual) +
                       t0 * a.e.residual_stride * dtype_bytes(a.e.residual_dtype);
    for (int i = 0; i < 2; ++i)
        if (a.e.pre[i]) a.e.pre[i] += done;
    a.n_tokens = tokens;
    a.features = c.out_features;
    void *params[] = {&a};
    return launch_kernel(c.n == 2 ? reinterpret_cast<const void *>(&df11_sum_slots_kernel<true>)
                                  : reinterpret_cast<const void *>(&df11_sum_slots_kernel<false>),
                         dim3(c.out_features / kPanelRows, (tokens + kSumTokens - 1) / kSumTokens), dim3(256), params,
                         0, stream, nullptr, nullptr);
}

uint64_t slots_bytes(const df11_device_stream *const *ws, uint32_t n, uint32_t n_tokens) {
    Partials p{};
    if (df11::partial_products(ws, n, nullptr, 0, std::min(n_tokens, kPartialTokens), nullptr, nullptr, p)) return 0;
    return p.slot_bytes;
}

uint64_t forward_workspace(const df11_device_stream *const *ws, uint32_t n, uint32_t n_tokens) {
    return slots_bytes(ws, n, n_tokens);
}

int forward(Call &c, const df11_epilogue *e, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    bool empty = false;
    int rc = check_call(c, e, workspace, empty);
    if (rc || empty) return rc;
    const uint64_t need = forward_workspace(c.w, c.n, c.n_tokens);
    if (!need) return DF11_E_HIP;
    if (!workspace) return DF11_E_INVALID_ARG;
    if (workspace_bytes < need) return DF11_E_BUFFER_TOO_SMALL;
    if (!workspace_clear(c, workspace, need)) return DF11_E_INVALID_ARG;
    for (uint32_t t0 = 0; t0 < c.n_tokens; t0 += kPartialTokens) {
        rc = slots_impl(c, t0, std::min(kPartialTokens, c.n_tokens - t0), workspace, stream);
        if (rc) return rc;
    }
    return DF11_OK;
}

}  // namespace

extern "C" {

uint64_t df11_epilogue_workspace(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens) {
    const df11_device_stream *ws[] = {w, up};
    const uint32_t n = up ? 2 : 1;
    if (!w || !n_tokens) return 0;
    for (uint32_t i = 0; i < n; ++i)
        if (df11::check_stream(ws[i]) || !ws[i]->h.n_elements || !ws[i]->tile_cols ||
            ws[i]->h.n_elements != w->h.n_elements || ws[i]->tile_cols != w->tile_cols)
            return 0;
    return forward_workspace(ws, n, n_tokens);
}

int df11_matmul_epilogue(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t n_tokens,
                         uint32_t in_features, uint32_t out_features, const df11_epilogue *e, void *workspace,
                         uint64_t workspace_bytes, void *hip_stream) {
    Call c{{w, nullptr}, 1, x, x_stride, n_tokens, in_features, out_features, {}};
    return forward(c, e, workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
}

int df11_gated_matmul(const df11_device_stream *gate, const df11_device_stream *up, const uint16_t *x,
                      uint64_t x_stride, uint32_t n_tokens, uint32_t in_features, uint32_t out_features,
                      const df11_epilogue *e, void *workspace, uint64_t workspace_bytes, void *hip_stream) {
    Call c{{gate, up}, 2, x, x_stride, n_tokens, in_features, out_features, {}};
    return forward(c, e, workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
