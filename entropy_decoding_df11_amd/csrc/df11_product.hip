// Products of compressed weights with an epilogue (gfx950):
//
//   y = act(x W^T + bias) + residual                        df11_matmul_epilogue
//   y = act(x Wg^T + bias0) * (x Wu^T + bias1) + residual   df11_gated_matmul
//
// The weights are DF11 streams in MFMA tile order.  Up to kPartialTokens
// tokens the decode is fused into the product (df11::partial_products):
// partial sums go to slots, and one kernel adds a panel's slots in the order
// of the stream, applies the epilogue and rounds once.  Beyond that the
// stream is decoded once into the workspace, in tile order as it is stored,
// and multiplied from there (df11::dense_product): every further sweep of the
// fused product would decode it again.
//
// The gradients go through the dense product too:
//
//   dz = dy * act'(z)   or   dzg = dy * zu * act'(zg), dzu = dy * act(zg)
//   dx = dz W           or   dx = dzg Wg + dzu Wu
//   dbias = sum over the tokens of dz
//
// with dz rounded to BF16, the matrix cores' operand type, for dx and kept in
// float for dbias.  That rounding is at most 2^-8 of each dz and as large as
// dx's own: dx is off by 0.0023 of its norm in place of 0.0017.  (dz as the sum
// of two BF16 would take it away and double the product's matrix work.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include <stdint.h>

#include "df11.h"
#include "df11_columns.h"
#include "df11_dense.h"
#include "df11_device.h"
#include "df11_epilogue.h"
#include "df11_partials.h"

namespace {

using df11::kPartialGroups;
using df11::kPartialTokens;
using df11::Partials;
using df11::PartialStream;

constexpr uint32_t kPanelRows = 64;  // output features of one panel

struct SumArgs {
    PartialStream s[2];
    const float *slots;
    Epilogue e;
    uint32_t n_tokens, features;
};

// Panel of element e of a tile-ordered stream.
__device__ __forceinline__ uint32_t panel_of(const PartialStream &s, uint32_t e) {
    return df11::panel_of_step(min(e, s.n_elements - 1u) >> 11, s.tile_magic);
}

__device__ __forceinline__ uint32_t out_pos_of(const PartialStream &s, uint32_t g) {
    return s.out_pos[min(g, s.n_groups)];
}

// First super-group of workgroup w's range: floor(w n_super / n_wg), as
// w * (n_super / n_wg) + floor(w * (n_super % n_wg) / n_wg) in 32 bits
// (n_wg is a grid size, far below 2^16).
__device__ __forceinline__ uint32_t range_begin(const PartialStream &s, uint32_t w) {
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
__device__ __forceinline__ void find_ranges(const PartialStream &s, uint32_t p, Found *f) {
    for (uint32_t w = threadIdx.x; w < s.n_wg; w += blockDim.x) {
        const uint32_t a = panel_of(s, out_pos_of(s, range_begin(s, w) * kPartialGroups));
        const uint32_t b = panel_of(s, max(out_pos_of(s, range_begin(s, w + 1u) * kPartialGroups), 1u) - 1u);
        if (a <= p && p <= b) {
            atomicMin(&f->lo, w);
            atomicMax(&f->hi, w + 1u);
            atomicMax(&f->skip, p - a);
        }
    }
}

// One workgroup adds the slots of one panel for up to TOKENS tokens: a lane
// per output feature, the slots split between the four waves, whose sums
// meet in LDS in wave order.  A wave takes several slots at once, so that
// more loads than one slot's are in flight.  What bounds it is the chain of a
// launch, the ranges' search and two rounds of loads: 4.5 us of a product's
// 45 for 4096 x 14336 at one token, whose slots are half a megabyte.
template <bool kGated, int TOKENS>
__global__ __launch_bounds__(256) void df11_sum_slots_kernel(SumArgs a) {
    constexpr int kStreams = kGated ? 2 : 1;
    constexpr int kAtOnce = TOKENS >= 4 ? 4 : 8;  // slots
    __shared__ Found s_found[kStreams];
    __shared__ float s_sum[kStreams][4][TOKENS][kWaveSize];
    const uint32_t p = blockIdx.x, t0 = blockIdx.y * TOKENS;
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t tokens = min(static_cast<uint32_t>(TOKENS), a.n_tokens - t0);
    const uint64_t slot = static_cast<uint64_t>(kPanelRows) * a.n_tokens;
    if (threadIdx.x < kStreams) s_found[threadIdx.x] = Found{~0u, 0u, 0u};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStreams; ++i) find_ranges(a.s[i], p, &s_found[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
        const PartialStream &s = a.s[i];
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
        const float *slots = a.slots + static_cast<uint64_t>(t0) * kPanelRows + lane;
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
    for (uint32_t t = wave; t < tokens; t += 4u) {
        float z[2] = {};
#pragma unroll
        for (int i = 0; i < kStreams; ++i)
            z[i] = (s_sum[i][0][t][lane] + s_sum[i][1][t][lane]) + (s_sum[i][2][t][lane] + s_sum[i][3][t][lane]);
        finish<kGated>(a.e, t0 + t, kPanelRows * p + lane, a.features, z[0], z[1]);
    }
}

// dz of every output, from dy and the sums before the activation.
struct SlopeArgs {
    const void *dy;
    const float *pre[2];
    uint16_t *dz[2];     // BF16, tokens x features; or null
    // Sums of dz over a chunk's tokens, or null: [chunk][features] of float,
    // or with one chunk the bias gradient itself, of sum_dtype.
    void *sums[2];
    uint64_t dy_stride;
    uint32_t dy_dtype, sum_dtype, dy_vec, act, tokens, features, chunk;
};

// A wave takes four columns per lane of every fourth token of the block's
// chunk of tokens (blockIdx.y); the four waves' column sums meet in LDS.
template <bool kGated>
__global__ __launch_bounds__(256) void df11_slope_kernel(SlopeArgs a) {
    __shared__ float s_sum[2][3][256];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wave = threadIdx.x / kWaveSize;
    const uint32_t col = 256u * blockIdx.x + 4u * lane;
    const uint32_t end = min((blockIdx.y + 1u) * a.chunk, a.tokens);
    constexpr int kMats = kGated ? 2 : 1;
    float sum[2][4] = {};
    for (uint32_t t = blockIdx.y * a.chunk + wave; t < end && col < a.features; t += 4u) {
        float dy[4], z0[4], z1[4], d[2][4];
        const uint64_t at = t * a.dy_stride + col, in = static_cast<uint64_t>(t) * a.features + col;
        if (a.dy_vec && a.dy_dtype == DF11_BF16) {
            load_vec<bf16_t, 4>(static_cast<const bf16_t *>(a.dy) + at, dy);
        } else if (a.dy_vec) {
            load_vec<float, 4>(static_cast<const float *>(a.dy) + at, dy);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) dy[e] = load_as(a.dy, at + e, a.dy_dtype);
        }
        if (a.pre[0]) load_vec<float, 4>(a.pre[0] + in, z0);
        if constexpr (kGated) load_vec<float, 4>(a.pre[1] + in, z1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kGated) {
                d[0][e] = dy[e] * z1[e] * slope(a.act, z0[e]);
                d[1][e] = dy[e] * activate(a.act, z0[e]);
            } else {
                d[0][e] = a.act == DF11_ACT_NONE ? dy[e] : dy[e] * slope(a.act, z0[e]);
            }
        }
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            if (a.dz[m]) store_vec<bf16_t, 4>(reinterpret_cast<bf16_t *>(a.dz[m]) + in, d[m]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[m][e] += d[m][e];
        }
    }
    if (!a.sums[0] && !a.sums[1]) return;
    for (int m = 0; m < kMats; ++m)
        for (int e = 0; e < 4 && wave; ++e) s_sum[m][wave - 1u][4u * lane + e] = sum[m][e];
    __syncthreads();
    if (wave || col >= a.features) return;
    for (int m = 0; m < kMats; ++m) {
        if (!a.sums[m]) continue;
        for (uint32_t e = 0; e < 4; ++e) {
            float v = sum[m][e];
            for (int w = 0; w < 3; ++w) v += s_sum[m][w][4u * lane + e];
            store_as(a.sums[m], static_cast<uint64_t>(blockIdx.y) * a.features + col + e, a.sum_dtype, v);
        }
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
// Longest row of x, of W and of an operand of the dense product, and largest
// stride between them: 256 of them then lie within a buffer resource's 32
// bits of offset.
constexpr uint64_t kMaxRow = 1ull << 22;

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
    if (in_features > kMaxRow || static_cast<uint64_t>(n_tokens) * std::max(in_features, out_features) >= (1ull << 32))
        return DF11_E_TOO_LARGE;
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
    if (!c.x || !aligned(c.x, 16) || c.x_stride % 8 || c.x_stride > kMaxRow || !e->out ||
        !aligned(e->out, out_bytes) || e->out_stride > kMaxStride ||
        (c.n_tokens > 1 && e->out_stride < c.out_features))
        return DF11_E_INVALID_ARG;
    if (e->residual && (!aligned(e->residual, res_bytes) || e->residual_stride > kMaxStride)) return DF11_E_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        if ((e->bias[i] && !aligned(e->bias[i], bias_bytes)) || (e->pre[i] && !aligned(e->pre[i], 16)))
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

int slots_impl(const Call &c, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    SumArgs a{};
    Partials p{};
    a.slots = static_cast<float *>(workspace);
    const int rc = df11::partial_products(c.w, c.n, c.x, c.x_stride, c.n_tokens, static_cast<float *>(workspace),
                                          workspace_bytes, stream, p);
    if (rc) return rc;
    a.s[0] = p.s[0];
    a.s[1] = p.s[1];
    a.e = c.e;
    a.n_tokens = c.n_tokens;
    a.features = c.out_features;
    void *params[] = {&a};
    // Tokens of a workgroup: one while two workgroups a CU have not come
    // together, then four, so that a panel's ranges are searched for less
    // often.  Whole products, one and four tokens a workgroup: 1024 x 4096 at
    // 16 tokens 14.1 and 14.9 us, 4096 x 4096 at 8 tokens 21.0 and 21.6, at 32
    // 30.3 and 28.7, 14336 x 4096 at 16 tokens 54.2 and 49.0.  (Sixteen tokens
    // a workgroup: 19.4, 24.3, 31.3 and 50.4.)
    const uint32_t panels = c.out_features / kPanelRows;
    const bool one = c.n_tokens == 1 || static_cast<uint64_t>(panels) * c.n_tokens <= 512;
    const uint32_t each = one ? 1 : 4;
    const auto pick = [one](auto gated) {
        constexpr bool kGated = decltype(gated)::value;
        return one ? reinterpret_cast<const void *>(&df11_sum_slots_kernel<kGated, 1>)
                   : reinterpret_cast<const void *>(&df11_sum_slots_kernel<kGated, 4>);
    };
    return launch_kernel(c.n == 2 ? pick(std::true_type{}) : pick(std::false_type{}),
                         dim3(panels, (c.n_tokens + each - 1) / each), dim3(256), params, 0,
                         stream, nullptr, nullptr);
}

uint64_t slots_bytes(const df11_device_stream *const *ws, uint32_t n, uint32_t n_tokens) {
    Partials p{};
    if (df11::partial_products(ws, n, nullptr, 0, n_tokens, nullptr, 0, nullptr, p)) return 0;
    return p.slot_bytes;
}

// Work counters of a decode.  Those of a weight are left alone: nothing orders
// this call after launches of the same weight by other threads, or a graph's
// replays after anything.  Two streams of kCounted weights or more decode by
// the dynamic schedule with counters of the workspace, zeroed first; shorter
// ones, and one alone, by the static schedule.  Gate and up of 64 tokens,
// counters against static: 14336 x 4096 each 131 against 136 us, 8192 x 4096
// 85 against 83, 4096 x 4096 56.0 against 54.4.
constexpr uint64_t kCounted = 3ull << 24;
constexpr uint32_t kCounterWords = 2 * DF11_SCHEDULE_WORDS;

__global__ void df11_zero_counters_kernel(uint32_t *p) {
    for (uint32_t i = threadIdx.x; i < kCounterWords; i += blockDim.x) p[i] = 0;
}

// Whether there are two different streams.  (Streams may share a buffer: those
// of a matrix and of its negative have the same exponents.)
bool two_streams(const df11_device_stream *const *ws, uint32_t n) {
    return n == 2 && (ws[1]->enc != ws[0]->enc || ws[1]->sm != ws[0]->sm);
}

// Bytes of the decoded weights (one copy of a stream given twice) and of the
// counters of their decode.
uint64_t decoded_bytes(const df11_device_stream *const *ws, uint32_t n) {
    const uint64_t one = round_up(2 * ws[0]->h.n_elements, 256);
    if (!two_streams(ws, n)) return one;
    return 2 * one + (ws[0]->h.n_elements >= kCounted ? round_up(4 * kCounterWords, 256) : 0);
}

// Decodes the streams into the workspace in tile order, as they are stored;
// out[i] receives where.
int decode_weights(const df11_device_stream *const *ws, uint32_t n, void *workspace, const uint16_t **out,
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

uint64_t forward_workspace(const df11_device_stream *const *ws, uint32_t n, uint32_t n_tokens, uint32_t cols) {
    if (n_tokens <= kPartialTokens) return slots_bytes(ws, n, n_tokens);
    const uint32_t rows = static_cast<uint32_t>(ws[0]->h.n_elements / cols);
    const uint64_t more = df11::dense_workspace(n == 2 ? df11::kDenseGated : df11::kDensePlain, n, n_tokens, rows, cols);
    return more == ~0ull ? 0 : decoded_bytes(ws, n) + more;
}

int dense_impl(const Call &c, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    const uint64_t need = forward_workspace(c.w, c.n, c.n_tokens, c.in_features);
    if (!need) return DF11_E_HIP;
    if (workspace_bytes < need) return DF11_E_BUFFER_TOO_SMALL;
    df11::DenseCall d{};
    d.mode = c.n == 2 ? df11::kDenseGated : df11::kDensePlain;
    d.left[0] = c.x;
    d.left_stride = c.x_stride;
    d.tokens = c.n_tokens;
    d.rows = c.out_features;
    d.cols = c.in_features;
    const int rc = decode_weights(c.w, c.n, workspace, d.w, stream);
    if (rc) return rc;
    return df11::dense_product(d, c.e, reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + decoded_bytes(c.w, c.n)),
                               stream);
}

int forward(Call &c, const df11_epilogue *e, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    bool empty = false;
    int rc = check_call(c, e, workspace, empty);
    if (rc || empty) return rc;
    if (!workspace) return DF11_E_INVALID_ARG;
    if (!workspace_clear(c, workspace, workspace_bytes)) return DF11_E_INVALID_ARG;
    return c.n_tokens <= kPartialTokens ? slots_impl(c, workspace, workspace_bytes, stream)
                                        : dense_impl(c, workspace, workspace_bytes, stream);
}

// ---- gradients

// Tokens of one block of the slopes' kernel: as many as leave about
// kSlopeBlocks blocks, between one and eight a wave, but at most
// kSlopeMaxChunks partial rows of a bias gradient.  (777 tokens of 1024
// features: 780 blocks of 4 tokens 5.7 us, 100 of 32 tokens 16.6.  1024
// tokens of 14336 gated move 206 MB: 44 us, 4.7 TB/s.)
// Up to kSlopeOneChunk tokens are one chunk, which needs no kernel to add the
// chunks, at 1.1 us for every four tokens of it (the bias gradient of 4096
// features: 8 tokens 4.5 us, 9 tokens in three chunks 5.4, 16 in one 6.8).
constexpr uint32_t kSlopeBlocks = 1024, kSlopeMaxChunks = 256, kSlopeOneChunk = 8;

uint32_t slope_chunk(uint32_t tokens, uint32_t rows) {
    if (tokens <= kSlopeOneChunk) return tokens;
    const uint64_t strips = (rows + 255) / 256;
    const uint32_t want = static_cast<uint32_t>(std::min<uint64_t>(32, tokens * strips / kSlopeBlocks));
    return std::max((std::max(want, 1u) + 3) / 4 * 4, (tokens + kSlopeMaxChunks - 1) / kSlopeMaxChunks);
}

// Where a gradient call's parts of the workspace begin.
struct GradPlan {
    uint64_t dz[2], partial[2], weights, split, end;
    uint32_t chunks;
    bool own_dz;  // dz is written (not dy itself)
};

bool grad_plan(const df11_device_stream *const *ws, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols,
               const df11_product_grad &g, GradPlan &p) {
    p.own_dz = n == 2 || g.activation != DF11_ACT_NONE || g.dy_dtype != DF11_BF16 || !aligned(g.dy, 16) ||
               g.dy_stride % 8 || g.dy_stride > kMaxRow;
    const uint32_t chunk = slope_chunk(tokens, rows);
    p.chunks = (tokens + chunk - 1) / chunk;
    uint64_t at = 0;
    for (uint32_t i = 0; i < 2; ++i) {
        p.dz[i] = at;
        if (i < n && g.dx && p.own_dz) at += round_up(2ull * tokens * rows, 256);
        p.partial[i] = at;
        if (i < n && g.dbias[i] && p.chunks > 1) at += round_up(4ull * p.chunks * rows, 256);
    }
    p.weights = at;
    if (g.dx) at += decoded_bytes(ws, n);
    p.split = at;
    if (g.dx) {
        const uint64_t more = df11::dense_workspace(df11::kDenseBack, n, tokens, rows, cols);
        if (more == ~0ull) return false;
        at += more;
    }
    p.end = at;
    return true;
}

int backward(const df11_device_stream *const *ws, uint32_t n, uint32_t tokens, uint32_t cols, uint32_t rows,
             const df11_product_grad *g, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    int rc = check_streams(ws, n, tokens, cols, rows);
    if (rc) return rc;
    if (!g || g->activation > DF11_ACT_GELU_TANH) return DF11_E_INVALID_ARG;
    const auto float_bytes = [](uint32_t dtype) { return dtype == DF11_FP16 ? 0u : dtype_bytes(dtype); };
    const uint32_t dy_bytes = float_bytes(g->dy_dtype), dx_bytes = float_bytes(g->dx_dtype);
    const uint32_t bias_bytes = float_bytes(g->bias_dtype);
    if (!dy_bytes || (g->dx && !dx_bytes) || ((g->dbias[0] || g->dbias[1]) && !bias_bytes)) return DF11_E_INVALID_ARG;
    if (n == 1 && (g->dbias[1] || g->pre[1])) return DF11_E_INVALID_ARG;
    if (rows == 0) return DF11_OK;
    if (rows > kMaxRow) return DF11_E_TOO_LARGE;
    const bool needs_pre = n == 2 || g->activation != DF11_ACT_NONE;
    if (tokens) {
        if (!g->dy || !aligned(g->dy, dy_bytes) || g->dy_stride > kMaxStride) return DF11_E_INVALID_ARG;
        for (uint32_t i = 0; i < n; ++i)
            if (needs_pre && (!g->pre[i] || !aligned(g->pre[i], 16))) return DF11_E_INVALID_ARG;
        if (g->dx && (!aligned(g->dx, dx_bytes) || g->dx_stride > kMaxStride || (tokens > 1 && g->dx_stride < cols)))
            return DF11_E_INVALID_ARG;
    }
    for (int i = 0; i < 2; ++i)
        if (g->dbias[i] && !aligned(g->dbias[i], bias_bytes)) return DF11_E_INVALID_ARG;
    // Outputs and the workspace stay clear of the inputs and of each other.
    const uint64_t dy_span = tokens ? rows_span(tokens, rows, g->dy_stride, dy_bytes) : 0;
    const uint64_t elems = static_cast<uint64_t>(tokens) * rows;
    GradPlan p{};
    uint64_t need = 0;
    if (tokens) {
        // (nothing below reads a pointer, so the overlap checks can wait for the plan)
        if (workspace && !aligned(workspace, 256)) return DF11_E_INVALID_ARG;
    }
    const void *outs[] = {tokens ? g->dx : nullptr, g->dbias[0], g->dbias[1], nullptr};
    uint64_t spans[] = {tokens && g->dx ? rows_span(tokens, cols, g->dx_stride, dx_bytes) : 0,
                        g->dbias[0] ? static_cast<uint64_t>(bias_bytes) * rows : 0,
                        g->dbias[1] ? static_cast<uint64_t>(bias_bytes) * rows : 0, 0};
    const auto clear = [&](int k) {
        for (int j = 0; j < k; ++j)
            if (overlaps(outs[k], spans[k], outs[j], spans[j])) return false;
        if (overlaps(outs[k], spans[k], g->dy, dy_span)) return false;
        for (int i = 0; i < 2; ++i)
            if (g->pre[i] && overlaps(outs[k], spans[k], g->pre[i], 4 * elems)) return false;
        for (uint32_t i = 0; i < n; ++i)
            if (df11::stream_overlaps(ws[i], outs[k], spans[k])) return false;
        return true;
    };
    for (int k = 0; k < 3; ++k)
        if (!clear(k)) return DF11_E_INVALID_ARG;
    if (tokens == 0) {
        for (uint32_t i = 0; i < n; ++i) {
            if (!g->dbias[i]) continue;
            rc = df11::column_sums(nullptr, 0, rows, g->dbias[i], g->bias_dtype, stream);
            if (rc) return rc;
        }
        return DF11_OK;
    }
    if (!g->dx && !g->dbias[0] && !g->dbias[1]) return DF11_OK;
    if (!grad_plan(ws, n, tokens, rows, cols, *g, p)) return DF11_E_HIP;
    need = p.end;
    if (!workspace && need) return DF11_E_INVALID_ARG;
    if (workspace_bytes < need) return DF11_E_BUFFER_TOO_SMALL;
    outs[3] = workspace;
    spans[3] = need;
    if (!clear(3)) return DF11_E_INVALID_ARG;

    uint8_t *base = static_cast<uint8_t *>(workspace);
    SlopeArgs a{};
    a.dy = g->dy;
    a.dy_stride = g->dy_stride;
    a.dy_dtype = g->dy_dtype;
    a.dy_vec = aligned(g->dy, 4 * dy_bytes) && g->dy_stride % 4 == 0;
    a.act = g->activation;
    a.tokens = tokens;
    a.features = rows;
    a.chunk = slope_chunk(tokens, rows);
    for (uint32_t i = 0; i < n; ++i) {
        a.pre[i] = needs_pre ? g->pre[i] : nullptr;
        if (g->dx && p.own_dz) a.dz[i] = reinterpret_cast<uint16_t *>(base + p.dz[i]);
        if (g->dbias[i]) a.sums[i] = p.chunks > 1 ? base + p.partial[i] : g->dbias[i];
    }
    a.sum_dtype = p.chunks > 1 ? static_cast<uint32_t>(DF11_FP32) : g->bias_dtype;
    (void)hipGetLastError();
    if (a.dz[0] || a.sums[0] || a.sums[1]) {
        void *params[] = {&a};
        rc = launch_kernel(n == 2 ? reinterpret_cast<const void *>(&df11_slope_kernel<true>)
                                  : reinterpret_cast<const void *>(&df11_slope_kernel<false>),
                           dim3((rows + 255) / 256, p.chunks), dim3(256), params, 0, stream, nullptr, nullptr);
        if (rc) return rc;
    }
    for (uint32_t i = 0; i < n; ++i) {
        if (!g->dbias[i] || p.chunks == 1) continue;
        rc = df11::column_sums(static_cast<const float *>(a.sums[i]), p.chunks, rows, g->dbias[i], g->bias_dtype, stream);
        if (rc) return rc;
    }
    if (!g->dx) return DF11_OK;
    df11::DenseCall d{};
    d.mode = df11::kDenseBack;
    d.tokens = tokens;
    d.rows = rows;
    d.cols = cols;
    rc = decode_weights(ws, n, base + p.weights, d.w, stream);
    if (rc) return rc;
    for (uint32_t i = 0; i < n; ++i) d.left[i] = p.own_dz ? a.dz[i] : static_cast<const uint16_t *>(g->dy);
    d.left_stride = p.own_dz ? rows : g->dy_stride;
    Epilogue e{};
    e.out = g->dx;
    e.out_stride = g->dx_stride;
    e.out_dtype = g->dx_dtype;
    return df11::dense_product(d, e, reinterpret_cast<float *>(base + p.split), stream);
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
    return forward_workspace(ws, n, n_tokens, w->tile_cols);
}

uint64_t df11_epilogue_grad_workspace(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens,
                                     const df11_product_grad *g) {
    const df11_device_stream *ws[] = {w, up};
    const uint32_t n = up ? 2 : 1;
    if (!w || !n_tokens || !g) return 0;
    for (uint32_t i = 0; i < n; ++i)
        if (df11::check_stream(ws[i]) || !ws[i]->h.n_elements || !ws[i]->tile_cols ||
            ws[i]->h.n_elements != w->h.n_elements || ws[i]->tile_cols != w->tile_cols)
            return 0;
    GradPlan p{};
    return grad_plan(ws, n, n_tokens, static_cast<uint32_t>(w->h.n_elements / w->tile_cols), w->tile_cols, *g, p) ? p.end
                                                                                                             : 0;
}

int df11_matmul_epilogue_grad(const df11_device_stream *w, const df11_device_stream *up, uint32_t n_tokens,
                          uint32_t in_features, uint32_t out_features, const df11_product_grad *g, void *workspace,
                          uint64_t workspace_bytes, void *hip_stream) {
    const df11_device_stream *ws[] = {w, up};
    return backward(ws, up ? 2 : 1, n_tokens, in_features, out_features, g, workspace, workspace_bytes,
                    static_cast<hipStream_t>(hip_stream));
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
