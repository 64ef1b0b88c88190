// Softmax cross entropy through a compressed output head (gfx950), without
// keeping the logits:
//
//   loss = log(sum_v exp(z_v)) - z_y,  z = x W^T
//   grad = sum_v p_v W_v - W_y
//
// A panel of 64 classes gives each token a pair (r, s): the sum s of
// 2^(z log2(e) - r) over the panel's classes but the target y, r the largest
// exponent rounded up.  With S and R the pairs' sum, and u = R ln 2 + ln S - z_y
// the others against the target,
//
//   loss = ln(1 + exp(u)),  sum_{v /= y} p_v = sigma(u),  p_y - 1 = -sigma(u)
//
// which lose nothing where the target is all but certain.
//
// The gradient comes in the same pass, piece by piece of the vocabulary: a
// piece's exponentials are the left operand of a second product with the same
// rows of W, whose sums A stay relative to the token's R:
//
//   grad = sigma(u) (A / S - W_y)
//
// so that the logits are computed once and W is decoded once (recomputing them
// in a backward pass of its own would take a third product and a second
// decode).  R begins as the target's own exponent, from a dot product of x with
// its row of W.  It is a whole number: where a logit passes it by 2^64 it moves, and
// the exponentials in BF16 and A are rescaled exactly.
//
// Up to kPartialTokens tokens without a gradient the decode is fused into the
// product, and its slots' sums end in the pairs; otherwise the head is decoded
// into the workspace, and the dense product's epilogue makes them.
//
// The matrix cores bound it, and the decode for few tokens.  24 tokens through 32000 x
// 4096: fused decode and product 102 us, slots' sums 13, tokens 5 (the floor, the
// compressed head's bytes, 37).  1000 tokens through 128256 x 4096: decode 353 us,
// product 854 to 880 (1.2 PFLOP/s).  2048 tokens through 32000 x 4096 with the gradient:
// decode 88, first references 28, logits and exponentials 460 (1.17 PFLOP/s), their
// product with W 380 (1.41), and all else 60.  (Once the clocks have settled, after
// some 100 passes; 5 to 15% more before.)  The logits alone would be 4 bytes a token and
// class, written once and read three times by the formulas one by one: 8.4 and 8.0 ms.
// The workspace has the decoded head, 2 bytes a weight: below in_features / 2 tokens
// more than the logits would have.
#include <hip/hip_runtime.h>

#include <algorithm>

#include <stdint.h>

#include "df11.h"
#include "df11_decoded.h"
#include "df11_dense.h"
#include "df11_device.h"
#include "df11_epilogue.h"
#include "df11_partials.h"
#include "df11_slots.h"
#include "df11_types.h"

namespace {

using df11::kLog2eHi;
using df11::kPartialTokens;
using df11::Partials;
using df11::PartialStream;

// Exponentials of a piece, tokens times classes: few pieces, since each reads A and
// writes it once more (8192 tokens, 32000 classes of 4096 columns with 16, 32, 64, 128
// and 256 M of them: 4623, 4066, 3709, 3593 and 3507 us), in 256 MB.  And the fewest
// classes of a piece (65536 tokens, 32000 classes of 512 columns with 2048, 4096 and
// 8192 of them: 7652, 6511 and 6012 us, for 0.27, 0.54 and 1.1 GB).
constexpr uint64_t kPieceExps = 128u << 20;
constexpr uint32_t kLeastPiece = 4096;
constexpr uint64_t kMaxRow = 1ull << 22;
// Tokens with a gradient: a workgroup of 256 threads each, and a dimension of a launch
// has fewer than 2^32.
constexpr uint32_t kMaxGradTokens = (1u << 24) - 1u;

constexpr float kLn2 = 0.69314718055994530942f;

struct SlotLossArgs {
    PartialStream s;
    const float *slots;
    const int64_t *targets;
    float *stats, *target_logit;
    uint32_t n_tokens, classes;
};

// A panel's pairs from the slots of up to TOKENS tokens.
template <int TOKENS>
__global__ __launch_bounds__(256) void df11_loss_slots_kernel(SlotLossArgs a) {
    __shared__ Found s_found[1];
    __shared__ float s_sum[1][4][TOKENS][kWaveSize];
    const uint32_t p = blockIdx.x, t0 = blockIdx.y * TOKENS;
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t tokens = min(static_cast<uint32_t>(TOKENS), a.n_tokens - t0);
    panel_sums<1, TOKENS>(&a.s, a.slots, a.n_tokens, p, t0, tokens, s_found, s_sum);
    const uint32_t v = kPanelRows * p + lane;
    for (uint32_t t = wave; t < tokens; t += 4u) {
        const uint32_t token = t0 + t;
        float z = (s_sum[0][0][t][lane] + s_sum[0][1][t][lane]) + (s_sum[0][2][t][lane] + s_sum[0][3][t][lane]);
        if (v >= a.classes) {
            z = -INFINITY;
        } else if (a.targets[token] == static_cast<int64_t>(v)) {
            a.target_logit[token] = z;
            z = -INFINITY;
        }
        float top = z;
#pragma unroll
        for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
        const float ref = ceilf(top * kLog2eHi), base = ref == -INFINITY ? 0.0f : ref;
        float sum = __builtin_amdgcn_exp2f(df11::class_exponent(z, base));
#pragma unroll
        for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
        if (lane == 0) {
            float *st = a.stats + 2u * (static_cast<uint64_t>(p) * a.n_tokens + token);
            st[0] = ref;
            st[1] = sum;
        }
    }
}

// What a token's end needs.
struct TokenArgs {
    const int64_t *targets;
    int64_t ignore_index;
    const float *stats, *target_logit;
    const float *rounded;      // [panel][token]
    float *ref, *sum, *sum_rounded, *scale;  // running, [token]
    uint16_t *exps;
    uint64_t exps_stride;
    float *loss;
    uint32_t n_tokens, classes, panels;
};

// 2^(r - to), 0 for no class.
__device__ __forceinline__ float ref_scale(float r, float to) {
    return r == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(r - to);
}

// Eight consecutive elements of row `row` of a decoded matrix in tile order.
__device__ __forceinline__ void load_row8(const uint16_t *w, uint32_t row, uint32_t c, uint32_t cols, float (&v)[8]) {
    const uint64_t block = (static_cast<uint64_t>(row / 64u) * (cols / 32u) + c / 32u) * 4u + row % 64u / 16u;
    load_vec<bf16_t, 8>(reinterpret_cast<const bf16_t *>(w) + block * 512u + (row % 16u + 2u * (c % 32u)) * 8u, v);
}

// Tokens of a workgroup of 1024 threads whose pairs lie next to each other, and the
// threads of each.
constexpr uint32_t kTokens = 8, kParts = 1024 / kTokens;

// The pairs (top, sum) of a token's threads joined in a fixed order, in its first.
// (N: sums that share the reference.)
template <int N>
__device__ __forceinline__ void join_pairs(float (*s_pair)[kTokens][1 + N], uint32_t part, uint32_t t, float &top,
                                           float (&sum)[N]) {
    s_pair[part][t][0] = top;
#pragma unroll
    for (int i = 0; i < N; ++i) s_pair[part][t][1 + i] = sum[i];
    __syncthreads();
    for (uint32_t half = kParts / 2u; half; half >>= 1) {
        if (part < half) {
            const float r = s_pair[part + half][t][0], to = fmaxf(top, r);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                sum[i] = sum[i] * ref_scale(top, to) + s_pair[part + half][t][1 + i] * ref_scale(r, to);
                s_pair[part][t][1 + i] = sum[i];
            }
            top = to;
            s_pair[part][t][0] = top;
        }
        __syncthreads();
    }
}

// The references that the tokens begin with: the exponent, rounded up, of their
// target's logit, or where the target is no class of another one's, which is as
// good a guess; none if it is not finite.  The targets' rows are kept for the
// gradient's end: in tile order a row's vectors lie in a line of memory each, and
// reading it again would take eight times what it has.  A workgroup a token.
__global__ __launch_bounds__(256) void df11_loss_first_kernel(TokenArgs a, const uint16_t *x, uint64_t x_stride,
                                                             const uint16_t *w, uint32_t cols, uint16_t *kept) {
    __shared__ float s_sum[4];
    const uint32_t token = blockIdx.x;
    const int64_t target = a.targets[token];
    const uint32_t row = target >= 0 && target < static_cast<int64_t>(a.classes) ? static_cast<uint32_t>(target) : 0u;
    float z = 0.0f;
#pragma unroll 2
    for (uint32_t c = 8u * threadIdx.x; c < cols; c += 8u * 256u) {
        float u[8], v[8];
        load_vec<bf16_t, 8>(reinterpret_cast<const bf16_t *>(x) + token * x_stride + c, u);
        load_row8(w, row, c, cols, v);
        store_vec<bf16_t, 8>(reinterpret_cast<bf16_t *>(kept) + static_cast<uint64_t>(token) * cols + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z += u[i] * v[i];
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) z += __shfl_xor(z, m);
    if (threadIdx.x % kWaveSize == 0) s_sum[threadIdx.x / kWaveSize] = z;
    __syncthreads();
    if (threadIdx.x) return;
    const float ref = ceilf((s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * kLog2eHi);
    a.ref[token] = fabsf(ref) < INFINITY ? ref : -INFINITY;
    a.sum[token] = 0.0f;
    a.sum_rounded[token] = 0.0f;
}

// A piece's pairs joined to what the tokens have.  Where the reference moves, or a
// panel has another, exponentials are brought to it.
__global__ __launch_bounds__(1024) void df11_loss_piece_kernel(TokenArgs a, uint32_t first_piece) {
    __shared__ float s_pair[kParts][kTokens][3];
    __shared__ float s_to[kTokens];
    __shared__ uint32_t s_other[kTokens];
    const uint32_t t = threadIdx.x % kTokens, part = threadIdx.x / kTokens, token = blockIdx.x * kTokens + t;
    const bool in = token < a.n_tokens;
    const float *st = a.stats + 2u * (in ? token : 0u);
    const uint64_t step = 2ull * a.n_tokens;
    const float was = in ? a.ref[token] : -INFINITY;
    if (threadIdx.x < kTokens) s_other[threadIdx.x] = 0;
    const float *rounded = a.rounded + (in ? token : 0u);
    float top = was, sum[2] = {0.0f, 0.0f};  // of the exponentials, and as they were rounded
    bool other = false;  // a reference that is not the token's
    for (uint32_t p = part; p < a.panels; p += kParts) {
        const float r = st[p * step], s = st[p * step + 1u], s2 = rounded[p * static_cast<uint64_t>(a.n_tokens)];
        const float to = fmaxf(top, r), old = ref_scale(top, to), f = ref_scale(r, to);
        sum[0] = sum[0] * old + s * f;
        sum[1] = sum[1] * old + s2 * f;
        top = to;
        other = other || (r != was && r != -INFINITY);
    }
    join_pairs(s_pair, part, t, top, sum);
    if (part == 0 && in) {
        // (the pairs of no class leave a token's first reference as it is)
        const float scale = first_piece ? 0.0f : ref_scale(was, top);
        a.ref[token] = top;
        a.sum[token] = a.sum[token] * scale + sum[0];
        a.sum_rounded[token] = a.sum_rounded[token] * scale + sum[1];
        a.scale[token] = scale;
        s_to[t] = top;
    }
    if (other && in) s_other[t] = 1;
    __syncthreads();
    // Eight lanes a panel, all of the workgroup one token after the other.
    for (uint32_t i = 0; i < kTokens; ++i) {
        if (!s_other[i]) continue;
        const uint32_t mine = blockIdx.x * kTokens + i;
        const float to = s_to[i];
        for (uint32_t p = threadIdx.x / 8u; p < a.panels; p += 1024u / 8u) {
            const float r = a.stats[2u * mine + p * step];
            if (r == to || r == -INFINITY) continue;
            const float f = ref_scale(r, to);
            bf16_t *e = reinterpret_cast<bf16_t *>(a.exps) + mine * a.exps_stride + 64u * p + 8u * (threadIdx.x % 8u);
            float v[8];
            load_vec<bf16_t, 8>(e, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= f;
            store_vec<bf16_t, 8>(e, v);
        }
    }
}

enum TokenKind { kScored = 0, kIgnored = 1, kNoClass = 2 };

__device__ __forceinline__ TokenKind kind_of(int64_t target, int64_t ignore_index, uint32_t classes) {
    if (target == ignore_index) return kIgnored;
    return target >= 0 && target < static_cast<int64_t>(classes) ? kScored : kNoClass;
}

// The others against the target (u above); nothing else in the vocabulary: -inf.
// (The target is in no sum: where its logit is not finite, which an infinity or a NaN
// in x always makes it, that has to be said here.)
__device__ __forceinline__ float others(float ref, float sum, float target_logit) {
    if (!(fabsf(target_logit) < INFINITY)) return __builtin_nanf("");
    return sum == 0.0f ? -INFINITY : ref * kLn2 + logf(sum) - target_logit;
}

__device__ __forceinline__ float loss_of(float u) { return u > 0.0f ? u + log1pf(expf(-u)) : log1pf(expf(u)); }

// The losses from the pairs of all panels.
__global__ __launch_bounds__(1024) void df11_loss_tokens_kernel(TokenArgs a) {
    __shared__ float s_pair[kParts][kTokens][2];
    const uint32_t t = threadIdx.x % kTokens, part = threadIdx.x / kTokens;
    const uint32_t token = (blockIdx.y * gridDim.x + blockIdx.x) * kTokens + t;
    const bool in = token < a.n_tokens;
    const float *st = a.stats + 2u * (in ? token : 0u);
    const uint64_t step = 2ull * a.n_tokens;
    float top = -INFINITY, sum[1] = {0.0f};
    for (uint32_t p = part; p < a.panels; p += kParts) {
        const float r = st[p * step], s = st[p * step + 1u], to = fmaxf(top, r);
        sum[0] = sum[0] * ref_scale(top, to) + s * ref_scale(r, to);
        top = to;
    }
    join_pairs(s_pair, part, t, top, sum);
    if (part || !in) return;
    const TokenKind kind = kind_of(a.targets[token], a.ignore_index, a.classes);
    a.loss[token] = kind == kIgnored   ? 0.0f
                    : kind == kNoClass ? __builtin_nanf("")
                                       : loss_of(others(top, sum[0], a.target_logit[token]));
}

// The gradient of an ignored token in every element, and no other's in any: what the
// loss's own gradient holds there, which need not be finite, reaches nothing.
constexpr float kNothing = -0.0f;

struct GradRowsArgs {
    TokenArgs t;
    const uint16_t *kept;  // the targets' rows, [token][cols]
    float *grad;        // A on entry
    uint32_t cols;
};

// The loss and grad = sigma(u) (A / S - W_y): a workgroup a token.  S is here the sum of
// the rounded exponentials, which A adds too: where few classes have most of the
// probability (and A is as large as W_y), their roundings cancel in the quotient.
__global__ __launch_bounds__(256) void df11_loss_rows_kernel(GradRowsArgs a) {
    const uint32_t token = blockIdx.x;
    const int64_t target = a.t.targets[token];
    const TokenKind kind = kind_of(target, a.t.ignore_index, a.t.classes);
    float u = 0.0f, inverse = 0.0f;
    if (kind == kScored) {
        const float sum = a.t.sum[token];
        u = others(a.t.ref[token], sum, a.t.target_logit[token]);
        const float rounded = a.t.sum_rounded[token];
        inverse = rounded == 0.0f ? 0.0f : 1.0f / rounded;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0)
        a.t.loss[token] = kind == kIgnored ? 0.0f : kind == kNoClass ? __builtin_nanf("") : loss_of(u);
    const float sigma = 1.0f / (1.0f + expf(-u));
    for (uint32_t c = 8u * (blockIdx.y * 256u + threadIdx.x); c < a.cols; c += 8u * 256u * gridDim.y) {
        float *g = a.grad + static_cast<uint64_t>(token) * a.cols + c;
        float v[8], wy[8];
        load_vec<float, 4>(g, *reinterpret_cast<float(*)[4]>(&v[0]));
        load_vec<float, 4>(g + 4, *reinterpret_cast<float(*)[4]>(&v[4]));
        if (kind == kScored) {
            load_vec<bf16_t, 8>(reinterpret_cast<const bf16_t *>(a.kept) + static_cast<uint64_t>(token) * a.cols + c, wy);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = sigma * (v[i] * inverse - wy[i]);
                if (v[i] == 0.0f) v[i] = 0.0f;  // (never kNothing)
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = kind == kIgnored ? kNothing : __builtin_nanf("");
        }
        store_vec<float, 4>(g, *reinterpret_cast<float(*)[4]>(&v[0]));
        store_vec<float, 4>(g + 4, *reinterpret_cast<float(*)[4]>(&v[4]));
    }
}

// The losses' sum or mean, in 64 bits and in an order that their number fixes.
__global__ __launch_bounds__(1024) void df11_loss_total_kernel(const float *loss, const int64_t *targets,
                                                              int64_t ignore_index, uint32_t n, uint32_t mean,
                                                              float *total, float *number) {
    __shared__ double s_sum[16];
    __shared__ uint32_t s_count[16];
    double sum = 0.0;
    uint32_t count = 0;
    for (uint32_t t = threadIdx.x; t < n; t += 1024u) {
        sum += loss[t];
        count += targets[t] != ignore_index ? 1u : 0u;
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        sum += __shfl_xor(sum, m);
        count += __shfl_xor(count, m);
    }
    if ((threadIdx.x & 63u) == 0) {
        s_sum[threadIdx.x / 64u] = sum;
        s_count[threadIdx.x / 64u] = count;
    }
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 16; ++w) {
        sum += s_sum[w];
        count += s_count[w];
    }
    if (total) *total = static_cast<float>(mean ? sum / count : sum);
    if (number) *number = static_cast<float>(count);
}

struct LossGradArgs {
    const float *grad, *dy, *count;
    void *dx;
    uint64_t dy_stride, dx_stride;
    uint32_t cols, dx_dtype, vec;
};

__global__ __launch_bounds__(256) void df11_loss_grad_kernel(LossGradArgs a) {
    const uint32_t token = blockIdx.x;
    float g = a.dy[token * a.dy_stride];
    if (a.count) g = *a.count > 0.0f ? g / *a.count : 0.0f;
    for (uint32_t c = 8u * (blockIdx.y * 256u + threadIdx.x); c < a.cols; c += 8u * 256u * gridDim.y) {
        const float *from = a.grad + static_cast<uint64_t>(token) * a.cols + c;
        float v[8];
        load_vec<float, 4>(from, *reinterpret_cast<float(*)[4]>(&v[0]));
        load_vec<float, 4>(from + 4, *reinterpret_cast<float(*)[4]>(&v[4]));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __float_as_uint(v[i]) == __float_as_uint(kNothing) ? 0.0f : v[i] * g;
        const uint64_t at = token * a.dx_stride + c;
        if (a.vec && a.dx_dtype == DF11_BF16) {
            store_vec<bf16_t, 8>(static_cast<bf16_t *>(a.dx) + at, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) store_as(a.dx, at + i, a.dx_dtype, v[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Host.

// Where a call's parts of the workspace begin.
struct LossPlan {
    bool slots;         // the fused product
    uint32_t piece;     // classes of a piece (the last one may have fewer)
    uint64_t weights, stats, rounded, logit, ref, sum, sum_rounded, scale, kept, exps, split, end;
};

// Classes of the piece that begins at class `from`.
uint32_t piece_at(uint32_t rows, uint32_t piece, uint32_t from) { return std::min(piece, rows - from); }

int loss_plan(const df11_device_stream *w, uint32_t tokens, bool grad, LossPlan &p) {
    const uint32_t cols = w->tile_cols, rows = static_cast<uint32_t>(w->h.n_elements / cols);
    p = LossPlan{};
    uint64_t at = 0;
    const auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    p.slots = !grad && tokens <= kPartialTokens;
    if (p.slots) {
        Partials parts{};
        if (df11::partial_products(&w, 1, nullptr, 0, tokens, nullptr, 0, nullptr, parts)) return DF11_E_HIP;
        p.weights = take(parts.slot_bytes);
    } else {
        p.weights = take(decoded_bytes(&w, 1));
    }
    p.logit = take(4ull * tokens);
    uint32_t most = rows;  // classes whose pairs are held at once
    if (!grad && !p.slots) {
        const int rc = df11::dense_fits(df11::kDenseStats, 1, tokens, rows, cols);
        if (rc) return rc;
    }
    if (grad) {
        if (tokens > kMaxGradTokens) return DF11_E_TOO_LARGE;
        // Pieces of about the same size.
        const uint64_t most_classes = std::max<uint64_t>(kLeastPiece, kPieceExps / tokens);
        const uint64_t pieces = (rows + most_classes - 1) / most_classes;
        p.piece = static_cast<uint32_t>(round_up((rows + pieces - 1) / pieces, 256));
        most = 0;
        uint64_t split = 0;
        for (uint32_t from = 0, n; from < rows; from += n) {
            n = piece_at(rows, p.piece, from);
            most = std::max(most, n);
            int rc = df11::dense_fits(df11::kDenseExp, 1, tokens, n, cols);
            if (!rc) rc = df11::dense_fits(df11::kDenseBackAdd, 1, tokens, n, cols);
            if (rc) return rc;
            const uint64_t more = df11::dense_workspace(df11::kDenseBackAdd, 1, tokens, n, cols);
            if (more == ~0ull) return DF11_E_HIP;
            split = std::max(split, more);
        }
        p.ref = take(4ull * tokens);
        p.sum = take(4ull * tokens);
        p.sum_rounded = take(4ull * tokens);
        p.rounded = take(4ull * (most / 64) * tokens);
        p.scale = take(4ull * tokens);
        p.kept = take(2ull * tokens * cols);
        p.exps = take(2ull * tokens * most);
        p.split = take(split);
    }
    p.stats = take(8ull * (most / 64) * tokens);
    p.end = at;
    return DF11_OK;
}

template <typename T>
T *at(void *workspace, uint64_t offset) {
    return reinterpret_cast<T *>(static_cast<uint8_t *>(workspace) + offset);
}

// The pairs of every panel, and the losses from them.
int loss_only(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t tokens, uint32_t cols,
              const LossPlan &p, TokenArgs t, void *ws, hipStream_t stream) {
    const uint32_t rows = static_cast<uint32_t>(w->h.n_elements / cols);
    int rc;
    if (p.slots) {
        Partials parts{};
        rc = df11::partial_products(&w, 1, x, x_stride, tokens, at<float>(ws, p.weights), p.logit - p.weights, stream, parts);
        if (rc) return rc;
        SlotLossArgs a{parts.s[0], at<float>(ws, p.weights), t.targets, at<float>(ws, p.stats), at<float>(ws, p.logit),
                       tokens, t.classes};
        void *params[] = {&a};
        // (tokens of a workgroup as for the products' sums, df11_product.hip)
        const bool one = tokens == 1 || static_cast<uint64_t>(rows / 64) * tokens <= 512;
        rc = launch_kernel(one ? reinterpret_cast<const void *>(&df11_loss_slots_kernel<1>)
                               : reinterpret_cast<const void *>(&df11_loss_slots_kernel<4>),
                           dim3(rows / 64, one ? tokens : (tokens + 3) / 4), dim3(256), params, 0, stream, nullptr, nullptr);
    } else {
        df11::DenseCall d{};
        rc = decode_weights(&w, 1, at<void>(ws, p.weights), d.w, stream);
        if (rc) return rc;
        d.mode = df11::kDenseStats;
        d.left[0] = x;
        d.left_stride = x_stride;
        d.tokens = tokens;
        d.rows = rows;
        d.cols = cols;
        d.loss.targets = t.targets;
        d.loss.stats = at<float>(ws, p.stats);
        d.loss.target_logit = at<float>(ws, p.logit);
        d.loss.classes = t.classes;
        rc = df11::dense_product(d, Epilogue{}, nullptr, stream);
    }
    if (rc) return rc;
    t.panels = rows / 64;
    void *params[] = {&t};
    // (in rows of 2^21 workgroups where one row of them would be too long for a launch)
    const uint32_t groups = (tokens + kTokens - 1) / kTokens, row = std::min(groups, 1u << 21);
    return launch_kernel(reinterpret_cast<const void *>(&df11_loss_tokens_kernel), dim3(row, (groups + row - 1) / row),
                         dim3(1024), params, 0, stream, nullptr, nullptr);
}

// Blocks of a token's columns, eight a thread.
uint32_t column_blocks(uint32_t cols) { return std::min(64u, (cols / 8 + 255) / 256); }

int loss_and_grad(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t tokens, uint32_t cols,
                  const LossPlan &p, TokenArgs t, float *grad, void *ws, hipStream_t stream) {
    const uint32_t rows = static_cast<uint32_t>(w->h.n_elements / cols);
    const uint16_t *decoded[2] = {};
    int rc = decode_weights(&w, 1, at<void>(ws, p.weights), decoded, stream);
    t.ref = at<float>(ws, p.ref);
    t.sum = at<float>(ws, p.sum);
    t.sum_rounded = at<float>(ws, p.sum_rounded);
    t.rounded = at<float>(ws, p.rounded);
    t.scale = at<float>(ws, p.scale);
    t.exps = at<uint16_t>(ws, p.exps);
    if (!rc) {
        const uint16_t *head = decoded[0];
        uint16_t *kept = at<uint16_t>(ws, p.kept);
        void *params[] = {&t, &x, &x_stride, &head, &cols, &kept};
        rc = launch_kernel(reinterpret_cast<const void *>(&df11_loss_first_kernel), dim3(tokens), dim3(256), params, 0,
                           stream, nullptr, nullptr);
    }
    for (uint32_t from = 0, n; !rc && from < rows; from += n) {
        n = piece_at(rows, p.piece, from);
        df11::DenseCall d{};
        d.mode = df11::kDenseExp;
        d.left[0] = x;
        d.left_stride = x_stride;
        d.w[0] = decoded[0] + static_cast<uint64_t>(from) * cols;  // (whole panels)
        d.tokens = tokens;
        d.rows = n;
        d.cols = cols;
        d.loss.targets = t.targets;
        d.loss.stats = at<float>(ws, p.stats);
        d.loss.target_logit = at<float>(ws, p.logit);
        d.loss.ref = t.ref;
        d.loss.rounded = at<float>(ws, p.rounded);
        d.loss.exps = t.exps;
        d.loss.exps_stride = n;
        d.loss.first_class = from;
        d.loss.classes = t.classes;
        rc = df11::dense_product(d, Epilogue{}, nullptr, stream);
        if (rc) break;
        t.panels = n / 64;
        t.exps_stride = n;
        uint32_t first = from == 0;
        void *params[] = {&t, &first};
        rc = launch_kernel(reinterpret_cast<const void *>(&df11_loss_piece_kernel), dim3((tokens + kTokens - 1) / kTokens), dim3(1024),
                           params, 0, stream, nullptr, nullptr);
        if (rc) break;
        d.mode = df11::kDenseBackAdd;
        d.left[0] = t.exps;
        d.left_stride = n;
        d.loss.scale = t.scale;
        Epilogue e{};
        e.out = grad;
        e.out_stride = cols;
        e.out_dtype = DF11_FP32;
        rc = df11::dense_product(d, e, at<float>(ws, p.split), stream);
    }
    if (rc) return rc;
    GradRowsArgs a{t, at<uint16_t>(ws, p.kept), grad, cols};
    void *params[] = {&a};
    return launch_kernel(reinterpret_cast<const void *>(&df11_loss_rows_kernel), dim3(tokens, column_blocks(cols)), dim3(256),
                         params, 0, stream, nullptr, nullptr);
}

int check_head(const df11_device_stream *w, uint32_t n_tokens, uint32_t in_features, uint32_t out_features) {
    if (!w) return DF11_E_INVALID_ARG;
    const int rc = df11::check_stream(w);
    if (rc) return rc;
    if (in_features < 32 || in_features % 32 || !out_features || out_features % kPanelRows ||
        static_cast<uint64_t>(in_features) * out_features != w->h.n_elements || w->tile_cols != in_features)
        return DF11_E_INVALID_ARG;
    if (in_features > kMaxRow || out_features > kMaxRow || static_cast<uint64_t>(n_tokens) * in_features >= (1ull << 32))
        return DF11_E_TOO_LARGE;
    return DF11_OK;
}

}  // namespace

extern "C" {

uint64_t df11_cross_entropy_workspace(const df11_device_stream *w, uint32_t n_tokens, int with_grad) {
    LossPlan p{};
    if (!w || !n_tokens || df11::check_stream(w) || !w->h.n_elements || !w->tile_cols) return 0;
    const uint64_t rows = w->h.n_elements / w->tile_cols;
    if (rows > kMaxRow || check_head(w, n_tokens, w->tile_cols, static_cast<uint32_t>(rows))) return 0;
    return loss_plan(w, n_tokens, with_grad != 0, p) ? 0 : p.end;
}

int df11_cross_entropy(const df11_device_stream *w, const uint16_t *x, uint64_t x_stride, uint32_t n_tokens,
                       uint32_t in_features, uint32_t out_features, const df11_loss *l, void *workspace,
                       uint64_t workspace_bytes, void *hip_stream) {
    int rc = check_head(w, n_tokens, in_features, out_features);
    if (rc) return rc;
    if (!l || !l->vocab || l->vocab > out_features || l->mean > 1 || (l->total && !aligned(l->total, 4)) ||
        (l->count && !aligned(l->count, 4)))
        return DF11_E_INVALID_ARG;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const uint64_t grad_span = l->grad ? 4ull * n_tokens * in_features : 0;
    if (n_tokens) {
        if (!x || !aligned(x, 16) || x_stride % 8 || x_stride > kMaxRow || !l->targets || !aligned(l->targets, 8) ||
            !l->loss || !aligned(l->loss, 4) || (l->grad && !aligned(l->grad, 16)))
            return DF11_E_INVALID_ARG;
    }
    // Everything that is written lies apart from the rest.
    const uint64_t x_span = n_tokens ? 2 * ((n_tokens - 1ull) * x_stride + in_features) : 0;
    const void *outs[] = {l->loss, l->total, l->count, l->grad, workspace};
    uint64_t spans[] = {4ull * n_tokens, l->total ? 4ull : 0ull, l->count ? 4ull : 0ull, grad_span, 0};
    const auto clear = [&](int i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], spans[i], outs[j], spans[j])) return false;
        return !overlaps(outs[i], spans[i], x, x_span) && !overlaps(outs[i], spans[i], l->targets, 8ull * n_tokens) &&
               !df11::stream_overlaps(w, outs[i], spans[i]);
    };
    for (int i = 0; i < 4; ++i)
        if (!clear(i)) return DF11_E_INVALID_ARG;
    (void)hipGetLastError();
    if (n_tokens) {
        LossPlan p{};
        rc = loss_plan(w, n_tokens, l->grad != nullptr, p);
        if (rc) return rc;
        if (!workspace || !aligned(workspace, 256)) return DF11_E_INVALID_ARG;
        if (workspace_bytes < p.end) return DF11_E_BUFFER_TOO_SMALL;
        spans[4] = p.end;
        if (!clear(4)) return DF11_E_INVALID_ARG;
        TokenArgs t{};
        t.targets = l->targets;
        t.ignore_index = l->ignore_index;
        t.stats = at<float>(workspace, p.stats);
        t.target_logit = at<float>(workspace, p.logit);
        t.loss = l->loss;
        t.n_tokens = n_tokens;
        t.classes = l->vocab;
        rc = l->grad ? loss_and_grad(w, x, x_stride, n_tokens, in_features, p, t, l->grad, workspace, stream)
                     : loss_only(w, x, x_stride, n_tokens, in_features, p, t, workspace, stream);
        if (rc) return rc;
    }
    if (!l->total && !l->count) return DF11_OK;
    const float *loss = l->loss;
    const int64_t *targets = l->targets;
    int64_t ignore_index = l->ignore_index;
    uint32_t n = n_tokens, mean = l->mean;
    float *total = l->total, *count = l->count;
    void *params[] = {&loss, &targets, &ignore_index, &n, &mean, &total, &count};
    return launch_kernel(reinterpret_cast<const void *>(&df11_loss_total_kernel), dim3(1), dim3(1024), params, 0, stream,
                         nullptr, nullptr);
}

int df11_cross_entropy_grad(const float *grad, const float *dy, uint64_t dy_stride, const float *count,
                            uint32_t n_tokens, uint32_t in_features, void *dx, uint64_t dx_stride, uint32_t dx_dtype,
                            void *hip_stream) {
    const uint32_t bytes = dx_dtype == DF11_FP16 ? 0 : dtype_bytes(dx_dtype);
    if (!bytes || in_features < 32 || in_features % 32) return DF11_E_INVALID_ARG;
    if (in_features > kMaxRow || static_cast<uint64_t>(n_tokens) * in_features >= (1ull << 32) || n_tokens > kMaxGradTokens)
        return DF11_E_TOO_LARGE;
    if (!n_tokens) return DF11_OK;
    if (!grad || !aligned(grad, 16) || !dy || !aligned(dy, 4) || dy_stride > (1ull << 31) || !dx || !aligned(dx, bytes) ||
        dx_stride > (1ull << 31) || (n_tokens > 1 && dx_stride < in_features) || (count && !aligned(count, 4)))
        return DF11_E_INVALID_ARG;
    const uint64_t span = ((n_tokens - 1ull) * dx_stride + in_features) * bytes;
    if (overlaps(dx, span, grad, 4ull * n_tokens * in_features) ||
        overlaps(dx, span, dy, 4 * ((n_tokens - 1ull) * dy_stride + 1)) || overlaps(dx, span, count, count ? 4 : 0))
        return DF11_E_INVALID_ARG;
    LossGradArgs a{grad, dy, count, dx, dy_stride, dx_stride, in_features, dx_dtype,
                   aligned(dx, 16) && dx_stride % 8 == 0 ? 1u : 0u};
    (void)hipGetLastError();
    void *params[] = {&a};
    return launch_kernel(reinterpret_cast<const void *>(&df11_loss_grad_kernel), dim3(n_tokens, column_blocks(in_features)),
                         dim3(256), params, 0, static_cast<hipStream_t>(hip_stream), nullptr, nullptr);
}

}  // extern "C"
