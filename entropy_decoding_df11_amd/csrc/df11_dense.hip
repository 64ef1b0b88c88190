// The dense products of df11_dense.h on the matrix cores (gfx950).
//
// A workgroup computes a tile of BM tokens x BN outputs in steps of 64 along
// K, from two LDS buffers that buffer_load ... lds fills without registers.
// A step has two halves of 32.  While the waves multiply the first half, they
// read the second half's operands from LDS; then one wait and one barrier
// (the next step has landed, and every wave has read all of this one); while
// they multiply the second half, the step after the next is sent for into
// the buffer just read, and the next step's first operands are read.  Loads
// thus have a whole step to land, and LDS reads half a step.
//
// Weights arrive in MFMA tile order: a 1 KB block is the operand of one
// v_mfma_f32_16x16x32_bf16 for 16 rows x 32 columns of W, lane l's 16 bytes
// at 16 l, so both the loads and the LDS reads of the forward product are
// linear.  The left operand's rows are 128 bytes in LDS, their eight 16-byte
// chunks permuted by the row (chunk c at c ^ (row mod 8)), which spreads the
// rows of an operand over all banks.  The backward product needs the
// transpose of the same blocks: column n of W, 8 consecutive rows, which
// ds_read_b64_tr_b16 gathers from 4 rows x 16 columns at a time.
//
// Rows past the last token and outputs past the last row of W lie past the
// end of their buffer resource by the lane's own offset, and are not read
// (df11_dense_tiles.h); what their places in LDS hold reaches no output.
//
// What the forms tried on a full chip showed: 4096 tokens, 14336 -> 4096 take
// 415 us (1.16 PFLOP/s) on random operands and 295 us (1.63 PFLOP/s) on
// zeros, with the same instructions, so the operands' values, and with them
// the clock that the power allows, decide; the MFMAs alone, without loads or
// LDS reads, take 264.  Every other form ends within 3% of the same time: four
// waves of 128 x 128 with the accumulators pinned by hand (which read a third
// less from LDS) 411 to 418 us, half-steps of 32 in a ring of four or five
// buffers 417 and 419, v_mfma_f32_32x32x16_bf16 416.  (Operands of W straight
// from memory to registers double the L1's traffic: 445.)  It is no limit of
// the card: the library's product of 1999 tokens, 4096 -> 28672 takes 339 us
// where this one takes 393 to 434 at MFMAs 64% busy.  What is left to look
// into is the work beside the MFMAs (595 MB read for 218 MB of operands; a
// quarter of the backward product's LDS reads in conflict).  With a fifth of
// the CUs busy a step of 256 x 256 takes 1.2 us against 0.85 of MFMAs.  128 x 128 tiles (two workgroups a CU, a quarter more LDS traffic a
// MFMA) take 505 us on that product and win where 256 x 256 leave CUs idle
// (2048 tokens, 4096 -> 4096: 64 against 92 us).  Tiles between the two, 128 x
// 256 or 256 x 128 in four waves, win nowhere (the same product 10 and 14 us
// more than 128 x 128): one wave a SIMD waits for its LDS reads.
#include <hip/hip_runtime.h>

#include <algorithm>

#include <stdint.h>

#include "df11.h"
#include "df11_dense.h"
#include "df11_dense_tiles.h"
#include "df11_device.h"

namespace {

using df11::DenseCall;
using df11::DenseMode;
using df11::kDenseBack;
using df11::kDenseGated;
using df11::kDensePlain;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
using Resource = __amdgpu_buffer_rsrc_t;

constexpr uint32_t kStep = df11::kDenseStep;
// Token tiles that follow each other before the next output tile: an XCD's 32
// (or 64) tiles at a time then read fewest distinct rows and columns.  8192
// tokens, 4096 -> 4096: 227 us against 241 without bands (128 x 128 tiles 263
// against 318); bands of 4 and 16 take 228 and 225 (266 and 276).
constexpr uint32_t kBand = 8;

struct DenseArgs {
    const uint16_t *left[2];
    const uint16_t *w[2];
    uint64_t left_stride;
    float *partial;        // split: [split][matrix][token][output]
    uint32_t tokens;
    uint32_t n_out;        // outputs per token
    uint32_t out0;         // first output of this launch
    uint32_t tile_ks;      // C / 32
    uint32_t panels;       // R / 64
    uint32_t k_steps;      // steps along K, all matrices of a backward product
    uint32_t k_steps_one;  // steps of one matrix
    uint32_t m_tiles, splits;
    uint32_t vec;          // the epilogue's out and residual allow 16-byte vectors
    Epilogue e;
};

// A buffer resource over a window of the operand at p (nothing past it is read).
__device__ __forceinline__ Resource resource(const uint16_t *p, df11::DenseWindow w) {
    const uint32_t n = w.bytes > 0xFFFFFFFFull ? 0xFFFFFFFFu : static_cast<uint32_t>(w.bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p + w.at / 2u), 0, n, 0x00020000);
}

// 16 bytes a lane from r, lane_at bytes on, to the wave-uniform LDS address
// dst + 16 lane.  (No scalar offset: df11_dense_tiles.h.)
__device__ __forceinline__ void load_to_lds(Resource r, uint8_t *dst, uint32_t lane_at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, lane_at, 0, 0, 0);
}

// Four rows x 16 columns of 2-byte elements, transposed across a quarter
// wave: lane i of the quarter passes the address of row i / 4, columns
// 4 (i mod 4) .. + 3, and receives column i of the four rows.
__device__ __forceinline__ shortx4 read_transposed(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4 *)p);
}

// Eight consecutive elements; `vec`: 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        load_vec<T, 4>(p, *reinterpret_cast<float(*)[4]>(&f[0]));
        load_vec<T, 4>(p + 4, *reinterpret_cast<float(*)[4]>(&f[4]));
    } else {
        load_vec<T, 8>(p, f);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        store_vec<T, 4>(p, *reinterpret_cast<const float(*)[4]>(&f[0]));
        store_vec<T, 4>(p + 4, *reinterpret_cast<const float(*)[4]>(&f[4]));
    } else {
        store_vec<T, 8>(p, f);
    }
}

__device__ __forceinline__ void load8_as(const void *p, uint64_t i, uint32_t dtype, bool vec, float (&f)[8]) {
    if (vec && dtype == DF11_FP32) {
        load8(static_cast<const float *>(p) + i, f);
    } else if (vec) {
        load8(static_cast<const bf16_t *>(p) + i, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = load_as(p, i + e, dtype);
    }
}

__device__ __forceinline__ void store8_as(void *p, uint64_t i, uint32_t dtype, bool vec, const float (&f)[8]) {
    if (vec && dtype == DF11_FP32) {
        store8(static_cast<float *>(p) + i, f);
    } else if (vec) {
        store8(static_cast<bf16_t *>(p) + i, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) store_as(p, i + e, dtype, f[e]);
    }
}

// The biases of eight outputs from col on.
template <int MODE>
__device__ __forceinline__ void load_biases(const DenseArgs &a, uint32_t col, float (&b0)[8], float (&b1)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b0[i] = b1[i] = 0.0f;
    if (a.e.bias[0]) load8_as(a.e.bias[0], col, a.e.bias_dtype, false, b0);
    if (MODE == kDenseGated && a.e.bias[1]) load8_as(a.e.bias[1], col, a.e.bias_dtype, false, b1);
}

// Eight sums of one token to their place (z0 and z1 without the biases).
template <uint32_t ACT, int MODE>
__device__ __forceinline__ void finish8(const DenseArgs &a, uint32_t token, uint32_t col, float (&z0)[8],
                                        float (&z1)[8], const float (&b0)[8], const float (&b1)[8]) {
    constexpr bool kGated = MODE == kDenseGated;
    const Epilogue &e = a.e;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z0[i] += b0[i];
        if constexpr (kGated) z1[i] += b1[i];
    }
    if (e.pre[0]) {
        store8(e.pre[0] + static_cast<uint64_t>(token) * a.n_out + col, z0);
        if constexpr (kGated) store8(e.pre[1] + static_cast<uint64_t>(token) * a.n_out + col, z1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = activate(ACT, z0[i]);
        if constexpr (kGated) y[i] *= z1[i];
    }
    if (e.residual) {
        float r[8];
        load8_as(e.residual, token * e.residual_stride + col, e.residual_dtype, a.vec, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += r[i];
    }
    store8_as(e.out, token * e.out_stride + col, e.out_dtype, a.vec, y);
}

// f.template operator()<ACT>() for the epilogue's activation: one branch
// around the loop over a tile's rows (a branch at every element took longer
// than the product's last steps).
template <int MODE, typename F>
__device__ __forceinline__ void with_activation(uint32_t act, F f) {
    switch (MODE == kDenseBack ? DF11_ACT_NONE : act) {
    case DF11_ACT_RELU: f.template run<DF11_ACT_RELU>(); break;
    case DF11_ACT_SILU: f.template run<DF11_ACT_SILU>(); break;
    case DF11_ACT_GELU: f.template run<DF11_ACT_GELU>(); break;
    case DF11_ACT_GELU_TANH: f.template run<DF11_ACT_GELU_TANH>(); break;
    default: f.template run<DF11_ACT_NONE>(); break;
    }
}

// The rows of a wave's staged sums (kStride floats a row, kOut outputs, of a
// gated product twice) through the epilogue, eight outputs a lane.
template <int MODE, int kStride, int kOut>
struct StagedRows {
    const DenseArgs &a;
    const float *staged;
    uint32_t rows, token0, col0, lane;

    template <uint32_t ACT>
    __device__ __forceinline__ void run() const {
        constexpr uint32_t kLanes = kOut / 8, kRows = kWaveSize / kLanes;
        const uint32_t c = 8u * (lane % kLanes), col = col0 + c;
        if (col >= a.n_out) return;
        float b0[8], b1[8];
        load_biases<MODE>(a, col, b0, b1);
#pragma unroll 2
        for (uint32_t r = lane / kLanes; r < rows; r += kRows) {
            if (token0 + r >= a.tokens) break;
            float z0[8], z1[8];
            load8(staged + r * kStride + c, z0);
            if constexpr (MODE == kDenseGated) load8(staged + r * kStride + kOut + c, z1);
            finish8<ACT, MODE>(a, token0 + r, col, z0, z1, b0, b1);
        }
    }
};

// Passes in which the waves' sums go through LDS (at most 140 KB at a time).
template <int W, int TM, int TN>
constexpr int kStagePasses = (W * TM * 16 * (TN * 16 + 4) * 4 + 139999) / 140000;

// Lane l holds outputs 4 (l / 16) .. + 3 of each block of 16 for token
// l mod 16; through LDS, eight consecutive outputs come to one lane and a
// token's outputs to neighbouring lanes.
// (P: the pass, a template argument so that the sums keep their registers.)
template <int P, int W, int TM, int TN, int MODE>
__device__ __forceinline__ void write_tile(const DenseArgs &a, const floatx4 (&acc)[TM][TN], uint8_t *lds,
                                           uint32_t wave, uint32_t lane, uint32_t token0, uint32_t col0,
                                           uint32_t split) {
    constexpr int kPasses = kStagePasses<W, TM, TN>, TP = TM / kPasses;
    static_assert(TP * kPasses == TM, "passes of whole token tiles");
    constexpr int kStride = TN * 16 + 4, kOut = MODE == kDenseGated ? TN * 8 : TN * 16;
    float *staged = reinterpret_cast<float *>(lds) + wave * (TP * 16 * kStride);
    const uint32_t quarter = lane >> 4, l16 = lane & 15u;
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<floatx4 *>(staged + (16 * i + l16) * kStride + 16 * j + 4 * quarter) =
                acc[P * TP + i][j];
    const uint32_t t0 = token0 + P * TP * 16;
    if (a.splits > 1u) {
        constexpr uint32_t kMats = MODE == kDenseGated ? 2u : 1u, kLanes = kOut / 4;
        const uint32_t c = 4u * (lane % kLanes);
        for (uint32_t r = lane / kLanes; r < TP * 16u; r += kWaveSize / kLanes) {
            if (t0 + r >= a.tokens || col0 + c >= a.n_out) break;
            float *q = a.partial + (static_cast<uint64_t>(split) * kMats * a.tokens + t0 + r) * a.n_out + col0 + c;
            *reinterpret_cast<floatx4 *>(q) = *reinterpret_cast<const floatx4 *>(staged + r * kStride + c);
            if constexpr (MODE == kDenseGated)
                *reinterpret_cast<floatx4 *>(q + static_cast<uint64_t>(a.tokens) * a.n_out) =
                    *reinterpret_cast<const floatx4 *>(staged + r * kStride + kOut + c);
        }
    } else {
        with_activation<MODE>(a.e.act, StagedRows<MODE, kStride, kOut>{a, staged, TP * 16u, t0, col0, lane});
    }
    if constexpr (P + 1 < kPasses) write_tile<P + 1, W, TM, TN, MODE>(a, acc, lds, wave, lane, token0, col0, split);
}

// Asks the scheduler to spread R LDS reads and L loads between M MFMAs
// instead of issuing them in a block, which the waves of a CU would do all
// at the same time.
template <int R, int M, int L>
__device__ __forceinline__ void interleave() {
    constexpr int kEach = (M * 3 / 4) / (R + L) > 0 ? (M * 3 / 4) / (R + L) : 1;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);     // a vector memory read
        __builtin_amdgcn_sched_group_barrier(0x8, kEach, 0);  // MFMAs
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
        __builtin_amdgcn_sched_group_barrier(0x8, kEach, 0);
    }
    if constexpr (M > kEach * (R + L)) __builtin_amdgcn_sched_group_barrier(0x8, M - kEach * (R + L), 0);
}

// WM x WN waves, each TM token tiles x TN output blocks of 16.
template <int WM, int WN, int TM, int TN>
constexpr int kDenseWavesPerSimd = (WM * TM + WN * TN) * 16 * 256 <= 65536 ? WM * WN / 2 : WM * WN / 4;

template <int WM, int WN, int TM, int TN, int MODE>
__global__ __launch_bounds__(64 * WM * WN)
__attribute__((amdgpu_waves_per_eu(kDenseWavesPerSimd<WM, WN, TM, TN>)))
void df11_dense_kernel(DenseArgs a) {
    constexpr int W = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
    constexpr uint32_t kOut = MODE == kDenseGated ? BN / 2 : BN;  // outputs of a tile
    constexpr int kLeftLoads = BM / 8 / W, kRightLoads = BN / 8 / W;
    constexpr int kLeftBytes = BM * 128, kStageBytes = (BM + BN) * 128;
    constexpr int kStaged = W * (TM / kStagePasses<W, TM, TN>) * 16 * (TN * 16 + 4) * 4;
    constexpr int kReads = MODE == kDenseBack ? TM + 2 * TN : TM + TN;
    __shared__ __align__(1024) uint8_t s_mem[2 * kStageBytes > kStaged ? 2 * kStageBytes : kStaged];

    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t wm = wave / WN, wn = wave % WN;

    // Tiles in runs per XCD (workgroup i runs on XCD i mod 8), in bands of up
    // to kBand token tiles: the tiles that an XCD works on at once then share
    // both their tokens and their part of W in its L2.
    const uint32_t total = gridDim.x, xcd = blockIdx.x % 8u, q = total / 8u, rest = total % 8u;
    const uint32_t tile = xcd * q + min(xcd, rest) + blockIdx.x / 8u;
    const uint32_t columns = total / a.m_tiles;  // output tiles times splits
    const uint32_t band = tile / (kBand * columns), in_band = tile % (kBand * columns);
    const uint32_t high = min(kBand, a.m_tiles - band * kBand);
    const uint32_t m_tile = band * kBand + in_band % high, column = in_band / high;
    const uint32_t split = column % a.splits, n_tile = column / a.splits;
    const uint32_t m0 = m_tile * BM, n0 = a.out0 + n_tile * kOut;
    // (every split has a step: the host gives no more splits than steps)
    const uint32_t k_begin = static_cast<uint32_t>(static_cast<uint64_t>(split) * a.k_steps / a.splits);
    const uint32_t k_end = static_cast<uint32_t>(static_cast<uint64_t>(split + 1u) * a.k_steps / a.splits);
    const uint64_t panel_bytes = static_cast<uint64_t>(a.tile_ks) * 4096u;

    const uint32_t rows_here = min(static_cast<uint32_t>(BM), a.tokens - m0);
    const uint32_t k_len = MODE == kDenseBack ? a.panels * 64u : a.tile_ks * 32u;
    const uint32_t stride = static_cast<uint32_t>(a.left_stride);
    const uint32_t left_at = df11::dense_left_lane(lane, stride);

    // Sends for one step.  (Forward, an odd last k-step: the upper half of
    // the step holds whatever follows, and its products are left out.)
    auto issue = [&](uint32_t step, uint8_t *stage) {
        const uint32_t one = MODE == kDenseBack && step >= a.k_steps_one ? 1u : 0u;
        const uint32_t ks = step - one * a.k_steps_one;  // step of this matrix
        const Resource left = resource(a.left[one], df11::dense_left_window(m0, rows_here, a.left_stride, k_len, ks));
#pragma unroll
        for (int i = 0; i < kLeftLoads; ++i)
            load_to_lds(left, stage + 1024u * (wave + W * i), left_at + df11::dense_left_group(wave + W * i, stride));
        stage += kLeftBytes;
        if constexpr (MODE == kDenseBack) {
            const Resource w = resource(a.w[one], df11::dense_back_window(n0, ks, panel_bytes));
#pragma unroll
            for (int i = 0; i < kRightLoads; ++i)
                load_to_lds(w, stage + 1024u * (wave + W * i), 16u * lane + df11::dense_back_block(wave + W * i));
        } else {
            const df11::DenseWindow window = df11::dense_right_window(n0, ks, a.panels, panel_bytes);
            const Resource w0 = resource(a.w[0], window);
            const Resource w1 = MODE == kDenseGated ? resource(a.w[1], window) : w0;
#pragma unroll
            for (int i = 0; i < kRightLoads; ++i) {
                const uint32_t b = wave + W * i, half = b / (BN / 16u), nb = b % (BN / 16u);
                // Of a gated product, the first half of each wave's blocks is
                // the gate's, the second up's (a tile may begin inside a panel).
                const bool second = MODE == kDenseGated && nb % TN >= TN / 2;
                const uint32_t r16 = MODE == kDenseGated
                                         ? (n0 & 63u) / 16u + (nb / TN) * (TN / 2) + nb % (TN / 2)
                                         : nb;
                load_to_lds(second ? w1 : w0, stage + 1024u * b,
                            16u * lane + df11::dense_right_block(r16, half, static_cast<uint32_t>(panel_bytes)));
            }
        }
    };

    floatx4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    // This lane's operands in a stage: tokens l mod 16 of each tile, chunk
    // 4 half + l / 16 of K; of W the same K.
    const uint32_t quarter = lane >> 4, l16 = lane & 15u;
    const uint32_t x_at = 128u * (wm * TM * 16u + l16) + 16u * (quarter ^ (l16 & 7u));
    const uint32_t w_at =
        kLeftBytes + (MODE == kDenseBack ? 1024u * (2u * TN * wn + (quarter >> 1)) + 8u * (l16 & 1u) +
                                               16u * (16u * ((l16 >> 1) & 1u) + 8u * (quarter & 1u) + (l16 >> 2))
                                         : 1024u * TN * wn + 16u * lane);
    auto read = [&](const uint8_t *stage, int half, bf16x8 (&fx)[TM], bf16x8 (&fw)[TN]) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (MODE == kDenseBack) {
                // outputs 16 (j mod 2) .. of k-step TN / 2 wn + j / 2; rows 32 half + 8 quarter ..
                const uint8_t *p = stage + w_at + 1024u * (4u * (j / 2) + 2u * half) + 512u * (j & 1);
                union {
                    shortx4 s[2];
                    bf16x8 v;
                } u;
                u.s[0] = read_transposed(p);
                u.s[1] = read_transposed(p + 64);  // four rows on
                fw[j] = u.v;
            } else {
                fw[j] = *reinterpret_cast<const bf16x8 *>(stage + w_at + 1024u * (half * (BN / 16) + j));
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fx[i] = *reinterpret_cast<const bf16x8 *>(stage + (x_at ^ (64u * half)) + 2048u * i);
    };
    auto multiply = [&](const bf16x8 (&fx)[TM], const bf16x8 (&fw)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[j], fx[i], acc[i][j], 0, 0, 0);
    };

    bf16x8 fx0[TM], fw0[TN], fx1[TM], fw1[TN];
    uint8_t *cur = s_mem, *next = s_mem + kStageBytes;
    auto first_half = [&]() {
        read(cur, 1, fx1, fw1);
        multiply(fx0, fw0);
        interleave<kReads, TM * TN, 0>();
        __builtin_amdgcn_sched_barrier(0);
    };
    // (steps past the last one are sent for again and never multiplied, so
    // that the counts of loads in flight are the same on every path)
    issue(k_begin, cur);
    issue(min(k_begin + 1u, k_end - 1u), next);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeftLoads + kRightLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(cur, 0, fx0, fw0);
    const bool odd = MODE != kDenseBack && (a.tile_ks & 1u) && k_end == a.k_steps;
    const uint32_t k_full = odd ? k_end - 1u : k_end;
    for (uint32_t step = k_begin; step < k_full; ++step) {
        first_half();
        // The next step has landed; this wave's reads of this one are back.
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(min(step + 2u, k_end - 1u), cur);
        read(next, 0, fx0, fw0);
        multiply(fx1, fw1);
        interleave<kReads, TM * TN, kLeftLoads + kRightLoads>();
        __builtin_amdgcn_sched_barrier(0);
        uint8_t *t = cur;
        cur = next;
        next = t;
    }
    if (odd) first_half();
    // (no load may land in LDS that the sums, or another workgroup, now use)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    write_tile<0, W, TM, TN, MODE>(a, acc, s_mem, wave, lane, m0 + wm * (TM * 16u),
                                n0 + wn * (MODE == kDenseGated ? TN * 8u : TN * 16u), split);
}

// Adds the splits' partial sums in order and applies the epilogue.
template <int MODE>
struct SplitRows {
    const DenseArgs &a;

    template <uint32_t ACT>
    __device__ __forceinline__ void run() const {
        constexpr uint32_t kMats = MODE == kDenseGated ? 2u : 1u;
        const uint32_t per_row = a.n_out / 8u;
        const uint64_t total = static_cast<uint64_t>(a.tokens) * per_row;
        const uint64_t plane = static_cast<uint64_t>(a.tokens) * a.n_out;
        for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
            const uint32_t token = static_cast<uint32_t>(i / per_row), col = 8u * static_cast<uint32_t>(i % per_row);
            float z[2][8], b0[8], b1[8];
            for (uint32_t m = 0; m < kMats; ++m) {
                const float *p = a.partial + m * plane + static_cast<uint64_t>(token) * a.n_out + col;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[m][e] = 0.0f;
                // (four splits' loads in flight; past the last one again, not added)
                for (uint32_t s = 0; s < a.splits; s += 4u) {
                    float more[4][8];
#pragma unroll
                    for (uint32_t k = 0; k < 4u; ++k) load8(p + min(s + k, a.splits - 1u) * kMats * plane, more[k]);
#pragma unroll
                    for (uint32_t k = 0; k < 4u; ++k)
                        if (s + k < a.splits)
#pragma unroll
                            for (int e = 0; e < 8; ++e) z[m][e] += more[k][e];
                }
            }
            load_biases<MODE>(a, col, b0, b1);
            finish8<ACT, MODE>(a, token, col, z[0], z[1], b0, b1);
        }
    }
};

template <int MODE>
__global__ __launch_bounds__(256) void df11_dense_sum_kernel(DenseArgs a) {
    with_activation<MODE>(a.e.act, SplitRows<MODE>{a});
}

// How a product is launched: outputs [0, large_out) in 256 x 256 tiles (one
// workgroup a CU), the rest in 128 x 128 tiles (two); all of it in one kind
// of tile if it is split along K.
struct DensePlan {
    uint32_t large_out;
    uint32_t splits;
};

// Picks the plan with the least time, by times in microseconds on 256 CUs
// fitted to 2400 products (33 to 2048 tokens, 640 to 14336 features, both
// kinds of tile in 1 to 32 splits): a round of small tiles takes 2.7 and, a
// step, 0.94 with two workgroups a CU and 0.72 with one (backward 4.4, 1.12
// and 0.97), a round of large tiles 4.5 and, a step, 1.25 (backward 6, and 1.9
// or, half of the CUs busy, 1.7); a split product writes and reads its partial
// sums at 6 TB/s, much of it cached, and takes 1.5 and 0.2 a split for the
// second kernel.  On the products of the fit the plan taken so is on average
// 0.4% slower than the best one tried (backward 0.2%), 5% at most; the plans
// of large tiles with a rest of small ones were not among them.  The times
// rank plans and foretell none: fitted to short runs, they fall short of long
// products on a full chip, whose steps of large tiles take 1.43 to 1.84 us
// (4096 tokens, 14336 -> 4096: 285 us here, 415 measured; in small tiles 426
// and 505), so that there the choice leans to large tiles.
DensePlan dense_plan(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols, int cus) {
    const bool back = mode == kDenseBack;
    const uint64_t n_out = back ? cols : rows, mats = mode == kDenseGated ? 2 : 1, room = static_cast<uint64_t>(cus);
    const uint32_t k_steps = back ? n * (rows / kStep) : (cols + kStep - 1) / kStep;
    const double large = back ? 6.0 : 4.5, large_full = back ? 1.9 : 1.25, large_half = back ? 1.7 : 1.25;
    const double small = back ? 4.4 : 2.7, small_full = back ? 1.12 : 0.94, small_half = back ? 0.97 : 0.72;
    const auto tiles = [&](uint64_t edge, uint64_t outs) {
        return (tokens + edge - 1) / edge * ((outs * mats + edge - 1) / edge);
    };
    // Time of `count` workgroups, `most` at once, each with `steps` steps.
    const auto time = [&](uint64_t count, uint64_t most, double base, double full, double half, double steps) {
        const uint64_t rest = count % most;
        return (count / most) * (base + full * steps) +
               (rest ? base + (2 * rest > most ? full : half) * steps : 0.0);
    };
    DensePlan best{0, 1};
    double least = 1e30;
    const auto consider = [&](double t, DensePlan p) {
        if (t < least) {
            least = t;
            best = p;
        }
    };
    for (uint32_t splits = 1; splits <= 32 && splits <= k_steps; splits *= 2) {
        const double steps = (k_steps + splits - 1) / splits;
        const double sum = splits > 1 ? 1.5 + 0.2 * splits + 8.0 * splits * mats * tokens * n_out / 6e6 : 0.0;
        consider(sum + time(tiles(128, n_out) * splits, 2 * room, small, small_full, small_half, steps), {0, splits});
        consider(sum + time(tiles(256, n_out) * splits, room, large, large_full, large_half, steps),
                 {static_cast<uint32_t>(n_out), splits});
    }
    // Whole rounds of large tiles, the rest small.
    const uint64_t m_tiles = (tokens + 255ull) / 256, outs = 256 / mats, n_tiles = (n_out + outs - 1) / outs;
    const uint64_t whole = m_tiles * n_tiles / room * room / m_tiles;
    if (whole && whole < n_tiles)
        consider(time(whole * m_tiles, room, large, large_full, large_half, k_steps) +
                     time(tiles(128, n_out - whole * outs), 2 * room, small, small_full, small_half, k_steps),
                 {static_cast<uint32_t>(whole * outs), 1});
    return best;
}

template <int WM, int WN, int TM, int TN>
const void *dense_kernel(DenseMode mode) {
    switch (mode) {
    case kDenseGated: return reinterpret_cast<const void *>(&df11_dense_kernel<WM, WN, TM, TN, kDenseGated>);
    case kDenseBack: return reinterpret_cast<const void *>(&df11_dense_kernel<WM, WN, TM, TN, kDenseBack>);
    default: return reinterpret_cast<const void *>(&df11_dense_kernel<WM, WN, TM, TN, kDensePlain>);
    }
}

}  // namespace

namespace df11 {

uint64_t dense_workspace(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols) {
    int dev = 0, cus = 0;
    if (device_cus(dev, cus)) return ~0ull;
    const DensePlan p = dense_plan(mode, n, tokens, rows, cols, cus);
    const uint64_t mats = mode == kDenseGated ? 2 : 1, n_out = mode == kDenseBack ? cols : rows;
    return p.splits > 1 ? 4ull * p.splits * mats * tokens * n_out : 0;
}

int dense_product(const DenseCall &c, const Epilogue &e, float *workspace, hipStream_t stream) {
    int dev = 0, cus = 0;
    if (device_cus(dev, cus)) return DF11_E_HIP;
    const uint32_t n = c.mode == kDensePlain || (c.mode == kDenseBack && !c.w[1]) ? 1 : 2;
    const DensePlan p = dense_plan(c.mode, n, c.tokens, c.rows, c.cols, cus);
    const uint32_t one = c.mode == kDenseBack ? c.rows / kStep : (c.cols + kStep - 1) / kStep;
    DenseArgs a{};
    for (int i = 0; i < 2; ++i) {
        a.left[i] = c.left[i];
        a.w[i] = c.w[i];
    }
    a.left_stride = c.left_stride;
    a.partial = workspace;
    a.tokens = c.tokens;
    a.n_out = c.mode == kDenseBack ? c.cols : c.rows;
    a.tile_ks = c.cols / 32;
    a.panels = c.rows / 64;
    a.k_steps = c.mode == kDenseBack ? n * one : one;
    a.k_steps_one = one;
    a.e = e;
    const uint32_t out_bytes = dtype_bytes(e.out_dtype), res_bytes = dtype_bytes(e.residual_dtype);
    a.vec = aligned(e.out, 16) && e.out_stride * out_bytes % 16 == 0 &&
            (!e.residual || (aligned(e.residual, 16) && e.residual_stride * res_bytes % 16 == 0));
    (void)hipGetLastError();
    void *params[] = {&a};
    a.splits = p.splits;
    // Outputs [from, to) in tiles of `edge` tokens.
    const auto part = [&](uint32_t edge, uint32_t from, uint32_t to) {
        const uint32_t outs = c.mode == kDenseGated ? edge / 2 : edge;
        a.out0 = from;
        a.m_tiles = (a.tokens + edge - 1) / edge;
        return launch_kernel(edge == 256 ? dense_kernel<2, 4, 8, 4>(c.mode) : dense_kernel<2, 2, 4, 4>(c.mode),
                             dim3(a.m_tiles * ((to - from + outs - 1) / outs) * p.splits), dim3(2 * edge), params, 0,
                             stream, nullptr, nullptr);
    };
    int rc = DF11_OK;
    if (p.large_out) rc = part(256, 0, p.large_out);
    if (!rc && p.large_out < a.n_out) rc = part(128, p.large_out, a.n_out);
    if (rc || p.splits == 1) return rc;
    const uint64_t items = static_cast<uint64_t>(a.tokens) * (a.n_out / 8u);
    const void *sum = c.mode == kDenseGated ? reinterpret_cast<const void *>(&df11_dense_sum_kernel<kDenseGated>)
                      : c.mode == kDenseBack ? reinterpret_cast<const void *>(&df11_dense_sum_kernel<kDenseBack>)
                                             : reinterpret_cast<const void *>(&df11_dense_sum_kernel<kDensePlain>);
    return launch_kernel(sum, dim3(static_cast<uint32_t>(std::min<uint64_t>((items + 255) / 256, 8ull * cus))), dim3(256),
                         params, 0, stream, nullptr, nullptr);
}

}  // namespace df11
