// The dense products of df11_dense.h on the matrix cores (gfx950).
//
// A workgroup computes a tile of BM tokens x BN outputs in steps of 64 along
// K, from two LDS buffers: while the waves multiply one step, the next one
// is on its way into the other buffer (global_load_lds, no registers), so a
// step costs one barrier and one wait for loads that a whole step of MFMAs
// has covered.
//
// Weights arrive in MFMA tile order: a 1 KB block is the operand of one
// v_mfma_f32_16x16x32_bf16 for 16 rows x 32 columns of W, lane l's 16 bytes
// at 16 l, so both the loads and the LDS reads of the forward product are
// linear.  The left operand's rows are 128 bytes in LDS, their eight 16-byte
// chunks permuted by the row (chunk c at c ^ (row mod 8)), which spreads the
// 16 rows of an operand over all banks.  The backward product needs the
// transpose of the same blocks: column n of W, 8 consecutive rows, which
// ds_read_b64_tr_b16 gathers from 4 rows x 16 columns at a time.
#include <hip/hip_runtime.h>

#include <algorithm>

#include <stdint.h>

#include "df11.h"
#include "df11_dense.h"
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

constexpr uint32_t kStep = 64;  // K elements of one step

struct DenseArgs {
    const uint16_t *left[2];
    const uint16_t *w[2];
    uint64_t left_stride;
    float *partial;       // split: [split][matrix][token][output]
    uint32_t tokens;
    uint32_t n_out;       // outputs per token
    uint32_t tile_ks;     // C / 32
    uint32_t panels;      // R / 64
    uint32_t k_steps;     // steps along K, all matrices of a backward product
    uint32_t k_steps_one; // steps of one matrix
    uint32_t m_tiles, n_tiles, splits;
    uint32_t vec;         // the epilogue's buffers allow vectors of four outputs
    Epilogue e;
};

__device__ __forceinline__ void load_to_lds(const uint16_t *src, uint8_t *dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Four rows x 16 columns of 2-byte elements, transposed across a quarter
// wave: lane i of the quarter passes the address of row i / 4, columns
// 4 (i mod 4) .. + 3, and receives column i of the four rows.
__device__ __forceinline__ shortx4 read_transposed(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4 *)p);
}

// Four consecutive outputs of one token.
template <int MODE>
__device__ __forceinline__ void finish4(const DenseArgs &a, uint32_t token, uint32_t col, const floatx4 &z0,
                                        const floatx4 &z1) {
    constexpr bool kGated = MODE == kDenseGated;
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) finish<kGated>(a.e, token, col + r, a.n_out, z0[r], kGated ? z1[r] : 0.0f);
}

template <int BM, int BN, int WM, int WN, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void df11_dense_kernel(DenseArgs a) {
    constexpr int kWavesAll = WM * WN;
    constexpr int TM = BM / WM / 16;  // token tiles of a wave
    static_assert(BN / WN == 64, "a wave's outputs are four blocks of 16");
    constexpr int kLeftBytes = BM * 128, kStageBytes = (BM + BN) * 128;
    constexpr int kLeftLoads = BM / 8, kLoads = (BM + BN) / 8;
    static_assert(kLoads % kWavesAll == 0 && kLeftLoads % kWavesAll == 0, "every wave loads alike");
    constexpr int kRowsTile = MODE == kDenseGated ? BN / 2 : BN;  // outputs of a tile
    __shared__ __align__(1024) uint8_t s_stage[2][kStageBytes];

    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t wm = wave / WN, wn = wave % WN;

    // Tiles in runs per XCD (workgroup i runs on XCD i mod 8): an XCD's L2
    // then serves the tokens of one column of tiles from one read of W.
    const uint32_t total = gridDim.x, xcd = blockIdx.x % 8u, q = total / 8u, rest = total % 8u;
    uint32_t tile = xcd * q + min(xcd, rest) + blockIdx.x / 8u;
    const uint32_t m_tile = tile % a.m_tiles;
    tile /= a.m_tiles;
    const uint32_t split = tile % a.splits, n_tile = tile / a.splits;
    const uint32_t m0 = m_tile * BM, n0 = n_tile * kRowsTile;
    const uint32_t k_begin = static_cast<uint32_t>(static_cast<uint64_t>(split) * a.k_steps / a.splits);
    const uint32_t k_end = static_cast<uint32_t>(static_cast<uint64_t>(split + 1u) * a.k_steps / a.splits);

    // This lane's row and chunk of each left load, and its element offset.
    const uint32_t chunk = (lane & 7u) ^ (lane >> 3);
    uint64_t left_at[kLeftLoads / kWavesAll];
#pragma unroll
    for (int i = 0; i < kLeftLoads / kWavesAll; ++i) {
        const uint32_t row = min(m0 + 8u * (wave + kWavesAll * i) + (lane >> 3), a.tokens - 1u);
        left_at[i] = row * a.left_stride;
    }

    auto issue = [&](uint32_t step, uint8_t *stage) {
        const uint32_t one = MODE == kDenseBack && step >= a.k_steps_one ? 1u : 0u;
        const uint32_t ks = step - one * a.k_steps_one;  // step of this matrix
        const uint16_t *left = a.left[one];
        // (forward, an odd last k-step: the upper half reads the lower's
        // columns and its products are left out)
        const uint32_t c = MODE != kDenseBack && 2u * ks + 1u >= a.tile_ks ? chunk & 3u : chunk;
        const uint32_t k0 = kStep * ks + 8u * c;
#pragma unroll
        for (int i = 0; i < kLeftLoads / kWavesAll; ++i)
            load_to_lds(left + left_at[i] + k0, stage + 1024u * (wave + kWavesAll * i));
#pragma unroll
        for (int i = kLeftLoads / kWavesAll; i < kLoads / kWavesAll; ++i) {
            const uint32_t b = wave + kWavesAll * i - kLeftLoads;  // block of the step
            const uint16_t *src;
            if constexpr (MODE == kDenseBack) {
                // panel ks, k-step n0 / 32 + b / 4 of it, block b mod 4
                const uint32_t at = min(n0 / 32u + b / 4u, a.tile_ks - 1u);
                src = a.w[one] + (static_cast<uint64_t>(ks * a.tile_ks + at) * 4u + (b & 3u)) * 512u;
            } else {
                const uint32_t half = b / (BN / 16u), nb = b % (BN / 16u);
                const uint32_t at = min(2u * ks + half, a.tile_ks - 1u);
                uint32_t r16;
                const uint16_t *w = a.w[0];
                if constexpr (MODE == kDenseGated) {
                    // blocks 0, 1 of each four from the gate, 2, 3 from up
                    r16 = n0 / 16u + 2u * (nb / 4u) + (nb & 1u);
                    w = a.w[(nb >> 1) & 1u];
                } else {
                    r16 = n0 / 16u + nb;
                }
                const uint32_t panel = min(r16 / 4u, a.panels - 1u);
                src = w + (static_cast<uint64_t>(panel * a.tile_ks + at) * 4u + (r16 & 3u)) * 512u;
            }
            load_to_lds(src + 8u * lane, stage + kLeftBytes + 1024u * b);
        }
    };

    floatx4 acc[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t quarter = lane >> 4, l16 = lane & 15u;
    auto multiply = [&](const uint8_t *stage, int half) {
        bf16x8 wf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (MODE == kDenseBack) {
                // outputs 16 (j mod 2) .. of k-step 2 wn + j / 2; rows 32 half + 8 quarter ..
                const uint8_t *block = stage + kLeftBytes + 1024u * (4u * (2u * wn + j / 2) + 2u * half + (quarter >> 1));
                const uint32_t row = 8u * (quarter & 1u) + (l16 >> 2);
                const uint8_t *p = block + 16u * (16u * (2u * (j & 1) + ((l16 >> 1) & 1u)) + row) + 8u * (l16 & 1u);
                union {
                    shortx4 s[2];
                    bf16x8 v;
                } u;
                u.s[0] = read_transposed(p);
                u.s[1] = read_transposed(p + 64);  // four rows on
                wf[j] = u.v;
            } else {
                wf[j] = *reinterpret_cast<const bf16x8 *>(stage + kLeftBytes + 1024u * (half * (BN / 16) + 4u * wn + j) +
                                                          16u * lane);
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const uint32_t row = wm * (BM / WM) + 16u * i + l16;
            const uint32_t c = (4u * half + quarter) ^ (row & 7u);
            const bf16x8 xf = *reinterpret_cast<const bf16x8 *>(stage + 128u * row + 16u * c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[j], xf, acc[i][j], 0, 0, 0);
        }
    };

    if (k_begin < k_end) issue(k_begin, s_stage[0]);
    for (uint32_t step = k_begin; step < k_end; ++step) {
        uint8_t *stage = s_stage[(step - k_begin) & 1u], *next = s_stage[(step - k_begin + 1u) & 1u];
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (step + 1u < k_end) issue(step + 1u, next);
        multiply(stage, 0);
        if (MODE == kDenseBack || 2u * step + 1u < a.tile_ks) multiply(stage, 1);
    }

    // Lane l holds outputs 4 (l / 16) .. + 3 of each block for token l mod 16.
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const uint32_t token = m0 + wm * (BM / WM) + 16u * i + l16;
        if (token >= a.tokens) continue;
        constexpr int kBlocks = MODE == kDenseGated ? 2 : 4;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const uint32_t col = n0 + (MODE == kDenseGated ? 32u : 64u) * wn + 16u * j + 4u * quarter;
            if (col >= a.n_out) continue;  // (outputs come in whole blocks of 16)
            if (a.splits > 1u) {
                constexpr uint32_t kMats = MODE == kDenseGated ? 2u : 1u;
                float *p = a.partial + ((static_cast<uint64_t>(split) * kMats) * a.tokens + token) * a.n_out + col;
                *reinterpret_cast<floatx4 *>(p) = acc[i][j];
                if constexpr (MODE == kDenseGated)
                    *reinterpret_cast<floatx4 *>(p + static_cast<uint64_t>(a.tokens) * a.n_out) = acc[i][j + 2];
            } else {
                finish4<MODE>(a, token, col, acc[i][j], MODE == kDenseGated ? acc[i][(j + 2) & 3] : acc[i][j]);
            }
        }
    }
}

// Adds the splits' partial sums in order and applies the epilogue.
template <int MODE>
__global__ __launch_bounds__(256) void df11_dense_sum_kernel(DenseArgs a) {
    constexpr uint32_t kMats = MODE == kDenseGated ? 2u : 1u;
    const uint32_t per_row = a.n_out / 4u;
    const uint64_t total = static_cast<uint64_t>(a.tokens) * per_row, plane = static_cast<uint64_t>(a.tokens) * a.n_out;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
        const uint32_t token = static_cast<uint32_t>(i / per_row), col = 4u * static_cast<uint32_t>(i % per_row);
        floatx4 z[2] = {};
        for (uint32_t m = 0; m < kMats; ++m) {
            const float *p = a.partial + m * plane + static_cast<uint64_t>(token) * a.n_out + col;
            z[m] = *reinterpret_cast<const floatx4 *>(p);
            for (uint32_t s = 1; s < a.splits; ++s)
                z[m] += *reinterpret_cast<const floatx4 *>(p + s * kMats * plane);
        }
        finish4<MODE>(a, token, col, z[0], z[1]);
    }
}

// Shape of one launch.
struct DenseShape {
    bool large;  // 256 x 256 tiles, one workgroup a CU; else 128 x 128, two
    uint32_t m_tiles, n_tiles, splits;
};

DenseShape dense_shape(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols, int cus) {
    const uint32_t n_out = mode == kDenseBack ? cols : rows;
    const uint32_t k_steps = mode == kDenseBack ? n * (rows / kStep) : (cols + kStep - 1) / kStep;
    DenseShape best{};
    double best_time = 0.0;
    for (int large = 0; large < 2; ++large) {
        const uint32_t bm = large ? 256u : 128u, bn = mode == kDenseGated ? bm / 2u : bm;
        const uint64_t mt = (tokens + bm - 1) / bm, nt = (n_out + bn - 1) / bn;
        const uint64_t room = static_cast<uint64_t>(cus) * (large ? 1u : 2u);
        for (uint32_t splits = 1; splits <= 16 && splits <= k_steps; splits *= 2) {
            const uint64_t turns = (mt * nt * splits + room - 1) / room;
            // Time in units of one 128 x 128 step of two workgroups on a CU.
            const double step = large ? 2.0 : 1.2;
            double t = turns * ((k_steps + splits - 1) / splits + 6.0) * step;
            if (splits > 1)  // partial sums written and read, about 4 bytes a nanosecond and CU
                t += 4.0 + 2.0 * 4.0 * splits * tokens * n_out * (mode == kDenseGated ? 2.0 : 1.0) / (cus * 5000.0);
            if (best.m_tiles == 0 || t < best_time) {
                best = DenseShape{large != 0, static_cast<uint32_t>(mt), static_cast<uint32_t>(nt), splits};
                best_time = t;
            }
        }
    }
    return best;
}

template <int BM, int BN, int WM, int WN>
const void *dense_kernel(DenseMode mode) {
    switch (mode) {
    case kDenseGated: return reinterpret_cast<const void *>(&df11_dense_kernel<BM, BN, WM, WN, kDenseGated>);
    case kDenseBack: return reinterpret_cast<const void *>(&df11_dense_kernel<BM, BN, WM, WN, kDenseBack>);
    default: return reinterpret_cast<const void *>(&df11_dense_kernel<BM, BN, WM, WN, kDensePlain>);
    }
}

}  // namespace

namespace df11 {

uint64_t dense_workspace(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols) {
    int dev = 0, cus = 0;
    if (device_cus(dev, cus)) return ~0ull;
    const DenseShape s = dense_shape(mode, n, tokens, rows, cols, cus);
    const uint64_t mats = mode == kDenseGated ? 2 : 1, n_out = mode == kDenseBack ? cols : rows;
    return s.splits > 1 ? 4ull * s.splits * mats * tokens * n_out : 0;
}

int dense_product(const DenseCall &c, const Epilogue &e, float *workspace, hipStream_t stream) {
    int dev = 0, cus = 0;
    if (device_cus(dev, cus)) return DF11_E_HIP;
    const uint32_t n = c.mode == kDensePlain || (c.mode == kDenseBack && !c.w[1]) ? 1 : 2;
    const DenseShape s = dense_shape(c.mode, n, c.tokens, c.rows, c.cols, cus);
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
    a.m_tiles = s.m_tiles;
    a.n_tiles = s.n_tiles;
    a.splits = s.splits;
    a.e = e;
    (void)hipGetLastError();
    void *params[] = {&a};
    const void *fn = s.large ? dense_kernel<256, 256, 2, 4>(c.mode) : dense_kernel<128, 128, 2, 2>(c.mode);
    const int rc = launch_kernel(fn, dim3(s.m_tiles * s.n_tiles * s.splits), dim3(s.large ? 512 : 256), params, 0,
                                 stream, nullptr, nullptr);
    if (rc || s.splits == 1) return rc;
    const uint64_t items = static_cast<uint64_t>(a.tokens) * (a.n_out / 4u);
    const void *sum = c.mode == kDenseGated ? reinterpret_cast<const void *>(&df11_dense_sum_kernel<kDenseGated>)
                                            : reinterpret_cast<const void *>(&df11_dense_sum_kernel<kDensePlain>);
    return launch_kernel(sum, dim3(static_cast<uint32_t>(std::min<uint64_t>((items + 255) / 256, 8ull * cus))), dim3(256),
                         params, 0, stream, nullptr, nullptr);
}

}  // namespace df11
