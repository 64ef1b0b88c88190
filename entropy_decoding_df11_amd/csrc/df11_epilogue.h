// The epilogue of the products: activations, their slopes, and the buffers
// that the last kernel of a product reads and writes.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11.h"
#include "df11_types.h"

namespace df11 {

// Kernel arguments of an epilogue (df11_epilogue with its checks done).
struct Epilogue {
    const void *bias[2];
    const void *residual;
    void *out;
    float *pre[2];
    uint64_t residual_stride, out_stride;
    uint32_t bias_dtype, residual_dtype, out_dtype, act;
};

}  // namespace df11

namespace {

using df11::Epilogue;

// act(z) in float.  Each form keeps its relative accuracy where the value is
// small (erfc and the logistic in place of 1 + erf and 1 + tanh, which cancel
// for negative z).
__device__ __forceinline__ float activate(uint32_t act, float z) {
    switch (act) {
    case DF11_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case DF11_ACT_SILU: return z / (1.0f + expf(-z));
    case DF11_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case DF11_ACT_GELU_TANH: {
        // 0.5 z (1 + tanh(u)) = z / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
        const float u2 = 1.5957691216057308f * z * (1.0f + 0.044715f * z * z);
        return z / (1.0f + expf(-u2));
    }
    default: return z;
    }
}

// d act(z) / dz in float.
__device__ __forceinline__ float slope(uint32_t act, float z) {
    switch (act) {
    case DF11_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case DF11_ACT_SILU: {
        const float p = 1.0f / (1.0f + expf(-z));
        return p * (1.0f + z * (1.0f / (1.0f + expf(z))));
    }
    case DF11_ACT_GELU:
        return 0.5f * erfcf(-0.70710678118654752f * z) + 0.39894228040143268f * z * expf(-0.5f * z * z);
    case DF11_ACT_GELU_TANH: {
        if (fabsf(z) > 16.0f) return z > 0.0f ? 1.0f : 0.0f;  // (exact in float, and z^2 cannot overflow)
        const float u2 = 1.5957691216057308f * z * (1.0f + 0.044715f * z * z);
        const float p = 1.0f / (1.0f + expf(-u2)), q = 1.0f / (1.0f + expf(u2));
        return p + z * p * q * 1.5957691216057308f * (1.0f + 0.134145f * z * z);
    }
    default: return 1.0f;
    }
}

// Sums of one output element (the second of a gated product) to its place.
// row: token, col: output feature, features: outputs per token.
template <bool kGated>
__device__ __forceinline__ void finish(const Epilogue &e, uint32_t row, uint32_t col, uint32_t features, float z0,
                                       float z1) {
    if (e.bias[0]) z0 += load_as(e.bias[0], col, e.bias_dtype);
    if constexpr (kGated) {
        if (e.bias[1]) z1 += load_as(e.bias[1], col, e.bias_dtype);
    }
    if (e.pre[0]) {
        e.pre[0][static_cast<uint64_t>(row) * features + col] = z0;
        if constexpr (kGated) e.pre[1][static_cast<uint64_t>(row) * features + col] = z1;
    }
    float y = activate(e.act, z0);
    if constexpr (kGated) y *= z1;
    if (e.residual) y += load_as(e.residual, row * e.residual_stride + col, e.residual_dtype);
    store_as(e.out, row * e.out_stride + col, e.out_dtype, y);
}

}  // namespace
