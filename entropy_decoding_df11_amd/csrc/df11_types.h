// Element types of the operators around the products, and their conversion
// to and from float in the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11.h"

namespace {

using bf16_t = __bf16;
using fp16_t = _Float16;

template <typename T, int N>
using vec_t = T __attribute__((ext_vector_type(N)));

// Bytes of one element, 0 for a value that names no type.
inline uint32_t dtype_bytes(uint32_t dtype) {
    return dtype == DF11_BF16 || dtype == DF11_FP16 ? 2u : dtype == DF11_FP32 ? 4u : 0u;
}

// N consecutive elements (N * sizeof(T) aligned) as floats, and back, each
// rounded once to nearest even.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = static_cast<float>(*p);
    } else {
        const vec_t<T, N> v = *reinterpret_cast<const vec_t<T, N> *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = static_cast<float>(v[i]);
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[N]) {
    if constexpr (N == 1) {
        *p = static_cast<T>(f[0]);
    } else {
        vec_t<T, N> v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = static_cast<T>(f[i]);
        *reinterpret_cast<vec_t<T, N> *>(p) = v;
    }
}

// One element of a buffer whose type is known at run time (wave-uniform).
__device__ __forceinline__ float load_as(const void *p, uint64_t i, uint32_t dtype) {
    if (dtype == DF11_FP32) return static_cast<const float *>(p)[i];
    if (dtype == DF11_BF16) return static_cast<float>(static_cast<const bf16_t *>(p)[i]);
    return static_cast<float>(static_cast<const fp16_t *>(p)[i]);
}

__device__ __forceinline__ void store_as(void *p, uint64_t i, uint32_t dtype, float v) {
    if (dtype == DF11_FP32) {
        static_cast<float *>(p)[i] = v;
    } else if (dtype == DF11_BF16) {
        static_cast<bf16_t *>(p)[i] = static_cast<bf16_t>(v);
    } else {
        static_cast<fp16_t *>(p)[i] = static_cast<fp16_t>(v);
    }
}

}  // namespace
