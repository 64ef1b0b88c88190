// The RMS norm with the residual's addition, forward and backward, and the
// column sums that bias and norm-weight gradients end in (gfx950).
//
//   s = round(x + residual)          rounded to the tensors' type: the value
//                                    that the residual stream carries on
//   y = s * rstd * weight            rstd = 1 / sqrt(mean(s^2) + eps)
//
// and, with h = s * rstd and the incoming gradients dy and ds,
//
//   dx = rstd * (dy * weight - h * mean(dy * weight * h)) + ds
//   dweight = sum over the rows of dy * h
//
// Both directions read each element once and write each result once: a row's
// threads hold its elements in registers between the sum and the output, so
// the row is not read again for the second use.  Sums are float, taken lane
// by lane, then across the wave by shuffles and across waves through LDS, in
// an order that depends on the width alone: results do not change from call
// to call.
#include <hip/hip_runtime.h>

#include <algorithm>

#include <stdint.h>

#include "df11.h"
#include "df11_columns.h"
#include "df11_device.h"
#include "df11_types.h"

namespace {

struct NormArgs {
    const void *x;
    const void *residual;  // or null
    const void *weight;    // or null
    void *sum;             // or null
    void *y;
    float *rstd;           // or null
    uint64_t x_stride, residual_stride, sum_stride, y_stride;  // elements
    uint32_t rows, cols;
    uint32_t weight_f32;   // weight is float32 (else the rows' own type)
    float eps;
};

// Sum of v over the TPR threads of a row, in every one of them.  One wave
// needs no LDS; the waves of a wider row meet in s_part (one float per wave
// of the block).
template <int TPR>
__device__ __forceinline__ float row_total(float v, float *s_part) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (TPR > static_cast<int>(kWaveSize)) {
        constexpr int kRowWaves = TPR / static_cast<int>(kWaveSize);
        if ((threadIdx.x & (kWaveSize - 1)) == 0) s_part[threadIdx.x / kWaveSize] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) v += s_part[w];
    }
    return v;
}

template <typename T, int VEC>
__device__ __forceinline__ void load_weight(const void *weight, uint32_t f32, uint32_t i, float (&w)[VEC]) {
    if (!weight) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 1.0f;
    } else if (f32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = static_cast<const float *>(weight)[i + e];
    } else {
        load_vec<T, VEC>(static_cast<const T *>(weight) + i, w);
    }
}

// TPR threads per row, NV vectors of VEC elements held per thread.  kWide:
// rows beyond TPR * NV vectors, whose elements past the held ones are read
// a second time for the output (from the sum where one is written).
template <typename T, int VEC, int NV, int TPR, bool kWide>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void df11_rms_norm_kernel(NormArgs a) {
    constexpr int kBlock = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kBlock / TPR;
    __shared__ float s_part[2][kBlock / kWaveSize];
    const uint32_t lid = threadIdx.x % TPR;
    uint32_t turn = 0;
    // (one row per group of threads, unless the rows outnumber the largest
    // grid; a row's waves leave the loop together)
    for (uint32_t row = blockIdx.x * kRows + threadIdx.x / TPR; row < a.rows; row += gridDim.x * kRows, turn ^= 1u) {
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
        T *sum = a.sum ? static_cast<T *>(a.sum) + row * a.sum_stride : nullptr;
        T *y = static_cast<T *>(a.y) + row * a.y_stride;

        float v[NV][VEC];
        float total = 0.0f;
        // One vector's s, written to the sum if there is one.
        auto take = [&](uint32_t i, float (&s)[VEC]) {
            load_vec<T, VEC>(x + i, s);
            if (res) {
                float r[VEC];
                load_vec<T, VEC>(res + i, r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] = static_cast<float>(static_cast<T>(s[e] + r[e]));
            }
            if (sum) store_vec<T, VEC>(sum + i, s);
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) {
                take(i, v[j]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) total += v[j][e] * v[j][e];
            }
        }
        if constexpr (kWide) {
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC) {
                float s[VEC];
                take(i, s);
#pragma unroll
                for (int e = 0; e < VEC; ++e) total += s[e] * s[e];
            }
        }
        total = row_total<TPR>(total, s_part[turn]);
        // (the quotient and the root are each rounded to float)
        const float r = 1.0f / sqrtf(total / static_cast<float>(a.cols) + a.eps);
        if (a.rstd && lid == 0) a.rstd[row] = r;
        auto put = [&](uint32_t i, const float (&s)[VEC]) {
            float w[VEC];
            load_weight<T, VEC>(a.weight, a.weight_f32, i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] *= s[e] * r;
            store_vec<T, VEC>(y + i, w);
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) put(i, v[j]);
        }
        if constexpr (kWide) {
            // Each thread reads back only what it wrote or read itself, so the
            // output may be x's or the residual's own buffer.
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC) {
                float s[VEC];
                load_vec<T, VEC>((sum ? static_cast<const T *>(sum) : x) + i, s);
                if (res && !sum) {
                    float q[VEC];
                    load_vec<T, VEC>(res + i, q);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s[e] = static_cast<float>(static_cast<T>(s[e] + q[e]));
                }
                put(i, s);
            }
        }
    }
}

struct NormGradArgs {
    const void *s;
    const void *weight;  // or null
    const float *rstd;
    const void *dy;
    const void *dsum;    // or null
    void *dx;
    float *partial;      // or null: [row groups][cols] sums of dy * h
    uint64_t s_stride, dy_stride, dsum_stride, dx_stride;
    uint32_t rows, cols;
    uint32_t weight_f32;
};

// A row group (the TPR threads of one row at a time) takes rows g, g + G,
// g + 2 G, ... of the G groups of the launch, and keeps its sums of dy * h
// for the columns its threads hold in registers; they leave once, at the end.
template <typename T, int VEC, int NV, int TPR, bool kWide>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void df11_rms_norm_grad_kernel(NormGradArgs a) {
    constexpr int kBlock = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kBlock / TPR;
    __shared__ float s_part[2][kBlock / kWaveSize];
    const uint32_t lid = threadIdx.x % TPR;
    const uint32_t group = blockIdx.x * kRows + threadIdx.x / TPR;
    const uint32_t groups = gridDim.x * kRows;
    const float inv = 1.0f / static_cast<float>(a.cols);
    float acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.0f;
    float *part = a.partial ? a.partial + static_cast<uint64_t>(group) * a.cols : nullptr;
    if constexpr (kWide) {
        if (part)
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC)
#pragma unroll
                for (int e = 0; e < VEC; ++e) part[i + e] = 0.0f;
    }
    uint32_t turn = 0;
    for (uint32_t row = group; row < a.rows; row += groups, turn ^= 1u) {
        const T *s = static_cast<const T *>(a.s) + row * a.s_stride;
        const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
        const T *ds = a.dsum ? static_cast<const T *>(a.dsum) + row * a.dsum_stride : nullptr;
        T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
        const float r = a.rstd[row];
        // (held packed, as loaded: the floats of a row of four vectors a
        // thread would not fit the registers of 1024 threads)
        Packed<T, VEC> sv[NV], dv[NV];
        float total = 0.0f;
        // h = s * rstd, d = dy * weight, raw = dy of one vector
        auto expand = [&](uint32_t i, const Packed<T, VEC> &ps, const Packed<T, VEC> &pd, float (&h)[VEC],
                          float (&d)[VEC], float (&raw)[VEC]) {
            float w[VEC];
            unpack<T, VEC>(ps, h);
            unpack<T, VEC>(pd, raw);
            load_weight<T, VEC>(a.weight, a.weight_f32, i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] *= r;
                d[e] = raw[e] * w[e];
            }
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) {
                sv[j] = load_packed<T, VEC>(s + i);
                dv[j] = load_packed<T, VEC>(dy + i);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) {
                float h[VEC], d[VEC], raw[VEC];
                expand(i, sv[j], dv[j], h, d, raw);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    total += d[e] * h[e];
                    acc[j][e] += raw[e] * h[e];
                }
            }
        }
        if constexpr (kWide) {
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC) {
                float h[VEC], d[VEC], raw[VEC];
                expand(i, load_packed<T, VEC>(s + i), load_packed<T, VEC>(dy + i), h, d, raw);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    total += d[e] * h[e];
                    if (part) part[i + e] += raw[e] * h[e];
                }
            }
        }
        // (two sets of wave sums, in turn: a wave may enter the next row's
        // sum while another still reads this one's)
        const float mean = row_total<TPR>(total, s_part[turn]) * inv;
        auto put = [&](uint32_t i, const Packed<T, VEC> &ps, const Packed<T, VEC> &pd) {
            float g[VEC], h[VEC], d[VEC], raw[VEC];
            if (ds) {
                load_vec<T, VEC>(ds + i, g);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[e] = 0.0f;
            }
            expand(i, ps, pd, h, d, raw);
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] += r * (d[e] - h[e] * mean);
            store_vec<T, VEC>(dx + i, g);
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) put(i, sv[j], dv[j]);
        }
        if constexpr (kWide) {
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC)
                put(i, load_packed<T, VEC>(s + i), load_packed<T, VEC>(dy + i));
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols)
#pragma unroll
                for (int e = 0; e < VEC; ++e) part[i + e] = acc[j][e];
        }
    }
}

// out[c] = sum over the rows of p[row][c], in row order within each of the
// block's 16 slices of rows, then over the slices.
__global__ __launch_bounds__(1024) void df11_column_sum_kernel(const float *p, uint32_t rows, uint32_t cols,
                                                               void *out, uint32_t dtype) {
    __shared__ float s_sum[16][kWaveSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), slice = threadIdx.x / kWaveSize;
    const uint32_t c = blockIdx.x * kWaveSize + lane;
    float v = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (uint32_t r = slice; r < rows; r += 16u) v += p[static_cast<uint64_t>(r) * cols + c];
    s_sum[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < cols) {
        for (uint32_t k = 1; k < 16u; ++k) v += s_sum[k][lane];
        store_as(out, c, dtype, v);
    }
}

// Threads per row and vectors per thread for a row of n vectors: the fewest
// threads that hold the row in at most four vectors each, so that rows of up
// to 256 vectors need no barrier.  1024 threads hold two vectors each (or
// eight single elements, where rows are not aligned to vectors): what their
// registers allow in the backward pass.  Past that the remainder is read twice.
struct RowShape {
    uint32_t threads, vectors;
    bool wide;
};

constexpr int kMostHeld(int vec) { return vec == 1 ? 8 : 2; }

RowShape row_shape(uint64_t n, uint32_t vec) {
    if (n <= 64) return {64, 1, false};
    if (n <= 128) return {64, 2, false};
    if (n <= 256) return {64, 4, false};
    if (n <= 512) return {256, 2, false};
    if (n <= 1024) return {256, 4, false};
    const uint32_t most = static_cast<uint32_t>(kMostHeld(static_cast<int>(vec)));
    return {1024, most, n > 1024ull * most};
}

// Elements per vector: 16 bytes where the rows of every tensor are aligned
// to that and the width is a whole number of vectors, else one element.
uint32_t row_vector(uint32_t bytes, uint32_t cols, const void *const *ptrs, const uint64_t *strides, int n) {
    const uint32_t per = 16u / bytes;
    bool whole = cols % per == 0;
    for (int i = 0; i < n; ++i)
        if (ptrs[i]) whole = whole && aligned(ptrs[i], 16) && strides[i] % per == 0;
    return whole ? per : 1u;
}

template <template <typename, int, int, int, bool> class Pick, typename T, int VEC>
const void *pick_shape(const RowShape &s) {
    if (s.wide) return Pick<T, VEC, kMostHeld(VEC), 1024, true>::get();
    if (s.threads == 1024) return Pick<T, VEC, kMostHeld(VEC), 1024, false>::get();
    if (s.threads == 256) return s.vectors == 2 ? Pick<T, VEC, 2, 256, false>::get() : Pick<T, VEC, 4, 256, false>::get();
    return s.vectors == 1   ? Pick<T, VEC, 1, 64, false>::get()
           : s.vectors == 2 ? Pick<T, VEC, 2, 64, false>::get()
                            : Pick<T, VEC, 4, 64, false>::get();
}

template <template <typename, int, int, int, bool> class Pick>
const void *pick_kernel(uint32_t dtype, uint32_t vec, const RowShape &s) {
    if (dtype == DF11_FP32) return vec > 1 ? pick_shape<Pick, float, 4>(s) : pick_shape<Pick, float, 1>(s);
    if (dtype == DF11_BF16) return vec > 1 ? pick_shape<Pick, bf16_t, 8>(s) : pick_shape<Pick, bf16_t, 1>(s);
    return vec > 1 ? pick_shape<Pick, fp16_t, 8>(s) : pick_shape<Pick, fp16_t, 1>(s);
}

template <typename T, int VEC, int NV, int TPR, bool kWide>
struct NormKernel {
    static const void *get() { return reinterpret_cast<const void *>(&df11_rms_norm_kernel<T, VEC, NV, TPR, kWide>); }
};
template <typename T, int VEC, int NV, int TPR, bool kWide>
struct NormGradKernel {
    static const void *get() {
        return reinterpret_cast<const void *>(&df11_rms_norm_grad_kernel<T, VEC, NV, TPR, kWide>);
    }
};

// Bytes from a row tensor's first to its last element.
uint64_t span_bytes(uint32_t rows, uint32_t cols, uint64_t stride, uint32_t bytes) {
    return rows && cols ? ((rows - 1ull) * stride + cols) * bytes : 0;
}

// Whether an output may lie where an input does: apart, or exactly on it
// (each thread reads an element before it writes the same one).
bool apart_or_same(const void *out, uint64_t out_stride, const void *in, uint64_t in_stride, uint32_t rows,
                   uint32_t cols, uint32_t bytes) {
    if (!in || (out == in && out_stride == in_stride)) return true;
    return !overlaps(out, span_bytes(rows, cols, out_stride, bytes), in, span_bytes(rows, cols, in_stride, bytes));
}

// Row groups of the backward pass when it sums the weight's gradient: a
// group's partial sums cost four bytes a column written and read again, so a
// group takes at least eight rows, and there are at most two blocks a CU.
constexpr uint32_t kGradRowsPerGroup = 4;
constexpr uint32_t kGradMaxGroups = 512;

uint32_t grad_groups(uint32_t rows, uint32_t per_block) {
    const uint32_t want = std::min(kGradMaxGroups, (rows + kGradRowsPerGroup - 1) / kGradRowsPerGroup);
    return std::max(1u, (want + per_block - 1) / per_block) * per_block;
}

// (for the largest number of row groups a block can hold)
uint32_t grad_groups_bound(uint32_t rows) { return grad_groups(rows, 256u / kWaveSize); }

// Most blocks of a launch (a grid's threads are counted in 32 bits); the rows
// past them are taken in further turns.
constexpr uint32_t kMaxBlocks = 1u << 20;

constexpr uint64_t kMaxRowElements = 1ull << 40;  // keeps row * stride * bytes within 64 bits

}  // namespace

namespace df11 {

int column_sums(const float *p, uint32_t rows, uint32_t cols, void *out, uint32_t dtype, hipStream_t stream) {
    void *params[] = {&p, &rows, &cols, &out, &dtype};
    return launch_kernel(reinterpret_cast<const void *>(&df11_column_sum_kernel),
                         dim3((cols + kWaveSize - 1) / kWaveSize), dim3(1024), params, 0, stream, nullptr, nullptr);
}

}  // namespace df11

extern "C" {

int df11_rms_norm(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                  const void *weight, uint32_t weight_dtype, uint32_t rows, uint32_t cols, uint32_t dtype, float eps,
                  void *sum, uint64_t sum_stride, void *y, uint64_t y_stride, float *rstd, void *hip_stream) {
    const uint32_t bytes = dtype_bytes(dtype);
    if (!bytes || cols == 0 || cols > (1u << 30) || rows > (1u << 30) || !(eps >= 0.0f)) return DF11_E_INVALID_ARG;
    if (weight && weight_dtype != dtype && weight_dtype != DF11_FP32) return DF11_E_INVALID_ARG;
    if (rows == 0) return DF11_OK;
    if (!x || !y) return DF11_E_INVALID_ARG;
    if (sum && !residual) return DF11_E_INVALID_ARG;  // (without a residual the sum is x itself)
    const void *ptrs[] = {x, residual, sum, y};
    const uint64_t strides[] = {x_stride, residual_stride, sum_stride, y_stride};
    for (int i = 0; i < 4; ++i) {
        if (!ptrs[i]) continue;
        if (!aligned(ptrs[i], bytes) || strides[i] > kMaxRowElements) return DF11_E_INVALID_ARG;
        // inputs may repeat a row (stride 0) or overlap themselves; outputs may not
        if (i >= 2 && strides[i] < cols && rows > 1) return DF11_E_INVALID_ARG;
    }
    const uint32_t wbytes = weight ? dtype_bytes(weight_dtype) : 0;
    if (weight && !aligned(weight, wbytes)) return DF11_E_INVALID_ARG;
    if (rstd && !aligned(rstd, 4)) return DF11_E_INVALID_ARG;
    const uint64_t y_span = span_bytes(rows, cols, y_stride, bytes);
    const uint64_t sum_span = sum ? span_bytes(rows, cols, sum_stride, bytes) : 0;
    const void *outs[] = {y, sum};
    const uint64_t out_strides[] = {y_stride, sum_stride}, out_spans[] = {y_span, sum_span};
    for (int i = 0; i < 2; ++i) {
        if (!outs[i]) continue;
        if (!apart_or_same(outs[i], out_strides[i], x, x_stride, rows, cols, bytes) ||
            !apart_or_same(outs[i], out_strides[i], residual, residual_stride, rows, cols, bytes) ||
            overlaps(outs[i], out_spans[i], weight, static_cast<uint64_t>(wbytes) * cols) ||
            overlaps(outs[i], out_spans[i], rstd, rstd ? 4ull * rows : 0))
            return DF11_E_INVALID_ARG;
    }
    if (overlaps(y, y_span, sum, sum_span)) return DF11_E_INVALID_ARG;
    if (rstd && (overlaps(rstd, 4ull * rows, x, span_bytes(rows, cols, x_stride, bytes)) ||
                 overlaps(rstd, 4ull * rows, residual, residual ? span_bytes(rows, cols, residual_stride, bytes) : 0) ||
                 overlaps(rstd, 4ull * rows, weight, static_cast<uint64_t>(wbytes) * cols)))
        return DF11_E_INVALID_ARG;
    NormArgs a{x, residual, weight, sum, y, rstd, x_stride, residual_stride, sum_stride, y_stride, rows, cols,
               weight && weight_dtype == DF11_FP32, eps};
    uint32_t vec = row_vector(bytes, cols, ptrs, strides, 4);
    if (weight && !aligned(weight, 16)) vec = 1;
    const RowShape shape = row_shape((cols + vec - 1) / vec, vec);
    const uint32_t block = std::max(256u, shape.threads), per_block = block / shape.threads;
    (void)hipGetLastError();
    void *params[] = {&a};
    return launch_kernel(pick_kernel<NormKernel>(dtype, vec, shape), dim3(std::min(kMaxBlocks, (rows + per_block - 1) / per_block)),
                         dim3(block), params, 0, static_cast<hipStream_t>(hip_stream), nullptr, nullptr);
}

uint64_t df11_rms_norm_grad_workspace(uint32_t rows, uint32_t cols) {
    return rows ? 4ull * grad_groups_bound(rows) * cols : 0;
}

int df11_rms_norm_grad(const void *s, uint64_t s_stride, const void *weight, uint32_t weight_dtype, const float *rstd,
                       const void *dy, uint64_t dy_stride, const void *dsum, uint64_t dsum_stride, uint32_t rows,
                       uint32_t cols, uint32_t dtype, void *dx, uint64_t dx_stride, void *dweight, void *workspace,
                       uint64_t workspace_bytes, void *hip_stream) {
    const uint32_t bytes = dtype_bytes(dtype);
    if (!bytes || cols == 0 || cols > (1u << 30) || rows > (1u << 30)) return DF11_E_INVALID_ARG;
    if (weight && weight_dtype != dtype && weight_dtype != DF11_FP32) return DF11_E_INVALID_ARG;
    if (dweight && !weight) return DF11_E_INVALID_ARG;
    const uint32_t wbytes = weight ? dtype_bytes(weight_dtype) : 0;
    const uint64_t w_span = static_cast<uint64_t>(wbytes) * cols;
    if ((weight && !aligned(weight, wbytes)) || (dweight && !aligned(dweight, wbytes))) return DF11_E_INVALID_ARG;
    if (rows && (!s || !rstd || !dy || !dx || !aligned(rstd, 4))) return DF11_E_INVALID_ARG;
    const void *ptrs[] = {s, dy, dsum, dx};
    const uint64_t strides[] = {s_stride, dy_stride, dsum_stride, dx_stride};
    for (int i = 0; i < 4 && rows; ++i)
        if (ptrs[i] && (!aligned(ptrs[i], bytes) || strides[i] > kMaxRowElements)) return DF11_E_INVALID_ARG;
    if (rows > 1 && dx_stride < cols) return DF11_E_INVALID_ARG;
    const uint64_t need = dweight ? df11_rms_norm_grad_workspace(rows, cols) : 0;
    if (need && (!workspace || !aligned(workspace, 16))) return DF11_E_INVALID_ARG;
    if (workspace_bytes < need) return DF11_E_BUFFER_TOO_SMALL;
    // outputs: dx (may lie exactly on s, dy or dsum), dweight, the workspace
    const uint64_t dx_span = span_bytes(rows, cols, dx_stride, bytes);
    if (rows && (!apart_or_same(dx, dx_stride, s, s_stride, rows, cols, bytes) ||
                 !apart_or_same(dx, dx_stride, dy, dy_stride, rows, cols, bytes) ||
                 !apart_or_same(dx, dx_stride, dsum, dsum_stride, rows, cols, bytes)))
        return DF11_E_INVALID_ARG;
    const void *outs[] = {dx, dweight, workspace};
    const uint64_t spans[] = {dx_span, dweight ? w_span : 0, need};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], spans[i], outs[j], spans[j])) return DF11_E_INVALID_ARG;
        if (overlaps(outs[i], spans[i], weight, w_span) || overlaps(outs[i], spans[i], rstd, 4ull * rows))
            return DF11_E_INVALID_ARG;
        for (int k = 0; k < 3 && i; ++k)
            if (ptrs[k] && overlaps(outs[i], spans[i], ptrs[k], span_bytes(rows, cols, strides[k], bytes)))
                return DF11_E_INVALID_ARG;
    }
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    uint32_t groups = 0;
    float *partial = dweight ? static_cast<float *>(workspace) : nullptr;
    (void)hipGetLastError();
    if (rows) {
        uint32_t vec = row_vector(bytes, cols, ptrs, strides, 4);
        if (weight && !aligned(weight, 16)) vec = 1;
        const RowShape shape = row_shape((cols + vec - 1) / vec, vec);
        const uint32_t block = std::max(256u, shape.threads), per_block = block / shape.threads;
        groups = dweight ? grad_groups(rows, per_block)
                         : std::min(kMaxBlocks, (rows + per_block - 1) / per_block) * per_block;
        NormGradArgs a{s, weight, rstd, dy, dsum, dx, partial, s_stride, dy_stride, dsum_stride, dx_stride, rows, cols,
                       weight && weight_dtype == DF11_FP32};
        void *params[] = {&a};
        const int rc = launch_kernel(pick_kernel<NormGradKernel>(dtype, vec, shape), dim3(groups / per_block),
                                     dim3(block), params, 0, stream, nullptr, nullptr);
        if (rc) return rc;
    }
    return dweight ? df11::column_sums(partial, groups, cols, dweight, weight_dtype, stream) : DF11_OK;
}

}  // extern "C"
