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
// an order that depends on the width and the type alone: results do not
// change from call to call.  (The rows' sums of the weight's gradient depend
// on the number of rows too.)
//
// What bounds them is memory.  bf16 with a residual, kernels' own times on
// buffers taken in turn (none cached): forward 8192 x 4096 (268 MB) 49.8 us,
// 5.4 TB/s; 2048 rows of it 15.8 us, 64 rows 4.3; backward with the weight's
// gradient, the column sums after it added, 44.6 + 4.0 (268 MB, 5.5 TB/s),
// 16.6 + 4.0 and 8.4 + 3.1.  A large copy reaches 4.7 TB/s.
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

// Rows are read and written in vectors of 16 bytes, at any alignment of their
// elements (the card loads and stores unaligned vectors); a row's last vector
// may be a part of one, `left` being the elements from its first to the end.
// (8192 x 4095 bf16 forward 85 to 94 us, where no row is aligned to more than
// its elements and nearly every vector lies across two aligned ones; one
// element at a time 183 us.)
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Unaligned {
    vec_t<T, kVec<T>> v;
};

template <typename T>
__device__ __forceinline__ vec_t<T, kVec<T>> load_row(const T *p, uint32_t left) {
    if (left >= static_cast<uint32_t>(kVec<T>)) return reinterpret_cast<const Unaligned<T> *>(p)->v;
    vec_t<T, kVec<T>> v = {};
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
        if (e < static_cast<int>(left)) v[e] = p[e];
    return v;
}

template <typename T>
__device__ __forceinline__ void store_row(T *p, uint32_t left, const float (&f)[kVec<T>]) {
    vec_t<T, kVec<T>> v;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) v[e] = static_cast<T>(f[e]);
    if (left >= static_cast<uint32_t>(kVec<T>)) {
        reinterpret_cast<Unaligned<T> *>(p)->v = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
        if (e < static_cast<int>(left)) p[e] = v[e];
}

// The weights of one vector of T (float32 weights may go with any T).
template <typename T>
__device__ __forceinline__ void load_weight(const void *weight, uint32_t f32, uint32_t i, uint32_t left,
                                            float (&w)[kVec<T>]) {
    if (!weight) {
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) w[e] = 1.0f;
    } else if (f32) {
#pragma unroll
        for (int q = 0; q < kVec<T>; q += 4) {
            const vec_t<float, 4> v =
                load_row(static_cast<const float *>(weight) + i + q, left > static_cast<uint32_t>(q) ? left - q : 0u);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[q + e] = v[e];
        }
    } else {
        const vec_t<T, kVec<T>> v = load_row(static_cast<const T *>(weight) + i, left);
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) w[e] = static_cast<float>(v[e]);
    }
}

// Threads of a block: one row, or as many rows as 256 threads hold where a
// row needs no more than a wave.
__host__ __device__ constexpr int block_threads(int tpr) { return tpr <= static_cast<int>(kWaveSize) ? 256 : tpr; }

// Sum of v over the TPR threads of a row, in every one of them.  Within a
// wave it needs no LDS; the waves of a wider row meet in s_part.
template <int TPR>
__device__ __forceinline__ float row_total(float v, float *s_part) {
#pragma unroll
    for (int m = (TPR < static_cast<int>(kWaveSize) ? TPR : static_cast<int>(kWaveSize)) / 2; m; m >>= 1)
        v += __shfl_xor(v, m);
    if constexpr (TPR > static_cast<int>(kWaveSize)) {
        if ((threadIdx.x & (kWaveSize - 1)) == 0) s_part[threadIdx.x / kWaveSize] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / static_cast<int>(kWaveSize); ++w) v += s_part[w];
    }
    return v;
}

// TPR threads per row, NV vectors held per thread.  kWide: rows beyond TPR *
// NV vectors, whose elements past the held ones are read a second time for
// the output (from the sum where one is written).
template <typename T, int NV, int TPR, bool kWide>
__global__ __launch_bounds__(block_threads(TPR)) void df11_rms_norm_kernel(NormArgs a) {
    constexpr int VEC = kVec<T>, kRows = block_threads(TPR) / TPR;
    using Vec = vec_t<T, VEC>;
    __shared__ float s_part[2][block_threads(TPR) / kWaveSize];
    const uint32_t lid = threadIdx.x % TPR;
    uint32_t turn = 0;
    // (one row per group of threads, unless the rows outnumber the largest
    // grid; a row's waves leave the loop together)
    for (uint32_t row = blockIdx.x * kRows + threadIdx.x / TPR; row < a.rows; row += gridDim.x * kRows, turn ^= 1u) {
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
        T *sum = a.sum ? static_cast<T *>(a.sum) + row * a.sum_stride : nullptr;
        T *y = static_cast<T *>(a.y) + row * a.y_stride;

        // One vector's s = round(x + residual).
        auto add = [&](const Vec &vx, const Vec &vr, float (&s)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[e] = static_cast<float>(vx[e]);
                if (res) s[e] = static_cast<float>(static_cast<T>(s[e] + static_cast<float>(vr[e])));
            }
        };
        auto put = [&](uint32_t i, const float (&s)[VEC], float r) {
            float w[VEC];
            load_weight<T>(a.weight, a.weight_f32, i, a.cols - i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] *= s[e] * r;
            store_row(y + i, a.cols - i, w);
        };
        Vec vx[NV], vr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            vx[j] = vr[j] = Vec{};
            if (i < a.cols) {
                vx[j] = load_row(x + i, a.cols - i);
                if (res) vr[j] = load_row(res + i, a.cols - i);
            }
        }
        float v[NV][VEC];
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            add(vx[j], vr[j], v[j]);
            if (sum && i < a.cols) store_row(sum + i, a.cols - i, v[j]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) total += v[j][e] * v[j][e];
        }
        if constexpr (kWide) {
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC) {
                float s[VEC];
                add(load_row(x + i, a.cols - i), res ? load_row(res + i, a.cols - i) : Vec{}, s);
                if (sum) store_row(sum + i, a.cols - i, s);
#pragma unroll
                for (int e = 0; e < VEC; ++e) total += s[e] * s[e];
            }
        }
        total = row_total<TPR>(total, s_part[turn]);
        // (the quotient and the root are each rounded to float)
        const float r = 1.0f / sqrtf(total / static_cast<float>(a.cols) + a.eps);
        if (a.rstd && lid == 0) a.rstd[row] = r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) put(i, v[j], r);
        }
        if constexpr (kWide) {
            // Each thread reads back only what it wrote or read itself, so the
            // output may be x's or the residual's own buffer.
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC) {
                float s[VEC];
                if (sum) {
                    const Vec back = load_row(static_cast<const T *>(sum) + i, a.cols - i);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s[e] = static_cast<float>(back[e]);
                } else {
                    add(load_row(x + i, a.cols - i), res ? load_row(res + i, a.cols - i) : Vec{}, s);
                }
                put(i, s, r);
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
    float *partial;      // or null: [blocks][cols] sums of dy * h
    uint64_t s_stride, dy_stride, dsum_stride, dx_stride;
    uint32_t rows, cols;
    uint32_t weight_f32;
};

// A row group (the TPR threads of one row at a time) takes rows g, g + G,
// g + 2 G, ... of the G groups of the launch, and keeps its sums of dy * h
// for the columns its threads hold in registers; at the end a block's groups
// add theirs in LDS, in order, and the block's sums leave once.
template <typename T, int NV, int TPR, bool kWide>
__global__ __launch_bounds__(block_threads(TPR)) void df11_rms_norm_grad_kernel(NormGradArgs a) {
    constexpr int VEC = kVec<T>, kRows = block_threads(TPR) / TPR;
    using Vec = vec_t<T, VEC>;
    __shared__ float s_part[2][block_threads(TPR) / kWaveSize];
    const uint32_t lid = threadIdx.x % TPR;
    const float inv = 1.0f / static_cast<float>(a.cols);
    float acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.0f;
    float *part = a.partial ? a.partial + static_cast<uint64_t>(blockIdx.x) * a.cols : nullptr;
    // (a wide row's block is that row's alone: the sums past the held columns
    // are kept where they will leave, each by one thread)
    if constexpr (kWide) {
        if (part)
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC)
                for (uint32_t e = 0; e < VEC && i + e < a.cols; ++e) part[i + e] = 0.0f;
    }
    uint32_t turn = 0;
    for (uint32_t row = blockIdx.x * kRows + threadIdx.x / TPR; row < a.rows; row += gridDim.x * kRows, turn ^= 1u) {
        const T *s = static_cast<const T *>(a.s) + row * a.s_stride;
        const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
        const T *ds = a.dsum ? static_cast<const T *>(a.dsum) + row * a.dsum_stride : nullptr;
        T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
        const float r = a.rstd[row];
        // (held packed, as loaded: the floats of four vectors a thread would
        // not fit the registers of 1024 threads)
        Vec sv[NV], dv[NV], gv[NV];
        float total = 0.0f;
        // h = s * rstd, d = dy * weight, raw = dy of one vector
        auto expand = [&](uint32_t i, const Vec &ps, const Vec &pd, float (&h)[VEC], float (&d)[VEC],
                          float (&raw)[VEC]) {
            float w[VEC];
            load_weight<T>(a.weight, a.weight_f32, i, a.cols - i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] = static_cast<float>(ps[e]) * r;
                raw[e] = static_cast<float>(pd[e]);
                d[e] = raw[e] * w[e];
            }
        };
        // the incoming gradients of the sum; zeros without them
        auto through = [&](uint32_t i) { return ds ? load_row(ds + i, a.cols - i) : Vec{}; };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) {
                sv[j] = load_row(s + i, a.cols - i);
                dv[j] = load_row(dy + i, a.cols - i);
                if constexpr (NV == 1) gv[j] = through(i);
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
                expand(i, load_row(s + i, a.cols - i), load_row(dy + i, a.cols - i), h, d, raw);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    total += d[e] * h[e];
                    if (part && i + e < a.cols) part[i + e] += raw[e] * h[e];
                }
            }
        }
        // (two sets of wave sums, in turn: a wave may enter the next row's
        // sum while another still reads this one's)
        const float mean = row_total<TPR>(total, s_part[turn]) * inv;
        auto put = [&](uint32_t i, const Vec &ps, const Vec &pd, const Vec &pg) {
            float g[VEC], h[VEC], d[VEC], raw[VEC];
            expand(i, ps, pd, h, d, raw);
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = static_cast<float>(pg[e]) + r * (d[e] - h[e] * mean);
            store_row(dx + i, a.cols - i, g);
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t i = (j * TPR + lid) * VEC;
            if (i < a.cols) {
                if constexpr (NV > 1) gv[j] = through(i);
                put(i, sv[j], dv[j], gv[j]);
            }
        }
        if constexpr (kWide) {
            for (uint32_t i = (NV * TPR + lid) * VEC; i < a.cols; i += TPR * VEC)
                put(i, load_row(s + i, a.cols - i), load_row(dy + i, a.cols - i), through(i));
        }
    }
    if (!part) return;
    if constexpr (kRows > 1) {
        static_assert(NV == 1);
        __shared__ float s_acc[VEC][kRows][TPR];
#pragma unroll
        for (int e = 0; e < VEC; ++e) s_acc[e][threadIdx.x / TPR][lid] = acc[0][e];
        __syncthreads();
        if (threadIdx.x >= TPR) return;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            for (int g = 1; g < kRows; ++g) acc[0][e] += s_acc[e][g][lid];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t i = (j * TPR + lid) * VEC;
#pragma unroll
        for (int q = 0; q < VEC; q += 4)
            if (i + q < a.cols) {
                const float f[4] = {acc[j][q], acc[j][q + 1], acc[j][q + 2], acc[j][q + 3]};
                store_row(part + i + q, a.cols - i - q, f);
            }
    }
}

// Most blocks of a launch (a grid's threads are counted in 32 bits); the rows
// or columns past them are taken in further turns.
constexpr uint32_t kMaxBlocks = 1u << 20;

// out[c] = sum over the rows of p[row][c], in row order within each of the
// block's 16 slices of rows, then over the slices.
__global__ __launch_bounds__(1024) void df11_column_sum_kernel(const float *p, uint32_t rows, uint32_t cols,
                                                               void *out, uint32_t dtype) {
    __shared__ float s_sum[16][kWaveSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), slice = threadIdx.x / kWaveSize;
    for (uint32_t c0 = blockIdx.x * kWaveSize; c0 < cols; c0 += gridDim.x * kWaveSize) {
        const uint32_t c = c0 + lane;
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
        __syncthreads();
    }
}

// Threads per row and vectors per thread for a row of n vectors: the fewest
// threads that hold it at a vector each, up to the 1024 of a block.  Several
// vectors a thread leave the loads of a row to fewer waves: bf16 rows of 2048,
// 64 threads of four vectors against 256 of one, 64 rows forward 4.4 against
// 3.0 us and backward 11.6 against 5.4, 16384 rows 55 against 49 and 156
// against 65.  More threads than vectors idle: 262144 rows of 128, 64 threads
// against 16, forward 88 against 50 us; 8192 rows of 4096, 1024 against 512,
// 72 against 50.  Past 4096 vectors the remainder of a row is read twice: four
// vectors held against two, 1024 rows of 32768, forward 54 against 58 us and
// backward 71 against 119; two held where they suffice, 2048 rows of 16384,
// 54.5 against 57.5 and 58.8 against 62.1.
struct RowShape {
    uint32_t threads, vectors;
    bool wide;
};

RowShape row_shape(uint64_t n) {
    for (uint32_t threads : {16u, 32u, 64u, 128u, 256u, 512u, 1024u})
        if (n <= threads) return {threads, 1, false};
    return {1024, n <= 2048 ? 2u : 4u, n > 4096};
}

template <template <typename, int, int, bool> class Pick, typename T>
const void *pick_shape(const RowShape &s) {
    if (s.wide) return Pick<T, 4, 1024, true>::get();
    if (s.vectors > 1) return s.vectors == 2 ? Pick<T, 2, 1024, false>::get() : Pick<T, 4, 1024, false>::get();
    switch (s.threads) {
    case 16: return Pick<T, 1, 16, false>::get();
    case 32: return Pick<T, 1, 32, false>::get();
    case 64: return Pick<T, 1, 64, false>::get();
    case 128: return Pick<T, 1, 128, false>::get();
    case 256: return Pick<T, 1, 256, false>::get();
    case 512: return Pick<T, 1, 512, false>::get();
    default: return Pick<T, 1, 1024, false>::get();
    }
}

template <template <typename, int, int, bool> class Pick>
const void *pick_kernel(uint32_t dtype, const RowShape &s) {
    if (dtype == DF11_FP32) return pick_shape<Pick, float>(s);
    return dtype == DF11_BF16 ? pick_shape<Pick, bf16_t>(s) : pick_shape<Pick, fp16_t>(s);
}

template <typename T, int NV, int TPR, bool kWide>
struct NormKernel {
    static const void *get() { return reinterpret_cast<const void *>(&df11_rms_norm_kernel<T, NV, TPR, kWide>); }
};
template <typename T, int NV, int TPR, bool kWide>
struct NormGradKernel {
    static const void *get() { return reinterpret_cast<const void *>(&df11_rms_norm_grad_kernel<T, NV, TPR, kWide>); }
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

// Blocks of the backward pass when it sums the weight's gradient: a block's
// sums cost four bytes a column written and read again, so each row group of
// a block takes at least kGradRows rows, and the launch has at most
// kGradThreads threads.  Bf16 rows of 4096, with the column sums after it: 64
// rows at one, two and four rows a group 6.3, 6.4 and 7.9 us, 512 rows 12.1,
// 10.1 and 10.3; 8192 rows in 2^18 threads 53.5 us, in 2^17 57.2.
constexpr uint32_t kGradRows = 2, kGradThreads = 1u << 18;

uint32_t grad_blocks(uint32_t rows, uint32_t per_block, uint32_t block) {
    const uint32_t each = kGradRows * per_block;
    return std::max(1u, std::min(kGradThreads / block, (rows + each - 1) / each));
}

// Whether the last row begins within 2^58 elements, so that its bytes and the
// extents that the overlap checks compare stay within 64 bits.
bool rows_fit(uint32_t rows, uint64_t stride) { return rows <= 1 || stride <= (1ull << 58) / (rows - 1ull); }

}  // namespace

namespace df11 {

int column_sums(const float *p, uint32_t rows, uint32_t cols, void *out, uint32_t dtype, hipStream_t stream) {
    void *params[] = {&p, &rows, &cols, &out, &dtype};
    return launch_kernel(reinterpret_cast<const void *>(&df11_column_sum_kernel),
                         dim3(std::min(kMaxBlocks, (cols + kWaveSize - 1) / kWaveSize)), dim3(1024), params, 0, stream,
                         nullptr, nullptr);
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
        if (!aligned(ptrs[i], bytes) || !rows_fit(rows, strides[i])) return DF11_E_INVALID_ARG;
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
    const RowShape shape = row_shape((static_cast<uint64_t>(cols) * bytes + 15) / 16);
    const uint32_t block = block_threads(static_cast<int>(shape.threads)), per_block = block / shape.threads;
    (void)hipGetLastError();
    void *params[] = {&a};
    return launch_kernel(pick_kernel<NormKernel>(dtype, shape), dim3(std::min(kMaxBlocks, (rows + per_block - 1) / per_block)),
                         dim3(block), params, 0, static_cast<hipStream_t>(hip_stream), nullptr, nullptr);
}

uint64_t df11_rms_norm_grad_workspace(uint32_t rows, uint32_t cols) {
    // (for the most blocks of any type's row shape)
    uint64_t blocks = 0;
    for (const uint32_t bytes : {2u, 4u}) {
        const RowShape shape = row_shape((static_cast<uint64_t>(cols) * bytes + 15) / 16);
        const uint32_t block = block_threads(static_cast<int>(shape.threads));
        blocks = std::max<uint64_t>(blocks, grad_blocks(rows, block / shape.threads, block));
    }
    return rows ? 4ull * blocks * cols : 0;
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
        if (ptrs[i] && (!aligned(ptrs[i], bytes) || !rows_fit(rows, strides[i]))) return DF11_E_INVALID_ARG;
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
    uint32_t blocks = 0;
    float *partial = dweight ? static_cast<float *>(workspace) : nullptr;
    (void)hipGetLastError();
    if (rows) {
        const RowShape shape = row_shape((static_cast<uint64_t>(cols) * bytes + 15) / 16);
        const uint32_t block = block_threads(static_cast<int>(shape.threads)), per_block = block / shape.threads;
        blocks = dweight ? grad_blocks(rows, per_block, block)
                         : std::min(kMaxBlocks, (rows + per_block - 1) / per_block);
        NormGradArgs a{s, weight, rstd, dy, dsum, dx, partial, s_stride, dy_stride, dsum_stride, dx_stride, rows, cols,
                       weight && weight_dtype == DF11_FP32};
        void *params[] = {&a};
        const int rc = launch_kernel(pick_kernel<NormGradKernel>(dtype, shape), dim3(blocks),
                                     dim3(block), params, 0, stream, nullptr, nullptr);
        if (rc) return rc;
    }
    return dweight ? df11::column_sums(partial, blocks, cols, dweight, weight_dtype, stream) : DF11_OK;
}

}  // extern "C"
