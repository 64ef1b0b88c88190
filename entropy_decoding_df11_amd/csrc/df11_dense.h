// Products with a matrix that has been decoded in MFMA tile order
// (df11_tile_order), for more tokens than one sweep of the fused product
// takes, and for gradients.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "df11_epilogue.h"

namespace df11 {

enum DenseMode {
    kDensePlain = 0,  // x W^T
    kDenseGated = 1,  // x Wg^T and x Wu^T, met in the epilogue
    kDenseBack = 2,   // d W (summed over one or two pairs): the gradient of x
    // Of the softmax cross entropy (df11_loss.hip), one weight's rows being
    // classes: statistics of x W^T without the sums themselves, the same with
    // their exponentials in BF16, and exponentials times W added to what is there.
    kDenseStats = 3,
    kDenseExp = 4,
    kDenseBackAdd = 5,
};

// What those modes read and write beside the operands.  A token's exponentials
// are 2^(z log2(e) - r) with a whole r, so that r changes without a rounding;
// the target's own is left out (zero).
struct DenseLoss {
    const int64_t *targets;
    float *stats;          // [panel of 64 classes][token][2]: r (-inf: no class) and the sum
    float *target_logit;   // [token], written where the target is among the rows
    const float *ref;      // kDenseExp: [token] r to use while no logit passes it by 2^kRefRoom
    float *rounded;        // kDenseExp: [panel][token], the sum of what exps holds
    uint16_t *exps;        // kDenseExp: [token][exps_stride]
    const float *scale;    // kDenseBackAdd: [token], of what is in e.out
    uint64_t exps_stride;  // a multiple of 8
    uint32_t first_class;  // class of the first row
    uint32_t classes;      // classes from there on are padding
};

// How far, in powers of two, a logit may pass the reference that its token has:
// the largest exponentials and their sums stay far from float's and BF16's range.
constexpr float kRefRoom = 64.0f;

// log2(e) in two floats.
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596303350001107901e-8f;

// The exponent z log2(e) - r of a class, r whole: to 2^-24 for a logit of 100.  r was
// rounded from z kLog2eHi; from logits of 2^24 on its last place is more than a whole
// number (many powers of two from 2^30 on), and the difference is taken of products
// that are rounded alike.
__device__ __forceinline__ float class_exponent(float z, float r) {
#pragma clang fp contract(off)
    const float rounded = z * kLog2eHi - r;
    return __builtin_fabsf(z) < 16777216.0f ? __builtin_fmaf(z, kLog2eLo, __builtin_fmaf(z, kLog2eHi, -r)) : rounded;
}

// One product.  R x C are a weight's rows and columns; tokens x K the left
// operand, K = C forward and R backward, tokens x N the output.
struct DenseCall {
    DenseMode mode;
    const uint16_t *left[2];  // BF16 rows, 16-byte aligned; [1] only backward with two weights
    uint64_t left_stride;     // elements, a multiple of 8
    const uint16_t *w[2];     // decoded weights in tile order
    uint32_t tokens, rows, cols;
    DenseLoss loss;           // kDenseStats, kDenseExp, kDenseBackAdd
};

// Workspace bytes of dense_product on the current device (partial sums of a
// split; 0 if it does not split), or ~0 if the device cannot be asked.
uint64_t dense_workspace(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols);

// Whether a launch holds the product's workgroups: DF11_OK, DF11_E_TOO_LARGE or
// DF11_E_HIP.  (dense_product asks too; a caller that launches something else first
// asks before that.)
int dense_fits(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols);

// Launches the product with its epilogue (e.pre as for the epilogue; the
// bias, activation and residual fields are unused backward, where kDenseBackAdd
// adds to the float e.out; all of it is unused by kDenseStats and kDenseExp).
int dense_product(const DenseCall &c, const Epilogue &e, float *workspace, hipStream_t stream);

}  // namespace df11
