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
};

// One product.  R x C are a weight's rows and columns; tokens x K the left
// operand, K = C forward and R backward, tokens x N the output.
struct DenseCall {
    DenseMode mode;
    const uint16_t *left[2];  // BF16 rows, 16-byte aligned; [1] only backward with two weights
    uint64_t left_stride;     // elements, a multiple of 8
    const uint16_t *w[2];     // decoded weights in tile order
    uint32_t tokens, rows, cols;
};

// Workspace bytes of dense_product on the current device (partial sums of a
// split; 0 if it does not split), or ~0 if the device cannot be asked.
uint64_t dense_workspace(DenseMode mode, uint32_t n, uint32_t tokens, uint32_t rows, uint32_t cols);

// Launches the product with its epilogue (e.pre as for the epilogue; the
// bias, activation and residual fields are unused backward).
int dense_product(const DenseCall &c, const Epilogue &e, float *workspace, hipStream_t stream);

}  // namespace df11
