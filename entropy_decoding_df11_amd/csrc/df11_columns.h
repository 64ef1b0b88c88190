// Column sums of float partial rows, the end of bias and norm-weight
// gradients.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace df11 {

// out[c] (cols elements of dtype) = sum over rows of p[row][c], rounded once,
// in an order that rows alone fixes.  With no rows the sums are zero.
int column_sums(const float *p, uint32_t rows, uint32_t cols, void *out, uint32_t dtype, hipStream_t stream);

}  // namespace df11
