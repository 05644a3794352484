// The orthogonalised update of small matrices (ortho_small.cu).
#pragma once

#include <cuda_runtime.h>

#include "../../include/psk.h"

namespace psk {

// The shorter and the longer side that one CTA takes.
constexpr int ORTHO_SMALL_M = 128, ORTHO_SMALL_N = 256;

// The factor in two: of matrices beyond 2^64 it would lose bits below f32's
// normal range.
__device__ __forceinline__ float2 ortho_factors(double f) {
  return f < 5.551115123125783e-17 ? make_float2(5.421010862427522e-20f, (float)(f * 18446744073709551616.0))
                                   : make_float2(1.0f, (float)f);
}

// copies: the x's one behind the other, or NULL: where the leaves have them.
int ortho_small_launch(const psk_ortho_leaf* leaves, const char* copies, int n_leaves, int64_t rows, int64_t cols, int32_t xt, int32_t yt,
                       const double* coefficients, int32_t steps, double eps, double scale, cudaStream_t stream);

}  // namespace psk
