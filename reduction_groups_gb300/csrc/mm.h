// The matrix product behind the linear layer and the orthogonalised update:
// the host's description of one launch (matmul.cu runs it).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace psk {

// A 16-bit operand in device memory: `outer` rows of `inner` contiguous
// elements, ld elements apart (16-byte aligned rows), in `planes` parts whose
// sum is the operand (plane after plane), one set of planes for each of the
// call's matrices.  k_inner: the contiguous direction is the summed one.
struct MMOperand {
  const void* p;
  int64_t inner, outer, ld, plane_stride;
  int planes;
  bool k_inner;
};

// Where a matrix of the orthogonalised update goes.
struct MMLeaf {
  void* y;
  int64_t ld, vec;
};

// An epilogue's kind: the orthogonalised update, the linear layer of any
// types, or of bf16 with an activation.
constexpr int MM_ORTHO = 16, MM_ANY = 17;

// What becomes of the accumulated product p(r, c).
struct MMEpilogue {
  // The linear layer: z = p + bias, y = act(z) + residual.  NULL: not there.
  const void *bias, *res;
  void *y, *z;
  int64_t ldr, ldy, ldz;
  int32_t bt, rt, yt, zt, act;
  // The orthogonalised update: v = alpha p + beta r, r and v matrices of fp16 planes (`ld`, a
  // multiple of 16, `plane_stride`, matrix after matrix), or v stored into leaves[matrix] (DEVICE, type yt).
  float alpha, beta;
  const uint16_t* from;
  uint16_t* to;
  int64_t ld, plane_stride;
  int32_t planes;
  const MMLeaf* leaves;
  int32_t transposed;                           // the leaves hold v's transpose
};

struct MMCall {
  int64_t m, n, k;
  MMOperand a, b;               // a: m x k, b: k x n
  bool f16;                     // operands fp16, else bf16
  int pairs;                    // products of planes, in the order they are added
  uint8_t pa[8], pb[8];
  int64_t matrices;
  bool symmetric;               // m == n, the result its own transpose: one triangle is computed
  bool ortho;
  MMEpilogue e;
};

// Sums of columns from their parts, `blocks` rows of `cols`, taken beside the
// products: out = [out +] the sum.
struct MMColumnSums {
  const float* parts;
  void* out;
  int64_t cols;
  int32_t blocks, dt, add;
};

// One product, or two (of no activation) whose tiles are shared out together
// (`count`), and column sums or NULL.
int mm_launch(const MMCall* calls, int count, const MMColumnSums* sums, cudaStream_t stream);

}  // namespace psk
