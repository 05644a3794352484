// psk_orthogonalize: Newton-Schulz products on a list of matrices of one
// shape.  With the shorter side m and the longer n (a tall matrix is taken
// transposed), X of m rows and n columns:
//   X = G / (||G||_F + eps);   A = X X^T,  B = b A + c A A,  X <- a X + B X.
// A and A A are symmetric: the product kernel computes one triangle of tiles
// and stores each tile twice.
//
// The iterates live in the workspace as fp16 times S = 2^10: X's singular
// values stay near 1 and its elements below that, so fp16's 11 bits are kept
// down to elements of 2^-24 and what is above 64 overflows.
//
// X is held in two fp16 parts (22 bits).  Directions of small singular values
// grow by a each step and carry X's rounding with them, but through the term
// a X alone: B, a polynomial without constant term, all but vanishes on them.
// So a X takes both parts, in the epilogue, and for a result stored in bf16
// the products take the first part, and A and B one part: the result's error
// is 3e-4 to 1e-3 of its size then (3e-3 to 4e-3 with X in one part; bf16's
// own rounding is 1.7e-3).  For a result stored in f32 A and B are two parts
// as well and every product three products of parts.
#include <algorithm>
#include <vector>

#include "common.cuh"
#include "vec8.cuh"
#include "mm.h"
#include "views.h"

namespace psk {

constexpr float ORTHO_SCALE = 1024.0f;
constexpr int ORTHO_MAX_LEAVES = PSK_ORTHO_MAX_LEAVES;
constexpr int ORTHO_PARTS = 2;                      // of X
constexpr int ORTHO_SUM_BLOCKS = 64;                // of a matrix's square sum, at most
constexpr int64_t ORTHO_MAX_SIDE = 1 << 20;

struct OrthoTable {
  const void* x[ORTHO_MAX_LEAVES];
  int64_t ldx[ORTHO_MAX_LEAVES];
};
struct OrthoTargets {
  void* y[ORTHO_MAX_LEAVES];
  int64_t ldy[ORTHO_MAX_LEAVES];
  uint8_t vec[ORTHO_MAX_LEAVES];
};

struct OrthoShape {
  int64_t rows, cols;           // of a leaf
  int64_t m, n, ldn, ldm;
  int32_t xt, tall, blocks, leaves;
  double eps;
  double* sums;                 // [leaf][block]
  MMLeaf* table;
  uint16_t* x;                  // [leaf][part][m][ldn]
};

// Where the results go, for the last product's epilogue.
__global__ void ortho_targets_kernel(const __grid_constant__ OrthoTargets T, MMLeaf* table, int leaves) {
  for (int i = threadIdx.x; i < leaves; i += blockDim.x) table[i] = MMLeaf{T.y[i], T.ldy[i], T.vec[i]};
}

// A block of rows' sum of squares: f32 within a thread's row, 64 bits beyond.
// Elements above 2^50, whose squares would leave f32, are taken times 2^-64.
__global__ void __launch_bounds__(256) ortho_sum_kernel(const __grid_constant__ OrthoTable T, OrthoShape S) {
  __shared__ double part[8];
  const int leaf = blockIdx.x / S.blocks, block = blockIdx.x % S.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const void* x = T.x[leaf];
  const int64_t ld = T.ldx[leaf];
  double total = 0.0;
  for (int64_t r = (int64_t)block * 8 + warp; r < S.rows; r += (int64_t)S.blocks * 8) {
    float s = 0.0f, big = 0.0f;
    for (int64_t c = lane; c < S.cols; c += 32) {
      const int64_t i = r * ld + c;
      const float v = S.xt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)x)[i]) : ((const float*)x)[i];
      if (fabsf(v) > 1.1e15f) {
        const float u = v * 5.421010862427522e-20f;
        big = fmaf(u, u, big);
      } else {
        s = fmaf(v, v, s);
      }
    }
    total += (double)s + (double)big * 3.402823669209385e38;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane == 0) part[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) total += part[w];
    S.sums[blockIdx.x] = total;
  }
}

__device__ __forceinline__ uint32_t to_f16(float f) {
  uint16_t h;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(f));
  return h;
}
__device__ __forceinline__ float from_f16(uint32_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)h));
  return f;
}

// The first iterate: 64 x 64 of it a CTA, through shared memory, so that the
// leaf's rows and the iterate's are both walked along.
__global__ void __launch_bounds__(256) ortho_begin_kernel(const __grid_constant__ OrthoTable T, OrthoShape S) {
  __shared__ float tile[64][65];
  __shared__ float factor;
  const int64_t tn = (S.ldn + 63) / 64, tm = (S.m + 63) / 64;
  const int64_t leaf = blockIdx.x / (tn * tm), at = blockIdx.x % (tn * tm);
  const int64_t r0 = at / tn * 64, c0 = at % tn * 64;
  const void* x = T.x[leaf];
  const int64_t ld = T.ldx[leaf];
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < S.blocks; ++i) s += S.sums[leaf * S.blocks + i];
    factor = (float)((double)ORTHO_SCALE / (sqrt(s) + S.eps));
  }
  __syncthreads();
  const float f = factor;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int a = i >> 6, b = i & 63;                      // b along the leaf's rows
    const int64_t r = r0 + (S.tall ? b : a), c = c0 + (S.tall ? a : b);
    float v = 0.0f;
    if (r < S.m && c < S.n) {
      const int64_t e = S.tall ? c * ld + r : r * ld + c;
      v = (S.xt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)x)[e]) : ((const float*)x)[e]) * f;
    }
    if (S.tall) tile[b][a] = v;
    else tile[a][b] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {
    const int a = i >> 3, g = (i & 7) * 8;
    if (r0 + a >= S.m || c0 + g >= S.ldn) continue;
    uint16_t* q = S.x + leaf * ORTHO_PARTS * S.m * S.ldn + (r0 + a) * S.ldn + c0 + g;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = tile[a][g + k];
#pragma unroll
    for (int p = 0; p < ORTHO_PARTS; ++p) {
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[k] = to_f16(v[k]);
        v[k] -= from_f16(h[k]);
      }
      *(uint4*)(q + p * S.m * S.ldn) = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                                  h[6] | h[7] << 16);
    }
  }
}

struct OrthoLayout {
  uint64_t sums, table, x0, x1, a, b, bytes;
  int64_t xsize, asize;         // elements of one plane
};

static int64_t ortho_up8(int64_t v) { return (v + 7) / 8 * 8; }

static OrthoLayout ortho_layout(int32_t leaves, int64_t rows, int64_t cols, int32_t yt) {
  OrthoLayout L{};
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  const int planes = yt == PSK_F32 ? 2 : 1;
  L.xsize = m * ortho_up8(n), L.asize = m * ortho_up8(m);
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  L.sums = take((uint64_t)leaves * ORTHO_SUM_BLOCKS * 8);
  L.table = take((uint64_t)leaves * sizeof(MMLeaf));
  L.x0 = take((uint64_t)leaves * ORTHO_PARTS * L.xsize * 2);
  L.x1 = take((uint64_t)leaves * ORTHO_PARTS * L.xsize * 2);
  L.a = take((uint64_t)leaves * planes * L.asize * 2);
  L.b = take((uint64_t)leaves * planes * L.asize * 2);
  L.bytes = at;
  return L;
}

static int ortho_check_sizes(int32_t leaves, int64_t rows, int64_t cols) {
  if (leaves < 0 || leaves > ORTHO_MAX_LEAVES) return fail(PSK_E_ARG, "%d matrices, at most %d", leaves, ORTHO_MAX_LEAVES);
  if (rows < 0 || cols < 0 || rows > ORTHO_MAX_SIDE || cols > ORTHO_MAX_SIDE)
    return fail(PSK_E_SHAPE, "rows %lld, cols %lld: not in [0, 2^20]", (long long)rows, (long long)cols);
  return PSK_OK;
}

}  // namespace psk

using namespace psk;

extern "C" int psk_orthogonalize_workspace(int32_t n_leaves, int64_t rows, int64_t cols, int32_t yt, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = ortho_check_sizes(n_leaves, rows, cols);
  if (rc) return rc;
  if (!dtype_ok(yt)) return fail(PSK_E_DTYPE, "y dtype %d", yt);
  *bytes = n_leaves && rows && cols ? ortho_layout(n_leaves, rows, cols, yt).bytes : 0;
  return PSK_OK;
}

extern "C" int psk_orthogonalize(const psk_ortho_leaf* leaves, int32_t n_leaves, int64_t rows, int64_t cols, int32_t xt,
                                 int32_t yt, const double* coefficients, int32_t steps, double eps, double scale,
                                 void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  int rc = ortho_check_sizes(n_leaves, rows, cols);
  if (rc) return rc;
  if (!dtype_ok(xt)) return fail(PSK_E_DTYPE, "x dtype %d", xt);
  if (!dtype_ok(yt)) return fail(PSK_E_DTYPE, "y dtype %d", yt);
  if (steps < 1 || steps > 64) return fail(PSK_E_ARG, "%d steps: not in [1, 64]", steps);
  if (!coefficients) return fail(PSK_E_NULL, "coefficients is NULL");
  for (int i = 0; i < 3 * steps; ++i)
    if (!(coefficients[i] >= -32.0 && coefficients[i] <= 32.0))
      return fail(PSK_E_ARG, "coefficient %d is not in [-32, 32]", i);
  if (!(eps >= 0.0 && eps <= 1e30)) return fail(PSK_E_ARG, "eps is not in [0, 1e30]");
  if (!(scale >= -1e30 && scale <= 1e30)) return fail(PSK_E_ARG, "scale is not in [-1e30, 1e30]");
  if (!n_leaves || !rows || !cols) return PSK_OK;
  if (!leaves) return fail(PSK_E_NULL, "leaves is NULL");
  const OrthoLayout L = ortho_layout(n_leaves, rows, cols, yt);
  if (!workspace) return fail(PSK_E_NULL, "workspace is NULL");
  if ((uintptr_t)workspace % 16) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
  if (workspace_bytes < L.bytes)
    return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                (unsigned long long)L.bytes);
  static thread_local OrthoTable T;
  static thread_local OrthoTargets Y;
  const View vws{(uintptr_t)workspace, 1, L.bytes, L.bytes};
  std::vector<View> out;
  try {
    out.reserve(n_leaves);
  } catch (...) {
    return fail(PSK_E_ARG, "out of host memory");
  }
  for (int i = 0; i < n_leaves; ++i) {
    const psk_ortho_leaf& f = leaves[i];
    if (!f.x || !f.y) return fail(PSK_E_NULL, "matrix %d: x or y is NULL", i);
    if ((uintptr_t)f.x % dtype_size(xt) || (uintptr_t)f.y % dtype_size(yt))
      return fail(PSK_E_ARG, "matrix %d is not aligned to its type", i);
    if (f.ldx < cols || f.ldy < cols) return fail(PSK_E_SHAPE, "matrix %d: leading dimension below cols", i);
    if (!rows_addressable(rows, f.ldx) || !rows_addressable(rows, f.ldy))
      return fail(PSK_E_SHAPE, "matrix %d: rows x leading dimension too large", i);
    const View vx = view_of(f.x, rows, cols, f.ldx, dtype_size(xt)), vy = view_of(f.y, rows, cols, f.ldy, dtype_size(yt));
    if (views_overlap(vx, vws) || views_overlap(vy, vws)) return fail(PSK_E_ALIAS, "matrix %d overlaps the workspace", i);
    out.push_back(vy);
    T.x[i] = f.x, T.ldx[i] = f.ldx;
    Y.y[i] = f.y, Y.ldy[i] = f.ldy, Y.vec[i] = rows_vec8(f.y, yt, f.ldy, rows);
  }
  std::sort(out.begin(), out.end(), [](const View& a, const View& b) { return a.p < b.p; });
  for (size_t i = 0; i < out.size(); ++i)
    for (size_t j = i + 1; j < out.size() && out[j].p < out[i].p + out[i].bytes(); ++j)
      if (views_overlap(out[i], out[j])) return fail(PSK_E_ALIAS, "two results overlap");

  cudaStream_t s = (cudaStream_t)stream;
  char* ws = (char*)workspace;
  OrthoShape S{};
  S.rows = rows, S.cols = cols;
  S.tall = rows > cols;
  S.m = S.tall ? cols : rows, S.n = S.tall ? rows : cols;
  S.ldn = ortho_up8(S.n), S.ldm = ortho_up8(S.m);
  S.xt = xt, S.leaves = n_leaves;
  const int planes = yt == PSK_F32 ? 2 : 1;
  int64_t blocks = (rows + 31) / 32;
  S.blocks = (int32_t)(blocks < ORTHO_SUM_BLOCKS ? blocks : ORTHO_SUM_BLOCKS);
  S.eps = eps;
  S.sums = (double*)(ws + L.sums), S.table = (MMLeaf*)(ws + L.table), S.x = (uint16_t*)(ws + L.x0);
  ortho_targets_kernel<<<1, 256, 0, s>>>(Y, S.table, n_leaves);
  ortho_sum_kernel<<<(unsigned)(n_leaves * S.blocks), 256, 0, s>>>(T, S);
  const int64_t tiles = (S.ldn + 63) / 64 * ((S.m + 63) / 64) * n_leaves;
  if (tiles > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many tiles");
  ortho_begin_kernel<<<(unsigned)tiles, 256, 0, s>>>(T, S);
  rc = check_launch("orthogonalisation's first kernels");
  uint16_t *x = S.x, *x2 = (uint16_t*)(ws + L.x1), *A = (uint16_t*)(ws + L.a), *B = (uint16_t*)(ws + L.b);
  const auto wide = [&](const uint16_t* p, bool k_inner) {
    return MMOperand{p, S.n, S.m, S.ldn, L.xsize, ORTHO_PARTS, k_inner};
  };
  const auto square = [&](const uint16_t* p) { return MMOperand{p, S.m, S.m, S.ldm, L.asize, planes, true}; };
  MMCall C{};
  C.f16 = true, C.matrices = n_leaves, C.kind = MM_ORTHO;
  if (planes == 1) {
    C.pairs = 1;
  } else {
    C.pairs = 3;
    C.pa[0] = 1, C.pb[0] = 0, C.pa[1] = 0, C.pb[1] = 1;     // the small products first
  }
  C.e.yt = yt;
  for (int i = 0; !rc && i < steps; ++i) {
    const double a = coefficients[3 * i], b = coefficients[3 * i + 1], c = coefficients[3 * i + 2];
    const bool last = i + 1 == steps;
    // A S = (X S)(X S)^T / S
    C.m = C.n = S.m, C.k = S.n, C.symmetric = true;
    C.a = wide(x, true), C.b = wide(x, true);
    C.e.alpha = 1.0f / ORTHO_SCALE, C.e.beta = 0.0f, C.e.from = nullptr, C.e.to = A;
    C.e.ld = S.ldm, C.e.plane_stride = L.asize, C.e.planes = planes;
    rc = mm_launch(C, s);
    if (rc) break;
    // B S = b (A S) + c (A S)(A S) / S
    C.k = S.m;
    C.a = square(A), C.b = square(A);
    C.e.alpha = (float)(c / ORTHO_SCALE), C.e.beta = (float)b, C.e.from = A, C.e.to = B;
    rc = mm_launch(C, s);
    if (rc) break;
    // X S <- a (X S) + (B S)(X S) / S
    C.n = S.n, C.symmetric = false, C.e.transposed = S.tall;
    C.a = square(B), C.b = wide(x, false);
    const double out_scale = last ? scale / ORTHO_SCALE : 1.0;
    C.e.alpha = (float)(out_scale / ORTHO_SCALE), C.e.beta = (float)(a * out_scale);
    C.e.from = x, C.e.to = last ? nullptr : x2, C.e.leaves = S.table;
    C.e.ld = S.ldn, C.e.plane_stride = L.xsize, C.e.planes = ORTHO_PARTS;
    rc = mm_launch(C, s);
    std::swap(x, x2);
  }
  return rc;
}
