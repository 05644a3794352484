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
// the products take the first part, and A and B one part.  The iteration
// amplifies their roundings: beside bf16's own rounding (1.7e-3 of the result's
// size) a Gaussian matrix is off by 1.1e-3 (4096 x 4096) to 3.7e-3 (64 x 192),
// shorter sides below 64 by up to 1e-2, below 8 by up to 3e-2; one of a few
// strong directions over noise by 2e-4 (4096 x 4096) to 2.4e-3 (64 x 192).  (X in
// one part: 3e-3 to 4e-3 where two give 3e-4 to 1e-3.)  For a result stored in
// f32 A and B are two parts as well and every product three products of parts:
// off by 1e-6 to 5e-6 (below 8 by up to 7e-5).
#include <algorithm>
#include <vector>

#include "common.cuh"
#include "vec8.cuh"
#include "mm.h"
#include "ortho.h"
#include "views.h"

namespace psk {

constexpr float ORTHO_SCALE = 1024.0f;
constexpr int ORTHO_MAX_LEAVES = PSK_ORTHO_MAX_LEAVES;
constexpr int ORTHO_PARTS = 2;                      // of X
constexpr int ORTHO_SUM_BLOCKS = 64;                // of a matrix's square sum, at most
constexpr int64_t ORTHO_MAX_SIDE = 1 << 20;

// The leaves, with room for CAP of them: a launch's parameters are copied for
// every one, so few leaves have a small table.
template <int CAP>
struct OrthoTable {
  const void* x[CAP];
  int64_t ldx[CAP];
};
template <int CAP>
struct OrthoTargets {
  void* y[CAP];
  int64_t ldy[CAP];
  uint8_t vec[CAP];
};
constexpr int ORTHO_FEW = 32;

struct OrthoShape {
  int64_t rows, cols;           // of a leaf
  int64_t m, n, ldn, ldm;
  int32_t xt, tall, blocks, leaves;
  double eps;
  double* sums;                 // [leaf][block]
  float2* factors;              // [leaf]: two, applied one after the other
  MMLeaf* table;
  uint16_t* x;                  // [leaf][part][m][ldn]
};

// A block's sum of squares: f32 within a thread's share of up to 1024 columns
// of a row, which are on their way at once, 64 bits beyond.  Warps take such
// pieces in turn (whole rows left few warps at work: 18 of [145, 4299] 58 us).
// A share whose squares leave f32 (elements above 2^60 or so) is taken again
// times 2^-80, which leaves room for 2^32 squares of the largest f32.
constexpr int ORTHO_PIECE = 1024;

template <int XT, bool VEC>
__device__ __forceinline__ float ortho_share(const void* x, int64_t row, int64_t c, int64_t cols, int lane, float scale) {
  float2 s = make_float2(0.0f, 0.0f);
  Piece<XT, VEC, 8> p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Columns<VEC, 8> C(c + j * 256, 32, lane, cols);
    C.template load<XT>(x, row, p[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float2 v = make_float2(p[j].get(k), p[j].get(k + 1));
      if (scale != 1.0f) v.x *= scale, v.y *= scale;
      s = __ffma2_rn(v, v, s);
    }
  return s.x + s.y;
}

template <int XT, bool VEC, int CAP>
__global__ void __launch_bounds__(256) ortho_sum_kernel(const __grid_constant__ OrthoTable<CAP> T, OrthoShape S) {
  __shared__ double part[8];
  const int leaf = blockIdx.x / S.blocks, block = blockIdx.x % S.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const void* x = T.x[leaf];
  const int64_t ld = T.ldx[leaf];
  double total = 0.0;
  const int64_t across = (S.cols + ORTHO_PIECE - 1) / ORTHO_PIECE, pieces = S.rows * across;
  for (int64_t i = (int64_t)block * 8 + warp; i < pieces; i += (int64_t)S.blocks * 8) {
    const int64_t r = i / across, c = (i - r * across) * ORTHO_PIECE;
    const float s = ortho_share<XT, VEC>(x, r * ld, c, S.cols, lane, 1.0f);
    if (s > 3.4028234663852886e38f)
      total += (double)ortho_share<XT, VEC>(x, r * ld, c, S.cols, lane, 8.271806125530277e-25f) * 1.461501637330903e48;
    else total += (double)s;
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

// A warp a leaf: the blocks' sums, the factor S / (norm + eps), and where the
// result goes, for the last product's epilogue.
template <int CAP>
__global__ void __launch_bounds__(256) ortho_factor_kernel(const __grid_constant__ OrthoTargets<CAP> T, OrthoShape S) {
  const int leaf = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (leaf >= S.leaves) return;
  double s = 0.0;
  for (int i = lane; i < S.blocks; i += 32) s += S.sums[leaf * S.blocks + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) {
    S.factors[leaf] = ortho_factors((double)ORTHO_SCALE / (sqrt(s) + S.eps));
    S.table[leaf] = MMLeaf{T.y[leaf], T.ldy[leaf], T.vec[leaf]};
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

// Eight columns of the iterate in its two parts.
__device__ __forceinline__ void ortho_store8(const OrthoShape& S, int64_t leaf, int64_t r, int64_t c, float* v) {
  uint16_t* q = S.x + leaf * ORTHO_PARTS * S.m * S.ldn + r * S.ldn + c;
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

// The first iterate.  64 x 64 of it a CTA: of a leaf whose rows are the
// iterate's, straight from rows to rows; of a tall one through shared memory,
// so that the leaf's rows and the iterate's are both walked along.
template <int XT, bool VEC, bool TALL, int CAP>
__global__ void __launch_bounds__(256) ortho_begin_kernel(const __grid_constant__ OrthoTable<CAP> T, OrthoShape S) {
  __shared__ float tile[TALL ? 64 : 1][65];
  const int64_t tn = (S.ldn + 63) / 64, tm = (S.m + 63) / 64;
  const int64_t leaf = blockIdx.x / (tn * tm), at = blockIdx.x % (tn * tm);
  const int64_t r0 = at / tn * 64, c0 = at % tn * 64;
  const void* x = T.x[leaf];
  const int64_t ld = T.ldx[leaf];
  const int i = threadIdx.x >> 3, g = (threadIdx.x & 7) * 8;           // a tile row, and 8 of its columns
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = (TALL ? c0 : r0) + i + 32 * h, c = (TALL ? r0 : c0) + g;
    const int64_t left = S.cols - c;
    load8<XT, VEC>(x, r * ld + c, r < S.rows && left > 0 ? (left < 8 ? (int)left : 8) : 0, v[h]);
  }
  const float2 f = S.factors[leaf];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[h][k] = v[h][k] * f.x * f.y;
      if constexpr (TALL) tile[g + k][i + 32 * h] = v[h][k];
    }
  if constexpr (TALL) __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int a = i + 32 * h;
    if constexpr (TALL) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[h][k] = tile[a][g + k];
    }
    if (r0 + a < S.m && c0 + g < S.ldn) ortho_store8(S, leaf, r0 + a, c0 + g, v[h]);
  }
}

// A leaf's rows, one behind the other.
__global__ void __launch_bounds__(256) ortho_copy_kernel(const __grid_constant__ OrthoTable<ORTHO_MAX_LEAVES> T, int rows, int cols, int32_t xt,
                                                         char* to) {
  const int leaf = blockIdx.x;
  const int64_t ld = T.ldx[leaf], at = (int64_t)leaf * rows * cols;
  for (int i = threadIdx.x; i < rows * cols; i += 256) {
    const int64_t e = (int64_t)(i / cols) * ld + i % cols;
    if (xt == PSK_BF16) ((uint16_t*)to)[at + i] = ((const uint16_t*)T.x[leaf])[e];
    else ((uint32_t*)to)[at + i] = ((const uint32_t*)T.x[leaf])[e];
  }
}

// Offsets from the workspace's first 32-byte boundary, and the bytes that hold
// them behind any 16-byte one.
struct OrthoLayout {
  uint64_t sums, factors, table, x0, x1, a, b, bytes;
  int64_t xsize, asize;         // elements of one plane
};
// The planes' rows go by 32 bytes at a time.
constexpr uint64_t ORTHO_ALIGN = 32;
static char* ortho_base(void* workspace) {
  return (char*)(((uintptr_t)workspace + ORTHO_ALIGN - 1) / ORTHO_ALIGN * ORTHO_ALIGN);
}

static int64_t ortho_up16(int64_t v) { return (v + 15) / 16 * 16; }      // rows of whole 32-byte sectors

static OrthoLayout ortho_layout(int32_t leaves, int64_t rows, int64_t cols, int32_t yt) {
  OrthoLayout L{};
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  const int planes = yt == PSK_F32 ? 2 : 1;
  L.xsize = m * ortho_up16(n), L.asize = m * ortho_up16(m);
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  L.sums = take((uint64_t)leaves * ORTHO_SUM_BLOCKS * 8);
  L.factors = take((uint64_t)leaves * 8);
  L.table = take((uint64_t)leaves * sizeof(MMLeaf));
  L.x0 = take((uint64_t)leaves * ORTHO_PARTS * L.xsize * 2);
  L.x1 = take((uint64_t)leaves * ORTHO_PARTS * L.xsize * 2);
  L.a = take((uint64_t)leaves * planes * L.asize * 2);
  L.b = take((uint64_t)leaves * planes * L.asize * 2);
  L.bytes = at + ORTHO_ALIGN - 16;
  return L;
}

// One CTA a matrix: fifteen dependent products of one tile or two are launches'
// latency otherwise ([64, 192] x 2 f32: 116 us, here 51).
static bool ortho_is_small(int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  return m <= ORTHO_SMALL_M && n <= ORTHO_SMALL_N;
}

// Whether a result lies on another matrix's x.  at: room for the x's, sorted by their beginnings.
static bool ortho_crossed(const std::vector<View>& in, const std::vector<View>& out,
                          std::vector<std::pair<uintptr_t, int>>& at) {
  uint64_t longest = 0;
  at.clear();
  for (size_t i = 0; i < in.size(); ++i) {
    at.push_back({in[i].p, (int)i});
    longest = longest > in[i].bytes() ? longest : in[i].bytes();
  }
  std::sort(at.begin(), at.end());
  for (size_t j = 0; j < out.size(); ++j) {
    const uintptr_t from = out[j].p > longest ? out[j].p - longest : 0, to = out[j].p + out[j].bytes();
    for (auto it = std::lower_bound(at.begin(), at.end(), std::make_pair(from, -1)); it != at.end() && it->first < to; ++it)
      if (it->second != (int)j && views_overlap(in[it->second], out[j])) return true;
  }
  return false;
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
  static thread_local OrthoTable<ORTHO_MAX_LEAVES> T;
  static thread_local OrthoTargets<ORTHO_MAX_LEAVES> Y;
  const View vws{(uintptr_t)workspace, 1, L.bytes, L.bytes};
  std::vector<View> out, in;
  std::vector<std::pair<uintptr_t, int>> starts;
  try {                                    // all that allocates: no exception leaves this entry
    out.reserve(n_leaves);
    in.reserve(n_leaves);
    starts.reserve(n_leaves);
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
    in.push_back(vx);
    T.x[i] = f.x, T.ldx[i] = f.ldx;
    Y.y[i] = f.y, Y.ldy[i] = f.ldy, Y.vec[i] = rows_vec8(f.y, yt, f.ldy, rows);
  }
  const bool crossed = ortho_is_small(rows, cols) && ortho_crossed(in, out, starts);
  std::sort(out.begin(), out.end(), [](const View& a, const View& b) { return a.p < b.p; });
  for (size_t i = 0; i < out.size(); ++i)
    for (size_t j = i + 1; j < out.size() && out[j].p < out[i].p + out[i].bytes(); ++j)
      if (views_overlap(out[i], out[j])) return fail(PSK_E_ALIAS, "two results overlap");

  cudaStream_t s = (cudaStream_t)stream;
  if (ortho_is_small(rows, cols)) {
    const char* copies = nullptr;
    if (crossed) {                       // every x is read before the first y is written
      char* to = ortho_base(workspace) + L.x0;
      copies = to;
      ortho_copy_kernel<<<n_leaves, 256, 0, s>>>(T, (int)rows, (int)cols, xt, to);
      rc = check_launch("orthogonalisation's copies");
      if (rc) return rc;
    }
    return ortho_small_launch(leaves, copies, n_leaves, rows, cols, xt, yt, coefficients, steps, eps, scale, s);
  }
  char* ws = ortho_base(workspace);
  OrthoShape S{};
  S.rows = rows, S.cols = cols;
  S.tall = rows > cols;
  S.m = S.tall ? cols : rows, S.n = S.tall ? rows : cols;
  S.ldn = ortho_up16(S.n), S.ldm = ortho_up16(S.m);
  S.xt = xt, S.leaves = n_leaves;
  const int planes = yt == PSK_F32 ? 2 : 1;
  const int64_t blocks = (rows * ((cols + ORTHO_PIECE - 1) / ORTHO_PIECE) + 15) / 16;     // two pieces a warp at least
  S.blocks = (int32_t)(blocks < ORTHO_SUM_BLOCKS ? blocks : ORTHO_SUM_BLOCKS);
  S.eps = eps;
  S.sums = (double*)(ws + L.sums), S.factors = (float2*)(ws + L.factors);
  S.table = (MMLeaf*)(ws + L.table), S.x = (uint16_t*)(ws + L.x0);
  bool vec = cols % 8 == 0;
  for (int i = 0; i < n_leaves; ++i) vec = vec && rows_vec8(leaves[i].x, xt, leaves[i].ldx, rows);
  const int64_t tiles = (S.ldn + 63) / 64 * ((S.m + 63) / 64) * n_leaves;
  if (tiles > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many tiles");
  const auto begin = [&](const auto& TT, const auto& YY) {
    constexpr int CAP = sizeof(TT.x) / sizeof(TT.x[0]);
    with_dtype(xt, [&](auto XT) {
      return with_bool(vec, [&](auto VEC) {
        ortho_sum_kernel<XT.value, VEC.value, CAP><<<(unsigned)(n_leaves * S.blocks), 256, 0, s>>>(TT, S);
        ortho_factor_kernel<CAP><<<(unsigned)((n_leaves + 7) / 8), 256, 0, s>>>(YY, S);
        if (S.tall) ortho_begin_kernel<XT.value, VEC.value, true, CAP><<<(unsigned)tiles, 256, 0, s>>>(TT, S);
        else ortho_begin_kernel<XT.value, VEC.value, false, CAP><<<(unsigned)tiles, 256, 0, s>>>(TT, S);
        return 0;
      });
    });
  };
  if (n_leaves <= ORTHO_FEW) {
    OrthoTable<ORTHO_FEW> t;
    OrthoTargets<ORTHO_FEW> y;
    for (int i = 0; i < n_leaves; ++i)
      t.x[i] = T.x[i], t.ldx[i] = T.ldx[i], y.y[i] = Y.y[i], y.ldy[i] = Y.ldy[i], y.vec[i] = Y.vec[i];
    begin(t, y);
  } else {
    begin(T, Y);
  }
  rc = check_launch("orthogonalisation's first kernels");
  uint16_t *x = S.x, *x2 = (uint16_t*)(ws + L.x1), *A = (uint16_t*)(ws + L.a), *B = (uint16_t*)(ws + L.b);
  const auto wide = [&](const uint16_t* p, bool k_inner) {
    return MMOperand{p, S.n, S.m, S.ldn, L.xsize, ORTHO_PARTS, k_inner};
  };
  const auto square = [&](const uint16_t* p) { return MMOperand{p, S.m, S.m, S.ldm, L.asize, planes, true}; };
  MMCall C{};
  C.f16 = true, C.matrices = n_leaves, C.ortho = true;
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
    rc = mm_launch(&C, 1, nullptr, s);
    if (rc) break;
    // B S = b (A S) + c (A S)(A S) / S
    C.k = S.m;
    C.a = square(A), C.b = square(A);
    C.e.alpha = (float)(c / ORTHO_SCALE), C.e.beta = (float)b, C.e.from = A, C.e.to = B;
    rc = mm_launch(&C, 1, nullptr, s);
    if (rc) break;
    // X S <- a (X S) + (B S)(X S) / S
    C.n = S.n, C.symmetric = false, C.e.transposed = S.tall;
    C.a = square(B), C.b = wide(x, false);
    const double out_scale = last ? scale / ORTHO_SCALE : 1.0;
    C.e.alpha = (float)(out_scale / ORTHO_SCALE), C.e.beta = (float)(a * out_scale);
    C.e.from = x, C.e.to = last ? nullptr : x2, C.e.leaves = S.table;
    C.e.ld = S.ldn, C.e.plane_stride = L.xsize, C.e.planes = ORTHO_PARTS;
    rc = mm_launch(&C, 1, nullptr, s);
    std::swap(x, x2);
  }
  return rc;
}
