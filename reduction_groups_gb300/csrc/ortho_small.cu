// psk_orthogonalize of matrices of up to 128 x 256: every step of a matrix in
// one launch, in one CTA.  X stays in shared memory in its two fp16 parts, A
// and B in theirs beside it, the products run from there into TMEM:
//   A = X X^T: both operands X's rows, K-major;
//   A A:       A's rows twice (A is its own transpose);
//   B X:       B's rows, and X's 128-byte rows read MN-major -- the same bytes.
// With three products and their epilogues a step the time is their latency:
// two of [64, 192] f32, five steps, took 116 us as 18 launches.
#include "common.cuh"
#include "vec8.cuh"
#include "act.cuh"
#include "tensor.cuh"
#include "ortho.h"
#include "trainops.h"

namespace psk {

constexpr int OS_THREADS = 256;
constexpr int OS_BLOCK = 128 * 128;        // bytes of 128 rows of 64 elements

struct OrthoSmallParams {
  const void* x[PSK_ORTHO_MAX_LEAVES];
  void* y[PSK_ORTHO_MAX_LEAVES];
  int64_t ldx[PSK_ORTHO_MAX_LEAVES], ldy[PSK_ORTHO_MAX_LEAVES];
  int32_t rows, cols, m, n, tall, xt, yt, steps;
  double eps, scale;
  float a[64], b[64], c[64];
};

__device__ __forceinline__ float os_load(const OrthoSmallParams& P, const void* x, int64_t ld, int r, int c) {
  const int64_t i = P.tall ? (int64_t)c * ld + r : (int64_t)r * ld + c;
  return P.xt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)x)[i]) : ((const float*)x)[i];
}

// Where 16 bytes (elements c .. c + 7 of row r) of a block of 64 columns stand, swizzled.
__device__ __forceinline__ uint32_t os_at(int r, int c) { return (uint32_t)(r * 128 + (((c & 63) * 2) ^ ((r & 7) << 4))); }

// Eight values in two fp16 parts, `apart` bytes apart (PARTS = 1: the first alone).
template <int PARTS>
__device__ __forceinline__ void os_store8(char* p, uint32_t apart, float* v) {
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = f32x2_to_f16x2(v[2 * k], v[2 * k + 1]);
      const float2 h = f16x2_to_f32(w[k]);
      v[2 * k] -= h.x, v[2 * k + 1] -= h.y;
    }
    *(uint4*)(p + q * apart) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// PLANES: of each factor of a product.
template <int PLANES>
__global__ void __launch_bounds__(OS_THREADS, 1) ortho_small_kernel(const __grid_constant__ OrthoSmallParams P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ double part[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char* base = (char*)smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  const int blocks = (P.n + 63) / 64;                       // of X's columns
  const uint32_t x_plane = blocks * OS_BLOCK, a_plane = 2 * OS_BLOCK;
  char* xs = base;                                          // [part][block][128 rows]
  char* as = base + 2 * x_plane;
  const uint32_t xa = smem_addr(xs), aa = smem_addr(as);
  const void* x = P.x[blockIdx.x];
  const int64_t ldx = P.ldx[blockIdx.x];
  if (warp == 0 && lane == 0) {
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<1>(&tmem_slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // An accumulator of up to 256 columns, and with two planes a second one for
  // their smaller products.
  constexpr uint32_t SMALL = 256;

  // ---- the norm, then X = G S / (norm + eps): rows by warps, lanes along the leaf's rows
  float s = 0.0f, big = 0.0f;
  for (int i = threadIdx.x; i < P.rows * P.cols; i += OS_THREADS) {
    const int r = i / P.cols;
    const int64_t e = (int64_t)r * ldx + (i - r * P.cols);
    const float v = P.xt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)x)[e]) : ((const float*)x)[e];
    if (fabsf(v) > 1.1e15f) {
      const float u = v * 5.421010862427522e-20f;           // squares that would leave f32
      big = fmaf(u, u, big);
    } else {
      s = fmaf(v, v, s);
    }
  }
  double total = (double)s + (double)big * 3.402823669209385e38;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane == 0) part[warp] = total;
  __syncthreads();
  total = 0.0;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += part[w];
  const float f = (float)(1024.0 / (sqrt(total) + P.eps));
  for (int i = threadIdx.x; i < 128 * blocks * 8; i += OS_THREADS) {
    // a leaf's row runs along c, a tall one's along r
    const int r = P.tall ? i & 127 : i / (blocks * 8), c = (P.tall ? i >> 7 : i % (blocks * 8)) * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r < P.m && c + k < P.n ? os_load(P, x, ldx, r, c + k) * f : 0.0f;
    os_store8<2>(xs + (c >> 6) * OS_BLOCK + os_at(r, c), x_plane, v);
  }

  const uint32_t idesc = (1u << 4) | ((uint32_t)(128 >> 4) << 24);                     // fp16, 128 rows, K-major
  const uint32_t square = idesc | ((uint32_t)(128 >> 3) << 17);
  const int wide_n = (P.n + 15) / 16 * 16;
  const uint32_t wide = idesc | (1u << 16) | ((uint32_t)(wide_n >> 3) << 17);          // B MN-major
  const int row = (warp & 3) * 32 + lane, half = warp >> 2;
  const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const float unit = 1.0f / 1024.0f;
  uint32_t phase = 0;
  bool ok = true;
  // The products of planes of A and B operands, K in sixteens, the smaller ones
  // into the second accumulator; then all threads wait for them.
  const auto multiply = [&](uint32_t a, uint32_t a_next, uint32_t b, uint32_t b_next, int sixteens, uint32_t desc,
                            bool b_rows) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");                       // operands written by threads
    fence_before();
    __syncthreads();
    if (warp == 0 && lane == 0) {
      fence_after();
#pragma unroll 1
      for (int p = PLANES == 2 ? 0 : 2; p < 3; ++p) {                                  // (1, 0), (0, 1), (0, 0)
        const uint32_t pa = a + (p == 0 ? a_next : 0), pb = b + (p == 1 ? b_next : 0);
        const uint32_t d = tmem + (p < 2 ? SMALL : 0);
#pragma unroll 1
        for (int k = 0; k < sixteens; ++k) {
          const uint64_t da = operand_desc(pa + (k >> 2) * OS_BLOCK + (k & 3) * 32, OS_BLOCK);
          const uint64_t db = operand_desc(b_rows ? pb + k * 2048 : pb + (k >> 2) * OS_BLOCK + (k & 3) * 32, OS_BLOCK);
          mma_16<1>(d, da, db, desc, k > 0 || p == 1);
        }
      }
      mma_commit<1>(&done);
    }
    __syncwarp();
    ok = __syncthreads_and(mbar_wait(&done, phase & 1)) && ok;
    ++phase;
    fence_after();
  };
  const auto take16 = [&](int c, float* v) {
    __syncwarp();
    tmem_load16(mine + c, v);
    if constexpr (PLANES == 2) {
      float w[16];
      tmem_load16(mine + SMALL + c, w);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] += w[k];
    }
  };

  for (int step = 0; step < P.steps && ok; ++step) {
    float af[64];                          // this thread's half row of A S
    multiply(xa, x_plane, xa, x_plane, (P.n + 15) / 16, square, false);
    if (!ok) break;
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      take16(half * 64 + c, af + c);
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = af[c + h + k] *= unit;
        os_store8<PLANES>(as + half * OS_BLOCK + os_at(row, c + h), a_plane, v);
      }
    }
    multiply(aa, a_plane, aa, a_plane, 8, square, false);
    if (!ok) break;
    const float b = P.b[step], cu = P.c[step] * unit;
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      float v[16];
      take16(half * 64 + c, v);
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h + k] = fmaf(b, af[c + h + k], v[h + k] * cu);
        os_store8<PLANES>(as + half * OS_BLOCK + os_at(row, c + h), a_plane, v + h);
      }
    }
    multiply(aa, a_plane, xa, x_plane, 8, wide, true);
    if (!ok) break;
    const bool last = step + 1 == P.steps;
    const float out = last ? (float)(P.scale / 1024.0) : 1.0f, a = P.a[step] * out, u = unit * out;
    void* y = P.y[blockIdx.x];
    const int64_t ldy = P.ldy[blockIdx.x];
#pragma unroll 1
    for (int c = half * 16; c < wide_n; c += 32) {
      float v[16];
      take16(c, v);
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        char* q = xs + ((c + h) >> 6) * OS_BLOCK + os_at(row, c + h);
        const uint4 w = *(const uint4*)q, l = *(const uint4*)(q + x_plane);
        const uint32_t hi[4] = {w.x, w.y, w.z, w.w}, lo[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 e = f16x2_to_f32(hi[k]), g = f16x2_to_f32(lo[k]);
          v[h + 2 * k] = fmaf(a, e.x, fmaf(a, g.x, v[h + 2 * k] * u));
          v[h + 2 * k + 1] = fmaf(a, e.y, fmaf(a, g.y, v[h + 2 * k + 1] * u));
        }
        if (!last) os_store8<2>(q, x_plane, v + h);
      }
      if (last && row < P.m) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c + k < P.n) {
            const int64_t i = P.tall ? (int64_t)(c + k) * ldy + row : (int64_t)row * ldy + c + k;
            if (P.yt == PSK_BF16) ((uint16_t*)y)[i] = f32_to_bf16_bits(v[k]);
            else ((float*)y)[i] = v[k];
          }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free<1>(tmem, 512);
}

int ortho_small_launch(const psk_ortho_leaf* leaves, const char* copies, int n_leaves, int64_t rows, int64_t cols, int32_t xt, int32_t yt,
                       const double* coefficients, int32_t steps, double eps, double scale, cudaStream_t stream) {
  static thread_local OrthoSmallParams P;
  for (int i = 0; i < n_leaves; ++i)
    P.x[i] = copies ? copies + i * rows * cols * dtype_size(xt) : leaves[i].x, P.ldx[i] = copies ? cols : leaves[i].ldx,
    P.y[i] = leaves[i].y, P.ldy[i] = leaves[i].ldy;
  P.rows = (int32_t)rows, P.cols = (int32_t)cols;
  P.tall = rows > cols;
  P.m = P.tall ? (int32_t)cols : (int32_t)rows, P.n = P.tall ? (int32_t)rows : (int32_t)cols;
  P.xt = xt, P.yt = yt, P.steps = steps, P.eps = eps, P.scale = scale;
  for (int i = 0; i < steps; ++i)
    P.a[i] = (float)coefficients[3 * i], P.b[i] = (float)coefficients[3 * i + 1], P.c[i] = (float)coefficients[3 * i + 2];
  const int blocks = (P.n + 63) / 64, planes = yt == PSK_F32 ? 2 : 1;
  const int smem = 2 * blocks * OS_BLOCK + planes * 2 * OS_BLOCK + 1024;
  static bool limit1[PSK_MAX_DEVICES] = {}, limit2[PSK_MAX_DEVICES] = {};
  constexpr int MOST = 2 * 4 * OS_BLOCK + 4 * OS_BLOCK + 1024;
  if (planes == 2) {
    smem_limit_once((const void*)ortho_small_kernel<2>, MOST, limit2);
    ortho_small_kernel<2><<<n_leaves, OS_THREADS, smem, stream>>>(P);
  } else {
    smem_limit_once((const void*)ortho_small_kernel<1>, MOST, limit1);
    ortho_small_kernel<1><<<n_leaves, OS_THREADS, smem, stream>>>(P);
  }
  return check_launch("small orthogonalisation kernel");
}

int ortho_small_status(unsigned int* v, bool reset) {
  if (cudaMemcpyFromSymbol(v, g_pipe_status, sizeof(*v)) != cudaSuccess) return check_launch("device status read");
  if (reset) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_pipe_status, &z, sizeof(z)) != cudaSuccess) return check_launch("device status reset");
  }
  return PSK_OK;
}

}  // namespace psk
