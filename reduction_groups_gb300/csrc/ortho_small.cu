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

constexpr int OS_THREADS = 512;            // four warps for each quarter of the rows
constexpr int OS_BLOCK = 128 * 128;        // bytes of 128 rows of 64 elements

struct OrthoSmallParams {
  int32_t rows, cols, m, n, tall, xt, yt, steps;
  double eps, scale;
  float a[64], b[64], c[64];
};
// The leaves, with room for CAP of them: the parameters of a launch are copied
// for every one.
template <int CAP>
struct OrthoSmallLeaves {
  const void* x[CAP];
  void* y[CAP];
  int64_t ldx[CAP], ldy[CAP];
};

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

// Calls f(row, column, element or 0) for a leaf's elements: rows by warps,
// columns by lanes, sixteen loads a thread on their way at once.  (The loops
// stay rolled: code that runs once or twice costs what it takes to fetch it.)
template <typename F>
__device__ __forceinline__ void os_each(const OrthoSmallParams& P, const void* x, int64_t ld, F&& f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r0 = warp; r0 < P.rows; r0 += 4 * (OS_THREADS / 32))
#pragma unroll 1
    for (int c0 = lane; c0 < P.cols; c0 += 128) {
      float v[4][4];
      const char* p = (const char*)x + ((int64_t)r0 * ld + c0) * (P.xt == PSK_BF16 ? 2 : 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] = 0.0f;
          if (r0 + i * (OS_THREADS / 32) < P.rows && c0 + 32 * j < P.cols) {
            const int64_t e = (int64_t)i * (OS_THREADS / 32) * ld + 32 * j;
            v[i][j] = P.xt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[e]) : ((const float*)p)[e];
          }
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) f(r0 + i * (OS_THREADS / 32), c0 + 32 * j, v[i][j]);
    }
}

// PLANES: of each factor of a product.
template <int PLANES, int CAP>
__global__ void __launch_bounds__(OS_THREADS, 1)
    ortho_small_kernel(const __grid_constant__ OrthoSmallParams P, const __grid_constant__ OrthoSmallLeaves<CAP> L) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ double part[OS_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char* base = (char*)smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  const int blocks = (P.n + 63) / 64;                       // of X's columns
  const uint32_t x_plane = blocks * OS_BLOCK, a_plane = 2 * OS_BLOCK;
  char* xs = base;                                          // [part][block][128 rows]
  char* as = base + 2 * x_plane;
  const uint32_t xa = smem_addr(xs), aa = smem_addr(as);
  const void* x = L.x[blockIdx.x];
  const int64_t ldx = L.ldx[blockIdx.x];
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

  // ---- X = G S / (norm + eps), zeros around it
  for (uint32_t i = threadIdx.x; i < 2 * x_plane / 16; i += OS_THREADS) ((uint4*)xs)[i] = make_uint4(0, 0, 0, 0);
  float s = 0.0f, big = 0.0f;
  os_each(P, x, ldx, [&](int, int, float v) {
    // squares that would leave f32 are taken times 2^-160 (64 of the largest: 2^102)
    const bool over = fabsf(v) > 1.1e15f;
    const float u = over ? v * 8.271806125530277e-25f : 0.0f, w = over ? 0.0f : v;
    big = fmaf(u, u, big), s = fmaf(w, w, s);
  });
  double total = (double)s + (double)big * 1.461501637330903e48;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane == 0) part[warp] = total;
  __syncthreads();
  total = 0.0;
  for (int w = 0; w < OS_THREADS / 32; ++w) total += part[w];
  const float2 f = ortho_factors(1024.0 / (sqrt(total) + P.eps));
  // Where element (row, column) of the leaf stands in X.
  const auto at = [&](int lr, int lc) {
    const int r = P.tall ? lc : lr, c = P.tall ? lr : lc;
    return xs + (c >> 6) * OS_BLOCK + os_at(r, c & ~7) + (c & 7) * 2;
  };
  os_each(P, x, ldx, [&](int lr, int lc, float v) {
    if (lr >= P.rows || lc >= P.cols) return;
    const float t = v * f.x * f.y;
    const uint32_t w = f32x2_to_f16x2(t, 0.0f);
    char* q = at(lr, lc);
    *(uint16_t*)q = (uint16_t)w;
    *(uint16_t*)(q + x_plane) = (uint16_t)f32x2_to_f16x2(t - f16x2_to_f32(w).x, 0.0f);
  });

  const uint32_t idesc = (1u << 4) | ((uint32_t)(128 >> 4) << 24);                     // fp16, 128 rows, K-major
  const uint32_t square = idesc | ((uint32_t)(128 >> 3) << 17);
  const int wide_n = (P.n + 15) / 16 * 16;
  const uint32_t wide = idesc | (1u << 16) | ((uint32_t)(wide_n >> 3) << 17);          // B MN-major
  const int row = (warp & 3) * 32 + lane, share = (warp >> 2) * 32;
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
    float af[32];                          // this thread's share of a row of A S
    multiply(xa, x_plane, xa, x_plane, (P.n + 15) / 16, square, false);
    if (!ok) break;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
      take16(share + c, af + c);
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = af[c + h + k] *= unit;
        os_store8<PLANES>(as + (share >> 6) * OS_BLOCK + os_at(row, share + c + h), a_plane, v);
      }
    }
    multiply(aa, a_plane, aa, a_plane, 8, square, false);
    if (!ok) break;
    const float b = P.b[step], cu = P.c[step] * unit;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
      float v[16];
      take16(share + c, v);
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h + k] = fmaf(b, af[c + h + k], v[h + k] * cu);
        os_store8<PLANES>(as + (share >> 6) * OS_BLOCK + os_at(row, share + c + h), a_plane, v + h);
      }
    }
    multiply(aa, a_plane, xa, x_plane, 8, wide, true);
    if (!ok) break;
    const bool last = step + 1 == P.steps;
    const float out = last ? (float)(P.scale / 1024.0) : 1.0f, a = P.a[step] * out, u = unit * out;
#pragma unroll 1
    for (int c = share / 2; c < wide_n; c += 64) {
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
        if (!last) {
          os_store8<2>(q, x_plane, v + h);
        } else {                           // f32 in two halves
          uint32_t top[4], low[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t e = __float_as_uint(v[h + 2 * k]), g = __float_as_uint(v[h + 2 * k + 1]);
            top[k] = e >> 16 | (g & 0xFFFF0000u), low[k] = (e & 0xFFFFu) | g << 16;
          }
          *(uint4*)q = make_uint4(top[0], top[1], top[2], top[3]);
          *(uint4*)(q + x_plane) = make_uint4(low[0], low[1], low[2], low[3]);
        }
      }
    }
  }
  // ---- the result: rows by warps, columns by lanes
  __syncthreads();
  if (ok) {
    void* y = L.y[blockIdx.x];
    const int64_t ldy = L.ldy[blockIdx.x];
    for (int lr = warp; lr < P.rows; lr += OS_THREADS / 32)
#pragma unroll 4
      for (int lc = lane; lc < P.cols; lc += 32) {
        const char* q = at(lr, lc);
        const float v = __uint_as_float((uint32_t) * (const uint16_t*)q << 16 | *(const uint16_t*)(q + x_plane));
        if (P.yt == PSK_BF16) ((uint16_t*)y)[lr * ldy + lc] = f32_to_bf16_bits(v);
        else ((float*)y)[lr * ldy + lc] = v;
      }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free<1>(tmem, 512);
}

template <int PLANES, int CAP>
static void launch_small(const OrthoSmallParams& P, const psk_ortho_leaf* leaves, const char* copies, int count, int smem,
                         cudaStream_t stream) {
  static thread_local OrthoSmallLeaves<CAP> L;
  for (int i = 0; i < count; ++i) {
    const psk_ortho_leaf& f = leaves[i];
    L.x[i] = copies ? copies + (int64_t)i * P.rows * P.cols * dtype_size(P.xt) : f.x;
    L.ldx[i] = copies ? P.cols : f.ldx;
    L.y[i] = f.y, L.ldy[i] = f.ldy;
  }
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)ortho_small_kernel<PLANES, CAP>, 12 * OS_BLOCK + 1024, limit);
  ortho_small_kernel<PLANES, CAP><<<count, OS_THREADS, smem, stream>>>(P, L);
}

int ortho_small_launch(const psk_ortho_leaf* leaves, const char* copies, int n_leaves, int64_t rows, int64_t cols, int32_t xt,
                       int32_t yt, const double* coefficients, int32_t steps, double eps, double scale,
                       cudaStream_t stream) {
  OrthoSmallParams P{};
  P.rows = (int32_t)rows, P.cols = (int32_t)cols;
  P.tall = rows > cols;
  P.m = P.tall ? (int32_t)cols : (int32_t)rows, P.n = P.tall ? (int32_t)rows : (int32_t)cols;
  P.xt = xt, P.yt = yt, P.steps = steps, P.eps = eps, P.scale = scale;
  for (int i = 0; i < steps; ++i)
    P.a[i] = (float)coefficients[3 * i], P.b[i] = (float)coefficients[3 * i + 1], P.c[i] = (float)coefficients[3 * i + 2];
  const int blocks = (P.n + 63) / 64, planes = yt == PSK_F32 ? 2 : 1;
  const int smem = 2 * blocks * OS_BLOCK + planes * 2 * OS_BLOCK + 1024;
  if (n_leaves <= 16) {
    if (planes == 2) launch_small<2, 16>(P, leaves, copies, n_leaves, smem, stream);
    else launch_small<1, 16>(P, leaves, copies, n_leaves, smem, stream);
  } else if (planes == 2) {
    launch_small<2, PSK_ORTHO_MAX_LEAVES>(P, leaves, copies, n_leaves, smem, stream);
  } else {
    launch_small<1, PSK_ORTHO_MAX_LEAVES>(P, leaves, copies, n_leaves, smem, stream);
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
