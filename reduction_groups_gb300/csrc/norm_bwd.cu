// The normalization regions' backward: with xh = (x - mu) / d (mu = 0 for
// RMSNorm), g = ct * gamma and means over a row's columns,
//   dx     = (g - [mean g] - xh mean(g xh)) / d     ([.] LayerNorm only)
//   dgamma = sum over rows of ct * xh,   dbeta = sum over rows of ct.
// Sums are held in f32 over trees fixed by the sizes: no atomics.
#include "vec8.cuh"

namespace psk {

constexpr int NB_THREADS = 256;
constexpr int NB_WARPS = NB_THREADS / 32;
constexpr int NB_MAX_COLS = 49152;         // as the forward regions
constexpr int NB_MAX_BLOCKS = 1024;        // row blocks of the column sums

struct NormBwdParams {
  const void* x;
  const void* ct;
  const void* gamma;      // NULL: ones
  void* dx;
  void* dgamma;           // NULL: not wanted
  void* dbeta;            // NULL: not wanted
  int64_t rows, cols, ldx, ldc, ldd;
  int32_t param_dtype, grad_dtype;
  float eps, inv_cols;
  float4* stats;          // per row: mu, 1/d, mean g, mean g xh
  float* part;            // [2][blocks][pcols]: row blocks' sums of ct * xh and ct
  int64_t pcols;
  int32_t blocks;
};

__device__ __forceinline__ float2 block_sum2(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  __syncthreads();                         // the last reduction's readers are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = red[0];
#pragma unroll
  for (int w = 1; w < NB_WARPS; ++w) s.x += red[w].x, s.y += red[w].y;
  return s;
}

// Row statistics, a CTA per row.  Rows are read once per reduction (two for
// LayerNorm, whose variance is taken about the mean); the later reads hit L1
// or L2.
template <int XT, int CT, int KIND, bool VEC>
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_stats_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float2 red[NB_WARPS];
  const int64_t groups = (P.cols + 7) / 8;
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const int64_t xo = r * P.ldx, co = r * P.ldc;
    float mu = 0.0f, mg = 0.0f;
    auto gated = [&](int64_t c, int n, float* g) {
      load8<CT, VEC>(P.ct, co + c, n, g);
      if (P.gamma) {
        float w[8];
        if (P.param_dtype == PSK_BF16) load8<PSK_BF16, VEC>(P.gamma, c, n, w);
        else load8<PSK_F32, VEC>(P.gamma, c, n, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] *= w[k];
      }
    };
    if (KIND == PSK_NORM_LAYER) {
      float s = 0.0f, t = 0.0f;
      for (int64_t q = threadIdx.x; q < groups; q += NB_THREADS) {
        const int64_t c = q * 8;
        const int n = P.cols - c < 8 ? (int)(P.cols - c) : 8;
        float x[8], g[8];
        load8<XT, VEC>(P.x, xo + c, n, x);
        gated(c, n, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += x[k], t += g[k];
      }
      const float2 v = block_sum2(s, t, red);
      mu = v.x * P.inv_cols;
      mg = v.y * P.inv_cols;
    }
    float s = 0.0f, t = 0.0f;
    for (int64_t q = threadIdx.x; q < groups; q += NB_THREADS) {
      const int64_t c = q * 8;
      const int n = P.cols - c < 8 ? (int)(P.cols - c) : 8;
      float x[8], g[8];
      load8<XT, VEC>(P.x, xo + c, n, x);
      gated(c, n, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = k < n ? x[k] - mu : 0.0f;
        s = fmaf(d, d, s);
        t = fmaf(d, g[k], t);
      }
    }
    const float2 v = block_sum2(s, t, red);
    const float rd = 1.0f / sqrtf(v.x * P.inv_cols + P.eps);
    if (threadIdx.x == 0) P.stats[r] = make_float4(mu, rd, mg, v.y * rd * P.inv_cols);
  }
}

// dx and the row blocks' column sums: a CTA takes a slice of 256 columns and
// one block of rows, its warps every eighth row; each element is read once
// and, in place, before it is written by the same thread.
template <int XT, int CT, int DT, int KIND, bool VEC>
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_apply_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float sums[2][NB_WARPS][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const SliceCols<VEC> sc((int)blockIdx.x, lane, P.cols);
  float gamma[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) gamma[k] = 1.0f;
  if (P.gamma) {
    if (P.param_dtype == PSK_BF16) sc.template load<PSK_BF16>(P.gamma, 0, gamma);
    else sc.template load<PSK_F32>(P.gamma, 0, gamma);
  }
  float dg[8] = {}, db[8] = {};
  const int64_t per = (P.rows + P.blocks - 1) / P.blocks;
  const int64_t r0 = (int64_t)blockIdx.y * per;
  const int64_t r1 = r0 + per < P.rows ? r0 + per : P.rows;
  for (int64_t r = r0 + warp; r < r1; r += NB_WARPS) {
    const float4 st = P.stats[r];
    float x[8], c[8];
    sc.template load<XT>(P.x, r * P.ldx, x);
    sc.template load<CT>(P.ct, r * P.ldc, c);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float xh = (x[k] - st.x) * st.y;
      const float g = c[k] * gamma[k];
      float t = KIND == PSK_NORM_LAYER ? g - st.z : g;
      t = fmaf(-xh, st.w, t);
      x[k] = t * st.y;
      dg[k] = fmaf(c[k], xh, dg[k]);
      db[k] += c[k];
    }
    sc.template store<DT>(P.dx, r * P.ldd, x);
  }
  if (!P.dgamma && !P.dbeta) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int at = VEC ? lane * 8 + k : lane + 32 * k;
    sums[0][warp][at] = dg[k];
    sums[1][warp][at] = db[k];
  }
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col < P.cols) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float s = sums[which][0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < NB_WARPS; ++w) s += sums[which][w][threadIdx.x];
      P.part[((int64_t)which * P.blocks + blockIdx.y) * P.pcols + col] = s;
    }
  }
}

// The row blocks' sums joined: 32 columns a CTA, warps over blocks in turn.
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_join_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float sums[NB_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int which = blockIdx.y;
  void* out = which ? P.dbeta : P.dgamma;
  if (!out) return;
  float s = 0.0f;
  if (col < P.cols) {
    const float* p = P.part + (int64_t)which * P.blocks * P.pcols + col;
    for (int b = warp; b < P.blocks; b += NB_WARPS) s += p[(int64_t)b * P.pcols];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < P.cols) {
#pragma unroll
    for (int w = 1; w < NB_WARPS; ++w) s += sums[w][lane];
    if (P.grad_dtype == PSK_BF16) ((uint16_t*)out)[col] = f32_to_bf16_bits(s);
    else ((float*)out)[col] = s;
  }
}

// dgamma and dbeta of no rows.
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_zero_kernel(const __grid_constant__ NormBwdParams P) {
  const int64_t col = (int64_t)blockIdx.x * NB_THREADS + threadIdx.x;
  void* out = blockIdx.y ? P.dbeta : P.dgamma;
  if (!out || col >= P.cols) return;
  if (P.grad_dtype == PSK_BF16) ((uint16_t*)out)[col] = 0;
  else ((float*)out)[col] = 0.0f;
}

// Row blocks of the column sums: enough CTAs to fill the GPU, at least 16
// rows each.
static int norm_bwd_blocks(int64_t rows, int64_t cols) {
  const int64_t slices = (cols + 255) / 256;
  int64_t b = (152 * 8 + slices - 1) / slices;
  if (b > (rows + 15) / 16) b = (rows + 15) / 16;
  return (int)(b < 1 ? 1 : b > NB_MAX_BLOCKS ? NB_MAX_BLOCKS : b);
}

static uint64_t norm_bwd_layout(int64_t rows, int64_t cols, uint64_t* part) {
  const uint64_t stats = ((uint64_t)rows * 16 + 255) / 256 * 256;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  *part = stats;
  return stats + 2ull * norm_bwd_blocks(rows, cols) * pcols * 4;
}

static int norm_bwd_check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return fail(PSK_E_SHAPE, "rows %lld, cols %lld", (long long)rows, (long long)cols);
  if (cols > NB_MAX_COLS) return fail(PSK_E_SHAPE, "cols %lld above %d", (long long)cols, NB_MAX_COLS);
  if (rows > (1LL << 40)) return fail(PSK_E_SHAPE, "rows %lld above 2^40", (long long)rows);
  return PSK_OK;
}

}  // namespace psk

using namespace psk;

extern "C" int psk_norm_backward_workspace(int64_t rows, int64_t cols, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = norm_bwd_check_sizes(rows, cols);
  if (rc) return rc;
  uint64_t part;
  *bytes = rows && cols ? norm_bwd_layout(rows, cols, &part) : 0;
  return PSK_OK;
}

extern "C" int psk_norm_backward(const void* x, int32_t xt, const void* ct, int32_t ct_t, void* dx, int32_t dxt,
                                 int64_t rows, int64_t cols, int64_t ldx, int64_t ldc, int64_t ldd, int32_t kind,
                                 double eps, const void* gamma, int32_t param_dtype, void* dgamma, void* dbeta,
                                 int32_t grad_dtype, void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  if (!dtype_ok(xt)) return fail(PSK_E_DTYPE, "x dtype %d", xt);
  if (!dtype_ok(ct_t)) return fail(PSK_E_DTYPE, "ct dtype %d", ct_t);
  if (!dtype_ok(dxt)) return fail(PSK_E_DTYPE, "dx dtype %d", dxt);
  if (kind != PSK_NORM_RMS && kind != PSK_NORM_LAYER) return fail(PSK_E_ARG, "norm kind %d", kind);
  if (!(eps == eps) || eps > 3.4e38 || eps < -3.4e38) return fail(PSK_E_ARG, "eps is not a finite f32 value");
  if (kind == PSK_NORM_RMS && dbeta) return fail(PSK_E_ARG, "RMSNorm takes no bias");
  if (gamma && !dtype_ok(param_dtype)) return fail(PSK_E_DTYPE, "parameter dtype %d", param_dtype);
  if ((dgamma || dbeta) && !dtype_ok(grad_dtype)) return fail(PSK_E_DTYPE, "parameter gradient dtype %d", grad_dtype);
  int rc = norm_bwd_check_sizes(rows, cols);
  if (rc) return rc;
  if (cols == 0) return PSK_OK;
  cudaStream_t s = (cudaStream_t)stream;
  NormBwdParams P{};
  P.gamma = gamma, P.dgamma = dgamma, P.dbeta = dbeta;
  P.cols = cols, P.rows = rows, P.param_dtype = param_dtype, P.grad_dtype = grad_dtype;
  const uint64_t pb = (uint64_t)cols * dtype_size(param_dtype), gb = (uint64_t)cols * dtype_size(grad_dtype);
  if (dgamma && dbeta && ranges_overlap(dgamma, gb, dbeta, gb)) return fail(PSK_E_ALIAS, "dgamma overlaps dbeta");
  for (const void* g : {(const void*)dgamma, (const void*)dbeta})
    if (g && gamma && ranges_overlap(g, gb, gamma, pb)) return fail(PSK_E_ALIAS, "dgamma or dbeta overlaps gamma");
  if (rows == 0) {
    if (!dgamma && !dbeta) return PSK_OK;
    norm_bwd_zero_kernel<<<dim3((unsigned)((cols + NB_THREADS - 1) / NB_THREADS), 2), NB_THREADS, 0, s>>>(P);
    return check_launch("norm backward zero kernel");
  }
  if (!x || !ct || !dx) return fail(PSK_E_NULL, "x, ct or dx is NULL");
  if ((uintptr_t)x % dtype_size(xt) || (uintptr_t)ct % dtype_size(ct_t) || (uintptr_t)dx % dtype_size(dxt) ||
      (gamma && (uintptr_t)gamma % dtype_size(param_dtype)) ||
      (dgamma && (uintptr_t)dgamma % dtype_size(grad_dtype)) || (dbeta && (uintptr_t)dbeta % dtype_size(grad_dtype)))
    return fail(PSK_E_ARG, "a tensor is not aligned to its type");
  if (ldx < cols || ldc < cols || ldd < cols) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(rows, ldx) || !rows_addressable(rows, ldc) || !rows_addressable(rows, ldd))
    return fail(PSK_E_SHAPE, "rows x leading dimension too large");
  uint64_t part = 0;
  const uint64_t need = norm_bwd_layout(rows, cols, &part);
  if (!workspace) return fail(PSK_E_NULL, "workspace is NULL");
  if ((uintptr_t)workspace % 16 != 0) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
  if (workspace_bytes < need)
    return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                (unsigned long long)need);
  const uint64_t xb = rows_bytes(rows, cols, ldx, xt), cb = rows_bytes(rows, cols, ldc, ct_t),
                 db = rows_bytes(rows, cols, ldd, dxt);
  if (ranges_overlap(x, xb, dx, db) && !(x == dx && xt == dxt && ldx == ldd))
    return fail(PSK_E_ALIAS, "dx overlaps x and is not the same buffer");
  if (ranges_overlap(ct, cb, dx, db) && !(ct == dx && ct_t == dxt && ldc == ldd))
    return fail(PSK_E_ALIAS, "dx overlaps ct and is not the same buffer");
  if (gamma && ranges_overlap(gamma, pb, dx, db)) return fail(PSK_E_ALIAS, "dx overlaps gamma");
  for (const void* g : {(const void*)dgamma, (const void*)dbeta})
    if (g && (ranges_overlap(g, gb, x, xb) || ranges_overlap(g, gb, ct, cb) || ranges_overlap(g, gb, dx, db) ||
              ranges_overlap(g, gb, workspace, need)))
      return fail(PSK_E_ALIAS, "dgamma or dbeta overlaps x, ct, dx or the workspace");
  if (ranges_overlap(workspace, need, x, xb) || ranges_overlap(workspace, need, ct, cb) ||
      ranges_overlap(workspace, need, dx, db) || (gamma && ranges_overlap(workspace, need, gamma, pb)))
    return fail(PSK_E_ALIAS, "the workspace overlaps x, ct, dx or gamma");
  P.x = x, P.ct = ct, P.dx = dx;
  P.ldx = ldx, P.ldc = ldc, P.ldd = ldd;
  P.eps = (float)eps, P.inv_cols = 1.0f / (float)cols;
  P.stats = (float4*)workspace;
  P.part = (float*)((char*)workspace + part);
  P.pcols = (cols + 7) / 8 * 8;
  P.blocks = norm_bwd_blocks(rows, cols);
  const bool vec = rows_vec8(x, xt, ldx, rows) && rows_vec8(ct, ct_t, ldc, rows) && rows_vec8(dx, dxt, ldd, rows) &&
                   (!gamma || rows_vec8(gamma, param_dtype, cols, 1));
  const int64_t most = (int64_t)device_sm_count() * 8;
  const unsigned rgrid = (unsigned)(rows < most ? rows : most);
  const dim3 agrid((unsigned)((cols + 255) / 256), (unsigned)P.blocks);
  with_dtype(xt, [&](auto XT) {
    return with_dtype(ct_t, [&](auto CT) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        constexpr int KIND = LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS;
        return with_bool(vec, [&](auto VEC) {
          norm_bwd_stats_kernel<XT.value, CT.value, KIND, VEC.value><<<rgrid, NB_THREADS, 0, s>>>(P);
          return with_dtype(dxt, [&](auto DT) {
            norm_bwd_apply_kernel<XT.value, CT.value, DT.value, KIND, VEC.value><<<agrid, NB_THREADS, 0, s>>>(P);
            return 0;
          });
        });
      });
    });
  });
  rc = check_launch("norm backward kernels");
  if (rc || (!dgamma && !dbeta)) return rc;
  norm_bwd_join_kernel<<<dim3((unsigned)((cols + 31) / 32), 2), NB_THREADS, 0, s>>>(P);
  return check_launch("norm backward join kernel");
}
