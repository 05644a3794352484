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

// ---------------------------------------------------------- the fused kernel
//
// One pass over rows of up to 8192 columns of one storage type: a team of T
// threads holds a row's x and ct in registers (NV groups of eight columns a
// thread) from the reductions to dx, while its next row's loads are in
// flight, and keeps its columns' dgamma and dbeta sums in registers over all
// of its rows.  The floor is one read of x and ct and one write of dx; a
// CTA's column sums go to the workspace once.
constexpr int NB_FUSED_COLS = 8192;
constexpr int NB_ROWS_PER_TEAM = 4;        // at least, where there are as many

// Eight of a thread's columns as loaded.
template <int TY, bool VEC>
struct Octet {
  static constexpr int W = VEC && TY == PSK_BF16 ? 4 : 8;
  uint32_t w[W];
  __device__ __forceinline__ float get(int k) const {
    if constexpr (VEC && TY == PSK_BF16) return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
    else return __uint_as_float(w[k]);
  }
};

// The columns of thread t: group j is columns (j T + t) 8 + k with 16-byte
// accesses, else j 8 T + k T + t (a warp's accesses then coalesce).
template <int TY, bool VEC>
struct TeamCols {
  int T, t, cols;
  __device__ __forceinline__ int col(int j, int k) const { return VEC ? (j * T + t) * 8 + k : (j * 8 + k) * T + t; }
  __device__ __forceinline__ bool has(int j, int k) const { return col(j, VEC ? 0 : k) < cols; }
  __device__ __forceinline__ void load(const void* p, int64_t row, int j, Octet<TY, VEC>& o) const {
    if constexpr (VEC) {
      const bool in = has(j, 0);
      if constexpr (TY == PSK_BF16) {
        const uint4 u = in ? __ldcs((const uint4*)((const uint16_t*)p + row + col(j, 0))) : make_uint4(0, 0, 0, 0);
        o.w[0] = u.x, o.w[1] = u.y, o.w[2] = u.z, o.w[3] = u.w;
      } else {
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4* q = (const uint4*)((const float*)p + row + col(j, 0));
        const uint4 a = in ? __ldcs(q) : z, b = in ? __ldcs(q + 1) : z;
        o.w[0] = a.x, o.w[1] = a.y, o.w[2] = a.z, o.w[3] = a.w, o.w[4] = b.x, o.w[5] = b.y, o.w[6] = b.z, o.w[7] = b.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o.w[k] = 0;
        if (has(j, k)) {
          if constexpr (TY == PSK_BF16) o.w[k] = (uint32_t)((const uint16_t*)p)[row + col(j, k)] << 16;
          else o.w[k] = ((const uint32_t*)p)[row + col(j, k)];
        }
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t row, int j, const float* v) const {
    if constexpr (VEC) {
      if (has(j, 0)) store8<TY, true>(p, row + col(j, 0), 8, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (has(j, k)) {
          if constexpr (TY == PSK_BF16) ((uint16_t*)p)[row + col(j, k)] = f32_to_bf16_bits(v[k]);
          else ((float*)p)[row + col(j, k)] = v[k];
        }
    }
  }
};

struct NormFusedParams {
  NormBwdParams B;
  int32_t team, teams;       // threads of a team, teams of a CTA
};

template <int TY, int KIND, bool VEC, int NV, int CTA>
__global__ void __launch_bounds__(CTA, 512 / CTA) norm_bwd_fused_kernel(const __grid_constant__ NormFusedParams Q) {
  extern __shared__ float colsum[];                       // [cols] of the CTA, added team by team
  __shared__ float2 red[2][CTA / 32];
  const NormBwdParams& P = Q.B;
  const int T = Q.team, team = threadIdx.x / T, t = threadIdx.x - team * T, nw = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const TeamCols<TY, VEC> tc{T, t, (int)P.cols};
  const int64_t step = (int64_t)gridDim.x * Q.teams;
  int flip = 0;
  // Sum two values over the team; one barrier (the buffers alternate).
  auto team_sum = [&](float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (nw == 1) return make_float2(a, b);
    flip ^= 1;
    if (lane == 0) red[flip][warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(T) : "memory");
    float2 s = red[flip][team * nw];
    for (int w = 1; w < nw; ++w) {
      const float2 u = red[flip][team * nw + w];
      s.x += u.x, s.y += u.y;
    }
    return s;
  };

  float gamma[NV][8], dg[NV][8], db[KIND == PSK_NORM_LAYER ? NV : 1][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = tc.col(j, k);
      gamma[j][k] = 1.0f;
      if (P.gamma && c < P.cols)
        gamma[j][k] = P.param_dtype == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)P.gamma)[c])
                                                : ((const float*)P.gamma)[c];
      dg[j][k] = 0.0f;
      if (KIND == PSK_NORM_LAYER) db[j][k] = 0.0f;
    }

  int64_t r = (int64_t)blockIdx.x * Q.teams + team;
  Octet<TY, VEC> x[NV], c[NV];
  if (r < P.rows) {
#pragma unroll
    for (int j = 0; j < NV; ++j) tc.load(P.x, r * P.ldx, j, x[j]), tc.load(P.ct, r * P.ldc, j, c[j]);
  }
  for (; r < P.rows; r += step) {
    float xv[NV][8], cv[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) xv[j][k] = x[j].get(k), cv[j][k] = c[j].get(k);
    if (r + step < P.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        tc.load(P.x, (r + step) * P.ldx, j, x[j]), tc.load(P.ct, (r + step) * P.ldc, j, c[j]);
    }
    float mg = 0.0f;
    if (KIND == PSK_NORM_LAYER) {
      float s = 0.0f, u = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) s += xv[j][k], u = fmaf(cv[j][k], gamma[j][k], u);
      const float2 v = team_sum(s, u);
      const float mu = v.x * P.inv_cols;
      mg = v.y * P.inv_cols;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) xv[j][k] = tc.has(j, k) ? xv[j][k] - mu : 0.0f;
    }
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s = fmaf(xv[j][k], xv[j][k], s);
        u = fmaf(xv[j][k], cv[j][k] * gamma[j][k], u);
      }
    const float2 v = team_sum(s, u);
    const float rd = 1.0f / sqrtf(v.x * P.inv_cols + P.eps);
    const float m2 = v.y * rd * P.inv_cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = xv[j][k] * rd;
        const float g = cv[j][k] * gamma[j][k];
        o[k] = fmaf(-xh, m2, KIND == PSK_NORM_LAYER ? g - mg : g) * rd;
        dg[j][k] = fmaf(cv[j][k], xh, dg[j][k]);
        if (KIND == PSK_NORM_LAYER) db[j][k] += cv[j][k];
      }
      tc.store(P.dx, r * P.ldd, j, o);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!P.dgamma && !P.dbeta) return;
  // The CTA's column sums: its teams' in turn, through shared memory.
#pragma unroll
  for (int which = 0; which < (KIND == PSK_NORM_LAYER ? 2 : 1); ++which) {
    float* part = P.part + ((int64_t)which * P.blocks + blockIdx.x) * P.pcols;
    for (int q = 0; q < Q.teams; ++q) {
      if (q > 0) __syncthreads();
      if (team == q) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = tc.col(j, k);
            if (col < P.cols) {
              float a = which == 0 ? dg[j][k] : db[KIND == PSK_NORM_LAYER ? j : 0][k];
              if (q > 0) a += colsum[col];
              if (q + 1 == Q.teams) part[col] = a;
              else colsum[col] = a;
            }
          }
      }
    }
    if (Q.teams > 1) __syncthreads();
  }
}

// The row blocks' sums joined: 32 columns a CTA, warps over blocks in turn.
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_join_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float sums[NB_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int which = blockIdx.y;
  void* out = which ? P.dbeta : P.dgamma;
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// Row blocks of the two-pass kernels' column sums: enough CTAs to fill the
// GPU, at least 16 rows each.
static int norm_bwd_blocks(int64_t rows, int64_t cols) {
  const int64_t slices = (cols + 255) / 256;
  int64_t b = (152 * 8 + slices - 1) / slices;
  if (b > (rows + 15) / 16) b = (rows + 15) / 16;
  return (int)(b < 1 ? 1 : b > NB_MAX_BLOCKS ? NB_MAX_BLOCKS : b);
}

// The fused kernel's shape: teams of the fewest threads that hold a row in
// one or two groups of eight columns each.
struct FusedShape {
  int team, teams, nv, cta;
};
static FusedShape fused_shape(int64_t cols) {
  FusedShape f{32, 1, 1, 256};
  const int64_t groups = (cols + 7) / 8;
  while (f.team < 256 && f.team < groups) f.team *= 2;
  if (groups > 256) f.nv = 2;
  if (groups > 512) f.team = f.cta = 512;
  f.teams = f.cta / f.team;
  return f;
}

// Most CTAs of the fused kernel (two of 256 threads an SM, or one of 512, on
// 160 SMs), at least NB_ROWS_PER_TEAM rows for each team.
static int fused_blocks(int64_t rows, int64_t cols) {
  const FusedShape f = fused_shape(cols);
  const int64_t most = 160 * (512 / f.cta), want = (rows + f.teams * NB_ROWS_PER_TEAM - 1) / (f.teams * NB_ROWS_PER_TEAM);
  return (int)(want < most ? want : most);
}

static uint64_t norm_bwd_layout(int64_t rows, int64_t cols, uint64_t* part) {
  const uint64_t stats = ((uint64_t)rows * 16 + 255) / 256 * 256;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  *part = stats;
  int blocks = norm_bwd_blocks(rows, cols);
  if (cols <= NB_FUSED_COLS && fused_blocks(rows, cols) > blocks) blocks = fused_blocks(rows, cols);
  return stats + 2ull * blocks * pcols * 4;
}

template <int TY, int KIND, bool VEC, int NV, int CTA>
static void fused_launch(const NormFusedParams& Q, cudaStream_t s) {
  norm_bwd_fused_kernel<TY, KIND, VEC, NV, CTA>
      <<<(unsigned)Q.B.blocks, CTA, Q.teams > 1 ? (size_t)Q.B.cols * 4 : 0, s>>>(Q);
}

// The column sums' join, launched so that its set-up overlaps the kernel
// before it.
static int norm_bwd_join(const NormBwdParams& P, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((P.cols + 31) / 32), P.dbeta ? 2 : 1);
  cfg.blockDim = dim3(NB_THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, norm_bwd_join_kernel, P);
  return check_launch("norm backward join kernel");
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
  if (cols <= NB_FUSED_COLS && xt == ct_t && xt == dxt) {
    const FusedShape f = fused_shape(cols);
    NormFusedParams Q{P, f.team, f.teams};
    const int64_t resident = (int64_t)device_sm_count() * (512 / f.cta);
    Q.B.blocks = fused_blocks(rows, cols);
    if (Q.B.blocks > resident) Q.B.blocks = (int)resident;
    with_dtype(xt, [&](auto TY) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        constexpr int KIND = LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS;
        return with_bool(vec && cols % 8 == 0, [&](auto VEC) {
          if (f.cta == 512) fused_launch<TY.value, KIND, VEC.value, 2, 512>(Q, s);
          else if (f.nv == 2) fused_launch<TY.value, KIND, VEC.value, 2, 256>(Q, s);
          else fused_launch<TY.value, KIND, VEC.value, 1, 256>(Q, s);
          return 0;
        });
      });
    });
    rc = check_launch("norm backward fused kernel");
    return rc || (!dgamma && !dbeta) ? rc : norm_bwd_join(Q.B, s);
  }
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
  return norm_bwd_join(P, s);
}
