// The normalization regions' backward: with xh = (x - mu) / d (mu = 0 for
// RMSNorm), g = ct * gamma and means over a row's columns,
//   dx     = (g - [mean g] - xh mean(g xh)) / d     ([.] LayerNorm only)
//   dgamma = sum over rows of ct * xh,   dbeta = sum over rows of ct.
// Sums are held in f32 over trees fixed by the sizes: no atomics.
#include "vec8.cuh"
#include "pair.cuh"
#include "pipe.cuh"
#include "trainops.h"

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
  const Columns<VEC, 8> sc((int64_t)blockIdx.x * 256, 32, lane, P.cols);
  float gamma[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) gamma[k] = 1.0f;
  if (P.gamma) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (sc.has(k))
        gamma[k] = P.param_dtype == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)P.gamma)[sc.col(k)])
                                             : ((const float*)P.gamma)[sc.col(k)];
  }
  float dg[8] = {}, db[8] = {};
  const int64_t per = (P.rows + P.blocks - 1) / P.blocks;
  const int64_t r0 = (int64_t)blockIdx.y * per;
  const int64_t r1 = r0 + per < P.rows ? r0 + per : P.rows;
  for (int64_t r = r0 + warp; r < r1; r += NB_WARPS) {
    const float4 st = P.stats[r];
    Piece<XT, VEC, 8> xp;
    Piece<CT, VEC, 8> cp;
    sc.load(P.x, r * P.ldx, xp);
    sc.load(P.ct, r * P.ldc, cp);
    float x[8], c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = xp.get(k), c[k] = cp.get(k);
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

struct NormFusedParams {
  NormBwdParams B;
  int32_t team, teams;       // threads of a team, teams of a CTA
};

template <int TY, int KIND, bool VEC, int NV, int CTA>
__global__ void __launch_bounds__(CTA, 512 / CTA) norm_bwd_fused_kernel(const __grid_constant__ NormFusedParams Q) {
  // gamma in f32, laid out as the threads read it; then the CTA's column sums.
  extern __shared__ __align__(16) float smem[];
  __shared__ float2 red[2][CTA / 32];
  const NormBwdParams& P = Q.B;
  constexpr bool LAYER = KIND == PSK_NORM_LAYER;
  const int T = Q.team, team = threadIdx.x / T, t = threadIdx.x - team * T, nw = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = (int64_t)gridDim.x * Q.teams;
  auto group = [&](int j) { return Columns<VEC, 8>((int64_t)j * T * 8, T, t, P.cols); };
  int flip = 0;
  // Sum two values over the team; one barrier (the buffers alternate).
  auto team_sum = [&](f2 a, f2 b) {
    float s = a.x + a.y, u = b.x + b.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    }
    if (nw == 1) return make_float2(s, u);
    flip ^= 1;
    if (lane == 0) red[flip][warp] = make_float2(s, u);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(T) : "memory");
    float2 v = red[flip][team * nw];
    for (int w = 1; w < nw; ++w) {
      const float2 q = red[flip][team * nw + w];
      v.x += q.x, v.y += q.y;
    }
    return v;
  };

  // gamma of group j, columns k..k+3: float4 number (2 j + k / 4) T + t.
  for (int i = threadIdx.x; i < NV * 8 * T; i += CTA) {
    const int at = i >> 2, who = at % T, piece = at / T, k = (piece & 1) * 4 + (i & 3);
    const int64_t c = Columns<VEC, 8>((int64_t)(piece >> 1) * T * 8, T, who, P.cols).col(k);
    float g = 1.0f;
    if (P.gamma && c < P.cols)
      g = P.param_dtype == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)P.gamma)[c]) : ((const float*)P.gamma)[c];
    smem[i] = g;
  }
  __syncthreads();
  const float4* gamma = (const float4*)smem;

  f2 dg[NV][4], db[LAYER ? NV : 1][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dg[j][k] = f2{0.0f, 0.0f};
      if (LAYER) db[j][k] = f2{0.0f, 0.0f};
    }
  int64_t r = (int64_t)blockIdx.x * Q.teams + team;
  Piece<TY, VEC, 8> x[NV], c[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) group(j).load(P.x, row * P.ldx, x[j]), group(j).load(P.ct, row * P.ldc, c[j]);
  };
  if (r < P.rows) fetch(r);
  for (; r < P.rows; r += step) {
    f2 xv[NV][4], cv[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xv[j][k] = f2{x[j].get(2 * k), x[j].get(2 * k + 1)};
        cv[j][k] = f2{c[j].get(2 * k), c[j].get(2 * k + 1)};
      }
    if (r + step < P.rows) fetch(r + step);
    auto gated = [&](int j, f2* g) {       // ct gamma
      const float4 a = gamma[(2 * j) * T + t], b = gamma[(2 * j + 1) * T + t];
      g[0] = f2_mul(cv[j][0], f2{a.x, a.y}), g[1] = f2_mul(cv[j][1], f2{a.z, a.w});
      g[2] = f2_mul(cv[j][2], f2{b.x, b.y}), g[3] = f2_mul(cv[j][3], f2{b.z, b.w});
    };
    float mg = 0.0f;
    if (LAYER) {
      f2 s{0.0f, 0.0f}, u{0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        f2 g[4];
        gated(j, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) s = f2_add(s, xv[j][k]), u = f2_add(u, g[k]);
      }
      const float2 v = team_sum(s, u);
      const f2 mu = f2_splat(-v.x * P.inv_cols);
      mg = v.y * P.inv_cols;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xv[j][k] = f2_add(xv[j][k], mu);
          if (!group(j).has(2 * k)) xv[j][k].x = 0.0f;
          if (!group(j).has(2 * k + 1)) xv[j][k].y = 0.0f;
        }
    }
    f2 s{0.0f, 0.0f}, u{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 g[4];
      gated(j, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) s = f2_fma(xv[j][k], xv[j][k], s), u = f2_fma(xv[j][k], g[k], u);
    }
    const float2 v = team_sum(s, u);
    const float rd = 1.0f / sqrtf(v.x * P.inv_cols + P.eps);
    const f2 rd2 = f2_splat(rd), m2 = f2_splat(-(v.y * rd * P.inv_cols)), nmg = f2_splat(-mg);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 g[4];
      gated(j, g);
      float o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f2 xh = f2_mul(xv[j][k], rd2);
        dg[j][k] = f2_fma(cv[j][k], xh, dg[j][k]);
        if (LAYER) db[j][k] = f2_add(db[j][k], cv[j][k]);
        const f2 y = f2_mul(f2_fma(xh, m2, LAYER ? f2_add(g[k], nmg) : g[k]), rd2);
        o[2 * k] = y.x, o[2 * k + 1] = y.y;
      }
      group(j).template store<TY>(P.dx, r * P.ldd, o);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!P.dgamma && !P.dbeta) return;
  // The CTA's column sums: its teams' in turn, through shared memory.
  float* colsum = smem + NV * 8 * T;
#pragma unroll
  for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
    float* part = P.part + ((int64_t)which * P.blocks + blockIdx.x) * P.pcols;
    for (int q = 0; q < Q.teams; ++q) {
      if (q > 0) __syncthreads();
      if (team == q) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (!group(j).has(k)) continue;
            const int64_t col = group(j).col(k);
            const f2 d = which == 0 ? dg[j][k / 2] : db[LAYER ? j : 0][k / 2];
            float a = k & 1 ? d.y : d.x;
            if (q > 0) a += colsum[col];
            if (q + 1 == Q.teams) part[col] = a;
            else colsum[col] = a;
          }
      }
    }
    if (Q.teams > 1) __syncthreads();
  }
}

// ----------------------------------------------------------- the ring kernel
//
// The same pass for rows of one storage type of 256 to 16384 columns that are
// 16-byte aligned: x and ct rows are copied by TMA into a ring of shared
// memory, several rows ahead (what keeps HBM busy: registers alone hold too
// few bytes in flight), and read from there for each reduction and for dx; a
// team's threads keep only their columns' dgamma and dbeta sums in registers.
// A team's first thread refills its own slots as soon as the team's warps have
// left them (a separate producer warp would leave 96 registers a thread):
// LayerNorm past a row's first barrier, which comes early in it; RMSNorm, whose
// only barrier comes halfway, as its warps report.
constexpr int RING_THREADS = 512;          // sixteen warps: 128 registers a thread
constexpr int RING_MAX_COLS = 16384;
constexpr int RING_MAX_SLOTS = 32;
constexpr int RING_MAX_BLOCKS = 160;
constexpr int RING_SMEM = 220 * 1024;

struct NormRingParams {
  NormBwdParams B;
  int32_t team, teams;       // threads of a team (the kernel's T), teams of a CTA
  int32_t slots;             // a multiple of teams: a slot's phases are one team's, in order
  int32_t row_bytes;         // of x and of ct; a slot holds one of each
};

// 1 / sqrt(v) by the unit's approximation and one Newton step (about one ulp;
// v = 0 gives +inf, NaN and negative v NaN, as the division would).
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float y = rsqrtf(v);
  const float h = 0.5f * v * y;
  const float z = fmaf(y, fmaf(-h, y, 0.5f), y);
  return v > 0.0f && v < INFINITY ? z : y;
}

template <int TY, int KIND, int NV, int T>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_bwd_ring_kernel(const __grid_constant__ NormRingParams Q) {
  // gamma in f32 as the threads read it (later the column sums), then the ring.
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ uint64_t full[RING_MAX_SLOTS], empty[RING_MAX_SLOTS];
  __shared__ __align__(16) float red[2][3][RING_THREADS / 32];
  __shared__ volatile int abort_flag;
  constexpr bool LAYER = KIND == PSK_NORM_LAYER;
  constexpr int E = TY == PSK_BF16 ? 8 : 4;              // elements of a 16-byte group
  constexpr int NG = NV * 8 / E;                         // groups of a thread
  const NormBwdParams& P = Q.B;
  constexpr int TEAMS = RING_THREADS / T, nw = T / 32;
  const int tid = threadIdx.x, slots = Q.slots;
  const int groups = (int)P.cols / E;
  float* gamma = (float*)ring_smem;
  unsigned char* ring = ring_smem + (size_t)(NG * E * T) * 4;
  const int slot_bytes = 2 * Q.row_bytes;
  const int n_local = blockIdx.x < P.rows ? (int)((P.rows - 1 - blockIdx.x) / gridDim.x + 1) : 0;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], T / 32);
    abort_flag = 0;
    fence_barrier_init();
  }
  // gamma of group j of thread t: float4 number (j E / 4 + i) T + t, i < E / 4.
  for (int i = tid; i < NG * E * T; i += RING_THREADS) {
    const int at = i >> 2, who = at % T, piece = at / T;
    const int64_t c = ((int64_t)(piece * 4 / E) * T + who) * E + (piece * 4) % E + (i & 3);
    float g = 1.0f;
    if (P.gamma && c < P.cols)
      g = P.param_dtype == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)P.gamma)[c]) : ((const float*)P.gamma)[c];
    gamma[i] = g;
  }
  __syncthreads();

  // After a timeout (`dead`) a thread skips waits and work but keeps meeting
  // its team's barriers.
  const int team = tid / T, t = tid - team * T, lane = tid & 31, warp = tid >> 5;
  bool dead = false;
  int flip = 0, issued = -1;
  const long long drop = g_pipe_drop_row;
  // The team's first thread copies local row i into its slot s.
  auto fetch = [&](int i, int s) {
    if (t != 0 || i >= n_local || dead || (drop >= 0 && i >= drop)) return;
    const int64_t r = blockIdx.x + (int64_t)i * gridDim.x;
    unsigned char* at = ring + (size_t)s * slot_bytes;
    mbar_arrive_expect_tx(&full[s], (uint32_t)slot_bytes);
    bulk_copy_g2s(at, (const unsigned char*)P.x + r * P.ldx * (16 / E), (uint32_t)Q.row_bytes, &full[s]);
    bulk_copy_g2s(at + Q.row_bytes, (const unsigned char*)P.ct + r * P.ldc * (16 / E), (uint32_t)Q.row_bytes, &full[s]);
    issued = i;
  };
  // Sums over the team, one barrier (the buffers alternate).
  auto team_sum = [&](float* v, int n) {
    flip ^= 1;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (q >= n) break;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[q] += __shfl_xor_sync(0xFFFFFFFFu, v[q], o);
      if (lane == 0) red[flip][q][warp] = v[q];
    }
    if (nw == 1) return;
    named_barrier(1 + team, T);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (q >= n) break;
      const float2* p = (const float2*)&red[flip][q][team * nw];     // nw: 2, 4, 8 or 16
      float2 s = p[0];
      #pragma unroll
      for (int w = 1; w < nw / 2; ++w) {
        const float2 u = p[w];
        s.x += u.x, s.y += u.y;
      }
      v[q] = s.x + s.y;
    }
  };
  for (int i = team; i < slots; i += TEAMS) fetch(i, i);
  const f2 zero{0.0f, 0.0f};
  f2 dg[NG][E / 2], db[LAYER ? NG : 1][E / 2];
#pragma unroll
  for (int j = 0; j < NG; ++j)
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      dg[j][k] = zero;
      if (LAYER) db[j][k] = zero;
    }
  int s = team, before = 0;                  // the row's slot, the last row's
  uint32_t parity = 0, parity_before = 0;    // of their phases
  for (int i = team; i < n_local; i += TEAMS) {
    const int64_t r = blockIdx.x + (int64_t)i * gridDim.x;
    dead = dead || abort_flag;
    if (!LAYER && i != team && t == 0 && !dead) {
      if (mbar_wait(&empty[before], parity_before)) fetch(i - TEAMS + slots, before);
      else abort_flag = 1, dead = true;
    }
    if (!dead && !mbar_wait(&full[s], parity)) { abort_flag = 1; dead = true; }
    const unsigned char* xs = ring + (size_t)s * slot_bytes;
    const unsigned char* cs = xs + Q.row_bytes;
    auto values = [&](const unsigned char* p, int j, f2* v) {
      const uint4 u = *(const uint4*)(p + (size_t)(j * T + t) * 16);
      if constexpr (TY == PSK_BF16) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = f2{__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)};
      } else {
        v[0] = f2{__uint_as_float(u.x), __uint_as_float(u.y)}, v[1] = f2{__uint_as_float(u.z), __uint_as_float(u.w)};
      }
    };
    auto gate = [&](int j, f2* g) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const float4 a = ((const float4*)gamma)[(j * (E / 4) + q) * T + t];
        g[2 * q] = f2_mul(g[2 * q], f2{a.x, a.y}), g[2 * q + 1] = f2_mul(g[2 * q + 1], f2{a.z, a.w});
      }
    };
    float sums[3];
    float mu = 0.0f;
    if (LAYER) {
      f2 a = zero;
      if (!dead) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          if (j * T + t >= groups) continue;
          f2 x[E / 2];
          values(xs, j, x);
#pragma unroll
          for (int k = 0; k < E / 2; ++k) a = f2_add(a, x[k]);
        }
      }
      sums[0] = a.x + a.y;
      team_sum(sums, 1);
      if (nw == 1) __syncwarp();
      if (i != team) fetch(i - TEAMS + slots, before);
      mu = sums[0] * P.inv_cols;
    }
    const f2 nmu = f2_splat(-mu);
    constexpr bool KEEP = !LAYER;            // widened values stay in registers for dx
    f2 kx[KEEP ? NG : 1][E / 2], kc[KEEP ? NG : 1][E / 2];
    f2 a = zero, b = zero, d = zero;
    if (!dead) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (j * T + t >= groups) continue;
        f2 x[E / 2], g[E / 2];
        values(xs, j, x);
        values(cs, j, g);
        if (KEEP) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) kx[KEEP ? j : 0][k] = x[k], kc[KEEP ? j : 0][k] = g[k];
        }
        gate(j, g);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          if (LAYER) x[k] = f2_add(x[k], nmu), d = f2_add(d, g[k]);
          a = f2_fma(x[k], x[k], a), b = f2_fma(x[k], g[k], b);
        }
      }
    }
    sums[0] = a.x + a.y, sums[1] = b.x + b.y, sums[2] = d.x + d.y;
    team_sum(sums, LAYER ? 3 : 2);
    const float mg = sums[2] * P.inv_cols;
    const float rd = rsqrt_newton(sums[0] * P.inv_cols + P.eps);
    const f2 rd2 = f2_splat(rd), m2 = f2_splat(-(sums[1] * rd * P.inv_cols)), nmg = f2_splat(-mg);
    if (!dead) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (j * T + t >= groups) continue;
        f2 x[E / 2], c[E / 2], g[E / 2], y[E / 2];
        if (KEEP) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) x[k] = kx[KEEP ? j : 0][k], c[k] = kc[KEEP ? j : 0][k];
        } else {
          values(xs, j, x);
          values(cs, j, c);
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) g[k] = c[k];
        gate(j, g);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          const f2 xh = f2_mul(LAYER ? f2_add(x[k], nmu) : x[k], rd2);
          dg[j][k] = f2_fma(c[k], xh, dg[j][k]);
          if (LAYER) db[j][k] = f2_add(db[j][k], c[k]);
          y[k] = f2_mul(f2_fma(xh, m2, LAYER ? f2_add(g[k], nmg) : g[k]), rd2);
        }
        unsigned char* o = (unsigned char*)P.dx + r * P.ldd * (16 / E) + (size_t)(j * T + t) * 16;
        if constexpr (TY == PSK_BF16)
          *(uint4*)o = make_uint4(f32x2_to_bf16x2(y[0].x, y[0].y), f32x2_to_bf16x2(y[1].x, y[1].y),
                                  f32x2_to_bf16x2(y[2].x, y[2].y), f32x2_to_bf16x2(y[3].x, y[3].y));
        else
          *(float4*)o = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
      }
    }
    __syncwarp();
    if (!LAYER && !dead && lane == 0) mbar_arrive(&empty[s]);
    before = s, parity_before = parity;
    s += TEAMS;
    if (s >= slots) s -= slots, parity ^= 1;
  }
  // After a timeout, copies still in flight land before the CTA retires.
  if (dead)
    for (int i = issued; i >= 0 && i > issued - slots; i -= TEAMS)
      mbar_wait(&full[i % slots], (uint32_t)(i / slots) & 1u);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!P.dgamma && !P.dbeta) return;
  // The CTA's column sums, its teams' in turn, in gamma's place.
#pragma unroll
  for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
    float* part = P.part + ((int64_t)which * P.blocks + blockIdx.x) * P.pcols;
    for (int q = 0; q < TEAMS; ++q) {
      if (TEAMS > 1) named_barrier(15, RING_THREADS);
      if (team != q) continue;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (j * T + t >= groups) continue;
#pragma unroll
        for (int h = 0; h < E / 4; ++h) {
          const f2 a = which == 0 ? dg[j][2 * h] : db[LAYER ? j : 0][2 * h];
          const f2 b = which == 0 ? dg[j][2 * h + 1] : db[LAYER ? j : 0][2 * h + 1];
          float4 sum = make_float4(a.x, a.y, b.x, b.y);
          float4* held = (float4*)gamma + (j * (E / 4) + h) * T + t;
          if (q > 0) {
            const float4 u = *held;
            sum.x += u.x, sum.y += u.y, sum.z += u.z, sum.w += u.w;
          }
          if (q + 1 == TEAMS) *(float4*)(part + (j * T + t) * E + 4 * h) = sum;
          else *held = sum;
        }
      }
    }
  }
}

// The row blocks' sums joined: 32 columns a CTA, 32 warps over the blocks in
// turn (the few sums a warp adds are all in flight at once).
constexpr int NB_JOIN_THREADS = 1024;
__global__ void __launch_bounds__(NB_JOIN_THREADS) norm_bwd_join_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float sums[NB_JOIN_THREADS / 32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int which = blockIdx.y;
  void* out = which ? P.dbeta : P.dgamma;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!out) return;
  float s = 0.0f;
  if (col < P.cols) {
    const float* p = P.part + (int64_t)which * P.blocks * P.pcols + col;
    for (int b0 = warp; b0 < P.blocks; b0 += 16 * (NB_JOIN_THREADS / 32)) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = b0 + i * (NB_JOIN_THREADS / 32);
        v[i] = b < P.blocks ? p[(int64_t)b * P.pcols] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s += v[i];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  // Column `warp`'s 32 sums, one a lane.
  s = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int64_t c = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && c < P.cols) {
    if (P.grad_dtype == PSK_BF16) ((uint16_t*)out)[c] = f32_to_bf16_bits(s);
    else ((float*)out)[c] = s;
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

// The ring kernel's shape for rows of this size, or false: teams of the fewest
// threads that hold a row's column sums in two (up to 512 columns) or four
// groups of eight a thread -- wide threads share a row's shuffles and barrier
// among more columns, and small teams overlap more rows -- and as many slots
// as fit, two rows a team at least.
static bool ring_shape(NormRingParams& Q, int* nv, int32_t dt, int64_t cols) {
  if (cols < 256 || cols > RING_MAX_COLS || cols % 8 != 0) return false;
  *nv = cols <= 512 ? 2 : 4;
  Q.team = 32;
  while (Q.team * *nv * 8 < cols) Q.team *= 2;
  Q.teams = RING_THREADS / Q.team;
  Q.row_bytes = (int32_t)cols * dtype_size(dt);
  const int fits = (RING_SMEM - *nv * 8 * Q.team * 4) / (2 * Q.row_bytes);
  Q.slots = (fits < RING_MAX_SLOTS ? fits : RING_MAX_SLOTS) / Q.teams * Q.teams;
  return Q.slots >= 2 * Q.teams;
}

static uint64_t norm_bwd_layout(int64_t rows, int64_t cols, uint64_t* part) {
  const uint64_t stats = ((uint64_t)rows * 16 + 255) / 256 * 256;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  *part = stats;
  int blocks = norm_bwd_blocks(rows, cols);
  if (cols <= NB_FUSED_COLS && fused_blocks(rows, cols) > blocks) blocks = fused_blocks(rows, cols);
  const int64_t ring = rows < RING_MAX_BLOCKS ? rows : RING_MAX_BLOCKS;
  if (ring > blocks) blocks = (int)ring;
  return stats + 2ull * blocks * pcols * 4;
}

template <int TY, int KIND, bool VEC, int NV, int CTA>
static void fused_launch(const NormFusedParams& Q, cudaStream_t s) {
  norm_bwd_fused_kernel<TY, KIND, VEC, NV, CTA>
      <<<(unsigned)Q.B.blocks, CTA, (size_t)(NV * 8 * Q.team + (Q.teams > 1 ? Q.B.cols : 0)) * 4, s>>>(Q);
}

template <int TY, int KIND, int NV, int T>
static int ring_launch_team(const NormRingParams& Q, cudaStream_t s) {
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)norm_bwd_ring_kernel<TY, KIND, NV, T>, RING_SMEM, limit);
  const size_t smem = (size_t)NV * 8 * T * 4 + (size_t)Q.slots * 2 * Q.row_bytes;
  norm_bwd_ring_kernel<TY, KIND, NV, T><<<(unsigned)Q.B.blocks, RING_THREADS, smem, s>>>(Q);
  return check_launch("norm backward ring kernel");
}

template <int TY, int KIND>
static int ring_launch(const NormRingParams& Q, int nv, cudaStream_t s) {
  if (nv == 2) return ring_launch_team<TY, KIND, 2, 32>(Q, s);
  switch (Q.team) {
    case 32: return ring_launch_team<TY, KIND, 4, 32>(Q, s);
    case 64: return ring_launch_team<TY, KIND, 4, 64>(Q, s);
    case 128: return ring_launch_team<TY, KIND, 4, 128>(Q, s);
    case 256: return ring_launch_team<TY, KIND, 4, 256>(Q, s);
    default: return ring_launch_team<TY, KIND, 4, 512>(Q, s);
  }
}

int norm_bwd_status(unsigned int* v, bool reset) {
  if (cudaMemcpyFromSymbol(v, g_pipe_status, sizeof(*v)) != cudaSuccess) return check_launch("device status read");
  if (reset) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_pipe_status, &z, sizeof(z)) != cudaSuccess) return check_launch("device status reset");
  }
  return PSK_OK;
}

int norm_bwd_set_drop_row(long long row) {
  if (cudaMemcpyToSymbol(g_pipe_drop_row, &row, sizeof(row)) != cudaSuccess) return check_launch("test hook write");
  return PSK_OK;
}

// The column sums' join, launched so that its set-up overlaps the kernel
// before it.
static int norm_bwd_join(const NormBwdParams& P, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((P.cols + 31) / 32), P.dbeta ? 2 : 1);
  cfg.blockDim = dim3(NB_JOIN_THREADS);
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
  const bool vec = cols % 8 == 0 && rows_vec8(x, xt, ldx, rows) && rows_vec8(ct, ct_t, ldc, rows) && rows_vec8(dx, dxt, ldd, rows) &&
                   (!gamma || rows_vec8(gamma, param_dtype, cols, 1));
  NormRingParams G{};
  int nv = 0;
  if (vec && xt == ct_t && xt == dxt && ring_shape(G, &nv, xt, cols)) {
    G.B = P;
    int64_t blocks = (rows + G.teams - 1) / G.teams;
    const int64_t sms = device_sm_count() < RING_MAX_BLOCKS ? device_sm_count() : RING_MAX_BLOCKS;
    G.B.blocks = (int)(blocks < sms ? blocks : sms);
    rc = with_dtype(xt, [&](auto TY) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        constexpr int KIND = LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS;
        return ring_launch<TY.value, KIND>(G, nv, s);
      });
    });
    return rc || (!dgamma && !dbeta) ? rc : norm_bwd_join(G.B, s);
  }
  if (cols <= NB_FUSED_COLS && xt == ct_t && xt == dxt) {
    const FusedShape f = fused_shape(cols);
    NormFusedParams Q{P, f.team, f.teams};
    const int64_t resident = (int64_t)device_sm_count() * (512 / f.cta);
    Q.B.blocks = fused_blocks(rows, cols);
    if (Q.B.blocks > resident) Q.B.blocks = (int)resident;
    with_dtype(xt, [&](auto TY) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        constexpr int KIND = LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS;
        return with_bool(vec, [&](auto VEC) {
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
