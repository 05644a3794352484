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
// or L2.  This kernel and the next serve what the kernels of one pass below do
// not: tensors of several types, rows beyond 16384 columns.  They read x and ct
// from HBM twice: [16384, 4096] f32 x, bf16 ct, f32 dx 184 us, 0.67 GB (0.4 GB of
// it once more); [4096, 20000] bf16 204 us.
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

// 1 / sqrt(v) by the unit's approximation and one Newton step (about one ulp;
// v = 0 gives +inf, NaN and negative v NaN, as the division would).
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float y = rsqrtf(v);
  const float h = 0.5f * v * y;
  const float z = fmaf(y, fmaf(-h, y, 0.5f), y);
  return v > 0.0f && v < INFINITY ? z : y;
}

// ------------------------------------------------------- the warp-a-row kernel
//
// One pass over rows of up to 255 columns of one storage type: a warp holds a
// row's x and ct in registers (eight columns a thread) from the reductions to
// dx, while its next row's loads are in flight, and keeps its columns' dgamma
// and dbeta sums in registers over all of its rows.  The floor is one read of
// x and ct and one write of dx; a CTA's column sums go to the workspace once.
// Rows this short are bound by their chains of shuffles (65536 x 200 bf16, 79
// MB: RMSNorm 27 us, 2.9 TB/s; f32 LayerNorm, 157 MB, 39 us, 4.0 TB/s); a
// second row in flight costs registers that more warps use better.
constexpr int NB_FUSED_COLS = 255;
constexpr int NB_ROWS_PER_WARP = 4;        // at least, where there are as many

template <int TY, int KIND, bool VEC>
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_warps_kernel(const __grid_constant__ NormBwdParams P) {
  __shared__ float colsum[2][NB_WARPS][256];
  constexpr bool LAYER = KIND == PSK_NORM_LAYER;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = (int64_t)gridDim.x * NB_WARPS;
  const Columns<VEC, 8> cols(0, 32, lane, P.cols);
  auto warp_sum = [&](f2 a) {
    float s = a.x + a.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
  };
  const f2 zero{0.0f, 0.0f};
  f2 gamma[4], dg[4], db[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float g = 1.0f;
    if (P.gamma && cols.has(k))
      g = P.param_dtype == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)P.gamma)[cols.col(k)])
                                    : ((const float*)P.gamma)[cols.col(k)];
    if (k & 1) gamma[k / 2].y = g;
    else gamma[k / 2].x = g;
    dg[k / 2] = zero, db[k / 2] = zero;
  }
  int64_t r = (int64_t)blockIdx.x * NB_WARPS + warp;
  Piece<TY, VEC, 8> x, c;
  if (r < P.rows) cols.load(P.x, r * P.ldx, x), cols.load(P.ct, r * P.ldc, c);
  for (; r < P.rows; r += step) {
    f2 xv[4], cv[4], g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      xv[k] = f2{x.get(2 * k), x.get(2 * k + 1)}, cv[k] = f2{c.get(2 * k), c.get(2 * k + 1)};
      g[k] = f2_mul(cv[k], gamma[k]);
    }
    if (r + step < P.rows) cols.load(P.x, (r + step) * P.ldx, x), cols.load(P.ct, (r + step) * P.ldc, c);
    float mg = 0.0f;
    if (LAYER) {
      const float mu = warp_sum(f2_add(f2_add(xv[0], xv[1]), f2_add(xv[2], xv[3]))) * P.inv_cols;
      mg = warp_sum(f2_add(f2_add(g[0], g[1]), f2_add(g[2], g[3]))) * P.inv_cols;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xv[k] = f2_add(xv[k], f2_splat(-mu));
        if (!cols.has(2 * k)) xv[k].x = 0.0f;
        if (!cols.has(2 * k + 1)) xv[k].y = 0.0f;
      }
    }
    f2 a = zero, b = zero;
#pragma unroll
    for (int k = 0; k < 4; ++k) a = f2_fma(xv[k], xv[k], a), b = f2_fma(xv[k], g[k], b);
    const float rd = rsqrt_newton(warp_sum(a) * P.inv_cols + P.eps);
    const f2 rd2 = f2_splat(rd), m2 = f2_splat(-(warp_sum(b) * rd * P.inv_cols)), nmg = f2_splat(-mg);
    float o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f2 xh = f2_mul(xv[k], rd2);
      dg[k] = f2_fma(cv[k], xh, dg[k]);
      if (LAYER) db[k] = f2_add(db[k], cv[k]);
      const f2 y = f2_mul(f2_fma(xh, m2, LAYER ? f2_add(g[k], nmg) : g[k]), rd2);
      o[2 * k] = y.x, o[2 * k + 1] = y.y;
    }
    cols.template store<TY>(P.dx, r * P.ldd, o);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!P.dgamma && !P.dbeta) return;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (cols.has(k)) {
      colsum[0][warp][cols.col(k)] = k & 1 ? dg[k / 2].y : dg[k / 2].x;
      if (LAYER) colsum[1][warp][cols.col(k)] = k & 1 ? db[k / 2].y : db[k / 2].x;
    }
  __syncthreads();
  if (threadIdx.x < P.cols) {
#pragma unroll
    for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
      float s = colsum[which][0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < NB_WARPS; ++w) s += colsum[which][w][threadIdx.x];
      P.part[((int64_t)which * P.blocks + blockIdx.x) * P.pcols + threadIdx.x] = s;
    }
  }
}

// ----------------------------------------------------------- the ring kernel
//
// The same pass for rows of one storage type of 256 to 16384 columns: x and ct rows are copied by TMA into a ring of shared
// memory, several rows ahead (what keeps HBM busy: registers alone hold too
// few bytes in flight), and read from there for each reduction and for dx; a
// team's threads keep only their columns' dgamma and dbeta sums in registers.
// A team's first thread refills its own slots as soon as the team's warps have
// left them (a separate producer warp would leave 96 registers a thread):
// LayerNorm past a row's first barrier, which comes early in it; RMSNorm, whose
// only barrier comes halfway, as its warps report.
//
// [32768, 4096] bf16, 805 MB: 133 us (RMSNorm) and 134 us (LayerNorm), 6.0 TB/s,
// bound by HBM with two reads to a write; [32768, 2048] 71 and 72 us; [16384, 4096] f32
// 139 and 150 us; [512, 2048] 13 us, launches; [4096, 16384] 83 and 104 us, one
// team whose two rows are all that fits beside gamma.  Rows beginning anywhere
// are bound by the instructions of their element-wise accesses: [32768, 1001]
// bf16 48 us, [16384, 3001] bf16 79 and 103 us (twice the warps at half the
// registers took as long); f32 [8192, 3001] 59 us, 5.0 TB/s, [8192, 7999] 149 us.
constexpr int RING_THREADS = 512;          // sixteen warps: 128 registers a thread
constexpr int RING_MAX_COLS = 16384;
constexpr int RING_MAX_SLOTS = 64;
constexpr int RING_MAX_BLOCKS = 160;
constexpr int RING_SMEM = 220 * 1024;

struct NormRingParams {
  NormBwdParams B;
  int32_t team, teams;       // threads of a team (the kernel's T), teams of a CTA
  int32_t slots;             // a multiple of teams: a slot's phases are one team's, in order
  int32_t row_bytes;         // of x and of ct; a slot holds one of each
};

// VEC: 16-byte aligned rows of whole 16-byte groups; group j of thread t begins
// at element (j T + t) E.  Else any rows: TMA copies the 16-byte blocks that a
// row lies in (what they hold of its neighbours is not used; the blocks in
// which the tensor begins and ends are left out, their few elements stored by
// the copying thread), so the row stands whole in its slot, and element k of
// group j is column (j E + k) T + t (the threads' columns must not move with a
// row's alignment, and neighbouring threads then read neighbouring elements).
template <int TY, int KIND, int NV, int T, bool VEC>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_bwd_ring_kernel(const __grid_constant__ NormRingParams Q) {
  // gamma in f32 as the threads read it, then the ring.
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ uint64_t full[RING_MAX_SLOTS], empty[RING_MAX_SLOTS];
  __shared__ __align__(16) float red[2][3][RING_THREADS / 32];
  __shared__ volatile int abort_flag;
  constexpr bool LAYER = KIND == PSK_NORM_LAYER;
  constexpr int ESZ = TY == PSK_BF16 ? 2 : 4;
  constexpr int E = VEC ? 16 / ESZ : NV == 2 ? 4 : 8;    // elements of a group
  constexpr int NG = NV * 8 / E;                         // groups of a thread
  constexpr int TEAMS = RING_THREADS / T, nw = T / 32;
  const NormBwdParams& P = Q.B;
  const int tid = threadIdx.x, slots = Q.slots;
  const int cols = (int)P.cols, groups = VEC ? cols / E : 0;
  float* gamma = (float*)ring_smem;
  unsigned char* ring = ring_smem + (size_t)(NG * E * T) * 4;
  const int slot_bytes = 2 * Q.row_bytes;
  const int n_local = blockIdx.x < P.rows ? (int)((P.rows - 1 - blockIdx.x) / gridDim.x + 1) : 0;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], T / 32);
    abort_flag = 0;
    fence_barrier_init();
  }
  // VEC: gamma of group j of thread t is float4 number (j E / 4 + i) T + t, i < E / 4.
  for (int i = tid; i < NG * E * T; i += RING_THREADS) {
    const int at = i >> 2, who = at % T, piece = at / T;
    const int c = VEC ? ((piece * 4 / E) * T + who) * E + (piece * 4) % E + (i & 3) : i;
    float g = 1.0f;
    if (P.gamma && c < cols)
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
  auto x_row = [&](int i) { return (const unsigned char*)P.x + (blockIdx.x + (int64_t)i * gridDim.x) * P.ldx * ESZ; };
  auto c_row = [&](int i) { return (const unsigned char*)P.ct + (blockIdx.x + (int64_t)i * gridDim.x) * P.ldc * ESZ; };
  // A row's bytes past the last 16-byte boundary before it.
  auto skew = [](const unsigned char* row) { return VEC ? 0 : (int)((uintptr_t)row & 15u); };
  // The team's first thread copies local row i into its slot s.
  auto fetch = [&](int i, int s) {
    if (t != 0 || i >= n_local || dead || (drop >= 0 && i >= drop)) return;
    unsigned char* at = ring + (size_t)s * slot_bytes;
    const unsigned char* from[2] = {x_row(i), c_row(i)};
    uint32_t lo[2] = {0, 0}, hi[2];                  // of the blocks' bytes, those copied
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t r = blockIdx.x + (int64_t)i * gridDim.x;
      const int off = skew(from[q]), end = off + cols * ESZ;
      hi[q] = (uint32_t)(end + 15) & ~15u;
      if constexpr (!VEC) {
        unsigned char* o = at + q * Q.row_bytes;
        const unsigned char* base = from[q] - off;
        auto keep = [&](int b) {
          if (ESZ == 2) *(uint16_t*)(o + b) = *(const uint16_t*)(base + b);
          else *(uint32_t*)(o + b) = *(const uint32_t*)(base + b);
        };
        if (r == 0 && off != 0) {
          lo[q] = 16;
          for (int b = off; b < 16; b += ESZ) keep(b);
        }
        if (r == P.rows - 1 && (end & 15) != 0) {
          hi[q] = (uint32_t)end & ~15u;
          for (int b = (int)hi[q]; b < end; b += ESZ) keep(b);
        }
        from[q] = base;
      }
    }
    mbar_arrive_expect_tx(&full[s], hi[0] - lo[0] + hi[1] - lo[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      bulk_copy_g2s(at + q * Q.row_bytes + lo[q], from[q] + lo[q], hi[q] - lo[q], &full[s]);
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
      if (nw > 1 && lane == 0) red[flip][q][warp] = v[q];
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
  // The row's widened values stay in registers for dx where RMSNorm has one pass
  // before it, and in narrow threads of unaligned rows.
  constexpr bool KEEP = !LAYER || (!VEC && NV == 2);
  // Whether the thread (VEC) or the team has nothing of a group; whether every
  // thread has all of it; if not, whether the thread lacks its element k.
  auto no_group = [&](int j) { return VEC ? j * T + t >= groups : j * E * T >= cols; };
  auto whole = [&](int j) { return VEC || (j + 1) * E * T <= cols; };
  auto absent = [&](int j, int k) { return !VEC && (j * E + k) * T + t >= cols; };
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
    const unsigned char* slot = ring + (size_t)s * slot_bytes;
    const unsigned char *xs = slot + skew(x_row(i)), *cs = slot + Q.row_bytes + skew(c_row(i));
    auto element = [&](const unsigned char* p) {
      return ESZ == 2 ? bf16_bits_to_f32(*(const uint16_t*)p) : *(const float*)p;
    };
    // Group j of x or ct, widened; columns past the row's end are 0.
    auto values = [&](const unsigned char* p, int j, f2* v) {
      if constexpr (VEC) {
        const uint4 u = *(const uint4*)(p + (size_t)(j * T + t) * 16);
        if constexpr (TY == PSK_BF16) {
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = f2{__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)};
        } else {
          v[0] = f2{__uint_as_float(u.x), __uint_as_float(u.y)}, v[1] = f2{__uint_as_float(u.z), __uint_as_float(u.w)};
        }
      } else {
        const unsigned char* q = p + (j * E * T + t) * ESZ;
        if (whole(j)) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) v[k] = f2{element(q + 2 * k * T * ESZ), element(q + (2 * k + 1) * T * ESZ)};
        } else {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) {
            v[k].x = absent(j, 2 * k) ? 0.0f : element(q + 2 * k * T * ESZ);
            v[k].y = absent(j, 2 * k + 1) ? 0.0f : element(q + (2 * k + 1) * T * ESZ);
          }
        }
      }
    };
    auto gate = [&](int j, f2* g) {
      if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
          const float4 a = ((const float4*)gamma)[(j * (E / 4) + q) * T + t];
          g[2 * q] = f2_mul(g[2 * q], f2{a.x, a.y}), g[2 * q + 1] = f2_mul(g[2 * q + 1], f2{a.z, a.w});
        }
      } else {
        const float* q = gamma + j * E * T + t;
#pragma unroll
        for (int k = 0; k < E / 2; ++k) g[k] = f2_mul(g[k], f2{q[2 * k * T], q[(2 * k + 1) * T]});
      }
    };
    f2 kx[KEEP ? NG : 1][E / 2], kc[KEEP ? NG : 1][E / 2];    // KEEP: the row's (centred) x and ct
    float sums[3];
    float mu = 0.0f;
    if (LAYER) {
      f2 a = zero;
      if (!dead) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          if (no_group(j)) continue;
          f2 x[E / 2];
          values(xs, j, x);
#pragma unroll
          for (int k = 0; k < E / 2; ++k) {
            a = f2_add(a, x[k]);
            if (KEEP) kx[KEEP ? j : 0][k] = x[k];
          }
        }
      }
      sums[0] = a.x + a.y;
      team_sum(sums, 1);
      if (nw == 1) __syncwarp();
      if (i != team) fetch(i - TEAMS + slots, before);
      mu = sums[0] * P.inv_cols;
    }
    const f2 nmu = f2_splat(-mu);
    // x - mu, 0 past the row's end.
    auto centre = [&](int j, f2* x) {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        x[k] = f2_add(x[k], nmu);
      }
      if (!whole(j)) {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          if (absent(j, 2 * k)) x[k].x = 0.0f;
          if (absent(j, 2 * k + 1)) x[k].y = 0.0f;
        }
      }
    };
    f2 a = zero, b = zero, d = zero;
    if (!dead) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (no_group(j)) continue;
        f2 x[E / 2], g[E / 2];
        if (KEEP && LAYER) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) x[k] = kx[KEEP ? j : 0][k];
        } else {
          values(xs, j, x);
        }
        values(cs, j, g);
        if (LAYER) centre(j, x);
        if (KEEP) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) kx[KEEP ? j : 0][k] = x[k], kc[KEEP ? j : 0][k] = g[k];
        }
        gate(j, g);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          if (LAYER) d = f2_add(d, g[k]);
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
        if (no_group(j)) continue;
        f2 x[E / 2], c[E / 2], g[E / 2], y[E / 2];
        if (KEEP) {
#pragma unroll
          for (int k = 0; k < E / 2; ++k) x[k] = kx[KEEP ? j : 0][k], c[k] = kc[KEEP ? j : 0][k];
        } else {
          values(xs, j, x);
          values(cs, j, c);
          if (LAYER) centre(j, x);
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) g[k] = c[k];
        gate(j, g);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          const f2 xh = f2_mul(x[k], rd2);
          dg[j][k] = f2_fma(c[k], xh, dg[j][k]);
          if (LAYER) db[j][k] = f2_add(db[j][k], c[k]);
          y[k] = f2_mul(f2_fma(xh, m2, LAYER ? f2_add(g[k], nmg) : g[k]), rd2);
        }
        if constexpr (VEC) {
          unsigned char* o = (unsigned char*)P.dx + r * P.ldd * ESZ + (size_t)(j * T + t) * 16;
          if constexpr (TY == PSK_BF16)
            *(uint4*)o = make_uint4(f32x2_to_bf16x2(y[0].x, y[0].y), f32x2_to_bf16x2(y[1].x, y[1].y),
                                    f32x2_to_bf16x2(y[2].x, y[2].y), f32x2_to_bf16x2(y[3].x, y[3].y));
          else
            *(float4*)o = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
        } else {
          unsigned char* o = (unsigned char*)P.dx + (r * P.ldd + j * E * T + t) * ESZ;
          auto put = [&](int k) {
            const float e = k & 1 ? y[k / 2].y : y[k / 2].x;
            if constexpr (TY == PSK_BF16) *(uint16_t*)(o + k * T * ESZ) = f32_to_bf16_bits(e);
            else *(float*)(o + k * T * ESZ) = e;
          };
          if (whole(j)) {
#pragma unroll
            for (int k = 0; k < E; ++k) put(k);
          } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
              if (!absent(j, k)) put(k);
          }
        }
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
  // The CTA's column sums: the teams' side by side in the ring, now free (its two
  // rows a team are at least as large), then
  // added in order, four (VEC) neighbouring columns or one a thread.
  constexpr int WIDE = NG * E * T;
  float* side = (float*)ring;
#pragma unroll
  for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
    float* part = P.part + ((int64_t)which * P.blocks + blockIdx.x) * P.pcols;
    named_barrier(15, RING_THREADS);
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int k = 0; k < E / 2; k += 2) {
        const f2 a = which == 0 ? dg[j][k] : db[LAYER ? j : 0][k];
        const f2 b = which == 0 ? dg[j][k + 1] : db[LAYER ? j : 0][k + 1];
        if constexpr (VEC) {
          ((float4*)side)[(team * WIDE) / 4 + (j * (E / 4) + k / 2) * T + t] = make_float4(a.x, a.y, b.x, b.y);
        } else {
          const int c = (j * E + 2 * k) * T + t;
          float* at = side + team * cols + c;
          if (c < cols) at[0] = a.x;
          if (c + T < cols) at[T] = a.y;
          if (c + 2 * T < cols) at[2 * T] = b.x;
          if (c + 3 * T < cols) at[3 * T] = b.y;
        }
      }
    named_barrier(15, RING_THREADS);
    if constexpr (VEC) {
      for (int q = tid; q < WIDE / 4; q += RING_THREADS) {
        const int c = ((q / T * 4 / E) * T + q % T) * E + (q / T * 4) % E;
        if (c >= cols) continue;
        float4 s = ((const float4*)side)[q];
#pragma unroll
        for (int m = 1; m < TEAMS; ++m) {
          const float4 u = ((const float4*)side)[m * (WIDE / 4) + q];
          s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
        }
        *(float4*)(part + c) = s;
      }
    } else {
      for (int c = tid; c < cols; c += RING_THREADS) {
        float s = side[c];
#pragma unroll
        for (int m = 1; m < TEAMS; ++m) s += side[m * cols + c];
        part[c] = s;
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
  int64_t b = (NOMINAL_SMS * 8 + slices - 1) / slices;
  if (b > (rows + 15) / 16) b = (rows + 15) / 16;
  return (int)(b < 1 ? 1 : b > NB_MAX_BLOCKS ? NB_MAX_BLOCKS : b);
}

// CTAs of the warp-a-row kernel: three an SM on 160 SMs at most, at least
// NB_ROWS_PER_WARP rows a warp.
static int warps_blocks(int64_t rows) {
  const int64_t want = (rows + NB_WARPS * NB_ROWS_PER_WARP - 1) / (NB_WARPS * NB_ROWS_PER_WARP);
  return (int)(want < 480 ? want : 480);
}

// The ring kernel's shape for rows of this size, or false: teams of the fewest
// threads that hold a row's column sums in four groups of eight (two for rows
// of up to 512 columns, and where four leave no two rows a team: f32 rows) --
// wide threads share a row's shuffles and barrier among more columns, and
// small teams overlap more rows.
static bool ring_shape(NormRingParams& Q, int* nv, int32_t dt, int32_t kind, bool vec, int64_t cols) {
  if (cols <= NB_FUSED_COLS || cols > RING_MAX_COLS) return false;
  const int64_t bytes = cols * dtype_size(dt);      // of a row, not vec: up to 14 before it in its first block
  Q.row_bytes = (int32_t)((bytes + (vec ? 0 : 14) + 15) / 16 * 16);
  for (*nv = cols > 512 ? 4 : 2; *nv >= 2; *nv -= 2) {
    Q.team = 32;
    while (Q.team * *nv * 8 < cols) Q.team *= 2;
    if (Q.team > RING_THREADS) return false;
    Q.teams = RING_THREADS / Q.team;
    int fits = (RING_SMEM - *nv * 8 * Q.team * 4) / (2 * Q.row_bytes);
    if (fits > RING_MAX_SLOTS) fits = RING_MAX_SLOTS;
    // RMSNorm is held to about 128 KB in flight: more reads ahead cost it DRAM
    // time (measured at [32768, 4096] bf16: 133 us with 128 KB, 146 with 192);
    // LayerNorm's two barriers want all there is (134 us with 192 KB, 141 with 128).
    if (kind == PSK_NORM_RMS) {
      const int enough = (128 * 1024) / (2 * Q.row_bytes), least = (Q.teams <= 2 ? 3 : 2) * Q.teams;
      if (fits > enough && fits > least) fits = enough > least ? enough : least;
    }
    Q.slots = fits / Q.teams * Q.teams;
    if (Q.slots >= 2 * Q.teams) return true;
  }
  return false;
}

static uint64_t norm_bwd_layout(int64_t rows, int64_t cols, uint64_t* part) {
  const uint64_t stats = ((uint64_t)rows * 16 + 255) / 256 * 256;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  *part = stats;
  int blocks = norm_bwd_blocks(rows, cols);
  if (cols <= NB_FUSED_COLS && warps_blocks(rows) > blocks) blocks = warps_blocks(rows);
  const int64_t ring = rows < RING_MAX_BLOCKS ? rows : RING_MAX_BLOCKS;
  if (cols > NB_FUSED_COLS && ring > blocks) blocks = (int)ring;
  return stats + 2ull * blocks * pcols * 4;
}

template <int TY, int KIND, int NV, int T, bool VEC>
static int ring_launch_team(const NormRingParams& Q, cudaStream_t s) {
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)norm_bwd_ring_kernel<TY, KIND, NV, T, VEC>, RING_SMEM, limit);
  const size_t smem = (size_t)NV * 8 * T * 4 + (size_t)Q.slots * 2 * Q.row_bytes;
  norm_bwd_ring_kernel<TY, KIND, NV, T, VEC><<<(unsigned)Q.B.blocks, RING_THREADS, smem, s>>>(Q);
  return check_launch("norm backward ring kernel");
}

template <int TY, int KIND, int NV, bool VEC>
static int ring_launch_shape(const NormRingParams& Q, cudaStream_t s) {
  switch (Q.team) {
    case 32: return ring_launch_team<TY, KIND, NV, 32, VEC>(Q, s);
    case 64: return ring_launch_team<TY, KIND, NV, 64, VEC>(Q, s);
    case 128: return ring_launch_team<TY, KIND, NV, 128, VEC>(Q, s);
    case 256: return ring_launch_team<TY, KIND, NV, 256, VEC>(Q, s);
    default: return ring_launch_team<TY, KIND, NV, 512, VEC>(Q, s);
  }
}

template <int TY, int KIND>
static int ring_launch(const NormRingParams& Q, int nv, bool vec, cudaStream_t s) {
  if (!vec) return nv == 2 ? ring_launch_shape<TY, KIND, 2, false>(Q, s) : ring_launch_shape<TY, KIND, 4, false>(Q, s);
  if (nv == 4) return ring_launch_shape<TY, KIND, 4, true>(Q, s);
  if constexpr (TY == PSK_F32) return ring_launch_shape<TY, KIND, 2, true>(Q, s);
  else return ring_launch_team<TY, KIND, 2, 32, true>(Q, s);
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
  const bool one_type = xt == ct_t && xt == dxt;
  if (one_type && ring_shape(G, &nv, xt, kind, vec, cols)) {
    G.B = P;
    const int64_t blocks = (rows + G.teams - 1) / G.teams;
    const int64_t sms = device_sm_count() < RING_MAX_BLOCKS ? device_sm_count() : RING_MAX_BLOCKS;
    G.B.blocks = (int)(blocks < sms ? blocks : sms);
    rc = with_dtype(xt, [&](auto TY) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        return ring_launch<TY.value, LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS>(G, nv, vec, s);
      });
    });
    return rc || (!dgamma && !dbeta) ? rc : norm_bwd_join(G.B, s);
  }
  if (one_type && cols <= NB_FUSED_COLS) {
    P.blocks = warps_blocks(rows);
    // As many CTAs as an SM holds at once by their registers: three of RMSNorm in
    // bf16 (65536 x 200: 27 us, four 34), else two (LayerNorm 65536 x 199 bf16: 34
    // us, four 40; three 38 with registers for them).
    const int per_sm = kind == PSK_NORM_RMS && xt == PSK_BF16 ? 3 : 2;
    if (P.blocks > per_sm * device_sm_count()) P.blocks = per_sm * device_sm_count();
    with_dtype(xt, [&](auto TY) {
      return with_bool(kind == PSK_NORM_LAYER, [&](auto LAYER) {
        return with_bool(vec, [&](auto VEC) {
          norm_bwd_warps_kernel<TY.value, LAYER.value ? PSK_NORM_LAYER : PSK_NORM_RMS, VEC.value>
              <<<(unsigned)P.blocks, NB_THREADS, 0, s>>>(P);
          return 0;
        });
      });
    });
    rc = check_launch("norm backward warp-a-row kernel");
    return rc || (!dgamma && !dbeta) ? rc : norm_bwd_join(P, s);
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
