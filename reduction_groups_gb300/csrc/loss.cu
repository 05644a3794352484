// Log-probabilities of given tokens and the clipped policy loss over rows of
// vocabulary logits, with the loss's gradient.  Per row, z = scale * x:
//   logp  = z_t - log sum_j exp(z_j)                       (t: the row's token)
//   ratio = exp(logp - old), term = -min(ratio A, clamp(ratio, 1 - lo, 1 + hi) A)
//   k     = e^q - q - 1, q = ref - logp                    (a KL estimate >= 0)
//   loss  = sum w (term + beta k)
//   dx_j  = scale w (dterm/dlogp - beta (e^q - 1)) ([j = t] - softmax_j)
// Sums of 2^(c (x - m)) about a running maximum m (c = scale log2 e; the
// maximum's own term is exactly 1), rescaled when the maximum grows: plain f32
// within a thread, joined across threads in pairs of floats (sum and rounding
// error).  So logp, and 1 - p of a nearly certain token, carry an absolute error
// of a few 2^-24; keeping more within a thread too would cost every step of
// sixteen logits its issue slots for digits that only the target's own entry has.
// logp is formed with its rounding error (a pair of floats, or 64 bits where
// f32 overflows and for long rows), and the loss's ratio and KL term from it in
// 64 bits with an exp of extra digits (exp_tier1_core), since their sum over
// rows cancels.  The gradient, whose entries do not, takes both in f32 in the
// resident kernel; within their rounding of a clip bound its case may differ
// from the loss's.
#include "vec8.cuh"
#include "crmath.cuh"
#include "pair.cuh"
#include "pipe.cuh"
#include "trainops.h"

namespace psk {

constexpr int LOSS_THREADS = 256;
constexpr int LOSS_WARPS = LOSS_THREADS / 32;
constexpr int LOSS_MAX_CTAS = 4096;

enum : int { LOSS_LOGP = 0, LOSS_VALUE = 1, LOSS_GRAD = 2 };

struct LossParams {
  const void* x;
  int64_t rows, cols, ldx, ldg;
  const void* targets;
  int32_t targets64;
  float scale;            // z = scale x
  float c;                // RN(scale log2 e): exp(scale t) = 2^(c t)
  const float* old_logp;
  const float* ref_logp;  // NULL: no KL term
  const float* adv;
  const float* weight;    // NULL: 1 / rows
  float uniform;          // RN(1 / rows)
  float low, high;        // 1 - lo, 1 + hi
  float beta;
  float* loss;            // loss, KL sum
  float* logp;            // may be NULL with a loss
  void* grad;
  double* part;           // per CTA: its rows' loss and KL sums
};

// 2^t by the multifunction unit (relative error below 2^-22, results below
// 2^-126 flushed to zero).
__device__ __forceinline__ float ex2_approx(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A partial sum relative to a maximum: sum 2^(c (x - m)) as s + e.
struct RowSum {
  float m, s, e;
};

__device__ __forceinline__ RowSum join(const RowSum& a, const RowSum& b, float c) {
  RowSum r;
  r.m = max_nan2(a.m, b.m);
  // Equal maxima (infinite ones too) scale by one; a NaN maximum gives NaN.
  const float fa = a.m == r.m ? 1.0f : ex2_approx((a.m - r.m) * c);
  const float fb = b.m == r.m ? 1.0f : ex2_approx((b.m - r.m) * c);
  float err;
  two_sum(a.s * fa, b.s * fb, r.s, err);
  r.e = err + (a.e * fa + b.e * fb);
  return r;
}

// Join the sums of aligned groups of `lanes` lanes (a power of two): the
// maximum first, one rescaling, then the sums with their rounding errors.
__device__ __forceinline__ RowSum lanes_join(RowSum v, float c, int lanes) {
  float m = v.m;
  for (int o = lanes >> 1; o > 0; o >>= 1) m = max_nan2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float f = v.m == m ? 1.0f : ex2_approx((v.m - m) * c);   // a NaN maximum gives NaN
  float s = v.s * f, e = v.e * f;
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    float err;
    two_sum(s, __shfl_xor_sync(0xFFFFFFFFu, s, o), s, err);
    e = (e + __shfl_xor_sync(0xFFFFFFFFu, e, o)) + err;
  }
  return RowSum{m, s, e};
}

__device__ __forceinline__ RowSum block_join(RowSum v, float c, RowSum* red) {
  v = lanes_join(v, c, 32);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  RowSum r = red[0];
#pragma unroll
  for (int w = 1; w < LOSS_WARPS; ++w) r = join(r, red[w], c);
  return r;
}

// Add eight logits (n of them) to a running sum.
__device__ __forceinline__ void add8(RowSum& v, const float* x, int n, float c) {
  float m = n > 0 ? x[0] : -INFINITY;
#pragma unroll
  for (int k = 1; k < 8; ++k)
    if (k < n) m = max_nan2(m, x[k]);
  if (!(m <= v.m)) {             // grows, or NaN
    const float f = ex2_approx((v.m - m) * c);
    v.s = v.s == 0.0f ? 0.0f : v.s * f;
    v.m = max_nan2(v.m, m);
  }
  if (v.m == -INFINITY) return;  // nothing but -inf so far
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) t += ex2_approx((x[k] - v.m) * c);
  v.s += t;
}

// e^q - q - 1 >= 0: its series where the difference would cancel.
__device__ __forceinline__ double kl_term(double q, double em1) {
  const float f = (float)q;
  if (em1 == INFINITY) return em1;
  if (!(fabsf(f) < 0.25f)) return em1 - q;
  float h = 1.0f / 362880.0f;    // sum q^(n-2) / n!, n = 2..9 (the next below 2^-36)
  h = fmaf(h, f, 1.0f / 40320.0f);
  h = fmaf(h, f, 1.0f / 5040.0f);
  h = fmaf(h, f, 1.0f / 720.0f);
  h = fmaf(h, f, 1.0f / 120.0f);
  h = fmaf(h, f, 1.0f / 24.0f);
  h = fmaf(h, f, 1.0f / 6.0f);
  h = fmaf(h, f, 0.5f);
  return q * q * (double)h;
}

// What a row's logp leads to.
struct RowLoss {
  double term, k;     // loss terms
  float d;            // d(term + beta k) / dlogp
};

// e^v to a relative error below 2^-40 for |v| <= 87: tier 1 of the correctly
// rounded exp, before its rounding, at v's f32 part, times 1 + the rest.
__device__ __forceinline__ double exp_wide(double v) {
  const float hi = (float)v;
  if (!(fabsf(hi) <= 87.0f)) return (double)expf(hi);
  const float lo = (float)(v - (double)hi);
  float R, d;
  int n;
  exp_tier1_core(hi, psk_exp_tab2, R, d, n);
  return ((double)R + (double)fmaf(R, lo, d)) * __hiloint2double((1023 + n) << 20, 0);
}

__device__ __forceinline__ double row_logp(float xt, const RowSum& v, float scale) {
  float R, d;
  if (!(v.s < INFINITY) || !(v.m < INFINITY) || v.m == -INFINITY) return (double)(v.s + (v.m - v.m));   // NaN
  log_tier1_core(v.s, 0, psk_log_tab, R, d);            // s >= 1: the maximum's own term
  return (double)scale * ((double)xt - (double)v.m) - ((double)R + (double)(d + v.e / v.s));
}

__device__ __forceinline__ RowLoss row_loss(const LossParams& P, double logp, float old, float ref, float adv) {
  RowLoss o;
  const double ratio = exp_wide(logp - (double)old), a = (double)adv;
  const double low = (double)P.low, high = (double)P.high;
  const double bound = ratio < low ? low : ratio > high ? high : ratio;
  // A zero advantage gives zero terms even where the ratio overflows.
  const double free_term = adv == 0.0f && ratio == ratio ? 0.0 : ratio * a, bound_term = bound * a;
  const bool clipped = bound_term < free_term;
  o.term = -(clipped ? bound_term : free_term);
  o.d = clipped ? 0.0f : -(float)free_term;
  o.k = 0.0;
  if (P.ref_logp) {
    const double q = (double)ref - logp;
    const double em1 = exp_wide(q) - 1.0;
    o.k = kl_term(q, em1);
    if (P.beta != 0.0f) o.d = fmaf(-P.beta, (float)em1, o.d);
  }
  return o;
}

// A row's logp as hi + lo (|lo| below half a step of hi), by error-free
// transforms; tab: the log table (or its copy in shared memory).
__device__ __forceinline__ void row_logp_pair(float xt, const RowSum& v, float scale, const float* tab, float& hi,
                                              float& lo) {
  lo = 0.0f;
  hi = v.s + (v.m - v.m);                               // NaN unless the sums are finite
  if (!(v.s < INFINITY) || !(fabsf(v.m) < INFINITY)) return;
  hi = xt;
  if (xt == -INFINITY) return;
  float R, d, th, tl, ph, pl;
  log_tier1_core(v.s, 0, tab, R, d);                    // s >= 1: the maximum's own term
  two_sum(xt, -v.m, th, tl);
  two_prod(scale, th, ph, pl);
  if (!(fabsf(ph) < INFINITY)) {                        // x_t - m or its product passes f32, whose error terms mean nothing then
    const double z = (double)scale * ((double)xt - (double)v.m) - ((double)R + (double)d);
    hi = (float)z;
    lo = fabsf(hi) < INFINITY ? (float)(z - (double)hi) : 0.0f;
    return;
  }
  pl = fmaf(scale, tl, pl);
  two_sum(ph, -R, hi, lo);
  lo += pl - (d + __fdividef(v.e, v.s));
  fast_two_sum(hi, lo, hi, lo);
}

// a - b for a pair a = hi + lo.
__device__ __forceinline__ float pair_minus(float hi, float lo, float b) {
  float s, e;
  two_sum(hi, -b, s, e);
  return fabsf(s) < INFINITY ? s + (e + lo) : s;
}

// d(term + beta k) / dlogp in f32 from the ratio and e^q - 1.
__device__ __forceinline__ float row_slope(const LossParams& P, float ratio, float em1, float adv) {
  const float bound = fminf(fmaxf(ratio, P.low), P.high);
  const float free_term = adv == 0.0f && ratio == ratio ? 0.0f : ratio * adv;
  const float d = bound * adv < free_term ? 0.0f : -free_term;
  return P.ref_logp && P.beta != 0.0f ? fmaf(-P.beta, em1, d) : d;
}

__device__ __forceinline__ int64_t row_target(const LossParams& P, int64_t r) {
  return P.targets64 ? ((const int64_t*)P.targets)[r] : (int64_t)((const int32_t*)P.targets)[r];
}

template <int LT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return LT == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
template <int LT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (LT == PSK_BF16) ((uint16_t*)p)[i] = f32_to_bf16_bits(v);
  else ((float*)p)[i] = v;
}

// Any row: a CTA per row, CTAs over rows in turn, the row read from global
// memory for its sums and (from L2) again for its gradient, four groups of
// eight columns a thread in flight (a lane's columns are 32 apart in unaligned
// rows).  Rows that the resident kernel below cannot take: longer than a
// cluster's shared memory, gradients of another type or alignment than the
// logits.  Bound by its loads' latency: [512, 300000] bf16 167 us, 3.7 TB/s (one
// group in flight for the gradient: 466); [4096, 32000] bf16 to f32 173 us, 4.5
// TB/s; unaligned, [4096, 32001], 367 us; 512 threads were slower.
template <int LT, int GT, int MODE, bool VEC>
__global__ void __launch_bounds__(LOSS_THREADS) loss_rows_kernel(const __grid_constant__ LossParams P) {
  __shared__ RowSum red[LOSS_WARPS];
  __shared__ float coef[2];
  const int64_t groups = VEC ? P.cols / 8 : (P.cols + 255) / 256 * 32;
  auto columns = [&](int64_t q) {
    return VEC ? Columns<VEC, 8>(q * 8, 1, 0, P.cols) : Columns<VEC, 8>(q / 32 * 256, 32, (int)(q % 32), P.cols);
  };
  double loss_sum = 0.0, kl_sum = 0.0;
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const int64_t t = row_target(P, r);
    const float w = MODE == LOSS_LOGP ? 1.0f : P.weight ? P.weight[r] : P.uniform;
    const bool live = t >= 0 && t < P.cols && !(w == 0.0f);
    if (!live) {                                        // left out: its logits are not read
      if (threadIdx.x == 0 && P.logp) P.logp[r] = 0.0f;
      if (MODE == LOSS_GRAD) {
        const float z[8] = {};
        for (int64_t q = threadIdx.x; q < groups; q += LOSS_THREADS) columns(q).template store<GT>(P.grad, r * P.ldg, z);
      }
      continue;
    }
    const int64_t xo = r * P.ldx;
    const float xt = load1<LT>(P.x, xo + t);       // read before the row may be overwritten in place
    RowSum v{-INFINITY, 0.0f, 0.0f};
    // Four of the thread's groups, all of their loads in flight.
    auto load4 = [&](int64_t q0, float (&x)[4][8], int (&n)[4]) {
      Piece<LT, VEC, 8> raw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto cols = columns(q0 + j * LOSS_THREADS);
        n[j] = cols.present;
        cols.load(P.x, xo, raw[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] = raw[j].get(k);
    };
    for (int64_t q0 = threadIdx.x; q0 < groups; q0 += 4 * LOSS_THREADS) {
      float x[4][8];
      int n[4];
      load4(q0, x, n);
#pragma unroll
      for (int j = 0; j < 4; ++j) add8(v, x[j], n[j], P.c);
    }
    v = block_join(v, P.c, red);
    if (threadIdx.x == 0) {
      const double logp = row_logp(xt, v, P.scale);
      if (P.logp) P.logp[r] = (float)logp;
      if (MODE != LOSS_LOGP) {
        const RowLoss o = row_loss(P, logp, P.old_logp[r], P.ref_logp ? P.ref_logp[r] : 0.0f, P.adv[r]);
        if (MODE == LOSS_GRAD) {
          const float a = w * o.d * P.scale;
          coef[0] = -a / v.s;                           // times 2^(c (x - m)): -a softmax
          coef[1] = a * -expm1f((float)logp);           // a (1 - softmax_t)
        }
        loss_sum += (double)w * (o.term + (P.beta != 0.0f ? (double)P.beta * o.k : 0.0));
        kl_sum += (double)w * o.k;
      }
    }
    __syncthreads();
    if (MODE == LOSS_GRAD) {
      const float f = coef[0], ft = coef[1];
      for (int64_t q0 = threadIdx.x; q0 < groups; q0 += 4 * LOSS_THREADS) {
        float x[4][8];
        int n[4];
        load4(q0, x, n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const auto cols = columns(q0 + j * LOSS_THREADS);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            x[j][k] = (VEC ? cols.first + k : cols.col(k)) == t ? ft : ex2_approx((x[j][k] - v.m) * P.c) * f;
          cols.template store<GT>(P.grad, r * P.ldg, x[j]);
        }
      }
    }
  }
  if (MODE != LOSS_LOGP && threadIdx.x == 0) {
    P.part[2 * blockIdx.x] = loss_sum;
    P.part[2 * blockIdx.x + 1] = kl_sum;
  }
}

// ------------------------------------------------------ the resident kernel
//
// A row is read from memory once: its body (the 16-byte groups between an
// unaligned head and tail of a few elements) is copied by TMA into shared
// memory, a row slice per CTA of a cluster (one CTA where the row fits, up to
// eight for rows of up to 8 x 72 KB or to spread a call of few rows), and
// stays there for the sums and for the gradient, which goes straight to
// memory: the floor of one read and one write per logit.  Teams of warps take
// rows in turn, each with slots of its own, so that one team's barriers and
// scalar section (logarithm, ratio, KL term) overlap another's exponentials.
// A slot is filled and freed in up to four chunks: the sums begin with the
// first chunk, and the next row's copy with the first chunk whose gradient is
// written.  A team's warps fetch the scalars of its next 32 rows at once.  A
// producer warp, a lane for each chunk of each slot, refills them as they fall
// free.  The CTAs of a cluster exchange their slices' maxima and sums through
// distributed shared memory.
//
// With gradient: [8192, 32000] bf16, an eighth of the rows left out, 983 MB: 169
// us, 5.8 TB/s; the same in f32, [4096, 32000]: 187 us, 5.6 TB/s; [2048, 131072]
// bf16, clusters of four (36 of them fit: 144 SMs work): 197 us, 5.3 TB/s;
// [8192, 9001] bf16, rows beginning anywhere: 74 us, 4.0 TB/s.  Without: [4096,
// 32000] bf16 48 us, 5.4 TB/s; [2048, 131072] 121 us, 4.4 TB/s.  HBM is about
// two thirds busy: the rest is the joins' and barriers' latency, which three
// teams of 256 threads do not all hide (two ex2 a logit alone would take about
// 50 of the 169 us).

constexpr int RES_CONSUMERS = 768;             // at most: teams of 32 to 512 threads
constexpr int RES_THREADS = RES_CONSUMERS + 32;
constexpr int RES_MAX_TEAMS = 24;
constexpr int RES_MAX_SLOTS = 32;
constexpr int RES_MAX_CHUNKS = 4;
constexpr int RES_ROWS_AHEAD = 3;              // slots of a team at most: rows a warp may be ahead of another
constexpr int RES_MAX_BARS = 32;               // slots x chunks
constexpr int RES_MAX_CLUSTER = 8;
constexpr int RES_SMEM = 210 * 1024;          // ring
constexpr int RES_SLICE = 70 * 1024;          // largest slice: three in the ring

struct ResParams {
  LossParams L;
  int32_t slice_groups;     // 16-byte groups of a CTA's slice (the last may be short)
  int32_t slots, slot_bytes;
  int32_t chunks, chunk_groups;  // of a slot
  int32_t team_threads, teams;   // slots is a multiple of teams: a slot's phases are all one team's, which
                                 // visits them in order (a parity wait must never run ahead of its barrier)
  int32_t cluster;
};

// A row's scalars.
struct RowInfo {
  int32_t target;
  float w, xt, old, ref, adv;
};

struct ResShared {
  uint64_t full[RES_MAX_BARS], empty[RES_MAX_BARS];      // slot x chunks + chunk
  uint64_t xbar[RES_MAX_TEAMS][2];
  uint64_t rbar[RES_MAX_TEAMS][RES_ROWS_AHEAD + 1];      // a row's warp sums are in
  RowSum red[RES_ROWS_AHEAD + 1][RES_CONSUMERS / 32];    // per warp
  uint32_t live[RES_MAX_TEAMS][2];              // which of a team's 32 rows are live, two batches in turn
  RowSum xchg[RES_MAX_TEAMS][2][RES_MAX_CLUSTER];
  float4 coef[RES_MAX_TEAMS];                   // -a / s (times 2^residue), a (1 - p_t), c m or m, the target
  float4 log_tab[512];                          // psk_log_tab: a lookup from L2 would stall every row
  double sums[RES_CONSUMERS / 32][2];           // per warp: its rows' loss and KL sums
  volatile int abort_flag;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait with the cluster's writes acquired.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  do {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
  } while (clock64() - t0 < PIPE_WAIT_CYCLES);
  atomicOr(&g_pipe_status, PIPE_TIMEOUT);
  return false;
}

// Whether the phase with this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Elements of a 16-byte group.
template <int LT>
struct GroupOf {
  static constexpr int N = LT == PSK_BF16 ? 8 : 4;
  static constexpr int PER_STEP = LT == PSK_BF16 ? 2 : 4;     // groups of a step: sixteen elements
};

__device__ __forceinline__ f2 unpack_bf16(uint32_t u) {
  return f2{__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)};
}

// A step's sixteen elements and their maximum; ALL: every group is there, else
// groups from n on are -inf.
template <int LT, bool ALL>
__device__ __forceinline__ void load_step(const unsigned char* s, int i, int n, int stride, f2* x, float& m) {
  if constexpr (LT == PSK_BF16) {
    uint4 u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!ALL) u[q] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
      if (ALL || i + q * stride < n) u[q] = *(const uint4*)(s + (size_t)(i + q * stride) * 16);
    }
    uint32_t h = bf16x2_max(bf16x2_max(bf16x2_max(u[0].x, u[0].y), bf16x2_max(u[0].z, u[0].w)),
                            bf16x2_max(bf16x2_max(u[1].x, u[1].y), bf16x2_max(u[1].z, u[1].w)));
    const f2 e = unpack_bf16(h);
    m = max_nan2(e.x, e.y);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      x[4 * q] = unpack_bf16(u[q].x), x[4 * q + 1] = unpack_bf16(u[q].y);
      x[4 * q + 2] = unpack_bf16(u[q].z), x[4 * q + 3] = unpack_bf16(u[q].w);
    }
  } else {
    m = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (ALL || i + q * stride < n) v = *(const float4*)(s + (size_t)(i + q * stride) * 16);
      x[2 * q] = f2{v.x, v.y}, x[2 * q + 1] = f2{v.z, v.w};
      m = max_nan2(m, max_nan2(max_nan2(v.x, v.y), max_nan2(v.z, v.w)));
    }
  }
}

// A step into the running maximum and sum.
template <int LT, bool ALL>
__device__ __forceinline__ void add_step(const unsigned char* s, int i, int n, int stride, float c, float& max, f2& sum) {
  f2 e[8];
  float m;
  load_step<LT, ALL>(s, i, n, stride, e, m);
  if (!(m <= max)) {                       // grows, or NaN
    m = max_nan2(m, max);
    const float f = ex2_approx((max - m) * c);
    sum.x *= f, sum.y *= f;
    max = m;
  }
  const f2 nm = f2_splat(max == -INFINITY ? 0.0f : -max);
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q] = f2_mul(f2_add(e[q], nm), f2_splat(c));
#pragma unroll
  for (int q = 0; q < 8; ++q) e[q].x = ex2_approx(e[q].x), e[q].y = ex2_approx(e[q].y);
#pragma unroll
  for (int q = 0; q < 4; ++q) e[q] = f2_add(e[q], e[q + 4]);
  sum = f2_add(sum, f2_add(f2_add(e[0], e[1]), f2_add(e[2], e[3])));
}

template <int LT, int MODE>
__global__ void __launch_bounds__(RES_THREADS, 1) loss_resident_kernel(const __grid_constant__ ResParams P) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) ResShared S;
  constexpr int G = GroupOf<LT>::N;
  constexpr int ESZ = 16 / G;
  const LossParams& L = P.L;
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t K = (uint32_t)P.cluster;
  const uint32_t rank = K > 1 ? cluster_rank() : 0;
  const int64_t cid = blockIdx.x / K, ncl = gridDim.x / K;
  const int n_local = cid < L.rows ? (int)((L.rows - 1 - cid) / ncl + 1) : 0;
  const int slots = P.slots, chunks = P.chunks, CG = P.chunk_groups, teams = P.teams;
  const int64_t cols = L.cols;
  const uintptr_t base = (uintptr_t)L.x;

  if (tid == 0) {
    for (int i = 0; i < slots * chunks; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], P.team_threads / 32);
    for (int t = 0; t < teams; ++t) {
      mbar_init(&S.xbar[t][0], K), mbar_init(&S.xbar[t][1], K);
      for (int b = 0; b <= RES_ROWS_AHEAD; ++b) mbar_init(&S.rbar[t][b], P.team_threads / 32);
    }
    S.abort_flag = 0;
    fence_barrier_init();
  }
  static_assert(sizeof(psk_log_tab) == sizeof(S.log_tab), "log table size");
  for (int i = tid; i < 512; i += blockDim.x) S.log_tab[i] = ((const float4*)psk_log_tab)[i];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the finishing kernel may be set up

  const int TT = P.team_threads, depth = slots / teams;
  const bool producer = tid >= teams * TT;
  // The producer's lane l fills chunk l % chunks of slot l / chunks.
  const int team = producer ? lane / chunks % teams : tid / TT;
  const int64_t first = (int64_t)rank * P.slice_groups;
  // The team's q-th row.
  auto row_of = [&](int q) { return cid + (int64_t)(team + q * teams) * ncl; };
  // Row r: elements before its first 16-byte boundary, full groups after.
  auto head_of = [&](int64_t r) {
    const int a = (int)(((base + (uintptr_t)(r * L.ldx) * ESZ) & 15u) / ESZ);
    const int64_t h = a ? G - a : 0;
    return (int)(h < cols ? h : cols);
  };
  auto groups_of = [&](int head) {                 // of the CTA's slice
    const int64_t n = (cols - head) / G - first;
    return (int)(n < 0 ? 0 : n < P.slice_groups ? n : P.slice_groups);
  };
  // Which of the team's rows q, .., q + 31 are live (the same in every warp, in
  // every CTA of a cluster); their scalars in the first warp's lanes.
  RowInfo batch{};
  auto live_rows = [&](int q, bool scalars) {
    bool live = false;
    if (team + (q + lane) * teams < n_local) {
      const int64_t r = row_of(q + lane), t = row_target(L, r);
      const float w = MODE == LOSS_LOGP ? 1.0f : L.weight ? L.weight[r] : L.uniform;
      live = t >= 0 && t < cols && !(w == 0.0f);
      if (scalars && live) {
        batch.target = (int32_t)t;
        batch.w = w;
        batch.xt = load1<LT>(L.x, r * L.ldx + t);
        if (MODE != LOSS_LOGP) {
          batch.old = L.old_logp[r], batch.adv = L.adv[r];
          batch.ref = L.ref_logp ? L.ref_logp[r] : 0.0f;
        }
      }
    }
    return __ballot_sync(0xFFFFFFFFu, live);
  };
  const int tt = tid - team * TT, tw = tt >> 5, nw = TT / 32;
  uint32_t live_now = 0;
  // The live rows of the batch that begins at row q, and of the next one for
  // the producer, which issues rows up to `depth` ahead.
  const bool any_warp = MODE != LOSS_GRAD && K == 1;   // takes scalar sections
  auto next_batch = [&](int q) {
    live_now = live_rows(q, any_warp || tw == 0);
    if (tw == 0) {
      const uint32_t next = live_rows(q + 32, false);
      if (lane == 0) S.live[team][(q / 32) & 1] = live_now, S.live[team][(q / 32 + 1) & 1] = next;
    }
  };
  if (!producer) next_batch(0);
  __syncthreads();
  if (K > 1) cluster_barrier();

  if (producer) {
    const long long drop = g_pipe_drop_row;
    const int slot = lane / chunks, h = lane % chunks;
    const bool mine = lane < slots * chunks;
    int q = slot / teams, issued = -1;             // the lane's next and last row
    uint32_t parity = 1;                           // of the slot's last phase; a fresh barrier passes 1
    long long t0 = clock64();
    while (true) {
      const bool pending = mine && team + q * teams < n_local && !(drop >= 0 && team + q * teams >= drop);
      if (!__any_sync(0xFFFFFFFFu, pending) || S.abort_flag) break;
      const bool ready = pending && mbar_test(&S.empty[lane], parity);
      if (ready) {
        const int64_t r = row_of(q);
        const int head = head_of(r);
        const bool live = (S.live[team][(q / 32) & 1] >> (q & 31)) & 1;
        int m = groups_of(head) - h * CG;
        m = !live || m < 0 ? 0 : m < CG ? m : CG;
        mbar_arrive_expect_tx(&S.full[lane], (uint32_t)m * 16u);
        if (m > 0)
          bulk_copy_g2s(ring + (size_t)slot * P.slot_bytes + (size_t)h * CG * 16,
                        (const unsigned char*)L.x + (r * L.ldx + head) * ESZ + (first + (int64_t)h * CG) * 16,
                        (uint32_t)m * 16u, &S.full[lane]);
        issued = q;
        q += depth;
        parity ^= 1;
      }
      if (__any_sync(0xFFFFFFFFu, ready)) {
        t0 = clock64();
      } else if (clock64() - t0 > PIPE_WAIT_CYCLES) {
        if (lane == 0) atomicOr(&g_pipe_status, PIPE_TIMEOUT);
        S.abort_flag = 1;
      } else {
        __nanosleep(64);
      }
    }
    __syncwarp();
    // After a timeout, copies still in flight land before the CTA retires.
    if (S.abort_flag && issued >= 0) mbar_wait(&S.full[lane], (uint32_t)(issued / depth) & 1u);
    __syncwarp();
    if (K > 1) cluster_barrier();
    return;
  }

  // ---------------- teams.  After a timeout (`dead`) a thread skips waits and
  // work but keeps meeting its team's barriers.
  const float c = L.c;
  bool dead = false;
  // The first warp's lane q holds the team's q-th row of 32 until their loss
  // terms are taken together: 64-bit arithmetic costs a warp's instruction
  // slots however few lanes need it.
  double loss_sum = 0.0, kl_sum = 0.0;
  float held_hi = 0.0f, held_lo = 0.0f;
  RowInfo held{};
  int n_held = 0;
  auto take_held = [&]() {
    if (lane < n_held) {
      const RowLoss o = row_loss(L, (double)held_hi + (double)held_lo, held.old, held.ref, held.adv);
      loss_sum += (double)held.w * (o.term + (L.beta != 0.0f ? (double)L.beta * o.k : 0.0));
      kl_sum += (double)held.w * o.k;
    }
    n_held = 0;
  };
  uint32_t exchanges = 0;
  auto team_barrier = [&]() {
    if (TT == 32) __syncwarp();
    else named_barrier(1 + team, TT);
  };
  int s = team;                                    // the row's slot
  uint32_t parity = 0;                             // of its phases
  int64_t r = row_of(0);
  const int64_t r_step = (int64_t)teams * ncl;
  // Where a row begins among 16-byte boundaries: the same for all rows of an
  // aligned leading dimension.
  const bool vary = (L.ldx * ESZ) % 16 != 0;
  int head = 0, n = 0;
  int64_t edge = -1;                               // the thread's element of the row's head or tail
  for (int q = 0; team + q * teams < n_local; ++q, r += r_step) {
    if (q > 0 && (q & 31) == 0) next_batch(q);
    const unsigned char* x = ring + (size_t)s * P.slot_bytes;
    if (vary || q == 0) {
      head = head_of(r);
      n = groups_of(head);
      // One each for the first threads of the first CTA's team.
      const int tail = (int)((cols - head) % G);
      edge = rank != 0 || tt >= 16 ? -1
             : tt < 8 ? (tt < head ? tt : -1)
                      : (tt - 8 < tail ? cols - tail + (tt - 8) : -1);
    }
    const bool live = (live_now >> (q & 31)) & 1;
    dead = dead || S.abort_flag;
    uint64_t* full = &S.full[s * chunks];
    uint64_t* empty = &S.empty[s * chunks];
    const float xe = live && edge >= 0 ? load1<LT>(L.x, r * L.ldx + edge) : -INFINITY;
    auto leave = [&](int h) {                       // the warp is past a chunk
      __syncwarp();
      if (!dead && lane == 0) mbar_arrive(empty + h);
    };

    RowSum v{-INFINITY, 0.0f, 0.0f};
    f2 sum{0.0f, 0.0f};
    for (int h = 0; h < chunks; ++h) {
      if (!dead && !mbar_wait(full + h, parity)) { S.abort_flag = 1; dead = true; }
      if (live && !dead) {
        constexpr int STEP = GroupOf<LT>::PER_STEP;
        const int hi = n < (h + 1) * CG ? n : (h + 1) * CG;
        int i = h * CG + tt;
        for (; i + (STEP - 1) * TT < hi; i += STEP * TT) add_step<LT, true>(x, i, hi, TT, c, v.m, sum);
        if (i < hi) add_step<LT, false>(x, i, hi, TT, c, v.m, sum);
      }
      if (MODE != LOSS_GRAD) leave(h);
    }
    if (live) {
      v.s = __fadd_rn(sum.x, sum.y);
      if (edge >= 0) {
        if (!(xe <= v.m)) {
          const float m = max_nan2(xe, v.m);
          v.s *= ex2_approx((v.m - m) * c);
          v.m = m;
        }
        v.s += v.m == -INFINITY ? 0.0f : ex2_approx((xe - v.m) * c);
      }
      __syncwarp();
      v = lanes_join(v, c, 32);
      if (lane == 0) S.red[q & RES_ROWS_AHEAD][tid >> 5] = v;
    }
    __syncwarp();
    // Without a gradient no warp needs the row's result: each reports its sum
    // and goes on, and the warps take the rows' scalar sections in turn (a warp
    // is at most RES_ROWS_AHEAD rows ahead of the one that reads its sums, since
    // a slot's refill waits for every warp).  In a cluster the first warp
    // keeps them all: the exchange's two buffers rest on its order.
    const bool turns = MODE != LOSS_GRAD && K == 1 && nw > 1;
    const int scalar_warp = turns ? q % nw : 0;
    if (turns) {
      uint64_t* rbar = &S.rbar[team][q & RES_ROWS_AHEAD];
      if (lane == 0) mbar_arrive(rbar);
      if (tw == scalar_warp && !dead && !mbar_wait(rbar, (uint32_t)(q / (RES_ROWS_AHEAD + 1)) & 1u)) {
        S.abort_flag = 1;
        dead = true;
      }
    } else {
      team_barrier();
    }
    if (tw == scalar_warp && live) {
      __syncwarp();
      v = lane < nw ? S.red[q & RES_ROWS_AHEAD][team * nw + lane] : RowSum{-INFINITY, 0.0f, 0.0f};
      if (nw > 1) v = lanes_join(v, c, nw);
      v.m = __shfl_sync(0xFFFFFFFFu, v.m, 0);
      v.s = __shfl_sync(0xFFFFFFFFu, v.s, 0);
      v.e = __shfl_sync(0xFFFFFFFFu, v.e, 0);
      if (K > 1) {
        const uint32_t p = exchanges & 1;
        if ((uint32_t)lane < K) {
          const uint32_t to = peer_addr(&S.xchg[team][p][rank], lane);
          peer_store(to, v.m);
          peer_store(to + 4, v.s);
          peer_store(to + 8, v.e);
          peer_arrive(peer_addr(&S.xbar[team][p], lane));
        }
        // every lane acquires what the peers wrote
        bool ok = dead || mbar_wait_cluster(&S.xbar[team][p], (exchanges >> 1) & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        ++exchanges;
        if (!ok) { S.abort_flag = 1; dead = true; }
        v = (uint32_t)lane < K ? S.xchg[team][p][lane] : RowSum{-INFINITY, 0.0f, 0.0f};
        v = lanes_join(v, c, (int)K);
        v.m = __shfl_sync(0xFFFFFFFFu, v.m, 0);
        v.s = __shfl_sync(0xFFFFFFFFu, v.s, 0);
        v.e = __shfl_sync(0xFFFFFFFFu, v.e, 0);
      }
      RowInfo info;
      const int from = q & 31;
      info.target = __shfl_sync(0xFFFFFFFFu, batch.target, from);
      info.xt = __shfl_sync(0xFFFFFFFFu, batch.xt, from);
      info.w = __shfl_sync(0xFFFFFFFFu, batch.w, from);
      info.old = __shfl_sync(0xFFFFFFFFu, batch.old, from);
      info.ref = __shfl_sync(0xFFFFFFFFu, batch.ref, from);
      info.adv = __shfl_sync(0xFFFFFFFFu, batch.adv, from);
      float hi, lo;
      row_logp_pair(info.xt, v, L.scale, (const float*)S.log_tab, hi, lo);
      if (lane == 0 && !dead && L.logp && rank == 0) L.logp[r] = hi;
      if (MODE == LOSS_GRAD) {
        // Two of the exponentials side by side: lane 1's for the KL term.
        const float d = pair_minus(-hi, -lo, -info.ref);
        const float em = expm1f(lane == 1 ? d : hi);
        const float em_q = __shfl_sync(0xFFFFFFFFu, em, 1);
        const float ratio = expf(pair_minus(hi, lo, info.old));
        const float a = info.w * row_slope(L, ratio, em_q, info.adv) * L.scale;
        // softmax_j = 2^(c x_j - RN(c m)) 2^(RN(c m) - c m) / s in one fma a
        // logit, where the product's rounding error, an exponent here, is at most
        // a half (from 2^31 on it can pass 127); else 2^(c (x_j - m)) / s.
        const float mc = v.m * c;
        const bool near = fabsf(mc) < 0x1p24f;
        const float f = __fdividef(-a, v.s);
        if (lane == 0)
          S.coef[team] = make_float4(near ? f * ex2_approx(fmaf(-v.m, c, mc)) : f, a * -em, near ? mc : v.m,
                                     __int_as_float(near ? info.target : ~info.target));
      }
      if (MODE != LOSS_LOGP && !dead) {
        if (lane == n_held) held_hi = hi, held_lo = lo, held = info;
        if (++n_held == 32) take_held();
      }
      __syncwarp();
    } else if (!live && tt == 0 && !dead && rank == 0 && L.logp) {
      L.logp[r] = 0.0f;                          // a row left out
    }
    if (MODE == LOSS_GRAD) {
      __syncwarp();
      team_barrier();
      unsigned char* g = (unsigned char*)L.grad + (r * L.ldg + head) * ESZ + first * 16;
      const float4 k = S.coef[team];
      const bool near = __float_as_int(k.w) >= 0;
      const int target = near ? __float_as_int(k.w) : ~__float_as_int(k.w);
      const f2 f = f2_splat(k.x), nm = f2_splat(-k.z), cc = f2_splat(c);
      auto grad = [&](auto NEAR, f2 e) {
        e = NEAR.value ? f2_fma(e, cc, nm) : f2_mul(f2_add(e, nm), cc);
        return f2_mul(f2{ex2_approx(e.x), ex2_approx(e.y)}, f);
      };
      auto chunk = [&](auto NEAR, int lo, int hi) {
        for (int i = lo + tt; i < hi; i += TT) {
          const uint4 u = *(const uint4*)(x + (size_t)i * 16);
          if constexpr (LT == PSK_BF16) {
            const f2 a = grad(NEAR, unpack_bf16(u.x)), b = grad(NEAR, unpack_bf16(u.y)),
                     d = grad(NEAR, unpack_bf16(u.z)), e = grad(NEAR, unpack_bf16(u.w));
            *(uint4*)(g + (size_t)i * 16) = make_uint4(f32x2_to_bf16x2(a.x, a.y), f32x2_to_bf16x2(b.x, b.y),
                                                       f32x2_to_bf16x2(d.x, d.y), f32x2_to_bf16x2(e.x, e.y));
          } else {
            const f2 a = grad(NEAR, f2{__uint_as_float(u.x), __uint_as_float(u.y)}),
                     b = grad(NEAR, f2{__uint_as_float(u.z), __uint_as_float(u.w)});
            *(float4*)(g + (size_t)i * 16) = make_float4(a.x, a.y, b.x, b.y);
          }
        }
      };
      for (int h = 0; h < chunks; ++h) {
        const int hi = dead ? 0 : n < (h + 1) * CG ? n : (h + 1) * CG;
        if (!live) {
          for (int i = h * CG + tt; i < hi; i += TT) *(uint4*)(g + (size_t)i * 16) = make_uint4(0, 0, 0, 0);
        } else if (near) {
          chunk(std::true_type{}, h * CG, hi);
        } else {
          chunk(std::false_type{}, h * CG, hi);
        }
        leave(h);
      }
      if (edge >= 0 && !dead) {
        const f2 e = near ? grad(std::true_type{}, f2{xe, xe}) : grad(std::false_type{}, f2{xe, xe});
        store1<LT>(L.grad, r * L.ldg + edge, !live ? 0.0f : edge == target ? k.y : e.x);
      }
      if (live && !dead && target >= head) {
        // The target's own element, over what its thread has just stored.
        const int64_t at = ((int64_t)target - head) / G - first;
        if (at >= 0 && at < n && ((int)at & (TT - 1)) == tt) store1<LT>(L.grad, r * L.ldg + target, k.y);
      }
    }
    s += teams;
    if (s >= slots) s -= slots, parity ^= 1;
  }
  __syncwarp();
  if (MODE != LOSS_LOGP && (any_warp || tw == 0)) {
    take_held();
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      loss_sum += __shfl_xor_sync(0xFFFFFFFFu, loss_sum, o);
      kl_sum += __shfl_xor_sync(0xFFFFFFFFu, kl_sum, o);
    }
    if (any_warp) {                                // the warps' sums in order, by the team's first
      if (lane == 0) S.sums[tid >> 5][0] = loss_sum, S.sums[tid >> 5][1] = kl_sum;
      team_barrier();
      for (int w = 1; tt == 0 && w < nw; ++w) loss_sum += S.sums[team * nw + w][0], kl_sum += S.sums[team * nw + w][1];
    }
    if (tt == 0 && rank == 0) {
      L.part[2 * (cid * teams + team)] = loss_sum;
      L.part[2 * (cid * teams + team) + 1] = kl_sum;
    }
  }
  __syncwarp();
  if (K > 1) cluster_barrier();     // no CTA leaves while a peer may still write to it
}

// The partial sums joined, 256 threads over them in turn for each of the two.
constexpr int FINISH_THREADS = 512;
__global__ void __launch_bounds__(FINISH_THREADS) loss_finish_kernel(const double* part, int n, float* loss) {
  __shared__ double sums[FINISH_THREADS / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int half = FINISH_THREADS / 2, which = threadIdx.x / half, t = threadIdx.x - which * half;
  double s = 0.0;
  for (int i = t; i < n; i += half) s += part[2 * i + which];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (t == 0) {
    const int w0 = which * (half / 32);
    for (int w = 1; w < half / 32; ++w) s += sums[w0 + w];
    loss[which] = (float)s;
  }
}

// Launched so that its set-up overlaps the kernel before it, whose sums it
// waits for.
static int loss_finish(const double* part, int n, float* loss, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(FINISH_THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, loss_finish_kernel, part, n, loss);
  return check_launch("policy loss finishing kernel");
}

static int loss_check_rows(const void* logits, int32_t lt, int64_t rows, int64_t cols, int64_t ldl, double scale,
                           const void* targets, int32_t tt) {
  if (!dtype_ok(lt)) return fail(PSK_E_DTYPE, "logits dtype %d", lt);
  if (tt != PSK_I32 && tt != PSK_I64) return fail(PSK_E_DTYPE, "target dtype %d", tt);
  if (rows < 0 || cols < 0) return fail(PSK_E_SHAPE, "rows %lld, cols %lld", (long long)rows, (long long)cols);
  if (rows > 0x7FFFFFFFll || cols > 0x7FFFFFFFll)
    return fail(PSK_E_SHAPE, "rows %lld or cols %lld above 2^31 - 1", (long long)rows, (long long)cols);
  if (rows > 0 && cols == 0) return fail(PSK_E_SHAPE, "rows of no logits");
  if (!(scale >= 1e-30 && scale <= 1e30)) return fail(PSK_E_ARG, "scale %g is not in [1e-30, 1e30]", scale);
  if (rows == 0) return PSK_OK;
  if (!logits || !targets) return fail(PSK_E_NULL, "logits or targets is NULL");
  if (ldl < cols) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(rows, ldl)) return fail(PSK_E_SHAPE, "rows x leading dimension too large");
  if ((uintptr_t)logits % dtype_size(lt) != 0) return fail(PSK_E_ARG, "logits are not aligned to their type");
  if ((uintptr_t)targets % (tt == PSK_I64 ? 8 : 4) != 0) return fail(PSK_E_ARG, "targets are not aligned to their type");
  return PSK_OK;
}

static LossParams loss_params(const void* logits, int64_t rows, int64_t cols, int64_t ldl, double scale,
                              const void* targets, int32_t tt) {
  LossParams P{};
  P.x = logits, P.rows = rows, P.cols = cols, P.ldx = ldl;
  P.targets = targets, P.targets64 = tt == PSK_I64;
  P.scale = (float)scale;
  P.c = (float)((double)P.scale * 1.4426950408889634074);
  return P;
}

// The resident kernel's shape for rows of this size, or false for rows beyond
// a cluster's shared memory.  The cluster is the smallest whose slices leave
// three in a CTA's ring; a call whose rows leave more than half of the SMs idle
// spreads each over a larger one while slices keep 2048 elements (a row of
// 32000 on one CTA is bound by that SM's copy and exponentials).  Teams take
// up to 128 elements a thread: a row's joins, barriers and scalar section cost
// every warp of its team, and more teams overlap them.
static bool resident_plan(ResParams& P, int32_t lt, int64_t rows, int64_t cols) {
  const int64_t g = lt == PSK_BF16 ? 8 : 4, groups = cols / g, sms = device_sm_count();
  int64_t k = 1;
  auto slice = [&](int64_t k) { return (groups + k - 1) / k; };
  while (k < RES_MAX_CLUSTER && slice(k) * 16 > RES_SLICE) k *= 2;
  if (slice(k) * 16 > RES_SLICE) return false;
  while (k < RES_MAX_CLUSTER && rows * k * 2 <= sms && slice(2 * k) * g >= 2048) k *= 2;
  P.cluster = (int32_t)k;
  P.slice_groups = (int32_t)(slice(k) > 0 ? slice(k) : 1);
  P.slot_bytes = (P.slice_groups * 16 + 127) / 128 * 128;
  const int fits = RES_SMEM / P.slot_bytes < RES_MAX_SLOTS ? RES_SMEM / P.slot_bytes : RES_MAX_SLOTS;
  const int64_t elements = P.slice_groups * g, each = (rows * k + sms - 1) / sms;
  P.team_threads = 32;
  while (P.team_threads < 256 && elements > 128 * P.team_threads) P.team_threads *= 2;
  // Fewer rows a cluster than teams: larger teams, down to 16 elements a thread.
  while (P.team_threads < 256 && RES_CONSUMERS / P.team_threads > each && elements > 16 * P.team_threads)
    P.team_threads *= 2;
  if (each == 1 && elements > 8192) P.team_threads = 512;
  P.teams = RES_CONSUMERS / P.team_threads;
  if (P.teams > fits) P.teams = fits;
  const int depth = fits / P.teams < RES_ROWS_AHEAD ? fits / P.teams : RES_ROWS_AHEAD;
  P.slots = depth * P.teams;
  // Chunks of whole steps (sixteen elements a thread).
  const int step = (int)(16 / g) * P.team_threads, steps = (P.slice_groups + step - 1) / step;
  int most = RES_MAX_BARS / P.slots < RES_MAX_CHUNKS ? RES_MAX_BARS / P.slots : RES_MAX_CHUNKS;
  if (most > steps) most = steps;
  P.chunk_groups = (steps + most - 1) / most * step;
  P.chunks = (P.slice_groups + P.chunk_groups - 1) / P.chunk_groups;
  return true;
}

// Clusters of `k` CTAs that run at once, asked once per device, kernel and size.
template <int LT, int MODE>
static int resident_clusters(int k) {
  static int cache[PSK_MAX_DEVICES][4] = {};
  static bool limit[PSK_MAX_DEVICES] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= PSK_MAX_DEVICES) dev = 0;
  const void* kernel = (const void*)loss_resident_kernel<LT, MODE>;
  smem_limit_once(kernel, RES_SMEM, limit);
  const int i = k == 1 ? 0 : k == 2 ? 1 : k == 4 ? 2 : 3;
  if (cache[dev][i] == 0) {
    int n = 0;
    if (k == 1) {
      n = device_sm_count();
    } else {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = k, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(k);
      cfg.blockDim = dim3(RES_THREADS);
      cfg.dynamicSmemBytes = RES_SMEM;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, loss_resident_kernel<LT, MODE>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 1;
      }
      if (n < 1) n = 1;
    }
    cache[dev][i] = n;
  }
  return cache[dev][i];
}

// Launch the resident kernel; *parts: the partial sums it leaves.
template <int LT, int MODE>
static int resident_launch(ResParams P, const LossParams& L, int* parts, cudaStream_t s) {
  P.L = L;
  int64_t n = resident_clusters<LT, MODE>(P.cluster);
  if (n > L.rows) n = L.rows;
  if (n * P.teams > LOSS_MAX_CTAS) n = LOSS_MAX_CTAS / P.teams;
  *parts = (int)n * P.teams;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = P.cluster, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(n * P.cluster));
  cfg.blockDim = dim3((unsigned)(P.teams * P.team_threads + 32));
  cfg.dynamicSmemBytes = RES_SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, loss_resident_kernel<LT, MODE>, P);
  return check_launch("resident loss kernel");
}

int loss_status(unsigned int* v, bool reset) {
  if (cudaMemcpyFromSymbol(v, g_pipe_status, sizeof(*v)) != cudaSuccess) return check_launch("device status read");
  if (reset) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_pipe_status, &z, sizeof(z)) != cudaSuccess) return check_launch("device status reset");
  }
  return PSK_OK;
}

int loss_set_drop_row(long long row) {
  if (cudaMemcpyToSymbol(g_pipe_drop_row, &row, sizeof(row)) != cudaSuccess) return check_launch("test hook write");
  return PSK_OK;
}

static unsigned loss_grid(int64_t rows) {
  int64_t most = (int64_t)device_sm_count() * 8;
  if (most > LOSS_MAX_CTAS) most = LOSS_MAX_CTAS;
  return (unsigned)(rows < most ? rows : most);
}

}  // namespace psk

using namespace psk;

extern "C" int psk_token_logp(const void* logits, int32_t lt, int64_t rows, int64_t cols, int64_t ldl, double scale,
                              const void* targets, int32_t tt, float* logp, void* stream) {
  clear_error();
  int rc = loss_check_rows(logits, lt, rows, cols, ldl, scale, targets, tt);
  if (rc || rows == 0) return rc;
  if (!logp) return fail(PSK_E_NULL, "logp is NULL");
  if ((uintptr_t)logp % 4 != 0) return fail(PSK_E_ARG, "logp is not 4-byte aligned");
  const uint64_t lb = (uint64_t)rows * 4;
  if (ranges_overlap(logp, lb, logits, rows_bytes(rows, cols, ldl, lt)) ||
      ranges_overlap(logp, lb, targets, (uint64_t)rows * (tt == PSK_I64 ? 8 : 4)))
    return fail(PSK_E_ALIAS, "logp overlaps the logits or the targets");
  LossParams P = loss_params(logits, rows, cols, ldl, scale, targets, tt);
  P.logp = logp;
  ResParams Q{};
  if (resident_plan(Q, lt, rows, cols)) {
    int parts = 0;
    return with_dtype(lt, [&](auto LT) {
      return resident_launch<LT.value, LOSS_LOGP>(Q, P, &parts, (cudaStream_t)stream);
    });
  }
  const bool vec = cols % 8 == 0 && rows_vec8(logits, lt, ldl, rows);
  with_dtype(lt, [&](auto LT) {
    return with_bool(vec, [&](auto VEC) {
      loss_rows_kernel<LT.value, PSK_F32, LOSS_LOGP, VEC.value>
          <<<loss_grid(rows), LOSS_THREADS, 0, (cudaStream_t)stream>>>(P);
      return 0;
    });
  });
  return check_launch("token log-probability kernel");
}

extern "C" int psk_policy_loss_workspace(int64_t rows, int64_t cols, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  if (rows < 0 || cols < 0) return fail(PSK_E_SHAPE, "rows %lld, cols %lld", (long long)rows, (long long)cols);
  *bytes = rows ? 16ull * LOSS_MAX_CTAS : 0;
  return PSK_OK;
}

extern "C" int psk_policy_loss(const void* logits, int32_t lt, int64_t rows, int64_t cols, int64_t ldl, double scale,
                               const void* targets, int32_t tt, const float* old_logp, const float* ref_logp,
                               const float* advantage, const float* weight, double clip_low, double clip_high,
                               double kl_coef, float* loss, float* logp, void* dlogits, int32_t gt, int64_t ldg,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  int rc = loss_check_rows(logits, lt, rows, cols, ldl, scale, targets, tt);
  if (rc) return rc;
  if (dlogits && !dtype_ok(gt)) return fail(PSK_E_DTYPE, "gradient dtype %d", gt);
  if (!(clip_low >= 0.0 && clip_low <= 1.0)) return fail(PSK_E_ARG, "clip_low %g is not in [0, 1]", clip_low);
  if (!(clip_high >= 0.0 && clip_high <= 1e30)) return fail(PSK_E_ARG, "clip_high %g is not in [0, 1e30]", clip_high);
  if (!(kl_coef >= -1e30 && kl_coef <= 1e30)) return fail(PSK_E_ARG, "kl_coef is not finite or above 1e30");
  if (kl_coef != 0.0 && rows > 0 && !ref_logp) return fail(PSK_E_NULL, "ref_logp is NULL with a KL term");
  if (!loss) return fail(PSK_E_NULL, "loss is NULL");
  if ((uintptr_t)loss % 4 != 0 || (uintptr_t)logp % 4 != 0 || (uintptr_t)old_logp % 4 != 0 ||
      (uintptr_t)ref_logp % 4 != 0 || (uintptr_t)advantage % 4 != 0 || (uintptr_t)weight % 4 != 0)
    return fail(PSK_E_ARG, "a vector of floats is not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    return loss_finish(nullptr, 0, loss, s);
  }
  if (!old_logp || !advantage) return fail(PSK_E_NULL, "old_logp or advantage is NULL");
  uint64_t need = 0;
  psk_policy_loss_workspace(rows, cols, &need);
  if (!workspace) return fail(PSK_E_NULL, "workspace is NULL");
  if ((uintptr_t)workspace % 16 != 0) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
  if (workspace_bytes < need)
    return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                (unsigned long long)need);
  const uint64_t xb = rows_bytes(rows, cols, ldl, lt), vb = (uint64_t)rows * 4;
  uint64_t gb = 0;
  if (dlogits) {
    if ((uintptr_t)dlogits % dtype_size(gt) != 0) return fail(PSK_E_ARG, "dlogits is not aligned to its type");
    if (ldg < cols) return fail(PSK_E_SHAPE, "gradient leading dimension below cols");
    if (!rows_addressable(rows, ldg)) return fail(PSK_E_SHAPE, "rows x leading dimension too large");
    gb = rows_bytes(rows, cols, ldg, gt);
    if (ranges_overlap(logits, xb, dlogits, gb) && !(logits == dlogits && lt == gt && ldl == ldg))
      return fail(PSK_E_ALIAS, "dlogits overlaps the logits and is not the same buffer");
  }
  // Each output against every input and every other output.
  struct Span { const void* p; uint64_t n; };
  const Span ins[] = {{targets, (uint64_t)rows * (tt == PSK_I64 ? 8 : 4)}, {old_logp, vb}, {ref_logp, vb},
                      {advantage, vb}, {weight, vb}};
  const Span outs[] = {{loss, 8}, {logp, vb}, {dlogits, gb}, {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i].p) continue;
    for (const Span& in : ins)
      if (in.p && ranges_overlap(outs[i].p, outs[i].n, in.p, in.n))
        return fail(PSK_E_ALIAS, "an output or the workspace overlaps a per-row input");
    if (i != 2 && ranges_overlap(outs[i].p, outs[i].n, logits, xb))
      return fail(PSK_E_ALIAS, "loss, logp or the workspace overlaps the logits");
    for (int j = 0; j < i; ++j)
      if (outs[j].p && ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return fail(PSK_E_ALIAS, "two outputs, or an output and the workspace, overlap");
  }
  LossParams P = loss_params(logits, rows, cols, ldl, scale, targets, tt);
  P.old_logp = old_logp, P.ref_logp = ref_logp, P.adv = advantage, P.weight = weight;
  P.uniform = (float)(1.0 / (double)rows);
  P.low = (float)(1.0 - clip_low), P.high = (float)(1.0 + clip_high);
  P.beta = (float)kl_coef;
  P.loss = loss, P.logp = logp, P.grad = dlogits, P.ldg = ldg;
  P.part = (double*)workspace;
  ResParams Q{};
  // Gradient rows must begin as far from a 16-byte boundary as their logits.
  const bool alike = !dlogits || (lt == gt && ((uintptr_t)logits - (uintptr_t)dlogits) % 16 == 0 &&
                                  (rows == 1 || ((ldl - ldg) * dtype_size(lt)) % 16 == 0));
  if (alike && resident_plan(Q, lt, rows, cols)) {
    int parts = 0;
    rc = with_dtype(lt, [&](auto LT) {
      return dlogits ? resident_launch<LT.value, LOSS_GRAD>(Q, P, &parts, s)
                     : resident_launch<LT.value, LOSS_VALUE>(Q, P, &parts, s);
    });
    return rc ? rc : loss_finish(P.part, parts, loss, s);
  }
  const unsigned grid = loss_grid(rows);
  const bool vec = cols % 8 == 0 && rows_vec8(logits, lt, ldl, rows) && (!dlogits || rows_vec8(dlogits, gt, ldg, rows));
  with_dtype(lt, [&](auto LT) {
    return with_bool(vec, [&](auto VEC) {
      if (!dlogits) {
        loss_rows_kernel<LT.value, PSK_F32, LOSS_VALUE, VEC.value><<<grid, LOSS_THREADS, 0, s>>>(P);
        return 0;
      }
      return with_dtype(gt, [&](auto GT) {
        loss_rows_kernel<LT.value, GT.value, LOSS_GRAD, VEC.value><<<grid, LOSS_THREADS, 0, s>>>(P);
        return 0;
      });
    });
  });
  rc = check_launch("policy loss kernel");
  return rc ? rc : loss_finish(P.part, (int)grid, loss, s);
}
