// Log-probabilities of given tokens and the clipped policy loss over rows of
// vocabulary logits, with the loss's gradient.  Per row, z = scale * x:
//   logp  = z_t - log sum_j exp(z_j)                       (t: the row's token)
//   ratio = exp(logp - old), term = -min(ratio A, clamp(ratio, 1 - lo, 1 + hi) A)
//   k     = e^q - q - 1, q = ref - logp                    (a KL estimate >= 0)
//   loss  = sum w (term + beta k)
//   dx_j  = scale w (dterm/dlogp - beta (e^q - 1)) ([j = t] - softmax_j)
// A row is one pass for its maximum and sum (each thread keeps a running
// maximum and rescales its sum when that grows) and, for the gradient, one
// more over the row, which then comes from L2.  Row sums are joined across
// threads in pairs of floats (sum and rounding error), so that 1 - p of a
// nearly certain token keeps its digits; logp is formed in 64 bits.
#include "vec8.cuh"
#include "crmath.cuh"

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

__device__ __forceinline__ RowSum block_join(RowSum v, float c, RowSum* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    RowSum u;
    u.m = __shfl_xor_sync(0xFFFFFFFFu, v.m, o);
    u.s = __shfl_xor_sync(0xFFFFFFFFu, v.s, o);
    u.e = __shfl_xor_sync(0xFFFFFFFFu, v.e, o);
    v = join(v, u, c);
  }
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
__device__ __forceinline__ float kl_term(float q, float em1) {
  if (em1 == INFINITY) return em1;
  if (!(fabsf(q) < 0.5f)) return em1 - q;
  float h = 1.0f / 3628800.0f;   // sum q^(n-2) / n!, n = 2..10
  h = fmaf(h, q, 1.0f / 362880.0f);
  h = fmaf(h, q, 1.0f / 40320.0f);
  h = fmaf(h, q, 1.0f / 5040.0f);
  h = fmaf(h, q, 1.0f / 720.0f);
  h = fmaf(h, q, 1.0f / 120.0f);
  h = fmaf(h, q, 1.0f / 24.0f);
  h = fmaf(h, q, 1.0f / 6.0f);
  h = fmaf(h, q, 0.5f);
  return q * q * h;
}

// What a row's logp leads to.
struct RowLoss {
  float term, k;      // loss terms
  float d;            // d(term + beta k) / dlogp
};

__device__ __forceinline__ double row_logp(float xt, const RowSum& v, float scale) {
  float R, d;
  if (!(v.s < INFINITY) || !(v.m < INFINITY) || v.m == -INFINITY) return (double)(v.s + (v.m - v.m));   // NaN
  log_tier1_core(v.s, 0, psk_log_tab, R, d);            // s >= 1: the maximum's own term
  return (double)scale * ((double)xt - (double)v.m) - ((double)R + (double)(d + v.e / v.s));
}

__device__ __forceinline__ RowLoss row_loss(const LossParams& P, double logp, float old, float ref, float adv) {
  RowLoss o;
  const float ratio = expf((float)(logp - (double)old));
  const float bound = fminf(fmaxf(ratio, P.low), P.high);
  // A zero advantage gives zero terms even where the ratio overflows.
  const float free_term = adv == 0.0f && ratio == ratio ? 0.0f : ratio * adv, bound_term = bound * adv;
  const bool clipped = bound_term < free_term;
  o.term = -(clipped ? bound_term : free_term);
  o.d = clipped ? 0.0f : -free_term;
  o.k = 0.0f;
  if (P.ref_logp) {
    const float q = (float)((double)ref - logp);
    const float em1 = expm1f(q);
    o.k = kl_term(q, em1);
    if (P.beta != 0.0f) o.d = fmaf(-P.beta, em1, o.d);
  }
  return o;
}

__device__ __forceinline__ int64_t row_target(const LossParams& P, int64_t r) {
  return P.targets64 ? ((const int64_t*)P.targets)[r] : (int64_t)((const int32_t*)P.targets)[r];
}

template <int LT, bool VEC>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return LT == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

// A CTA per row, CTAs over rows in turn.
template <int LT, int GT, int MODE, bool VEC>
__global__ void __launch_bounds__(LOSS_THREADS) loss_rows_kernel(const __grid_constant__ LossParams P) {
  __shared__ RowSum red[LOSS_WARPS];
  __shared__ float coef[3];
  const int64_t groups = (P.cols + 7) / 8;
  double loss_sum = 0.0, kl_sum = 0.0;
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const int64_t t = row_target(P, r);
    const float w = MODE == LOSS_LOGP ? 1.0f : P.weight ? P.weight[r] : P.uniform;
    const bool live = t >= 0 && t < P.cols && !(w == 0.0f);
    if (!live) {                                        // left out: its logits are not read
      if (threadIdx.x == 0 && P.logp) P.logp[r] = 0.0f;
      if (MODE == LOSS_GRAD) {
        const float z[8] = {};
        for (int64_t q = threadIdx.x; q < groups; q += LOSS_THREADS)
          store8<GT, VEC>(P.grad, r * P.ldg + q * 8, (int)(P.cols - q * 8 < 8 ? P.cols - q * 8 : 8), z);
      }
      continue;
    }
    const int64_t xo = r * P.ldx;
    const float xt = load1<LT, VEC>(P.x, xo + t);       // read before the row may be overwritten in place
    RowSum v{-INFINITY, 0.0f, 0.0f};
    for (int64_t q0 = threadIdx.x; q0 < groups; q0 += 4 * LOSS_THREADS) {
      float x[4][8];
      int n[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t left = P.cols - (q0 + j * LOSS_THREADS) * 8;
        n[j] = left <= 0 ? 0 : left < 8 ? (int)left : 8;
        if (n[j] > 0) load8<LT, VEC>(P.x, xo + (q0 + j * LOSS_THREADS) * 8, n[j], x[j]);
      }
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
        loss_sum += (double)w * ((double)o.term + (P.beta != 0.0f ? (double)P.beta * (double)o.k : 0.0));
        kl_sum += (double)w * (double)o.k;
      }
    }
    __syncthreads();
    if (MODE == LOSS_GRAD) {
      const float f = coef[0], ft = coef[1];
      for (int64_t q = threadIdx.x; q < groups; q += LOSS_THREADS) {
        const int64_t c0 = q * 8;
        const int n = P.cols - c0 < 8 ? (int)(P.cols - c0) : 8;
        float x[8];
        load8<LT, VEC>(P.x, xo + c0, n, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = c0 + k == t ? ft : ex2_approx((x[k] - v.m) * P.c) * f;
        store8<GT, VEC>(P.grad, r * P.ldg + c0, n, x);
      }
    }
  }
  if (MODE != LOSS_LOGP && threadIdx.x == 0) {
    P.part[2 * blockIdx.x] = loss_sum;
    P.part[2 * blockIdx.x + 1] = kl_sum;
  }
}

// The CTAs' sums joined: two warps, lanes over CTAs in turn.
__global__ void __launch_bounds__(64) loss_finish_kernel(const double* part, int n, float* loss) {
  const int lane = threadIdx.x & 31, which = threadIdx.x >> 5;
  double s = 0.0;
  for (int i = lane; i < n; i += 32) s += part[2 * i + which];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) loss[which] = (float)s;
}

static int loss_check_rows(const void* logits, int32_t lt, int64_t rows, int64_t cols, int64_t ldl, double scale,
                           const void* targets, int32_t tt) {
  if (!dtype_ok(lt)) return fail(PSK_E_DTYPE, "logits dtype %d", lt);
  if (tt != PSK_I32 && tt != PSK_I64) return fail(PSK_E_DTYPE, "target dtype %d", tt);
  if (rows < 0 || cols < 0) return fail(PSK_E_SHAPE, "rows %lld, cols %lld", (long long)rows, (long long)cols);
  if (cols > (1LL << 31)) return fail(PSK_E_SHAPE, "cols %lld above 2^31", (long long)cols);
  if (rows > 0 && cols == 0) return fail(PSK_E_SHAPE, "rows of no logits");
  if (!(scale >= 1e-30 && scale <= 1e30)) return fail(PSK_E_ARG, "scale %g is not in [1e-30, 1e30]", scale);
  if (rows == 0) return PSK_OK;
  if (!logits || !targets) return fail(PSK_E_NULL, "logits or targets is NULL");
  if (ldl < cols) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(rows, ldl)) return fail(PSK_E_SHAPE, "rows x leading dimension too large");
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
  const bool vec = rows_vec8(logits, lt, ldl, rows);
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
  *bytes = 16ull * (uint64_t)(rows < LOSS_MAX_CTAS ? rows : LOSS_MAX_CTAS);
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
    loss_finish_kernel<<<1, 64, 0, s>>>(nullptr, 0, loss);
    return check_launch("policy loss finishing kernel");
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
  const unsigned grid = loss_grid(rows);
  const bool vec = rows_vec8(logits, lt, ldl, rows) && (!dlogits || rows_vec8(dlogits, gt, ldg, rows));
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
  if (rc) return rc;
  loss_finish_kernel<<<1, 64, 0, s>>>(P.part, (int)grid, loss);
  return check_launch("policy loss finishing kernel");
}
