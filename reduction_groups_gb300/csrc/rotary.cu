// psk_qk_norm_rotary: the norm of every query and key head and the rotation
// by its token's position in one pass, and the backward.
//
// A head of D columns: u = x / sqrt(mean(x^2) + eps) gamma (or u = x), then
// each pair of its first `rot` columns turns by pos f_j:
//   (u_a, u_b) -> (u_a cos - u_b sin, u_b cos + u_a sin).
// The angle is reduced exactly: f_j / 2 pi is held as a 64-bit fraction of a
// turn, its product with the position taken mod 2^64 is the fraction of a turn
// at that position (off by 2^-64 a position), and sincospi does the rest.  A
// warp forms its token's cosines and sines once for all heads.
//
// Memory-bound: x is read once and y written once.  Heads are taken by teams
// of lanes, a lane holding groups of V pairs (V = 8: 16-byte accesses), several
// heads of a token in flight in a warp.
#include "common.cuh"
#include "vec8.cuh"
#include "views.h"

namespace psk {

constexpr int ROT_THREADS = 256;
constexpr int ROT_WARPS = ROT_THREADS / 32;
constexpr int ROT_MAX_DIM = 512;
constexpr int ROT_MAX_BLOCKS = 304;

struct RotSide {
  const void *x, *ct, *gamma;
  void *y, *dgamma;
  int64_t xt, xh, ct_t, ct_h, yt, yh;      // element strides of a token and a head
  int32_t heads;
};

struct RotParams {
  RotSide side[2];
  const void* pos;
  const float* freqs;
  float* part;                             // [block][2][dim]
  int64_t tokens;
  int32_t dim, rot, pos64, rms, neighbours;
  int32_t x_type, ct_type, y_type, gamma_type, dgamma_type;
  int32_t chunks, per;                     // a token's heads in `chunks` shares of `per` warp steps
  int32_t blocks;
  float eps, inv_dim;
};

// f / 2 pi as a fraction of 2^64 (mod 1): the quotient as a pair of doubles.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const double H = 0.15915494309189535, L = -9.839338337591243e-18;
  const double x = (double)f;
  const double hi = x * H, lo = fma(x, H, -hi) + x * L;
  const double frac = hi - floor(hi);
  return __double2ull_rd(frac * 18446744073709551616.0) + (uint64_t)__double2ll_rn(lo * 18446744073709551616.0);
}

struct RotTable {
  uint64_t turn[ROT_MAX_DIM / 2];
  float bad[ROT_MAX_DIM / 2];              // NaN where the frequency is not finite
};

__device__ __forceinline__ void rot_table(RotTable& T, const RotParams& P) {
  for (int j = threadIdx.x; j < (P.tokens ? P.rot / 2 : 0); j += ROT_THREADS) {
    const float f = P.freqs[j];
    T.turn[j] = turn_fraction(f);
    T.bad[j] = f * 0.0f;
  }
  __syncthreads();
}

__device__ __forceinline__ void rot_angles(float2* cs, const RotTable& T, const RotParams& P, int64_t token, int lane) {
  const int64_t pos = P.pos64 ? ((const int64_t*)P.pos)[token] : (int64_t)((const int32_t*)P.pos)[token];
  __syncwarp();
  for (int j = lane; j < P.rot / 2; j += 32) {
    const int64_t frac = (int64_t)((uint64_t)pos * T.turn[j]);
    float s, c;
    sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &s, &c);     // 2 turns 2^-64
    cs[j] = make_float2(c + T.bad[j], s + T.bad[j]);
  }
  __syncwarp();
}

// A lane's group g of V pairs of a head: its columns, in two runs of V (pairs
// of halves) or as 2 V neighbours.
template <int V, bool NEIGH>
struct RotGroup {
  int first[2];                            // of each run
  int pair;                                // its first pair
  bool turns, has[2];
  __device__ __forceinline__ RotGroup(int g, const RotParams& P) {
    pair = g * V;
    turns = pair < P.rot / 2;
    if constexpr (NEIGH) {
      first[0] = 2 * pair, first[1] = 2 * pair + V;
    } else if (turns) {
      first[0] = pair, first[1] = pair + P.rot / 2;
    } else {
      const int i = pair - P.rot / 2;
      first[0] = P.rot + i, first[1] = P.rot + (P.dim - P.rot + 1) / 2 + i;
    }
    const int pairs = P.rot / 2 + (P.dim - P.rot + 1) / 2;
    has[0] = pair < pairs;
    has[1] = has[0] && first[1] < P.dim;
  }
  // Element index of the members of pair i in the 2 V values.
  static __device__ __forceinline__ constexpr int a(int i) { return NEIGH ? 2 * i : i; }
  static __device__ __forceinline__ constexpr int b(int i) { return NEIGH ? 2 * i + 1 : i + V; }
  __device__ __forceinline__ void load(const void* p, int32_t dt, int64_t at, float* v) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (V == 8) {
        const int n = has[k] ? 8 : 0;
        if (dt == PSK_BF16) {
          if (n) load8<PSK_BF16, true>(p, at + first[k], 8, v + 8 * k);
        } else {
          if (n) load8<PSK_F32, true>(p, at + first[k], 8, v + 8 * k);
        }
        if (!n) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * k + i] = 0.0f;
        }
      } else {
        v[k] = !has[k] ? 0.0f
               : dt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[at + first[k]])
                                : ((const float*)p)[at + first[k]];
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int32_t dt, int64_t at, const float* v) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!has[k]) continue;
      if constexpr (V == 8) {
        const float* w = v + 8 * k;
        if (dt == PSK_BF16) {
          *(uint4*)((uint16_t*)p + at + first[k]) = make_uint4(f32x2_to_bf16x2(w[0], w[1]), f32x2_to_bf16x2(w[2], w[3]),
                                                               f32x2_to_bf16x2(w[4], w[5]), f32x2_to_bf16x2(w[6], w[7]));
        } else {
          float4* q = (float4*)((float*)p + at + first[k]);
          q[0] = make_float4(w[0], w[1], w[2], w[3]);
          q[1] = make_float4(w[4], w[5], w[6], w[7]);
        }
      } else if (dt == PSK_BF16) {
        ((uint16_t*)p)[at + first[k]] = f32_to_bf16_bits(v[k]);
      } else {
        ((float*)p)[at + first[k]] = v[k];
      }
    }
  }
  // Turn the pairs by sign times their angle.
  __device__ __forceinline__ void turn(const float2* cs, float sign, float* v) const {
    if (!turns || !has[0]) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 t = cs[pair + i];
      const float x = v[a(i)], y = v[b(i)], s = sign * t.y;
      v[a(i)] = fmaf(x, t.x, -(y * s));
      v[b(i)] = fmaf(y, t.x, x * s);
    }
  }
};

__device__ __forceinline__ float team_sum(float s, int team) {
  for (int o = team >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// Lanes of a team (a power of two): one for each group of V pairs, a warp at most.
template <int V>
static int rot_team(const RotParams& P) {
  const int pairs = P.rot / 2 + (P.dim - P.rot + 1) / 2, groups = (pairs + V - 1) / V;
  int t = 1;
  while (t < 32 && t < groups) t *= 2;
  return t;
}

template <int V, int NG, bool NEIGH, int XT, int YT>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ RotTable T;
  __shared__ float2 angles[ROT_WARPS][ROT_MAX_DIM / 2];
  __shared__ float gammas[2][ROT_MAX_DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int xt = XT < 0 ? P.x_type : XT, yt = YT < 0 ? P.y_type : YT;
  rot_table(T, P);
  for (int i = threadIdx.x; i < 2 * P.dim; i += ROT_THREADS) {
    const int s = i >= P.dim, c = i - s * P.dim;
    const void* g = P.side[s].gamma;
    gammas[s][c] = !g ? 1.0f : P.gamma_type == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)g)[c]) : ((const float*)g)[c];
  }
  __syncthreads();
  const int slots = 32 / team, slot = lane / team, in = lane % team;
  const int heads = P.side[0].heads + P.side[1].heads;
  float2* cs = angles[warp];
  const int64_t units = P.tokens * P.chunks;
  for (int64_t u = (int64_t)blockIdx.x * ROT_WARPS + warp; u < units; u += (int64_t)gridDim.x * ROT_WARPS) {
    const int64_t token = u / P.chunks;
    const int h0 = (int)(u - token * P.chunks) * P.per * slots;
    rot_angles(cs, T, P, token, lane);
    for (int i = 0; i < P.per; ++i) {
      const int head = h0 + i * slots + slot;
      const bool live = head < heads;
      const int sd = head >= P.side[0].heads;
      const RotSide& S = P.side[sd];
      const int h = head - (sd ? P.side[0].heads : 0);
      float v[NG][2 * V];
      float sum = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        RotGroup<V, NEIGH> G(in + g * team, P);
        if (live) G.load(S.x, xt, token * S.xt + h * S.xh, v[g]);
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
          if (!live) v[g][k] = 0.0f;
          sum = fmaf(v[g][k], v[g][k], sum);
        }
      }
      if (P.rms) {
        sum = team_sum(sum, team);
        const float r = __frsqrt_rn(fmaf(sum, P.inv_dim, P.eps));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          RotGroup<V, NEIGH> G(in + g * team, P);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (G.has[k]) {
#pragma unroll
              for (int j = 0; j < V; ++j) v[g][k * V + j] = v[g][k * V + j] * r * gammas[sd][G.first[k] + j];
            }
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        RotGroup<V, NEIGH> G(in + g * team, P);
        G.turn(cs, 1.0f, v[g]);
        if (live) G.store(S.y, yt, token * S.yt + h * S.yh, v[g]);
      }
    }
  }
}

// The backward: the cotangent turned back, then the norm's.  A CTA's dgamma
// sums stay in registers over all its tokens, side after side.
template <int V, int NG, bool NEIGH, int XT, int CT, int YT>
__global__ void __launch_bounds__(ROT_THREADS) rotary_backward_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ RotTable T;
  __shared__ float2 angles[ROT_WARPS][ROT_MAX_DIM / 2];
  __shared__ float gammas[2][ROT_MAX_DIM];
  __shared__ float sums[ROT_WARPS][ROT_MAX_DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int xt = XT < 0 ? P.x_type : XT, ct = CT < 0 ? P.ct_type : CT, yt = YT < 0 ? P.y_type : YT;
  rot_table(T, P);
  for (int i = threadIdx.x; i < 2 * P.dim; i += ROT_THREADS) {
    const int s = i >= P.dim, c = i - s * P.dim;
    const void* g = P.side[s].gamma;
    gammas[s][c] = !g ? 1.0f : P.gamma_type == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)g)[c]) : ((const float*)g)[c];
  }
  __syncthreads();
  const int slots = 32 / team, slot = lane / team, in = lane % team;
  float2* cs = angles[warp];
  float dg[2][NG][2 * V];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) dg[s][g][k] = 0.0f;
  for (int64_t token = (int64_t)blockIdx.x * ROT_WARPS + warp; token < P.tokens;
       token += (int64_t)gridDim.x * ROT_WARPS) {
    rot_angles(cs, T, P, token, lane);
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const RotSide& S = P.side[sd];
      for (int h0 = 0; h0 < S.heads; h0 += slots) {
        const int h = h0 + slot;
        const bool live = h < S.heads;
        float v[NG][2 * V], x[NG][2 * V];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          RotGroup<V, NEIGH> G(in + g * team, P);
          if (live) G.load(S.ct, ct, token * S.ct_t + h * S.ct_h, v[g]);
          if (live && P.rms) G.load(S.x, xt, token * S.xt + h * S.xh, x[g]);
          if (!live || !P.rms) {
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) x[g][k] = 0.0f;
          }
          if (!live) {
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) v[g][k] = 0.0f;
          }
        }
        float r = 1.0f, m = 0.0f;
        if (P.rms) {
          float sum = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) sum = fmaf(x[g][k], x[g][k], sum);
          r = __frsqrt_rn(fmaf(team_sum(sum, team), P.inv_dim, P.eps));
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          RotGroup<V, NEIGH> G(in + g * team, P);
          G.turn(cs, -1.0f, v[g]);
          if (P.rms) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (G.has[k] && live) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                  const int e = k * V + j;
                  x[g][e] *= r;
                  dg[sd][g][e] = fmaf(v[g][e], x[g][e], dg[sd][g][e]);
                  v[g][e] *= gammas[sd][G.first[k] + j];
                  m = fmaf(v[g][e], x[g][e], m);
                }
              }
          }
        }
        if (P.rms) {
          m = team_sum(m, team) * P.inv_dim;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) v[g][k] = fmaf(-x[g][k], m, v[g][k]) * r;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          RotGroup<V, NEIGH> G(in + g * team, P);
          if (live) G.store(S.y, yt, token * S.yt + h * S.yh, v[g]);
        }
      }
    }
  }
  if (!P.part) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
    // teams of a warp joined by shuffles, warps through shared memory
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int k = 0; k < 2 * V; ++k)
        for (int o = team; o < 32; o <<= 1) dg[sd][g][k] += __shfl_xor_sync(0xFFFFFFFFu, dg[sd][g][k], o);
    __syncthreads();
    if (slot == 0) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        RotGroup<V, NEIGH> G(in + g * team, P);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (G.has[k]) {
#pragma unroll
            for (int j = 0; j < V; ++j) sums[warp][G.first[k] + j] = dg[sd][g][k * V + j];
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < P.dim; c += ROT_THREADS) {
      float s = sums[0][c];
#pragma unroll
      for (int w = 1; w < ROT_WARPS; ++w) s += sums[w][c];
      P.part[((int64_t)blockIdx.x * 2 + sd) * P.dim + c] = s;
    }
  }
}

// dgamma from the CTAs' sums: 32 columns of one side a CTA, 32 warps the blocks in turn.
__global__ void __launch_bounds__(1024) rotary_join_kernel(const __grid_constant__ RotParams P) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, sd = blockIdx.y;
  void* out = P.side[sd].dgamma;
  if (!out) return;
  float s = 0.0f;
  if (c < P.dim)
    for (int b = warp; b < P.blocks; b += 32) s += P.part[((int64_t)b * 2 + sd) * P.dim + c];
  part[warp][lane] = s;
  __syncthreads();
  s = part[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < P.dim) {
    if (P.dgamma_type == PSK_BF16) ((uint16_t*)out)[col] = f32_to_bf16_bits(s);
    else ((float*)out)[col] = s;
  }
}

// ---------------------------------------------------------------------- host

static int64_t rot_blocks(int64_t tokens) {
  const int64_t b = (tokens + ROT_WARPS - 1) / ROT_WARPS;
  return b < 1 ? 1 : b < ROT_MAX_BLOCKS ? b : ROT_MAX_BLOCKS;
}

static int rot_check_sizes(int64_t tokens, int64_t hq, int64_t hk, int64_t dim) {
  if (tokens < 0 || tokens >= 1LL << 40) return fail(PSK_E_SHAPE, "tokens %lld", (long long)tokens);
  if (hq < 0 || hk < 0 || hq > 1 << 20 || hk > 1 << 20)
    return fail(PSK_E_SHAPE, "heads %lld, %lld", (long long)hq, (long long)hk);
  if (dim < 1 || dim > ROT_MAX_DIM) return fail(PSK_E_SHAPE, "head size %lld is not in [1, %d]", (long long)dim, ROT_MAX_DIM);
  return PSK_OK;
}

// A tensor [tokens, heads, dim]; empty when it has no elements.
struct Heads {
  const char* name;
  const void* p;
  int32_t dt;
  int64_t tokens, heads, dim, ts, hs;
  bool there() const { return tokens && heads; }
  int64_t of_token() const { return (heads > 1 ? (heads - 1) * hs : 0) + dim; }     // first to last element
  int64_t of_head() const { return (tokens > 1 ? (tokens - 1) * ts : 0) + dim; }
  bool token_major() const { return tokens <= 1 || ts >= of_token(); }
};

static int heads_check(const Heads& h) {
  if (!dtype_ok(h.dt)) return fail(PSK_E_DTYPE, "%s dtype %d", h.name, h.dt);
  if (!h.there()) return PSK_OK;
  if (!h.p) return fail(PSK_E_NULL, "%s is NULL", h.name);
  if ((uintptr_t)h.p % dtype_size(h.dt)) return fail(PSK_E_ARG, "%s is not aligned to its type", h.name);
  if ((h.heads > 1 && h.hs < h.dim) || (h.tokens > 1 && h.ts < h.dim))
    return fail(PSK_E_SHAPE, "%s: a stride below the head's size", h.name);
  if ((h.heads > 1 && !rows_addressable(h.heads, h.hs)) || (h.tokens > 1 && !rows_addressable(h.tokens, h.ts)))
    return fail(PSK_E_SHAPE, "%s: stride too large", h.name);
  if (!h.token_major() && !(h.heads <= 1 || h.hs >= h.of_head()))
    return fail(PSK_E_SHAPE, "%s: neither a token's heads nor a head's tokens are apart", h.name);
  return PSK_OK;
}

// The tensor as one stretch a token, or a head where heads are apart.
static View heads_view(const Heads& h) {
  if (!h.there() || !h.p) return View{0, 0, 0, 0};
  if (h.token_major()) return view_of(h.p, h.tokens, h.of_token(), h.ts, dtype_size(h.dt));
  return view_of(h.p, h.heads, h.of_head(), h.hs, dtype_size(h.dt));
}

static bool heads_same(const Heads& a, const Heads& b) {
  return a.p == b.p && a.dt == b.dt && (a.heads <= 1 || a.hs == b.hs) && (a.tokens <= 1 || a.ts == b.ts);
}

static bool heads_vec(const Heads& h) {
  const int64_t e = 16 / dtype_size(h.dt);
  return !h.there() || ((uintptr_t)h.p % 16 == 0 && (h.tokens <= 1 || h.ts % e == 0) && (h.heads <= 1 || h.hs % e == 0));
}

static View span_view(const void* p, uint64_t bytes) { return View{(uintptr_t)p, p && bytes ? 1 : 0, bytes, bytes}; }

static int rot_check_common(int64_t tokens, const void* pos, int32_t pt, const float* freqs, int64_t dim, int64_t rot,
                            int32_t pairs, int32_t norm, double eps, const void* gq, const void* gk, int32_t gt) {
  if (rot < 0 || rot > dim || rot % 2) return fail(PSK_E_SHAPE, "%lld rotating columns of %lld", (long long)rot, (long long)dim);
  if (pt != PSK_I32 && pt != PSK_I64) return fail(PSK_E_DTYPE, "position dtype %d", pt);
  if (pairs != PSK_PAIRS_HALVES && pairs != PSK_PAIRS_NEIGHBOURS) return fail(PSK_E_ARG, "pairs %d", pairs);
  if (norm != PSK_HEAD_NORM_NONE && norm != PSK_HEAD_NORM_RMS) return fail(PSK_E_ARG, "norm %d", norm);
  if (norm == PSK_HEAD_NORM_RMS && !(eps >= 0.0 && eps <= 3.4e38)) return fail(PSK_E_ARG, "eps is not in [0, 3.4e38]");
  if (norm == PSK_HEAD_NORM_NONE && (gq || gk)) return fail(PSK_E_ARG, "scales without a norm");
  if ((gq || gk) && !dtype_ok(gt)) return fail(PSK_E_DTYPE, "scale dtype %d", gt);
  if ((gq && (uintptr_t)gq % dtype_size(gt)) || (gk && (uintptr_t)gk % dtype_size(gt)))
    return fail(PSK_E_ARG, "a scale is not aligned to its type");
  if (tokens && rot && !pos) return fail(PSK_E_NULL, "positions is NULL");
  if (tokens && rot && !freqs) return fail(PSK_E_NULL, "freqs is NULL");
  if ((uintptr_t)pos % (pt == PSK_I64 ? 8 : 4) || (uintptr_t)freqs % 4)
    return fail(PSK_E_ARG, "positions or freqs is not aligned to its type");
  return PSK_OK;
}

static bool rot_vec(int64_t dim, int64_t rot) { return dim % 16 == 0 && rot % 16 == 0; }

template <typename F>
static int rot_shape(const RotParams& P, bool vec, F&& f) {
  const int pairs = P.rot / 2 + (P.dim - P.rot + 1) / 2;
  const auto with_pairs = [&](auto V, auto NG) {
    return with_bool(P.neighbours != 0, [&](auto N) { return f(V, NG, N); });
  };
  using std::integral_constant;
  if (vec) return with_pairs(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (pairs <= 32) return with_pairs(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (pairs <= 64) return with_pairs(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (pairs <= 128) return with_pairs(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  return with_pairs(integral_constant<int, 1>{}, integral_constant<int, 8>{});
}

}  // namespace psk

using namespace psk;

extern "C" int psk_qk_norm_rotary(const void* q, const void* k, int32_t xt, int64_t q_token, int64_t q_head,
                                  int64_t k_token, int64_t k_head, void* yq, void* yk, int32_t yt, int64_t yq_token,
                                  int64_t yq_head, int64_t yk_token, int64_t yk_head, int64_t tokens, int64_t hq,
                                  int64_t hk, int64_t dim, int64_t rot, const void* positions, int32_t pt,
                                  const float* freqs, int32_t pairs, int32_t norm, double eps, const void* gamma_q,
                                  const void* gamma_k, int32_t gt, void* stream) {
  clear_error();
  int rc = rot_check_sizes(tokens, hq, hk, dim);
  if (!rc) rc = rot_check_common(tokens, positions, pt, freqs, dim, rot, pairs, norm, eps, gamma_q, gamma_k, gt);
  if (rc) return rc;
  const Heads in[2] = {{"q", q, xt, tokens, hq, dim, q_token, q_head}, {"k", k, xt, tokens, hk, dim, k_token, k_head}};
  const Heads out[2] = {{"yq", yq, yt, tokens, hq, dim, yq_token, yq_head},
                        {"yk", yk, yt, tokens, hk, dim, yk_token, yk_head}};
  for (int i = 0; !rc && i < 2; ++i) {
    rc = heads_check(in[i]);
    if (!rc) rc = heads_check(out[i]);
  }
  if (rc || !tokens || !(hq + hk)) return rc;
  const View plain[4] = {span_view(positions, (uint64_t)tokens * (pt == PSK_I64 ? 8 : 4)),
                         span_view(freqs, (uint64_t)rot * 2), span_view(gamma_q, (uint64_t)dim * dtype_size(gt)),
                         span_view(gamma_k, (uint64_t)dim * dtype_size(gt))};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 2; ++j)
      if (views_overlap(heads_view(out[i]), heads_view(in[j])) && !(i == j && heads_same(out[i], in[j])))
        return fail(PSK_E_ALIAS, "%s overlaps %s and is not the same tensor", out[i].name, in[j].name);
    for (const View& v : plain)
      if (views_overlap(heads_view(out[i]), v)) return fail(PSK_E_ALIAS, "%s overlaps positions, freqs or a scale", out[i].name);
  }
  if (views_overlap(heads_view(out[0]), heads_view(out[1]))) return fail(PSK_E_ALIAS, "yq overlaps yk");
  RotParams P{};
  P.side[0] = RotSide{q, nullptr, gamma_q, yq, nullptr, q_token, q_head, 0, 0, yq_token, yq_head, (int32_t)hq};
  P.side[1] = RotSide{k, nullptr, gamma_k, yk, nullptr, k_token, k_head, 0, 0, yk_token, yk_head, (int32_t)hk};
  P.pos = positions, P.freqs = freqs, P.tokens = tokens, P.dim = (int32_t)dim, P.rot = (int32_t)rot;
  P.pos64 = pt == PSK_I64, P.rms = norm == PSK_HEAD_NORM_RMS, P.neighbours = pairs == PSK_PAIRS_NEIGHBOURS;
  P.x_type = xt, P.y_type = yt, P.gamma_type = gt;
  P.eps = (float)eps, P.inv_dim = 1.0f / (float)dim;
  const bool vec = rot_vec(dim, rot) && heads_vec(in[0]) && heads_vec(in[1]) && heads_vec(out[0]) && heads_vec(out[1]);
  cudaStream_t s = (cudaStream_t)stream;
  return rot_shape(P, vec, [&](auto V, auto NG, auto N) {
    const int team = rot_team<V.value>(P), slots = 32 / team;
    const int64_t steps = (hq + hk + slots - 1) / slots, warps = (int64_t)device_sm_count() * 8 * ROT_WARPS;
    // A token's heads go to one warp where tokens alone fill the GPU, else to several.
    int64_t chunks = tokens >= warps ? 1 : (warps + tokens - 1) / tokens;
    if (chunks > steps) chunks = steps;
    P.per = (int32_t)((steps + chunks - 1) / chunks);
    P.chunks = (int32_t)((steps + P.per - 1) / P.per);
    const int64_t ctas = (tokens * P.chunks + ROT_WARPS - 1) / ROT_WARPS, most = (int64_t)device_sm_count() * 8;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    if (V.value == 8 && xt == yt)
      with_dtype(xt, [&](auto TY) {
        rotary_kernel<V.value, NG.value, N.value, TY.value, TY.value><<<grid, ROT_THREADS, 0, s>>>(P, team);
        return 0;
      });
    else rotary_kernel<V.value, NG.value, N.value, -1, -1><<<grid, ROT_THREADS, 0, s>>>(P, team);
    return check_launch("rotary kernel");
  });
}

extern "C" int psk_qk_norm_rotary_backward_workspace(int64_t tokens, int64_t hq, int64_t hk, int64_t dim,
                                                     uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = rot_check_sizes(tokens, hq, hk, dim);
  if (rc) return rc;
  *bytes = (uint64_t)rot_blocks(tokens) * 2 * dim * 4;
  return PSK_OK;
}

extern "C" int psk_qk_norm_rotary_backward(
    const void* cq, const void* ck, int32_t ct, int64_t cq_token, int64_t cq_head, int64_t ck_token, int64_t ck_head,
    const void* q, const void* k, int32_t xt, int64_t q_token, int64_t q_head, int64_t k_token, int64_t k_head,
    void* dq, void* dk, int32_t dt, int64_t dq_token, int64_t dq_head, int64_t dk_token, int64_t dk_head,
    int64_t tokens, int64_t hq, int64_t hk, int64_t dim, int64_t rot, const void* positions, int32_t pt,
    const float* freqs, int32_t pairs, int32_t norm, double eps, const void* gamma_q, const void* gamma_k, int32_t gt,
    void* dgamma_q, void* dgamma_k, int32_t dgt, void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  int rc = rot_check_sizes(tokens, hq, hk, dim);
  if (!rc) rc = rot_check_common(tokens, positions, pt, freqs, dim, rot, pairs, norm, eps, gamma_q, gamma_k, gt);
  if (rc) return rc;
  const bool rms = norm == PSK_HEAD_NORM_RMS;
  const bool sums = dgamma_q || dgamma_k;
  if (sums && !rms) return fail(PSK_E_ARG, "scale gradients without a norm");
  if (sums && !dtype_ok(dgt)) return fail(PSK_E_DTYPE, "scale gradient dtype %d", dgt);
  if ((dgamma_q && (uintptr_t)dgamma_q % dtype_size(dgt)) || (dgamma_k && (uintptr_t)dgamma_k % dtype_size(dgt)))
    return fail(PSK_E_ARG, "a scale gradient is not aligned to its type");
  const int64_t xtok = rms ? tokens : 0;      // without a norm x is not read
  const Heads cts[2] = {{"cq", cq, ct, tokens, hq, dim, cq_token, cq_head}, {"ck", ck, ct, tokens, hk, dim, ck_token, ck_head}};
  const Heads xs[2] = {{"q", q, rms ? xt : PSK_F32, xtok, hq, dim, q_token, q_head},
                       {"k", k, rms ? xt : PSK_F32, xtok, hk, dim, k_token, k_head}};
  const Heads out[2] = {{"dq", dq, dt, tokens, hq, dim, dq_token, dq_head}, {"dk", dk, dt, tokens, hk, dim, dk_token, dk_head}};
  for (int i = 0; !rc && i < 2; ++i) {
    rc = heads_check(cts[i]);
    if (!rc) rc = heads_check(xs[i]);
    if (!rc) rc = heads_check(out[i]);
  }
  if (rc || (!sums && (!tokens || !(hq + hk)))) return rc;
  const uint64_t need = sums ? (uint64_t)rot_blocks(tokens) * 2 * dim * 4 : 0;
  if (sums) {
    if (!workspace) return fail(PSK_E_NULL, "workspace is NULL");
    if ((uintptr_t)workspace % 16) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                  (unsigned long long)need);
  }
  const uint64_t gb = (uint64_t)dim * dtype_size(gt), dgb = (uint64_t)dim * dtype_size(dgt);
  const View plain[4] = {span_view(positions, (uint64_t)tokens * (pt == PSK_I64 ? 8 : 4)),
                         span_view(freqs, (uint64_t)rot * 2), span_view(gamma_q, gb), span_view(gamma_k, gb)};
  const View grads[3] = {span_view(dgamma_q, dgb), span_view(dgamma_k, dgb), span_view(sums ? workspace : nullptr, need)};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 2; ++j) {
      if (views_overlap(heads_view(out[i]), heads_view(cts[j])) && !(i == j && heads_same(out[i], cts[j])))
        return fail(PSK_E_ALIAS, "%s overlaps %s and is not the same tensor", out[i].name, cts[j].name);
      if (views_overlap(heads_view(out[i]), heads_view(xs[j])) && !(i == j && heads_same(out[i], xs[j])))
        return fail(PSK_E_ALIAS, "%s overlaps %s and is not the same tensor", out[i].name, xs[j].name);
    }
    for (const View& v : plain)
      if (views_overlap(heads_view(out[i]), v)) return fail(PSK_E_ALIAS, "%s overlaps positions, freqs or a scale", out[i].name);
  }
  if (views_overlap(heads_view(out[0]), heads_view(out[1]))) return fail(PSK_E_ALIAS, "dq overlaps dk");
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (views_overlap(grads[i], grads[j])) return fail(PSK_E_ALIAS, "the scale gradients and the workspace overlap");
    for (const View& v : plain)
      if (views_overlap(grads[i], v)) return fail(PSK_E_ALIAS, "a scale gradient or the workspace overlaps positions, freqs or a scale");
    for (int j = 0; j < 2; ++j)
      if (views_overlap(grads[i], heads_view(out[j])) || views_overlap(grads[i], heads_view(cts[j])) ||
          views_overlap(grads[i], heads_view(xs[j])))
        return fail(PSK_E_ALIAS, "a scale gradient or the workspace overlaps a tensor");
  }
  RotParams P{};
  P.side[0] = RotSide{q, cq, gamma_q, dq, dgamma_q, q_token, q_head, cq_token, cq_head, dq_token, dq_head, (int32_t)hq};
  P.side[1] = RotSide{k, ck, gamma_k, dk, dgamma_k, k_token, k_head, ck_token, ck_head, dk_token, dk_head, (int32_t)hk};
  P.pos = positions, P.freqs = freqs, P.tokens = tokens, P.dim = (int32_t)dim, P.rot = (int32_t)rot;
  P.pos64 = pt == PSK_I64, P.rms = rms, P.neighbours = pairs == PSK_PAIRS_NEIGHBOURS;
  P.x_type = xt, P.ct_type = ct, P.y_type = dt, P.gamma_type = gt, P.dgamma_type = dgt;
  P.eps = (float)eps, P.inv_dim = 1.0f / (float)dim;
  P.part = sums ? (float*)workspace : nullptr;
  P.blocks = (int32_t)rot_blocks(tokens);
  const bool vec = rot_vec(dim, rot) && heads_vec(cts[0]) && heads_vec(cts[1]) && heads_vec(out[0]) &&
                   heads_vec(out[1]) && (!rms || (heads_vec(xs[0]) && heads_vec(xs[1])));
  cudaStream_t s = (cudaStream_t)stream;
  rc = rot_shape(P, vec, [&](auto V, auto NG, auto N) {
    const int team = rot_team<V.value>(P);
    const unsigned grid = (unsigned)P.blocks;
    if (V.value == 8 && ct == dt && (!rms || xt == ct))
      with_dtype(ct, [&](auto TY) {
        rotary_backward_kernel<V.value, NG.value, N.value, TY.value, TY.value, TY.value>
            <<<grid, ROT_THREADS, 0, s>>>(P, team);
        return 0;
      });
    else rotary_backward_kernel<V.value, NG.value, N.value, -1, -1, -1><<<grid, ROT_THREADS, 0, s>>>(P, team);
    return check_launch("rotary backward kernel");
  });
  if (rc || !sums) return rc;
  rotary_join_kernel<<<dim3((unsigned)((dim + 31) / 32), 2), 1024, 0, s>>>(P);
  return check_launch("rotary join kernel");
}
