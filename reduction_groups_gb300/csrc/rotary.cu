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
// of lanes, several heads of a token by a warp at once, and the loads of the
// steps to come are in flight while one is worked on.
#include "common.cuh"
#include "vec8.cuh"
#include "views.h"

namespace psk {

constexpr int ROT_THREADS = 256;
constexpr int ROT_WARPS = ROT_THREADS / 32;
constexpr int ROT_MAX_DIM = 512;
// CTAs an SM, by registers: of the forward with four pairs a lane and two or
// four heads a team at once, and of the rest.
template <int TY, int SUB>
constexpr int ROT_FWD_CTAS = TY == PSK_BF16 && SUB == 2 ? 3 : 2;
constexpr int ROT_BWD_CTAS = 2;
constexpr int ROT_MAX_BLOCKS = 4 * NOMINAL_SMS;      // CTAs of the backward, at most

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
// Of |f|, whose fraction of a turn is exact (of a small negative one it would
// be 1 - a little, rounded to 2^-53), and negated in integers.  L is off by
// 2^-110, so up to 2^40 radians the fraction is off by about a step of 2^-64.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const double H = 0.15915494309189535, L = -9.839338337591243e-18;
  const double x = fabs((double)f);
  const double hi = x * H, lo = fma(x, H, -hi) + x * L;
  const double frac = hi - floor(hi);
  const uint64_t turn =
      __double2ull_rd(frac * 18446744073709551616.0) + (uint64_t)__double2ll_rn(lo * 18446744073709551616.0);
  return f < 0.0f ? 0 - turn : turn;
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

// (Without turning columns there need be no positions.)
__device__ __forceinline__ int64_t rot_position(const RotParams& P, int64_t token) {
  if (!P.rot) return 0;
  return P.pos64 ? ((const int64_t*)P.pos)[token] : (int64_t)((const int32_t*)P.pos)[token];
}

__device__ __forceinline__ void rot_angles(float2* cs, const RotTable& T, const RotParams& P, int64_t token, int lane) {
  const int64_t pos = rot_position(P, token);
  __syncwarp();
  for (int j = lane; j < P.rot / 2; j += 32) {
    const int64_t frac = (int64_t)((uint64_t)pos * T.turn[j]);
    float s, c;
    sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &s, &c);     // 2 turns 2^-64
    cs[j] = make_float2(c + T.bad[j], s + T.bad[j]);
  }
  __syncwarp();
}

// ------------------------------------------------- heads of any size and type
//
// A lane holds NG pairs of a head, `team` lanes apart, loaded and stored
// element by element.

struct RotPair {
  int col[2], pair;
  bool turns, has[2];
  __device__ __forceinline__ void place(int p, bool neighbours, const RotParams& P) {
    pair = p;
    turns = p < P.rot / 2;
    const int rest = (P.dim - P.rot + 1) / 2;          // pairs of columns that do not turn
    if (turns) {
      col[0] = neighbours ? 2 * p : p, col[1] = neighbours ? 2 * p + 1 : p + P.rot / 2;
    } else {
      col[0] = P.rot + p - P.rot / 2, col[1] = col[0] + rest;
    }
    has[0] = p < P.rot / 2 + rest;
    has[1] = has[0] && col[1] < P.dim;
  }
  template <int DT>
  __device__ __forceinline__ void load(const void* p, bool live, float (&v)[2]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      v[k] = 0.0f;
      if (live && has[k]) v[k] = DT == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[col[k]]) : ((const float*)p)[col[k]];
    }
  }
  template <int DT>
  __device__ __forceinline__ void store(void* p, const float (&v)[2]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!has[k]) continue;
      if (DT == PSK_BF16) ((uint16_t*)p)[col[k]] = f32_to_bf16_bits(v[k]);
      else ((float*)p)[col[k]] = v[k];
    }
  }
  __device__ __forceinline__ float2 angle(const float2* cs) const { return turns ? cs[pair] : make_float2(1.0f, 0.0f); }
  __device__ __forceinline__ void turn(float2 t, float (&v)[2]) const {
    if (!turns) return;
    const float x = v[0], y = v[1];
    v[0] = fmaf(x, t.x, -(y * t.y));
    v[1] = fmaf(y, t.x, x * t.y);
  }
};

// A lane's pairs of one head (at: the head's first element); the type is looked
// up once for all of them.
template <int NG>
__device__ __forceinline__ void load_pairs(const RotPair (&G)[NG], const void* p, int32_t dt, int64_t at, bool live,
                                           float (&v)[NG][2]) {
  if (dt == PSK_BF16) {
#pragma unroll
    for (int g = 0; g < NG; ++g) G[g].template load<PSK_BF16>((const uint16_t*)p + at, live, v[g]);
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) G[g].template load<PSK_F32>((const float*)p + at, live, v[g]);
  }
}
template <int NG>
__device__ __forceinline__ void store_pairs(const RotPair (&G)[NG], void* p, int32_t dt, int64_t at,
                                            const float (&v)[NG][2]) {
  if (dt == PSK_BF16) {
#pragma unroll
    for (int g = 0; g < NG; ++g) G[g].template store<PSK_BF16>((uint16_t*)p + at, v[g]);
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) G[g].template store<PSK_F32>((float*)p + at, v[g]);
  }
}

__device__ __forceinline__ float team_sum(float s, int team) {
  for (int o = team >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

__device__ __forceinline__ void rot_scales(float (&gammas)[2][ROT_MAX_DIM], const RotParams& P) {
  for (int i = threadIdx.x; i < 2 * P.dim; i += ROT_THREADS) {
    const int s = i >= P.dim, c = i - s * P.dim;
    const void* g = P.side[s].gamma;
    gammas[s][c] = !g ? 1.0f : P.gamma_type == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)g)[c]) : ((const float*)g)[c];
  }
  __syncthreads();
}

// A CTA's sums of one side: its warps' joined.
__device__ __forceinline__ void rot_part(const float (&sums)[ROT_WARPS][ROT_MAX_DIM], int sd, const RotParams& P) {
  __syncthreads();
  for (int c = threadIdx.x; c < P.dim; c += ROT_THREADS) {
    float s = sums[0][c];
#pragma unroll
    for (int w = 1; w < ROT_WARPS; ++w) s += sums[w][c];
    P.part[((int64_t)blockIdx.x * 2 + sd) * P.dim + c] = s;
  }
}

template <int NG>
__global__ void __launch_bounds__(ROT_THREADS, 3) rotary_any_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ RotTable T;
  __shared__ float2 angles[ROT_WARPS][ROT_MAX_DIM / 2];
  __shared__ float gammas[2][ROT_MAX_DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  rot_table(T, P);
  rot_scales(gammas, P);
  const int slots = 32 / team, slot = lane / team, in = lane % team;
  const int qsteps = (P.side[0].heads + slots - 1) / slots, steps = qsteps + (P.side[1].heads + slots - 1) / slots;
  RotPair G[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) G[g].place(in + g * team, P.neighbours, P);
  constexpr int U = NG == 2 ? 4 : NG == 4 ? 2 : 1;             // steps in flight together
  const int64_t units = P.tokens * P.chunks;
  for (int64_t u = (int64_t)blockIdx.x * ROT_WARPS + warp; u < units; u += (int64_t)gridDim.x * ROT_WARPS) {
    const int64_t token = u / P.chunks;
    const int s0 = (int)(u - token * P.chunks) * P.per, s1 = s0 + P.per < steps ? s0 + P.per : steps;
    for (int i = s0; i < s1; i += U) {
      float v[U][NG][2];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int sd = i + j >= qsteps, h = (i + j - sd * qsteps) * slots + slot;
        const RotSide& S = P.side[sd];
        load_pairs(G, S.x, P.x_type, token * S.xt + h * S.xh, i + j < s1 && h < S.heads, v[j]);
      }
      if (i == s0) rot_angles(angles[warp], T, P, token, lane);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (i + j >= s1) break;
        const int sd = i + j >= qsteps, h = (i + j - sd * qsteps) * slots + slot;
        const RotSide& S = P.side[sd];
        float r = 1.0f;
        if (P.rms) {
          float sum = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) sum = fmaf(v[j][g][0], v[j][g][0], fmaf(v[j][g][1], v[j][g][1], sum));
          r = __frsqrt_rn(fmaf(team_sum(sum, team), P.inv_dim, P.eps));
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (P.rms) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (G[g].has[k]) v[j][g][k] = v[j][g][k] * r * gammas[sd][G[g].col[k]];
          }
          G[g].turn(G[g].angle(angles[warp]), v[j][g]);
        }
        if (h < S.heads) store_pairs(G, S.y, P.y_type, token * S.yt + h * S.yh, v[j]);
      }
    }
  }
}

// The backward: the cotangent turned back, then the norm's.  A CTA's dgamma
// sums stay in registers over all its tokens, side after side.
template <int NG>
__global__ void __launch_bounds__(ROT_THREADS, 2) rotary_any_backward_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ RotTable T;
  __shared__ float2 angles[ROT_WARPS][ROT_MAX_DIM / 2];
  __shared__ float gammas[2][ROT_MAX_DIM];
  __shared__ float sums[ROT_WARPS][ROT_MAX_DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  rot_table(T, P);
  rot_scales(gammas, P);
  const int slots = 32 / team, slot = lane / team, in = lane % team;
  RotPair G[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) G[g].place(in + g * team, P.neighbours, P);
  float dg[2][NG][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int g = 0; g < NG; ++g) dg[s][g][0] = dg[s][g][1] = 0.0f;
  for (int64_t token = (int64_t)blockIdx.x * ROT_WARPS + warp; token < P.tokens;
       token += (int64_t)gridDim.x * ROT_WARPS) {
    bool fresh = true;
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const RotSide& S = P.side[sd];
      for (int h = slot; h - slot < S.heads; h += slots) {
        float v[NG][2], x[NG][2];
        load_pairs(G, S.ct, P.ct_type, token * S.ct_t + h * S.ct_h, h < S.heads, v);
        load_pairs(G, S.x, P.x_type, token * S.xt + h * S.xh, P.rms && h < S.heads, x);
        if (fresh) {
          fresh = false;
          rot_angles(angles[warp], T, P, token, lane);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 t = G[g].angle(angles[warp]);
          G[g].turn(make_float2(t.x, -t.y), v[g]);
        }
        if (P.rms) {
          float sum = 0.0f, m = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = G[g].has[k] ? gammas[sd][G[g].col[k]] : 0.0f;
              sum = fmaf(x[g][k], x[g][k], sum);
              m = fmaf(v[g][k] * w, x[g][k], m);
            }
          sum = team_sum(sum, team), m = team_sum(m, team);
          const float r = __frsqrt_rn(fmaf(sum, P.inv_dim, P.eps));
          m = m * r * P.inv_dim;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = G[g].has[k] ? gammas[sd][G[g].col[k]] : 0.0f, xh = x[g][k] * r;
              if (h < S.heads) dg[sd][g][k] = fmaf(v[g][k], xh, dg[sd][g][k]);
              v[g][k] = fmaf(-xh, m, v[g][k] * w) * r;
            }
        }
        if (h < S.heads) store_pairs(G, S.y, P.y_type, token * S.yt + h * S.yh, v);
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
      for (int k = 0; k < 2; ++k)
        for (int o = team; o < 32; o <<= 1) dg[sd][g][k] += __shfl_xor_sync(0xFFFFFFFFu, dg[sd][g][k], o);
    __syncthreads();
    if (slot == 0) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (G[g].has[k]) sums[warp][G[g].col[k]] = dg[sd][g][k];
    }
    rot_part(sums, sd, P);
  }
}

// --------------------------------------- heads of 8-column groups, one type
//
// A lane holds NP pairs of a head (four, or eight where four would need more
// lanes than a warp has), first and second members apart, as float2 for packed
// arithmetic; memory is accessed 8 or 16 bytes at a time and pairs that are
// neighbours come apart as they are widened.  Cosines, sines and scales stand
// in shared memory by pair.  Both kernels walk a token's heads step after step
// (a step: one head a team, in the forward up to four) and have the next steps'
// loads under way while one is worked on, across tokens too.  Four pairs a lane
// rather than eight halve its registers, and the warps that this admits hide the
// latencies of a short pass.

template <int TY, int NP>
struct RotRaw {
  static constexpr int W = TY == PSK_BF16 ? NP : 2 * NP;       // words
  uint32_t w[W];
};

// The pairs' members.
template <int NP>
struct RotPairs {
  float2 a[NP / 2], b[NP / 2];
};

struct RotTables {
  uint64_t turn[ROT_MAX_DIM / 2];                              // as RotTable
  float bad[ROT_MAX_DIM / 2];
  float cosine[ROT_WARPS][ROT_MAX_DIM / 2], sine[ROT_WARPS][ROT_MAX_DIM / 2];
  float gamma[2][2][ROT_MAX_DIM / 2];                          // [side][member][pair]
};

template <bool NEIGH, int NP>
struct RotLane {
  int first[2], pair;                      // the columns of the two runs of NP, the first pair
  bool turns, there;
  __device__ __forceinline__ RotLane(int g, const RotParams& P) {
    pair = NP * g;
    turns = pair < P.rot / 2;
    there = 2 * pair < P.dim;
    if (NEIGH) first[0] = 2 * pair, first[1] = 2 * pair + NP;
    else if (turns) first[0] = pair, first[1] = pair + P.rot / 2;
    else first[0] = P.rot / 2 + pair, first[1] = first[0] + (P.dim - P.rot) / 2;
  }
  // The column of a member of pair `pair + i`.
  __device__ __forceinline__ int column(int member, int i) const {
    return NEIGH ? first[0] + 2 * i + member : first[member] + i;
  }
  template <int TY>
  __device__ __forceinline__ void load(const char* p, bool live, RotRaw<TY, NP>& o) const {
    constexpr int N = RotRaw<TY, NP>::W / 2;           // words of a run
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) o.w[i] = 0;
    if (!live || !there) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const char* q = p + (k ? (first[1] - first[0]) * (TY == PSK_BF16 ? 2 : 4) : 0);
      if constexpr (N == 2) {
        const uint2 u = *(const uint2*)q;
        o.w[2 * k] = u.x, o.w[2 * k + 1] = u.y;
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const uint4 u = *(const uint4*)(q + 4 * i);
          uint32_t* w = o.w + k * N + i;
          w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        }
      }
    }
  }
  template <int TY>
  __device__ __forceinline__ void widen(const RotRaw<TY, NP>& o, RotPairs<NP>& v) const {
    // element e of the lane's 2 NP, in memory order
    const auto at = [&](int e) {
      if constexpr (TY == PSK_BF16) return __uint_as_float(e & 1 ? o.w[e >> 1] & 0xFFFF0000u : o.w[e >> 1] << 16);
      else return __uint_as_float(o.w[e]);
    };
#pragma unroll
    for (int j = 0; j < NP / 2; ++j) {
      v.a[j] = NEIGH ? make_float2(at(4 * j), at(4 * j + 2)) : make_float2(at(2 * j), at(2 * j + 1));
      v.b[j] = NEIGH ? make_float2(at(4 * j + 1), at(4 * j + 3)) : make_float2(at(NP + 2 * j), at(NP + 1 + 2 * j));
    }
  }
  template <int TY>
  __device__ __forceinline__ void store(char* p, const RotPairs<NP>& v) const {
    if (!there) return;
    float e[2 * NP];                                   // in memory order
#pragma unroll
    for (int j = 0; j < NP / 2; ++j) {
      e[NEIGH ? 4 * j : 2 * j] = v.a[j].x, e[NEIGH ? 4 * j + 2 : 2 * j + 1] = v.a[j].y;
      e[NEIGH ? 4 * j + 1 : NP + 2 * j] = v.b[j].x, e[NEIGH ? 4 * j + 3 : NP + 1 + 2 * j] = v.b[j].y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      char* q = p + (k ? (first[1] - first[0]) * (TY == PSK_BF16 ? 2 : 4) : 0);
      const float* w = e + NP * k;
      if constexpr (TY == PSK_F32) {
#pragma unroll
        for (int i = 0; i < NP; i += 4) *(float4*)(q + 4 * i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      } else if constexpr (NP == 4) {
        *(uint2*)q = make_uint2(f32x2_to_bf16x2(w[0], w[1]), f32x2_to_bf16x2(w[2], w[3]));
      } else {
        *(uint4*)q = make_uint4(f32x2_to_bf16x2(w[0], w[1]), f32x2_to_bf16x2(w[2], w[3]), f32x2_to_bf16x2(w[4], w[5]),
                                f32x2_to_bf16x2(w[6], w[7]));
      }
    }
  }
  // NP values of a table by pair.
  __device__ __forceinline__ void of_pairs(const float* table, float2 (&o)[NP / 2]) const {
#pragma unroll
    for (int i = 0; i < NP; i += 4) {
      const float4 x = *(const float4*)(table + pair + i);
      o[i / 2] = make_float2(x.x, x.y), o[i / 2 + 1] = make_float2(x.z, x.w);
    }
  }
};

template <bool NEIGH>
__device__ __forceinline__ void rot_tables(RotTables& T, const RotParams& P) {
  const int half = P.rot / 2, pairs = P.dim / 2;
  // A team of more lanes than the head has groups reads scales past its pairs:
  // zeros, for whatever an earlier kernel left there times zero may be NaN.
  for (int j = pairs + threadIdx.x; j < ROT_MAX_DIM / 2; j += ROT_THREADS)
    T.gamma[0][0][j] = T.gamma[0][1][j] = T.gamma[1][0][j] = T.gamma[1][1][j] = 0.0f;
  for (int j = threadIdx.x; j < pairs; j += ROT_THREADS) {
    if (j < half) {
      const float f = P.tokens ? P.freqs[j] : 0.0f;
      T.turn[j] = turn_fraction(f);
      T.bad[j] = f * 0.0f;
    }
    for (int w = 0; w < ROT_WARPS; ++w) T.cosine[w][j] = 1.0f, T.sine[w][j] = 0.0f;
    for (int s = 0; s < 2; ++s)
      for (int m = 0; m < 2; ++m) {
        const void* g = P.side[s].gamma;
        const int rest = j - half, c = j < half ? (NEIGH ? 2 * j + m : j + m * half)
                                                : (NEIGH ? 2 * j + m : P.rot + rest + m * (pairs - half));
        T.gamma[s][m][j] = !g ? 1.0f
                           : P.gamma_type == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)g)[c])
                                                      : ((const float*)g)[c];
      }
  }
  __syncthreads();
}

__device__ __forceinline__ void rot_angles_at(RotTables& T, const RotParams& P, int64_t pos, int warp, int lane) {
  __syncwarp();
  for (int j = lane; j < P.rot / 2; j += 32) {
    const int64_t frac = (int64_t)((uint64_t)pos * T.turn[j]);
    float s, c;
    sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &s, &c);     // 2 turns 2^-64
    T.cosine[warp][j] = c + T.bad[j], T.sine[warp][j] = s + T.bad[j];
  }
  __syncwarp();
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// A lane's way through one side's heads in one tensor, in bytes: from the
// tensor's beginning to its columns in its first head, from step to step.  The
// launch has seen to it that a token's stretch and the distance of tokens stay
// below 2^31 bytes.
struct RotWalk {
  const char* base;
  uint32_t offset, sub, step, token;       // sub: between the heads of one step
  __device__ __forceinline__ RotWalk(const void* p, int64_t ts, int64_t hs, int slot, int slots, int column, int size,
                                     int subs = 1)
      : base((const char*)p), offset(((uint32_t)hs * slot + column) * size), sub((uint32_t)hs * slots * size), step(sub * subs),
        token((uint32_t)ts * size) {}
  __device__ __forceinline__ const char* at(uint32_t t, int i) const {
    return base + (uint64_t)t * token + (offset + i * step);
  }
};

// 1 / sqrt to 2^-22.9.
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The scale is folded into a token's cosines and sines, once for all its
// heads, so a head's pass is a sum of squares, y = r (x p + x' q) with x' the
// pair's other member, and its loads and stores.  A team works on SUB heads at
// once (a step's bookkeeping serves them all, and their chains of dependent
// operations overlap) while the next AHEAD steps' loads are under way.
template <bool NEIGH, int TY, int NP, int SUB>
__global__ void __launch_bounds__(ROT_THREADS, ROT_FWD_CTAS<TY, SUB>) rotary_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ __align__(16) RotTables T;
  constexpr int SIZE = TY == PSK_BF16 ? 2 : 4, AHEAD = NP == 8 && TY == PSK_BF16 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = 32 / team, slot = lane / team;
  const RotLane<NEIGH, NP> G(lane % team, P);
  // steps of both sides, and those in which this lane's team has a head
  const int nq = (P.side[0].heads + SUB * slots - 1) / (SUB * slots), nk = (P.side[1].heads + SUB * slots - 1) / (SUB * slots);
  int lq[SUB], lk[SUB];
#pragma unroll
  for (int j = 0; j < SUB; ++j) {
    lq[j] = (P.side[0].heads - slot - j * slots + SUB * slots - 1) / (SUB * slots);
    lk[j] = (P.side[1].heads - slot - j * slots + SUB * slots - 1) / (SUB * slots);
  }
  const uint32_t jump = gridDim.x * ROT_WARPS, units = (uint32_t)P.tokens * P.chunks;
  const auto walk = [&](int sd, bool y) {
    const RotSide& S = P.side[sd];
    return y ? RotWalk(S.y, S.yt, S.yh, slot, slots, G.first[0], SIZE, SUB) : RotWalk(S.x, S.xt, S.xh, slot, slots, G.first[0], SIZE, SUB);
  };
  const RotWalk Xq = walk(0, false), Xk = walk(1, false), Yq = walk(0, true), Yk = walk(1, true);
  // What is fetched next: step `fi` of unit `fu` (token `ft`), a unit being a
  // token's steps [s0, s0 + per) of both sides, queries first.
  uint32_t fu = blockIdx.x * ROT_WARPS + warp, ft = 0;
  int fi = 0, fend = 0;
  const auto enter = [&]() {
    if (fu >= units) return;
    if (P.chunks == 1) {
      ft = fu, fi = 0, fend = nq + nk;
    } else {
      ft = fu / (uint32_t)P.chunks, fi = (int)(fu - ft * P.chunks) * P.per;
      fend = fi + P.per < nq + nk ? fi + P.per : nq + nk;
    }
  };
  RotRaw<TY, NP> raw[AHEAD][SUB];
  const auto fetch = [&](RotRaw<TY, NP> (&o)[SUB]) {
    if (fu >= units) return;
    if (fi < nq) {
      const char* p = Xq.at(ft, fi);
#pragma unroll
      for (int j = 0; j < SUB; ++j) G.load(p + (uint32_t)(j * Xq.sub), fi < lq[j], o[j]);
    } else {
      const char* p = Xk.at(ft, fi - nq);
#pragma unroll
      for (int j = 0; j < SUB; ++j) G.load(p + (uint32_t)(j * Xk.sub), fi - nq < lk[j], o[j]);
    }
    if (++fi == fend) fu += jump, enter();
  };
  enter();
  int64_t pos = fu < units ? rot_position(P, ft) : 0;
  uint32_t u = fu;
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) fetch(raw[j]);
  rot_tables<NEIGH>(T, P);
  uint32_t token = 0;
  int i = 0, end = 0;
  bool fresh = true, keys = false;
  float2 pa[NP / 2], qa[NP / 2], pb[NP / 2], qb[NP / 2];
  while (u < units) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (u >= units) break;
      RotPairs<NP> v[SUB];
#pragma unroll
      for (int h = 0; h < SUB; ++h) G.widen(raw[j][h], v[h]);
      fetch(raw[j]);
      if (fresh) {
        if (P.chunks == 1) token = u, i = 0, end = nq + nk;
        else {
          token = u / (uint32_t)P.chunks, i = (int)(u - token * P.chunks) * P.per;
          end = i + P.per < nq + nk ? i + P.per : nq + nk;
        }
        rot_angles_at(T, P, pos, warp, lane);
        if (u + jump < units) pos = rot_position(P, P.chunks == 1 ? u + jump : (u + jump) / (uint32_t)P.chunks);
      }
      if (fresh || (i >= nq) != keys) {
        fresh = false, keys = i >= nq;
        float2 c[NP / 2], s[NP / 2], ga[NP / 2], gb[NP / 2];
        G.of_pairs(T.cosine[warp], c), G.of_pairs(T.sine[warp], s);
        G.of_pairs(T.gamma[keys][0], ga), G.of_pairs(T.gamma[keys][1], gb);
#pragma unroll
        for (int m = 0; m < NP / 2; ++m) {
          pa[m] = __fmul2_rn(ga[m], c[m]), pb[m] = __fmul2_rn(gb[m], c[m]);
          qa[m] = __fmul2_rn(gb[m], make_float2(-s[m].x, -s[m].y)), qb[m] = __fmul2_rn(ga[m], s[m]);
        }
      }
      float2 r[SUB];
#pragma unroll
      for (int h = 0; h < SUB; ++h) r[h] = splat(1.0f);
      if (P.rms) {
        float sums[SUB];
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
          float2 sum = splat(0.0f);
#pragma unroll
          for (int m = 0; m < NP / 2; ++m) sum = __ffma2_rn(v[h].a[m], v[h].a[m], __ffma2_rn(v[h].b[m], v[h].b[m], sum));
          sums[h] = sum.x + sum.y;
        }
        for (int o = team >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int h = 0; h < SUB; ++h) sums[h] += __shfl_xor_sync(0xFFFFFFFFu, sums[h], o);
#pragma unroll
        for (int h = 0; h < SUB; ++h) r[h] = splat(rsqrt_approx(fmaf(sums[h], P.inv_dim, P.eps)));
      }
#pragma unroll
      for (int h = 0; h < SUB; ++h)
#pragma unroll
        for (int m = 0; m < NP / 2; ++m) {
          const float2 a = __fmul2_rn(v[h].a[m], r[h]), b = __fmul2_rn(v[h].b[m], r[h]);
          v[h].a[m] = __fmul2_rn(a, pa[m]), v[h].b[m] = __fmul2_rn(b, pb[m]);
          if (G.turns) v[h].a[m] = __ffma2_rn(b, qa[m], v[h].a[m]), v[h].b[m] = __ffma2_rn(a, qb[m], v[h].b[m]);
        }
      if (keys) {
        char* p = (char*)Yk.at(token, i - nq);
#pragma unroll
        for (int h = 0; h < SUB; ++h)
          if (i - nq < lk[h]) G.template store<TY>(p + (uint32_t)(h * Yk.sub), v[h]);
      } else {
        char* p = (char*)Yq.at(token, i);
#pragma unroll
        for (int h = 0; h < SUB; ++h)
          if (i < lq[h]) G.template store<TY>(p + (uint32_t)(h * Yq.sub), v[h]);
      }
      if (++i == end) u += jump, fresh = true;
    }
  }
}

template <bool NEIGH, int TY, int NP>
__global__ void __launch_bounds__(ROT_THREADS, NP == 4 ? ROT_BWD_CTAS : 2) rotary_backward_kernel(const __grid_constant__ RotParams P, int team) {
  __shared__ __align__(16) RotTables T;
  __shared__ float sums[ROT_WARPS][ROT_MAX_DIM];
  constexpr int SIZE = TY == PSK_BF16 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = 32 / team, slot = lane / team;
  const RotLane<NEIGH, NP> G(lane % team, P);
  const int nq = (P.side[0].heads + slots - 1) / slots, nk = (P.side[1].heads + slots - 1) / slots;
  const int lq = (P.side[0].heads - slot + slots - 1) / slots, lk = (P.side[1].heads - slot + slots - 1) / slots;
  const uint32_t jump = gridDim.x * ROT_WARPS, tokens = (uint32_t)P.tokens;
  uint32_t token = blockIdx.x * ROT_WARPS + warp;
  RotPairs<NP> dg[2];
#pragma unroll
  for (int j = 0; j < NP / 2; ++j) dg[0].a[j] = dg[0].b[j] = dg[1].a[j] = dg[1].b[j] = splat(0.0f);
  RotRaw<TY, NP> craw, xraw;
  const auto walk = [&](int sd, int which) {
    const RotSide& S = P.side[sd];
    if (which == 0) return RotWalk(S.ct, S.ct_t, S.ct_h, slot, slots, G.first[0], SIZE);
    if (which == 1) return RotWalk(S.x, S.xt, S.xh, slot, slots, G.first[0], SIZE);
    return RotWalk(S.y, S.yt, S.yh, slot, slots, G.first[0], SIZE);
  };
  const auto first = [&](int sd, uint32_t t) {
    G.load(walk(sd, 0).at(t, 0), 0 < (sd ? lk : lq), craw);
    G.load(walk(sd, 1).at(t, 0), P.rms && 0 < (sd ? lk : lq), xraw);
  };
  if (token < tokens) {
    if (nq) first(0, token);
    else first(1, token);
  }
  rot_tables<NEIGH>(T, P);
  int64_t pos = token < tokens ? rot_position(P, token) : 0;
  for (; token < tokens; token += jump) {
    rot_angles_at(T, P, pos, warp, lane);
    if (token + jump < tokens) pos = rot_position(P, token + jump);
    float2 c[NP / 2], s[NP / 2];
    G.of_pairs(T.cosine[warp], c), G.of_pairs(T.sine[warp], s);
    const auto side = [&](auto SD) {
      constexpr int sd = SD.value;
      const int n = sd ? nk : nq, mine = sd ? lk : lq;
      if (!n) return;
      const RotWalk C = walk(sd, 0), X = walk(sd, 1), Y = walk(sd, 2);
      const char *pc = C.at(token, 0), *px = X.at(token, 0);
      char* py = (char*)Y.at(token, 0);
      for (int i = 0; i < n; ++i) {
        RotPairs<NP> v, x;
        G.widen(craw, v), G.widen(xraw, x);
        // the next step's, the other side's first, or the next token's
        if (i + 1 < n) {
          pc += C.step, px += X.step;
          G.load(pc, i + 1 < mine, craw);
          G.load(px, P.rms && i + 1 < mine, xraw);
        } else if (sd == 0 && nk) {
          first(1, token);
        } else if (token + jump < tokens) {
          if (nq) first(0, token + jump);
          else first(1, token + jump);
        }
        if (G.turns) {
#pragma unroll
          for (int j = 0; j < NP / 2; ++j) {
            const float2 a = v.a[j], b = v.b[j];
            v.a[j] = __ffma2_rn(a, c[j], __fmul2_rn(b, s[j]));
            v.b[j] = __ffma2_rn(b, c[j], __fmul2_rn(a, make_float2(-s[j].x, -s[j].y)));
          }
        }
        if (P.rms) {
          float2 ga[NP / 2], gb[NP / 2], sum = splat(0.0f), m = splat(0.0f);
          G.of_pairs(T.gamma[sd][0], ga), G.of_pairs(T.gamma[sd][1], gb);
#pragma unroll
          for (int j = 0; j < NP / 2; ++j) {
            ga[j] = __fmul2_rn(v.a[j], ga[j]), gb[j] = __fmul2_rn(v.b[j], gb[j]);
            sum = __ffma2_rn(x.a[j], x.a[j], __ffma2_rn(x.b[j], x.b[j], sum));
            m = __ffma2_rn(ga[j], x.a[j], __ffma2_rn(gb[j], x.b[j], m));
          }
          float s1 = sum.x + sum.y, s2 = m.x + m.y;
          for (int o = team >> 1; o > 0; o >>= 1) {
            s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
            s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
          }
          const float r = rsqrt_approx(fmaf(s1, P.inv_dim, P.eps));
          const float2 r2 = splat(r), mean = splat(-(s2 * r * P.inv_dim));
#pragma unroll
          for (int j = 0; j < NP / 2; ++j) {
            const float2 xa = __fmul2_rn(x.a[j], r2), xb = __fmul2_rn(x.b[j], r2);
            if (i < mine) {
              dg[sd].a[j] = __ffma2_rn(v.a[j], xa, dg[sd].a[j]);
              dg[sd].b[j] = __ffma2_rn(v.b[j], xb, dg[sd].b[j]);
            }
            v.a[j] = __fmul2_rn(__ffma2_rn(xa, mean, ga[j]), r2);
            v.b[j] = __fmul2_rn(__ffma2_rn(xb, mean, gb[j]), r2);
          }
        }
        if (i < mine) G.template store<TY>(py, v);
        py += Y.step;
      }
    };
    side(std::integral_constant<int, 0>{});
    side(std::integral_constant<int, 1>{});
  }
  if (!P.part) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
    // teams of a warp joined by shuffles, warps through shared memory
    const auto join = [&](float v) {
      for (int o = team; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    };
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 da = dg[sd].a[i >> 1], db = dg[sd].b[i >> 1];
      const float a = join(i & 1 ? da.y : da.x), b = join(i & 1 ? db.y : db.x);
      if (slot == 0 && G.there) sums[warp][G.column(0, i)] = a, sums[warp][G.column(1, i)] = b;
    }
    rot_part(sums, sd, P);
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

// Whether a token's stretch and the distance of tokens stay below 2^31 bytes.
static bool heads_near(const Heads& h) {
  const int64_t most = (1LL << 31) / dtype_size(h.dt) - 1;
  return !h.there() || ((h.tokens <= 1 || h.ts <= most) && h.of_token() <= most - 32 * (h.heads > 1 ? h.hs : 0));
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

// The fast kernels' groups of columns, of four pairs or eight.
static int rot_group(int64_t dim, int64_t rot) {
  if (dim <= 256) return dim % 8 == 0 && rot % 8 == 0 ? 4 : 0;
  return dim % 16 == 0 && rot % 16 == 0 ? 8 : 0;
}

// Lanes of a team (a power of two): one for each group of V pairs, a warp at most.
static int rot_team(const RotParams& P, int V) {
  const int pairs = P.rot / 2 + (P.dim - P.rot + 1) / 2, groups = (pairs + V - 1) / V;
  int t = 1;
  while (t < 32 && t < groups) t *= 2;
  return t;
}

// Pairs a lane of the general kernels: as many as the head needs, two at least
// in the forward and four in the backward (fewer lanes a head and more heads a
// warp save instructions: [16384, 6 + 6, 50] bf16 with one, two and four pairs
// 50, 39 and 42 us forward, 102, 88 and 77 backward; 33 and 68 since a head's
// type is looked up once and not for every element).
template <int LEAST, typename F>
static int rot_pairs(const RotParams& P, F&& f) {
  const int pairs = P.rot / 2 + (P.dim - P.rot + 1) / 2;
  using std::integral_constant;
  if constexpr (LEAST <= 2)
    if (pairs <= 64) return f(integral_constant<int, 2>{});
  if (pairs <= 128) return f(integral_constant<int, 4>{});
  return f(integral_constant<int, 8>{});
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
  const int np = rot_group(dim, rot);
  const bool vec = np && tokens * (hq + hk) < 1LL << 31 && heads_near(in[0]) && heads_near(in[1]) &&
                   heads_near(out[0]) && heads_near(out[1]) && heads_vec(in[0]) && heads_vec(in[1]) && heads_vec(out[0]) && heads_vec(out[1]);
  cudaStream_t s = (cudaStream_t)stream;
  const bool fast = vec && xt == yt;
  const int team = rot_team(P, fast ? np : rot_pairs<2>(P, [](auto NG) { return (int)NG.value; })), teams = 32 / team;
  // Heads a team takes at once: two, or four of bf16 where no more of them are
  // left empty ([4096, 32 + 8, 128] bf16: one 21.8 us, two 18.9, four 15.4;
  // [16384, 4 + 1, 256] 19.5, 18.7, 21.7; [16384, 32 + 4, 64] f32 64, 50).
  const auto padded = [&](int64_t n) { return ((hq + n - 1) / n + (hk + n - 1) / n) * n; };
  const int subs = !fast || np == 8 ? 1 : xt == PSK_BF16 && padded(4 * teams) <= padded(2 * teams) ? 4 : 2;
  const int slots = teams * subs, per_sm = !fast || (xt == PSK_BF16 && subs == 2) ? 3 : 2;
  const int64_t steps = (hq + slots - 1) / slots + (hk + slots - 1) / slots;
  const int64_t most = (int64_t)device_sm_count() * per_sm, warps = most * ROT_WARPS;
  // A token's heads go to one warp where tokens alone fill the GPU, else to several.
  int64_t chunks = tokens >= warps ? 1 : (warps + tokens - 1) / tokens;
  if (chunks > steps) chunks = steps;
  P.per = (int32_t)((steps + chunks - 1) / chunks);
  P.chunks = (int32_t)((steps + P.per - 1) / P.per);
  const int64_t ctas = (tokens * P.chunks + ROT_WARPS - 1) / ROT_WARPS;
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  if (fast)
    with_dtype(xt, [&](auto TY) {
      return with_bool(P.neighbours != 0, [&](auto N) {
        if (subs == 1) rotary_kernel<N.value, TY.value, 8, 1><<<grid, ROT_THREADS, 0, s>>>(P, team);
        else if (subs == 2) rotary_kernel<N.value, TY.value, 4, 2><<<grid, ROT_THREADS, 0, s>>>(P, team);
        else rotary_kernel<N.value, PSK_BF16, 4, 4><<<grid, ROT_THREADS, 0, s>>>(P, team);
        return 0;
      });
    });
  else
    rot_pairs<2>(P, [&](auto NG) {
      rotary_any_kernel<NG.value><<<grid, ROT_THREADS, 0, s>>>(P, team);
      return 0;
    });
  return check_launch("rotary kernel");
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
  const int np = rot_group(dim, rot);
  const bool vec = np && tokens * (hq + hk) < 1LL << 31 && heads_near(cts[0]) && heads_near(cts[1]) &&
                   heads_near(out[0]) && heads_near(out[1]) && heads_near(xs[0]) && heads_near(xs[1]) && heads_vec(cts[0]) && heads_vec(cts[1]) && heads_vec(out[0]) &&
                   heads_vec(out[1]) && (!rms || (heads_vec(xs[0]) && heads_vec(xs[1])));
  cudaStream_t s = (cudaStream_t)stream;
  const bool fast = vec && ct == dt && (!rms || xt == ct);
  const int team = rot_team(P, fast ? np : rot_pairs<4>(P, [](auto NG) { return (int)NG.value; }));
  const int64_t most = (int64_t)device_sm_count() * (fast && np == 4 ? ROT_BWD_CTAS : 2);
  if (P.blocks > most) P.blocks = (int32_t)most;
  const unsigned grid = (unsigned)P.blocks;
  if (fast)
    with_dtype(ct, [&](auto TY) {
      return with_bool(P.neighbours != 0, [&](auto N) {
        if (np == 4) rotary_backward_kernel<N.value, TY.value, 4><<<grid, ROT_THREADS, 0, s>>>(P, team);
        else rotary_backward_kernel<N.value, TY.value, 8><<<grid, ROT_THREADS, 0, s>>>(P, team);
        return 0;
      });
    });
  else
    rot_pairs<4>(P, [&](auto NG) {
      rotary_any_backward_kernel<NG.value><<<grid, ROT_THREADS, 0, s>>>(P, team);
      return 0;
    });
  rc = check_launch("rotary backward kernel");
  if (rc || !sums) return rc;
  rotary_join_kernel<<<dim3((unsigned)((dim + 31) / 32), 2), 1024, 0, s>>>(P);
  return check_launch("rotary join kernel");
}
