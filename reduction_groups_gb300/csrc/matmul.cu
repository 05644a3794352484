// D = A B of 16-bit operands (bf16 or fp16) on the tensor cores with f32
// accumulators, and the epilogues of the linear layer and of the
// orthogonalised update.
//
// One persistent CTA (or pair of CTAs, CG = 2) an SM takes output tiles in
// turn.  Warp 0 fills a ring of shared-memory stages by TMA (64 summed
// elements of both operands, 128-byte swizzled), warp 1 issues tcgen05.mma
// from one thread into one of two accumulators in TMEM, the warps from 4 on take
// finished accumulators out of TMEM and run the epilogue on them while the
// next tile's products are running.  A pair shares one tile of 256 rows: each
// CTA brings half of A's rows and half of B's columns, the first issues the
// products for both.
//
// Either operand may lie with the summed direction contiguous (K-major) or
// the other one (MN-major): the shared-memory descriptors and the bit in the
// instruction descriptor say which, so no operand is transposed in memory.
//
// f32 operands come as planes of 16-bit parts; the launch lists the products
// of planes to be added, the smallest first: a stage holds every plane of its
// part of the summed axis, the products of planes but the last go into an
// accumulator of their own.
//
// The tensor core's additions truncate, so sums of f32 operands, and long ones
// of 16-bit operands, leave their accumulators piece by piece and are added up
// in the epilogue warps' registers (MM_PARTS, MM_PIECES; [8192, 4096] x 4096,
// f32 result, by pieces: 188 us under ncu, tensor pipe 63 % of cycles, as with
// whole sums of bf16 results).
//
// Every wait is bounded: a role that gives up records it in the device status
// and leaves its loop, all meet at the end of the kernel.
#include <cuda.h>

#include "common.cuh"
#include "pipe.cuh"
#include "vec8.cuh"
#include "act.cuh"
#include "tensor.cuh"
#include "mm.h"
#include "trainops.h"

namespace psk {

// How a tile's sum is taken (SUM): whole, in one accumulator; by pieces of the
// summed axis, which the epilogue's warps add up in registers; or by pieces of
// the products of several planes, the smaller ones in an accumulator beside.
constexpr int MM_WHOLE = 0, MM_PIECES = 1, MM_PARTS = 2;

// Warps of the epilogue: sixteen, or eight where each keeps its sums in registers.
template <int SUM>
struct MMWarps {
  static constexpr int EPI = SUM ? 8 : 16, THREADS = 128 + 32 * EPI;
};
constexpr int MM_A_BYTES = 128 * MM_BK * 2;

struct MMProblem {
  CUtensorMap ta, tb;
  MMEpilogue e;
  int64_t m, n;
  int32_t kblocks, pairs, planes_a, planes_b;
  int32_t chunk;                           // blocks of the summed axis that one accumulator takes
  int32_t na, nb;                          // planes of A and B in a stage (one each but with MM_PARTS)
  int32_t a_k, b_k, tiles_m, tiles_n, tiles, symmetric;      // tiles: of one matrix
  uint8_t pa[8], pb[8];
};

// One launch: one product or two, the second's tiles after the first's.
struct MMParams {
  MMProblem q[2];
  int32_t split, total;                    // tiles of the first, of both
  int32_t f16, stages, slot_bytes;         // of the ring
  MMColumnSums sums;
};

// --------------------------------------------------------------- tile order

struct Tile {
  int32_t matrix, tm, tn;
};

// Tiles of one matrix after another's; within one, groups of eight tile rows
// walk through the columns together, so that the tiles running at one time
// share operand rows in L2.  Symmetric: the lower triangle, row after row.
template <int Q>
__device__ __forceinline__ Tile tile_at(const MMProblem& P, int32_t t) {
  Tile o;
  const int32_t per = P.tiles;
  o.matrix = t / per;
  t -= o.matrix * per;
  if (P.symmetric) {
    // row i of tiles has q (i + 1) of them, q = BM / BN (the last may have fewer)
    const int32_t u = t / Q;
    int32_t i = (int32_t)((sqrtf(8.0f * (float)u + 1.0f) - 1.0f) * 0.5f);
    while ((int64_t)i * (i + 1) / 2 > u) --i;
    while ((int64_t)(i + 1) * (i + 2) / 2 <= u) ++i;
    o.tm = i, o.tn = t - (int32_t)((int64_t)i * (i + 1) / 2) * Q;
    return o;
  }
  const int32_t band = 8 * P.tiles_n, g = t / band, first = g * 8;
  const int32_t rows = P.tiles_m - first < 8 ? P.tiles_m - first : 8;
  const int32_t in = t - g * band;
  o.tm = first + in % rows, o.tn = in / rows;
  return o;
}

// ----------------------------------------------------------------- epilogue

__device__ __forceinline__ void store8_rt(void* p, int32_t dt, int64_t i, int n, bool vec, const float* v) {
  if (dt == PSK_BF16) {
    uint16_t* q = (uint16_t*)p + i;
    if (vec && n >= 8) {
      *(uint4*)q = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                              f32x2_to_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = f32_to_bf16_bits(v[k]);
    }
  } else {
    float* q = (float*)p + i;
    if (vec && n >= 8) {
      *(float4*)q = make_float4(v[0], v[1], v[2], v[3]);
      *(float4*)(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = v[k];
    }
  }
}

__device__ __forceinline__ void store1_rt(void* p, int32_t dt, int64_t i, float v) {
  if (dt == PSK_BF16) ((uint16_t*)p)[i] = f32_to_bf16_bits(v);
  else ((float*)p)[i] = v;
}

// Sixteen bf16 of a 32-byte aligned row: one sector an access, so that lanes
// on different rows fetch and write whole sectors.  The reads leave L1 alone,
// whose 30 KB beside the ring hold few such rows' lines (22 orthogonalised
// 2048 x 2048 bf16 on one machine: 3247 us without the hint, 3092 with it).
__device__ __forceinline__ void load16_bf16(const void* p, int64_t i, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"((const uint16_t*)p + i));
}
__device__ __forceinline__ void store16(void* p, int64_t i, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"((uint16_t*)p + i), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store16_bf16(void* p, int64_t i, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = f32x2_to_bf16x2(v[2 * k], v[2 * k + 1]);
  store16(p, i, w);
}

// Sixteen columns of a half warp's sixteen rows turned: lane l of a half gets
// column l of its rows.  Four exchanges, of lanes 8, 4, 2 and 1 apart.
__device__ __forceinline__ void turn16(float* v, int lane) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k & d) continue;
      const float give = up ? v[k] : v[k + d], got = __shfl_xor_sync(0xFFFFFFFFu, give, d);
      if (up) v[k] = got;
      else v[k + d] = got;
    }
  }
}

template <int ACT, bool FINE, int N>
__device__ __forceinline__ void act_all(float* v) {
  if constexpr (ACT != ACT_NONE) {
    if constexpr (ACT == ACT_SILU) {       // one test for all: values this far out are rare
      float low = v[0];
#pragma unroll
      for (int k = 1; k < N; ++k) low = fminf(low, v[k]);
      if (low < SILU_FAR) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          v[k] = v[k] < SILU_FAR ? silu_far(v[k]) : act_value<ACT, FINE>(make_float2(v[k], v[k])).x;
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const float2 a = act_value<ACT, FINE>(make_float2(v[k], v[k + 1]));
      v[k] = a.x, v[k + 1] = a.y;
    }
  }
}

__device__ __forceinline__ float load1_rt(const void* p, int32_t dt, int64_t i) {
  return dt == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

template <int N>
__device__ __forceinline__ void act_rt(float* v, int32_t act) {
  switch (act) {
    case ACT_RELU: act_all<ACT_RELU, true, N>(v); break;
    case ACT_GELU: act_all<ACT_GELU, true, N>(v); break;
    case ACT_SILU: act_all<ACT_SILU, true, N>(v); break;
    default: break;
  }
}

// Eight elements `step` bytes apart, those below n.
template <int DT>
__device__ __forceinline__ void gather8(const char* p, int64_t step, int n, float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k, p += step) {
    v[k] = 0.0f;
    if (k < n) v[k] = DT == PSK_BF16 ? bf16_bits_to_f32(*(const uint16_t*)p) : *(const float*)p;
  }
}
template <int DT>
__device__ __forceinline__ void scatter8(char* p, int64_t step, int n, const float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k, p += step)
    if (k < n) {
      if (DT == PSK_BF16) *(uint16_t*)p = f32_to_bf16_bits(v[k]);
      else *(float*)p = v[k];
    }
}
__device__ __forceinline__ void scatter8_rt(void* p, int32_t dt, int64_t i, int64_t ld, int n, const float* v) {
  if (dt == PSK_BF16) scatter8<PSK_BF16>((char*)p + 2 * i, 4 * ld, n, v);
  else scatter8<PSK_F32>((char*)p + 4 * i, 8 * ld, n, v);
}

// Sixteen columns of a warp's 32 rows, of any types and strides: turned
// through shared memory, so that lanes hold neighbouring columns (two rows at
// a time) and what they load and store is coalesced wherever rows begin.  Few
// instructions: in a small call a warp is alone on its scheduler, each costs
// its latency (unrolled throughout and with types and bounds looked up for
// every element, a tile of [1003, 771] x [771, 1501] f32 spent 10 us here).
__device__ __forceinline__ void linear_any16(const MMProblem& P, int64_t row0, int64_t c0, int lane, float* stage,
                                             const float* v) {
  const MMEpilogue& E = P.e;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 16; ++k) stage[lane * 17 + k] = v[k];
  __syncwarp();
  const int64_t c = c0 + (lane & 15);
  if (c >= P.n) return;
  const float bias = E.bias ? load1_rt(E.bias, E.bt, c) : 0.0f;
  const float* from = stage + (lane >> 4) * 17 + (lane & 15);
  int64_t r = row0 + (lane >> 4);
#pragma unroll 1
  for (int half = 0; half < 2; ++half, r += 16, from += 16 * 17) {     // eight rows, two apart
    const int n = P.m - r >= 16 ? 8 : P.m > r ? (int)((P.m - r + 1) / 2) : 0;
    float t[8], res[8];
    if (E.res) {
      if (E.rt == PSK_BF16) gather8<PSK_BF16>((const char*)E.res + 2 * (r * E.ldr + c), 4 * E.ldr, n, res);
      else gather8<PSK_F32>((const char*)E.res + 4 * (r * E.ldr + c), 8 * E.ldr, n, res);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = from[2 * k * 17] + bias;
    if (E.z) scatter8_rt(E.z, E.zt, r * E.ldz + c, E.ldz, n, t);
    act_rt<8>(t, E.act);
    if (E.res) {
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] += res[k];
    }
    scatter8_rt(E.y, E.yt, r * E.ldy + c, E.ldy, n, t);
  }
}

// What the epilogue of 16 columns reads from memory, fetched while the
// columns before them are worked on: the residual and the bias (both bf16,
// on 32-byte boundaries), or the two parts of the update's own term.
struct Fetched {
  uint32_t a[8], b[8];
};

__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], float* t) {
#pragma unroll
  for (int k = 0; k < 8; ++k) t[2 * k] = __uint_as_float(w[k] << 16), t[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
}
__device__ __forceinline__ void add16(const uint32_t (&w)[8], float* v) {
  float t[16];
  unpack16(w, t);
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const float2 s = __fadd2_rn(make_float2(v[k], v[k + 1]), make_float2(t[k], t[k + 1]));
    v[k] = s.x, v[k + 1] = s.y;
  }
}

// Sixteen columns of one row, every matrix in bf16 with 32-byte aligned rows.
template <int ACT>
__device__ __forceinline__ void linear_row16(const MMEpilogue& E, int64_t r, int64_t c, const Fetched& F, float* v) {
  if (E.bias) add16(F.b, v);
  if (E.z) store16_bf16(E.z, r * E.ldz + c, v);
  act_all<ACT, false, 16>(v);
  if (E.res) add16(F.a, v);
  store16_bf16(E.y, r * E.ldy + c, v);
}

// Sixteen columns of a warp's rows of the orthogonalised update: v = alpha v +
// beta from, stored in fp16 planes (and mirrored) or into a leaf.  The planes'
// rows are padded to 32 bytes; their padding may be written.
__device__ __forceinline__ void ortho_row16(const MMProblem& P, int32_t matrix, int64_t row0, int lane, int64_t c,
                                            bool mirrored, const Fetched& F, float* v) {
  const int64_t r = row0 + lane;
  const bool live = r < P.m;
  const MMEpilogue& E = P.e;
  const int64_t at = (int64_t)matrix * E.planes * E.plane_stride;
  const int64_t left = P.n - c;
  const float2 alpha = pair_of(E.alpha), beta = pair_of(E.beta);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float2 x = __fmul2_rn(make_float2(v[2 * k], v[2 * k + 1]), alpha);
    if (E.from) {
      if (E.planes == 2) x = __ffma2_rn(beta, f16x2_to_f32(F.b[k]), x);
      x = __ffma2_rn(beta, f16x2_to_f32(F.a[k]), x);
    }
    v[2 * k] = x.x, v[2 * k + 1] = x.y;
  }
  if (E.to) {
    if (!live) return;
    for (int p = 0; p < E.planes; ++p) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k] = f32x2_to_f16x2(v[2 * k], v[2 * k + 1]);
        const float2 h = f16x2_to_f32(w[k]);
        v[2 * k] -= h.x, v[2 * k + 1] -= h.y;
      }
      uint16_t* to = E.to + at + p * E.plane_stride;
      store16(to, r * E.ld + c, w);
      if (mirrored) {
        uint16_t* o = to + c * E.ld + r;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k < left) o[(int64_t)k * E.ld] = (uint16_t)(k & 1 ? w[k >> 1] >> 16 : w[k >> 1]);
      }
    }
    return;
  }
  const MMLeaf L = E.leaves[matrix];
  if (!E.transposed && !L.vec) {           // rows that begin anywhere: lanes along them
    turn16(v, lane);
    const int64_t col = c + (lane & 15), first = row0 + (lane & 16);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (first + k < P.m && col < P.n) store1_rt(L.y, E.yt, (first + k) * L.ld + col, v[k]);
    return;
  }
  if (!live) return;
  if (E.transposed) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < left) store1_rt(L.y, E.yt, (c + k) * L.ld + r, v[k]);
  } else {
#pragma unroll
    for (int h = 0; h < 16; h += 8)
      if (h < left) store8_rt(L.y, E.yt, r * L.ld + c + h, left - h < 8 ? (int)(left - h) : 8, L.vec != 0, v + h);
  }
}

template <int KIND>
__device__ __forceinline__ void fetch16(const MMProblem& P, int32_t matrix, int64_t r, int64_t c, Fetched& F) {
  const MMEpilogue& E = P.e;
  if (KIND == MM_ANY || r >= P.m || c >= P.n) return;
  if constexpr (KIND == MM_ORTHO) {
    if (!E.from) return;
    const uint16_t* from = E.from + (int64_t)matrix * E.planes * E.plane_stride + r * E.ld + c;
    load16_bf16(from, 0, F.a);
    if (E.planes == 2) load16_bf16(from, E.plane_stride, F.b);
  } else {
    if (E.res) load16_bf16(E.res, r * E.ldr + c, F.a);
    if (E.bias) load16_bf16(E.bias, c, F.b);
  }
}

// The epilogue of 16 neighbouring accumulators, from column c on, of row0 + lane.
template <int KIND>
__device__ __forceinline__ void finish16(const MMProblem& P, int32_t matrix, int64_t row0, int lane, int64_t c,
                                         bool mirrored, const Fetched& F, float* stage, float* v) {
  if (c >= P.n) return;
  if constexpr (KIND == MM_ANY) {
    linear_any16(P, row0, c, lane, stage, v);
  } else if constexpr (KIND == MM_ORTHO) {
    ortho_row16(P, matrix, row0, lane, c, mirrored, F, v);
  } else if (row0 + lane < P.m) {
    linear_row16<KIND>(P.e, row0 + lane, c, F, v);
  }
}

// Columns first, first + step, ... of the sums.
__device__ __forceinline__ void column_sums(const MMColumnSums& J, int64_t first, int64_t step) {
  if (!J.out) return;
  for (int64_t c = first; c < J.cols; c += step) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int b = 0;
    for (; b + 4 <= J.blocks; b += 4)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += J.parts[(int64_t)(b + i) * J.cols + c];
    for (; b < J.blocks; ++b) s[0] += J.parts[(int64_t)b * J.cols + c];
    const float v = (s[0] + s[1]) + (s[2] + s[3]);
    if (J.dt == PSK_BF16) {
      uint16_t* q = (uint16_t*)J.out + c;
      *q = f32_to_bf16_bits(J.add ? bf16_bits_to_f32(*q) + v : v);
    } else {
      float* q = (float*)J.out + c;
      *q = J.add ? *q + v : v;
    }
  }
}

// ------------------------------------------------------------------- kernel

// KIND: an activation with every matrix in bf16, 32-byte aligned rows and n a
// multiple of 16; MM_ANY: the linear layer with any types; MM_ORTHO.
template <int CG, int BN, int KIND, int SUM>
struct MMShape {
  static constexpr bool PARTS = SUM == MM_PARTS;
  static constexpr int BM = 128 * CG;
  static constexpr int B_ROWS = BN / CG;                        // of B's tile in one CTA
  static constexpr int B_BYTES = B_ROWS * MM_BK * 2;
  static constexpr int STAGE = MM_A_BYTES + B_BYTES;            // of one plane each
  static constexpr int TURN = KIND == MM_ANY ? MMWarps<SUM>::EPI * 32 * 17 * 4 : 0;     // of the epilogue
  static constexpr int STAGES = (225 * 1024 - TURN) / STAGE < 8 ? (225 * 1024 - TURN) / STAGE : 8;
  static constexpr int RING = PARTS ? (225 * 1024 - TURN) / 1024 * 1024 : STAGES * STAGE;
  static constexpr int SMEM = RING + TURN + 1024;               // and what aligns the ring to 1024 bytes
  // Columns of one accumulator: the last product of planes has its own, beside
  // that of the others.
  static constexpr int ACC = PARTS ? 2 * BN : BN;
};

template <int CG, int BN, int KIND, int SUM, int COUNT>
__global__ void __launch_bounds__(MMWarps<SUM>::THREADS, 1) mm_kernel(const __grid_constant__ MMParams G) {
  using S = MMShape<CG, BN, KIND, SUM>;
  constexpr bool PARTS = S::PARTS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[S::STAGES], empty[S::STAGES], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int32_t first = blockIdx.x / CG, step = gridDim.x / CG;
  const int32_t total = G.total;
  const int stages = PARTS ? G.stages : S::STAGES;
  const uint32_t slot_bytes = PARTS ? G.slot_bytes : S::STAGE;

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], MMWarps<SUM>::EPI * CG);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<CG>(&tmem_slot, 2 * S::ACC);
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // set up beside the kernel before it; its results, and the memory it reads, from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0 && lane == 0) {
    // ---- producer
    const long long drop = g_pipe_drop_row;
    long long issued = 0;
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    for (int32_t t = first; ok && t < total; t += step) {
      const int q = COUNT == 2 && t >= G.split;
      const MMProblem& P = G.q[q];
      const Tile tile = tile_at<S::BM / BN>(P, q ? t - G.split : t);
      const int na = PARTS ? P.na : 1, nb = PARTS ? P.nb : 1;
      const int32_t am = tile.tm * S::BM + (int32_t)rank * 128;
      const int32_t bn = tile.tn * BN + (int32_t)rank * S::B_ROWS;
      for (int32_t kb = 0; kb < P.kblocks; ++kb) {
        if (!mbar_wait(&empty[slot], (round & 1) ^ 1) || (drop >= 0 && issued >= drop)) {      // the test hook's lost copies
          ok = false;
          break;
        }
        if (rank == 0) mbar_arrive_expect_tx(&full[slot], (na * MM_A_BYTES + nb * S::B_BYTES) * CG);
        uint32_t at = ring + slot * slot_bytes;
        const uint32_t bar = smem_addr(&full[slot]);
        const int32_t k0 = kb * MM_BK;
        for (int p = 0; p < na; ++p, at += MM_A_BYTES) {
          const int32_t z = tile.matrix * P.planes_a + p;
          if (P.a_k) {
            tma_box<CG>(at, &P.ta, k0, am, z, bar);
          } else {
            tma_box<CG>(at, &P.ta, am, k0, z, bar);
            tma_box<CG>(at + MM_A_BYTES / 2, &P.ta, am + 64, k0, z, bar);
          }
        }
        for (int p = 0; p < nb; ++p, at += S::B_BYTES) {
          const int32_t z = tile.matrix * P.planes_b + p;
          if (P.b_k) {
            tma_box<CG>(at, &P.tb, k0, bn, z, bar);
          } else {
#pragma unroll
            for (int j = 0; j < S::B_ROWS / 64; ++j)
              tma_box<CG>(at + j * (64 * MM_BK * 2), &P.tb, bn + j * 64, k0, z, bar);
          }
        }
        ++issued;
        if (++slot == stages) slot = 0, ++round;
      }
    }
    if (!ok && rank == 0)        // copies in flight land before the kernel's memory is given up
      for (long long i = issued > stages ? issued - stages : 0; i < issued; ++i)
        mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    uint32_t n = 0, round = 0;
    int slot = 0;
    bool ok = true;
    for (int32_t t = first; ok && t < total; t += step) {
      const MMProblem& P = G.q[COUNT == 2 && t >= G.split];
      const uint32_t idesc = (1u << 4) | (G.f16 ? 0u : (1u << 7) | (1u << 10)) | (P.a_k ? 0u : 1u << 15) |
                             (P.b_k ? 0u : 1u << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(S::BM >> 4) << 24);
      const uint32_t a_step = (P.a_k ? 32u : 2048u) >> 4, b_step = (P.b_k ? 32u : 2048u) >> 4;
      const int32_t b_first = (PARTS ? P.na : 1) * MM_A_BYTES;
      for (int32_t k = 0; ok && k < P.kblocks; k += P.chunk, ++n) {
        const int buf = n & 1;
        if (!mbar_wait(&acc_empty[buf], ((n >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t d = tmem + buf * S::ACC;
        const int32_t blocks = P.kblocks - k < P.chunk ? P.kblocks - k : P.chunk;
        for (int32_t i = 0; i < blocks; ++i) {
          if (!mbar_wait(&full[slot], round & 1)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t at = ring + slot * slot_bytes;
          for (int p = 0; p < (PARTS ? P.pairs : 1); ++p) {
            const uint32_t a = at + (PARTS ? P.pa[p] : 0) * MM_A_BYTES, b = at + b_first + (PARTS ? P.pb[p] : 0) * S::B_BYTES;
            const uint64_t da = operand_desc(a, MM_A_BYTES / 2), db = operand_desc(b, 64 * MM_BK * 2);
#pragma unroll
            for (int j = 0; j < MM_BK / 16; ++j)
              mma_16<CG>(PARTS && p + 1 < P.pairs ? d + BN : d, da + (uint64_t)(j * a_step), db + (uint64_t)(j * b_step), idesc,
                         (i | j) != 0 || (PARTS && p > 0 && p + 1 < P.pairs));
          }
          mma_commit<CG>(&empty[slot]);
          if (++slot == stages) slot = 0, ++round;
        }
        if (ok) mma_commit<CG>(&acc_full[buf]);
      }
    }
    if (!ok) {                   // products in flight end before the memory is given up
      mma_commit<CG>(&drain);
      mbar_wait(&drain, 0);
    }
  } else if (warp == 3) {
    // ---- columns' sums joined, beside the products
    column_sums(G.sums, (int64_t)blockIdx.x * 32 + lane, (int64_t)gridDim.x * 32);
  } else if (warp >= 4) {
    // ---- epilogue: a warp's 32 accumulator rows (set by its number), a share of the columns
    constexpr int COLS = BN * 4 / MMWarps<SUM>::EPI;
    const int rows = (warp & 3) * 32, share = (warp - 4) >> 2;
    float* stage = (float*)(smem_raw + (ring - smem_addr(smem_raw)) + S::RING) + (warp - 4) * (32 * 17);
    const uint32_t mine = tmem + ((uint32_t)rows << 16) + share * COLS;
    uint32_t n = 0;
    // One tile of a product; false if a wait gave up.
    const auto finish = [&](const MMProblem& P, int32_t t) {
      const Tile tile = tile_at<S::BM / BN>(P, t);
      const int64_t row0 = (int64_t)tile.tm * S::BM + rank * 128 + rows, r = row0 + lane;
      const int64_t col = (int64_t)tile.tn * BN + share * COLS;
      const bool mirrored = P.symmetric && (tile.tn + 1) * BN <= tile.tm * S::BM;
      bool ok = true;
      if constexpr (SUM) {
        float sum[COLS];
        if constexpr (!PARTS) {
#pragma unroll
          for (int i = 0; i < COLS; ++i) sum[i] = 0.0f;
        }
        for (int32_t k = 0; k < P.kblocks; k += P.chunk, ++n) {
          const int buf = n & 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], (n >> 1) & 1));
          if (!ok) return false;
          fence_after();
#pragma unroll
          for (int c = 0; c < COLS; c += 16) {
            float v[16];
            if constexpr (PARTS) {
              float w[16];
              tmem_load16(mine + buf * S::ACC + BN + c, w);
              tmem_load16(mine + buf * S::ACC + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c + i] = k ? sum[c + i] + (v[i] + w[i]) : v[i] + w[i];
            } else {
              tmem_load16(mine + buf * S::ACC + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c + i] += v[i];
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
        }
#pragma unroll 1
        for (int c = 0; c < COLS; c += 16) {
          Fetched F;
          fetch16<KIND>(P, tile.matrix, r, col + c, F);
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = sum[i];
#pragma unroll
            for (int q = 16; q < COLS; q += 16) v[i] = c == q ? sum[q + i] : v[i];
          }
          finish16<KIND>(P, tile.matrix, row0, lane, col + c, mirrored, F, stage, v);
        }
      } else {
        const int buf = n & 1;
        Fetched F;
        fetch16<KIND>(P, tile.matrix, r, col, F);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], (n >> 1) & 1));
        if (!ok) return false;
        ++n;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < COLS; c += 16) {
          float v[16];
          __syncwarp();
          tmem_load16(mine + buf * S::ACC + c, v);
          if (c + 16 >= COLS) {      // the accumulator is read: the next tile but one may have it
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
          }
          const Fetched now = F;
          if (c + 16 < COLS) fetch16<KIND>(P, tile.matrix, r, col + c + 16, F);
          finish16<KIND>(P, tile.matrix, row0, lane, col + c, mirrored, now, stage, v);
        }
      }
      return true;
    };
    for (int32_t t = first; t < total; t += step) {
      // (each product's parameters are read as constants)
      if (!(COUNT == 2 && t >= G.split ? finish(G.q[COUNT - 1], t - G.split) : finish(G.q[0], t))) break;
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  fence_after();
  if (warp == 2) tmem_free<CG>(tmem, 2 * S::ACC);
}

// -------------------------------------------------------------- few tiles
//
// A CTA is fed at 64 bytes a clock, so a product of few tiles takes what one
// tile's operands take, while most SMs idle.  Here the CTAs of a cluster share
// a tile's summed axis, so that more SMs have a part of it on the way at once.
// Their accumulators meet in shared memory and are added in the cluster's
// order; a CTA finishes its share of the elements.  The product is taken the
// other way round, 128 columns of the second operand as the tensor core's rows
// and BN rows of the first as its N: for few rows of x the weights' bytes are
// the time, and lanes hold neighbouring columns of y.
template <int BN, int SUM>
struct SplitShape {
  static constexpr bool PARTS = SUM == MM_PARTS;
  static constexpr int B_BYTES = BN * MM_BK * 2, STAGE = MM_A_BYTES + B_BYTES;
  static constexpr int STAGES = BN < 128 ? 8 : 6;                // with planes as many as they leave room for
  static constexpr int RING = PARTS ? 224 * 1024 : STAGES * STAGE;
  static constexpr int SMEM = RING + 1024;
  static constexpr int ACC = PARTS ? 2 * BN : BN, BUFS = SUM ? 2 : 1;
  static constexpr int TMEM_COLS = BUFS * ACC < 32 ? 32 : BUFS * ACC;
};
constexpr int SPLIT_THREADS = 320;
constexpr int SPLIT_ROW = 132;             // floats of a column of the accumulator in shared memory

struct SplitParams {
  MMProblem q;                             // a: the columns' operand, b: the rows'
  MMColumnSums sums;
  int32_t split, row_tiles, tiles, stages, slot_bytes, f16;      // tiles: of one matrix
};

__device__ __forceinline__ float4 load_cluster(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

__device__ __forceinline__ void load4_rt(const void* p, int32_t dt, int64_t i, int n, float* v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = k < n ? load1_rt(p, dt, i + k) : 0.0f;
}
__device__ __forceinline__ void store4_rt(void* p, int32_t dt, int64_t i, int n, const float* v) {
  if (dt == PSK_BF16) {
    uint16_t* q = (uint16_t*)p + i;
    if (n == 4 && (uintptr_t)q % 8 == 0) {
      *(uint2*)q = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) q[k] = f32_to_bf16_bits(v[k]);
  } else {
    float* q = (float*)p + i;
    if (n == 4 && (uintptr_t)q % 16 == 0) {
      *(float4*)q = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) q[k] = v[k];
  }
}

// Four columns of a row of the orthogonalised update, into fp16 planes.
__device__ __forceinline__ void ortho_row4(const MMEpilogue& E, int32_t matrix, int64_t r, int64_t c, float* t) {
  const int64_t at = (int64_t)matrix * E.planes * E.plane_stride + r * E.ld + c;
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = E.alpha * t[k];
  if (E.from)
    for (int p = E.planes - 1; p >= 0; --p) {
      const uint2 w = *(const uint2*)(E.from + at + p * E.plane_stride);
      const float2 x = f16x2_to_f32(w.x), y = f16x2_to_f32(w.y);
      v[0] = fmaf(E.beta, x.x, v[0]), v[1] = fmaf(E.beta, x.y, v[1]);
      v[2] = fmaf(E.beta, y.x, v[2]), v[3] = fmaf(E.beta, y.y, v[3]);
    }
  for (int p = 0; p < E.planes; ++p) {
    const uint2 w = make_uint2(f32x2_to_f16x2(v[0], v[1]), f32x2_to_f16x2(v[2], v[3]));
    const float2 x = f16x2_to_f32(w.x), y = f16x2_to_f32(w.y);
    v[0] -= x.x, v[1] -= x.y, v[2] -= y.x, v[3] -= y.y;
    *(uint2*)(E.to + at + p * E.plane_stride) = w;
  }
}

template <int BN, int SUM, bool ORTHO>
__global__ void __launch_bounds__(SPLIT_THREADS, 1) mm_split_kernel(const __grid_constant__ SplitParams G) {
  using S = SplitShape<BN, SUM>;
  constexpr bool PARTS = S::PARTS;
  const MMProblem& P = G.q;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[S::STAGES], empty[S::STAGES], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = G.split;
  const uint32_t rank = cluster_rank();
  const int32_t unit = blockIdx.x / split, matrix = ORTHO ? unit / G.tiles : 0, tile = unit - matrix * G.tiles;
  const int32_t tc = tile / G.row_tiles, tr = tile - tc * G.row_tiles;
  const int32_t za = matrix * P.planes_a, zb = matrix * P.planes_b;
  const int32_t k0 = (int32_t)((int64_t)P.kblocks * rank / split), k1 = (int32_t)((int64_t)P.kblocks * (rank + 1) / split);
  const int stages = PARTS ? G.stages : S::STAGES, na = PARTS ? P.na : 1, nb = PARTS ? P.nb : 1;
  const uint32_t slot_bytes = PARTS ? G.slot_bytes : S::STAGE;
  const int32_t chunk = SUM ? P.chunk : P.kblocks;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], SPLIT_THREADS / 32 - 2);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<1>(&tmem_slot, S::TMEM_COLS);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // set up beside the kernel before it; its results, and the memory it reads, from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0 && lane == 0) {
    const long long drop = g_pipe_drop_row;
    int issued = 0;
    bool ok = true;
    for (int32_t kb = k0; kb < k1; ++kb, ++issued) {
      const int s = issued % stages;
      if (!mbar_wait(&empty[s], ((issued / stages) & 1) ^ 1) || (drop >= 0 && issued >= drop)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&full[s], na * MM_A_BYTES + nb * S::B_BYTES);
      uint32_t at = ring + s * slot_bytes;
      const uint32_t bar = smem_addr(&full[s]);
      for (int p = 0; p < na; ++p, at += MM_A_BYTES) {
        if (P.a_k) {
          tma_box<1>(at, &P.ta, kb * MM_BK, tc * 128, za + p, bar);
        } else {
          tma_box<1>(at, &P.ta, tc * 128, kb * MM_BK, za + p, bar);
          tma_box<1>(at + MM_A_BYTES / 2, &P.ta, tc * 128 + 64, kb * MM_BK, za + p, bar);
        }
      }
      for (int p = 0; p < nb; ++p, at += S::B_BYTES) {
        if (P.b_k) {
          tma_box<1>(at, &P.tb, kb * MM_BK, tr * BN, zb + p, bar);
        } else {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j)
            tma_box<1>(at + j * (64 * MM_BK * 2), &P.tb, tr * BN + j * 64, kb * MM_BK, zb + p, bar);
        }
      }
    }
    if (!ok)
      for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) mbar_wait(&full[i % stages], (i / stages) & 1);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = (1u << 4) | (G.f16 ? 0u : (1u << 7) | (1u << 10)) | (P.a_k ? 0u : 1u << 15) | (P.b_k ? 0u : 1u << 16) |
                           ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    const uint32_t a_step = (P.a_k ? 32u : 2048u) >> 4, b_step = (P.b_k ? 32u : 2048u) >> 4;
    bool ok = true;
    int i = 0;
    for (int n = 0; ok && i < k1 - k0; ++n) {
      const int buf = SUM ? n & 1 : 0;
      if (SUM && !mbar_wait(&acc_empty[buf], ((n >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
      fence_after();
      const uint32_t d = tmem + buf * S::ACC;
      const int end = k1 - k0 - i < chunk ? k1 - k0 : i + chunk;
      for (bool fresh = true; i < end; ++i, fresh = false) {
        const int s = i % stages;
        if (!mbar_wait(&full[s], (i / stages) & 1)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t at = ring + s * slot_bytes;
        for (int p = 0; p < (PARTS ? P.pairs : 1); ++p) {
          const bool small = PARTS && p + 1 < P.pairs;
          const uint64_t da = operand_desc(at + (PARTS ? P.pa[p] : 0) * MM_A_BYTES, MM_A_BYTES / 2);
          const uint64_t db = operand_desc(at + na * MM_A_BYTES + (PARTS ? P.pb[p] : 0) * S::B_BYTES, 64 * MM_BK * 2);
#pragma unroll
          for (int j = 0; j < MM_BK / 16; ++j)
            mma_16<1>(small ? d + BN : d, da + (uint64_t)(j * a_step), db + (uint64_t)(j * b_step), idesc,
                      !fresh || j != 0 || (small && p > 0));
        }
        mma_commit<1>(&empty[s]);
      }
      if (ok) mma_commit<1>(&acc_full[buf]);
    }
    if (!ok) {
      mma_commit<1>(&drain);
      mbar_wait(&drain, 0);
    }
  }
  __syncwarp();
  // Every part of the ring has been used up once the last accumulator is there:
  // it takes the sums, column after column.
  float* part = (float*)(smem_raw + (ring - smem_addr(smem_raw)));
  if (warp >= 2) {
    constexpr int MINE = BN < 32 ? 1 : BN / 32;          // sixteens of columns of this warp's
    const int row = (warp & 3) * 32, share = (warp - 2) / 4;
    const uint32_t mine = tmem + ((uint32_t)row << 16);
    if constexpr (SUM) {
      float sum[MINE * 16];
      if constexpr (!PARTS) {
#pragma unroll
        for (int j = 0; j < MINE * 16; ++j) sum[j] = 0.0f;
      }
      bool ok = true;
      int n = 0;
      for (int32_t k = k0; k < k1; k += chunk, ++n) {
        const int buf = n & 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], (n >> 1) & 1));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int c = 0; c < MINE; ++c) {
          float v[16];
          const int at = (share + 2 * c) * 16;
          if (at >= BN) break;             // (of 16 columns the second four warps have none)
          if constexpr (PARTS) {
            float w[16];
            tmem_load16(mine + buf * S::ACC + BN + at, w);
            tmem_load16(mine + buf * S::ACC + at, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[16 * c + j] = n ? sum[16 * c + j] + (v[j] + w[j]) : v[j] + w[j];
          } else {
            tmem_load16(mine + buf * S::ACC + at, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[16 * c + j] += v[j];
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      }
      // (all of them: the ring is another's until every warp has its last sums)
      __syncwarp();
      named_barrier(1, SPLIT_THREADS - 64);
      if (ok) {
#pragma unroll
        for (int c = 0; c < MINE && (share + 2 * c) * 16 < BN; ++c)
#pragma unroll
          for (int j = 0; j < 16; ++j) part[((share + 2 * c) * 16 + j) * SPLIT_ROW + row + lane] = sum[16 * c + j];
      }
    } else if (__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[0], 0))) {
      fence_after();
#pragma unroll 1
      for (int c = share * 16; c < BN; c += 32) {
        float v[16];
        __syncwarp();
        tmem_load16(mine + c, v);
#pragma unroll
        for (int k = 0; k < 16; ++k) part[(c + k) * SPLIT_ROW + row + lane] = v[k];
      }
      fence_before();
    }
  }
  cluster_sync_all();
  fence_after();
  if (warp == 1) tmem_free<1>(tmem, S::TMEM_COLS);
  const MMEpilogue& E = P.e;
  // P.m: columns of y, P.n: its rows; four columns a thread
  const int rows = P.n - (int64_t)tr * BN < BN ? (int)(P.n - (int64_t)tr * BN) : BN, total = 32 * rows;
  const int from = total * (int)rank / split, to = total * (int)(rank + 1) / split;
#pragma unroll 1
  for (int i = from + threadIdx.x; i < to; i += SPLIT_THREADS) {
    const int64_t c = (int64_t)tc * 128 + (i & 31) * 4, r = (int64_t)tr * BN + (i >> 5);
    if (c >= P.m) continue;
    const int n = P.m - c < 4 ? (int)(P.m - c) : 4;
    const uint32_t at = smem_addr(part + (i >> 5) * SPLIT_ROW + (i & 31) * 4);
    float4 parts[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < split) parts[q] = load_cluster(at, q);
    float res[4], t[4];
    if (!ORTHO && E.res) load4_rt(E.res, E.rt, r * E.ldr + c, n, res);
    t[0] = parts[0].x, t[1] = parts[0].y, t[2] = parts[0].z, t[3] = parts[0].w;
#pragma unroll
    for (int q = 1; q < 8; ++q)
      if (q < split) t[0] += parts[q].x, t[1] += parts[q].y, t[2] += parts[q].z, t[3] += parts[q].w;
    if constexpr (ORTHO) {
      ortho_row4(E, matrix, r, c, t);
      continue;
    }
    if (E.bias) {
      float b[4];
      load4_rt(E.bias, E.bt, c, n, b);
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] += b[k];
    }
    if (E.z) store4_rt(E.z, E.zt, r * E.ldz + c, n, t);
    act_rt<4>(t, E.act);
    if (E.res) {
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] += res[k];
    }
    store4_rt(E.y, E.yt, r * E.ldy + c, n, t);
  }
  column_sums(G.sums, (int64_t)blockIdx.x * SPLIT_THREADS + threadIdx.x, (int64_t)gridDim.x * SPLIT_THREADS);
  cluster_sync_all();
}

// --------------------------------------------------------------------- host

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static const EncodeFn fn = []() -> EncodeFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// Boxes of 64 contiguous elements by `rows` rows, zeros outside the operand.
static int encode_operand(CUtensorMap* map, const MMOperand& o, int64_t matrices, bool f16, int rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return fail(PSK_E_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)(o.planes * matrices)};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2u, (cuuint64_t)o.plane_stride * 2u};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const auto encode = [&] {
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) bind_context(), r = encode();
  if (r != CUDA_SUCCESS) return fail(PSK_E_CUDA, "tensor map encoding failed (CUresult %d)", (int)r);
  return PSK_OK;
}

// Blocks of the summed axis that one accumulator takes where the sum is taken
// by pieces: the tensor core's additions truncate, always to one side (terms of
// one sign: 2048 are off by 2.4e-6 of their sum, 8192 by 9e-6, 65536 by up to
// 3.4e-4), so the accumulator is added to a register with one rounding instead.
// With an f32 operand every 256 terms; and the small products of planes have an
// accumulator of their own: added into the large one, each would truncate it
// again (1.5e-6 of the result's size, apart 1.5e-7).  bf16 operands every 1024
// terms, which keeps f32 results to 1e-6 at any length and hides the last piece's
// epilogue behind the next tile's products (16384 x 2048 x 5632, f32 result, in
// pieces of 256 terms 453 us, 512 391, 1024 301, 2048 285, whole 231).
constexpr int MM_SUM_BLOCKS = 4, MM_PIECE_BLOCKS = 16;

// By pieces go the sums of f32 operands; those of bf16 ones above 2048 terms
// (that one CTA takes) whose result is stored in f32 (8192 x 2048 x 5632's
// gradients with an f32 dw 286 us for 270, off by 1e-6 instead of 9e-6); and
// those so long that truncations would come near bf16's rounding of the result
// (half a step is 2e-3 to 4e-3).
constexpr int64_t MM_WHOLE_F32 = 2048, MM_WHOLE_BF16 = 65536;
static int sum_of(const MMCall& C, int64_t terms) {
  if (C.pairs > 1) return MM_PARTS;
  const bool f32 = !C.ortho && (C.e.yt == PSK_F32 || (C.e.z && C.e.zt == PSK_F32));
  return terms > (f32 ? MM_WHOLE_F32 : MM_WHOLE_BF16) ? MM_PIECES : MM_WHOLE;
}
static int piece_of(int sum) { return sum == MM_PARTS ? MM_SUM_BLOCKS : MM_PIECE_BLOCKS; }

// Absent, or bf16 rows that begin on 32-byte boundaries.
static bool rows_32(const void* p, int32_t dt, int64_t ld) {
  return !p || (dt == PSK_BF16 && (uintptr_t)p % 32 == 0 && ld % 16 == 0);
}

template <int CG, int BN, int KIND, int SUM, int COUNT>
static int launch_shape(const MMCall* calls, const MMColumnSums* sums, cudaStream_t stream) {
  using S = MMShape<CG, BN, KIND, SUM>;
  MMParams G{};
  int64_t all = 0;
  for (int q = 0; q < COUNT; ++q) {
    const MMCall& C = calls[q];
    MMProblem& P = G.q[q];
    int rc = encode_operand(&P.ta, C.a, C.matrices, C.f16, C.a.k_inner ? 128 : 64);
    if (!rc) rc = encode_operand(&P.tb, C.b, C.matrices, C.f16, C.b.k_inner ? S::B_ROWS : 64);
    if (rc) return rc;
    P.e = C.e;
    P.m = C.m, P.n = C.n;
    P.kblocks = (int32_t)((C.k + MM_BK - 1) / MM_BK), P.pairs = C.pairs;
    P.chunk = sum_of(C, C.k) == MM_WHOLE ? P.kblocks : piece_of(SUM);
    P.planes_a = C.a.planes, P.planes_b = C.b.planes;
    P.a_k = C.a.k_inner, P.b_k = C.b.k_inner;
    for (int i = 0; i < C.pairs; ++i) {
      P.pa[i] = C.pa[i], P.pb[i] = C.pb[i];
      P.na = C.pa[i] + 1 > P.na ? C.pa[i] + 1 : P.na;
      P.nb = C.pb[i] + 1 > P.nb ? C.pb[i] + 1 : P.nb;
    }
    const int32_t slot = P.na * MM_A_BYTES + P.nb * S::B_BYTES;
    if (slot > G.slot_bytes) G.slot_bytes = slot;
    const int64_t tm = (C.m + S::BM - 1) / S::BM, tn = (C.n + BN - 1) / BN;
    int64_t tiles = tm * tn;
    if (C.symmetric) {               // the last row of tiles may end before the diagonal block does
      constexpr int Q = S::BM / BN;
      tiles = Q * (tm * (tm - 1) / 2) + (Q * tm < tn ? Q * tm : tn);
    }
    all += tiles * C.matrices;
    if (all > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many output tiles");
    P.tiles_m = (int32_t)tm, P.tiles_n = (int32_t)tn, P.tiles = (int32_t)tiles, P.symmetric = C.symmetric;
    if (q == 0) G.split = (int32_t)all;
    G.f16 = C.f16;
  }
  G.total = (int32_t)all;
  G.stages = S::RING / G.slot_bytes < S::STAGES ? S::RING / G.slot_bytes : S::STAGES;
  if (sums) G.sums = *sums;
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)mm_kernel<CG, BN, KIND, SUM, COUNT>, S::SMEM, limit);
  const int64_t most = device_sm_count() / CG;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((all < most ? all : most) * CG));
  cfg.blockDim = dim3(MMWarps<SUM>::THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, mm_kernel<CG, BN, KIND, SUM, COUNT>, G);
  return check_launch("matrix product kernel");
}

// CTAs that share a tile of 128 columns and `rows` rows: what fills the SMs
// once, two blocks of the summed axis each at least, as long as all clusters
// find their place at one time: of eight CTAs up to eight tiles (512 x 2048 x
// 512, 16 tiles: 12.6 us by eight, 7.2 by four; the gradients of 16384 x 128 x
// 128, 1 and 128: 32.5 and 42.2), of four up to 36 (768 x 2048 x 768, 36: 8.6 us,
// by three 9.1; 2432 x 2048 x 256, 38: 15.0 and 9.1), of three up to 42 (1280 x
// 4096 x 512, 40: 12.4 us, by two 15.8; the gradients of 2000 x 304 x 2000, 48:
// 35.1 and 20.4).
static int split_of(const MMCall& C, int rows) {
  const int64_t tiles = ((C.n + 127) / 128) * ((C.m + rows - 1) / rows) * C.matrices, blocks = (C.k + MM_BK - 1) / MM_BK;
  int64_t split = device_sm_count() / tiles;
  const int64_t most = tiles <= 8 ? 8 : tiles <= 36 ? 4 : tiles <= 42 ? 3 : 2;
  split = split < 1 ? 1 : split > most ? most : split;
  while (split > 1 && blocks < 2 * split) --split;
  return (int)split;
}

template <int BN, int SUM, bool ORTHO = false>
static int launch_split(const MMCall& C, const MMColumnSums* sums, cudaStream_t stream) {
  using S = SplitShape<BN, SUM>;
  SplitParams G{};
  MMProblem& P = G.q;
  int rc = encode_operand(&P.ta, C.b, C.matrices, C.f16, C.b.k_inner ? 128 : 64);
  if (!rc) rc = encode_operand(&P.tb, C.a, C.matrices, C.f16, C.a.k_inner ? BN : 64);
  if (rc) return rc;
  P.e = C.e;
  P.m = C.n, P.n = C.m;
  P.kblocks = (int32_t)((C.k + MM_BK - 1) / MM_BK), P.chunk = piece_of(SUM), P.pairs = C.pairs;
  P.a_k = C.b.k_inner, P.b_k = C.a.k_inner, P.planes_a = C.b.planes, P.planes_b = C.a.planes;
  for (int i = 0; i < C.pairs; ++i) {
    P.pa[i] = C.pb[i], P.pb[i] = C.pa[i];
    P.na = C.pb[i] + 1 > P.na ? C.pb[i] + 1 : P.na;
    P.nb = C.pa[i] + 1 > P.nb ? C.pa[i] + 1 : P.nb;
  }
  G.slot_bytes = P.na * MM_A_BYTES + P.nb * S::B_BYTES;
  G.stages = S::RING / G.slot_bytes < S::STAGES ? S::RING / G.slot_bytes : S::STAGES;
  if (sums) G.sums = *sums;
  G.split = split_of(C, BN), G.row_tiles = (int32_t)((C.m + BN - 1) / BN);
  const int64_t each = ((C.n + 127) / 128) * G.row_tiles, tiles = each * C.matrices;
  if (tiles * G.split > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many output tiles");
  G.tiles = (int32_t)each, G.f16 = C.f16;
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)mm_split_kernel<BN, SUM, ORTHO>, S::SMEM, limit);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)G.split, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * G.split));
  cfg.blockDim = dim3(SPLIT_THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, mm_split_kernel<BN, SUM, ORTHO>, G);
  return check_launch("matrix product kernel of few tiles");
}

// Rows of the split kernel's tile for a product of planes (0: it gains nothing):
// 64 or 128, by the time of the blocks that one CTA takes in turn, 20 and 23 by
// measure (1 x 1024 x 1024's update 300 us by 64, 215 by 128; 509 x 771 x 1003's
// gradients, with both in one launch 35, apart 29; 300 x 3000 x 400 the same).
static int split_rows_sum(const MMCall& C) {
  const int64_t blocks = (C.k + MM_BK - 1) / MM_BK;
  const int s64 = split_of(C, 64), s128 = split_of(C, 128);
  const bool wide = (blocks + s128 - 1) / s128 * 23 < (blocks + s64 - 1) / s64 * 20;
  return (wide ? s128 : s64) < 2 ? 0 : wide ? 128 : 64;
}

// The same of any product.
static int split_rows(const MMCall& C) {
  if (C.ortho) {
    // Of f32 results wherever they can (1 x 512 x 512, five steps: 201 us, 111);
    // else, where both triangles are more tiles than one, if a tile's summed axis
    // shrinks by 12 blocks at least (8 x 64 x 4096 162 us, 92; 1 x 512 x 1024 105,
    // 97; by 8 or less 1 x 1024 x 1024 132, 150, and 1 x 512 x 512 95, 101).
    if (!C.e.to || C.pairs > 1) return C.e.to ? split_rows_sum(C) : 0;
    const int rows = C.m <= 64 ? 64 : 128, split = split_of(C, rows);
    const int64_t blocks = (C.k + MM_BK - 1) / MM_BK;
    return split >= 2 && blocks - blocks / split >= 12 ? rows : 0;
  }
  if (C.pairs > 1) return split_rows_sum(C);
  // (the rows' operand is read along the summed axis, or in boxes of 64 rows)
  if (C.m <= 64) return C.m > 32 || !C.a.k_inner ? 64 : C.m > 16 ? 32 : 16;
  return split_of(C, 128) >= 2 ? 128 : 0;
}

// Pairs of CTAs on tiles of 256 x 256, or single ones on 128 x 128: by the
// time of the tiles that one SM takes in turn.  64 summed elements of a tile
// take about 0.34 us of a pair and 0.30 us of one CTA, whose 128 columns are
// bound by shared memory (operands read and filled in: 2048^3 16.8 and 24.3 us,
// 512 x 2048 x 5632 15.9 and 23.8, 1024^3 11.4 and 9.0, 128 x 2048 x 5632 15.6
// and 13.4).  With planes always the latter: two accumulators of 256 columns would
// leave no second pair of them, and pairs on 256 x 128 gain nothing (4096 x 2048
// x 2048 f32 199 us, single ones 195).  The update's products take 128 x 64 where
// those still fit the SMs once (512 x 512, five steps: 114 us, 95).
template <int KIND, int SUM>
static int launch_kind(const MMCall* calls, const MMColumnSums* sums, cudaStream_t stream) {
  const MMCall& C = calls[0];
  const int64_t sms = device_sm_count(), pairs = sms / 2;
  const auto waves = [&](int64_t side, int64_t units) {
    const int64_t tm = (C.m + side - 1) / side, tn = (C.n + side - 1) / side;
    return ((C.symmetric ? tm * (tm + 1) / 2 : tm * tn) * C.matrices + units - 1) / units;
  };
  if constexpr (SUM == MM_WHOLE || (SUM == MM_PIECES && KIND == MM_ANY))
    if (pairs > 0 && waves(256, pairs) * 34 < waves(128, sms) * 30)
      return launch_shape<2, 256, KIND, SUM, 1>(calls, sums, stream);
  if constexpr (KIND == MM_ORTHO && SUM == MM_WHOLE)
    if (waves(128, 1) * 2 <= sms) return launch_shape<1, 64, KIND, MM_WHOLE, 1>(calls, sums, stream);
  return launch_shape<1, 128, KIND, SUM, 1>(calls, sums, stream);
}

static bool is_wide(const MMCall& C) {
  const MMEpilogue& E = C.e;
  return C.n % 16 == 0 && rows_32(E.y, E.yt, E.ldy) && rows_32(E.z, E.zt, E.ldz) && rows_32(E.res, E.rt, E.ldr) &&
         rows_32(E.bias, E.bt, 0);
}

// rows: split_rows' answer.
template <int SUM>
static int launch_one(const MMCall* calls, int rows, const MMColumnSums* sums, cudaStream_t stream) {
  const MMCall& C = calls[0];
  if (C.ortho) {
    if (rows == 64) return launch_split<64, SUM, true>(C, sums, stream);
    if (rows == 128) return launch_split<128, SUM, true>(C, sums, stream);
    return launch_kind<MM_ORTHO, SUM>(calls, sums, stream);
  }
  if constexpr (SUM != MM_PARTS) {
    if (rows == 16) return launch_split<16, SUM>(C, sums, stream);
    if (rows == 32) return launch_split<32, SUM>(C, sums, stream);
  }
  if (rows == 64) return launch_split<64, SUM>(C, sums, stream);
  if (rows == 128) return launch_split<128, SUM>(C, sums, stream);
  if constexpr (SUM == MM_WHOLE)
    if (is_wide(C)) switch (C.e.act) {
        case ACT_RELU: return launch_kind<ACT_RELU, SUM>(calls, sums, stream);
        case ACT_GELU: return launch_kind<ACT_GELU, SUM>(calls, sums, stream);
        case ACT_SILU: return launch_kind<ACT_SILU, SUM>(calls, sums, stream);
        default: return launch_kind<ACT_NONE, SUM>(calls, sums, stream);
      }
  return launch_kind<MM_ANY, SUM>(calls, sums, stream);
}

int mm_launch(const MMCall* calls, int count, const MMColumnSums* sums, cudaStream_t stream) {
  const MMCall& C = calls[0];
  if (count == 2) {
    const int sum = sum_of(C, C.k), other = sum_of(calls[1], calls[1].k);
    // One launch where one kernel serves both, their tiles together fill the SMs
    // once at most, and the longer tile takes less than the two launches with
    // their summed axes shared among CTAs (2000 x 304 x 2000 bf16: 20 us as one, 35
    // as two by threes; 509 x 771 x 1003 f32: 78 as two unshared ones, 35 as one,
    // 29 as two shared; 16384 x 128 x 128 bf16: 106 as one, 33 as two shared).
    // More tiles run better one product after the other (8192 x 2048 x 5632: 252
    // us, together 275).
    int64_t tiles = 0, longest = 0, apart = 0;
    for (int q = 0; q < 2; ++q) {
      const MMCall& D = calls[q];
      tiles += ((D.m + 127) / 128) * ((D.n + 127) / 128);
      const int64_t blocks = (D.k + MM_BK - 1) / MM_BK;
      const int rows = split_rows(D);
      longest = longest > blocks ? longest : blocks;
      apart += blocks / (rows ? split_of(D, rows) : 1);
    }
    const bool parts = sum == MM_PARTS, whole = sum == MM_WHOLE && other == MM_WHOLE, wide = whole && is_wide(C);
    // a launch more costs what eight blocks take, with planes three
    if (tiles > device_sm_count() || longest > apart + (parts ? 3 : 8) || (other == MM_PARTS) != parts ||
        (whole && is_wide(calls[1]) != wide)) {
      const int rc = mm_launch(calls, 1, sums, stream);
      return rc ? rc : mm_launch(calls + 1, 1, nullptr, stream);
    }
    if (calls[1].k * calls[1].pairs > C.k * C.pairs) {      // the longer tiles first
      const MMCall turned[2] = {calls[1], calls[0]};
      return mm_launch(turned, 2, sums, stream);
    }
    if (parts) return launch_shape<1, 128, MM_ANY, MM_PARTS, 2>(calls, sums, stream);
    if (!whole) return launch_shape<1, 128, MM_ANY, MM_PIECES, 2>(calls, sums, stream);
    if (!wide) return launch_shape<1, 128, MM_ANY, MM_WHOLE, 2>(calls, sums, stream);
    return launch_shape<1, 128, ACT_NONE, MM_WHOLE, 2>(calls, sums, stream);
  }
  const int rows = split_rows(C);
  const int64_t blocks = (C.k + MM_BK - 1) / MM_BK, split = rows ? split_of(C, rows) : 1;
  switch (sum_of(C, split == 1 ? C.k : (blocks + split - 1) / split * MM_BK)) {
    case MM_PARTS: return launch_one<MM_PARTS>(calls, rows, sums, stream);
    case MM_PIECES: return launch_one<MM_PIECES>(calls, rows, sums, stream);
    default: return launch_one<MM_WHOLE>(calls, rows, sums, stream);
  }
}

int mm_status(unsigned int* v, bool reset) {
  if (cudaMemcpyFromSymbol(v, g_pipe_status, sizeof(*v)) != cudaSuccess) return check_launch("device status read");
  if (reset) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_pipe_status, &z, sizeof(z)) != cudaSuccess) return check_launch("device status reset");
  }
  return PSK_OK;
}

int mm_set_drop_row(long long row) {
  if (cudaMemcpyToSymbol(g_pipe_drop_row, &row, sizeof(row)) != cudaSuccess) return check_launch("test hook write");
  return PSK_OK;
}

}  // namespace psk
