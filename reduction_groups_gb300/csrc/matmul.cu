// D = A B of 16-bit operands (bf16 or fp16) on the tensor cores with f32
// accumulators, and the epilogues of the linear layer and of the
// orthogonalised update.
//
// One persistent CTA (or pair of CTAs, CG = 2) an SM takes output tiles in
// turn.  Warp 0 fills a ring of shared-memory stages by TMA (64 summed
// elements of both operands, 128-byte swizzled), warp 1 issues tcgen05.mma
// from one thread into one of two accumulators in TMEM, warps 4 to 11 take
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
// of planes to be added, the smallest first, and each is a pass over the
// summed axis into the same accumulator.
//
// Every wait is bounded: a role that gives up records it in the device status
// and leaves its loop, all meet at the end of the kernel.
#include <cuda.h>

#include "common.cuh"
#include "pipe.cuh"
#include "vec8.cuh"
#include "act.cuh"
#include "mm.h"
#include "trainops.h"

namespace psk {

constexpr int MM_THREADS = 384;
constexpr int MM_EPI_WARPS = 8;
constexpr int MM_BK = 64;                  // summed elements a stage: one 128-byte swizzled row
constexpr int MM_A_BYTES = 128 * MM_BK * 2;

struct MMParams {
  CUtensorMap ta, tb;
  MMEpilogue e;
  int64_t m, n;
  int32_t kblocks, pairs, matrices;
  int32_t planes_a, planes_b;
  int32_t a_k, b_k, f16;
  int32_t tiles_m, tiles_n, tiles, symmetric;
  int32_t chunk;                           // blocks of the summed axis that one accumulator takes
  uint8_t pa[8], pb[8];
};

// ------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
  }
}

template <int CG>
__device__ __forceinline__ void mma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Arrive on `bar` (of both CTAs of a pair) when every product issued so far is done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// A box of the tensor map into shared memory; of a pair, the first CTA's barrier counts both CTAs' bytes.
template <int CG>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                        uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar & 0xFEFFFFFFu)
        : "memory");
}

// A 128-byte swizzled operand tile.  K-major: rows of 128 bytes, groups of
// eight 1024 bytes apart.  MN-major: 64 of M or N by 8 of K in 1024 bytes,
// `lbo` bytes to the next 64 of M or N.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on the barrier at this address in the first CTA of the pair.
template <int CG>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if constexpr (CG == 1) {
    mbar_arrive(bar);
  } else {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
  }
}

// --------------------------------------------------------------- tile order

struct Tile {
  int32_t matrix, tm, tn;
};

// Tiles of one matrix after another's; within one, groups of eight tile rows
// walk through the columns together, so that the tiles running at one time
// share operand rows in L2.  Symmetric: the lower triangle, row after row.
template <int Q>
__device__ __forceinline__ Tile tile_at(const MMParams& P, int32_t t) {
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

__device__ __forceinline__ void load8_rt(const void* p, int32_t dt, int64_t i, int n, bool vec, float* v) {
  if (dt == PSK_BF16) {
    if (vec) load8<PSK_BF16, true>(p, i, n, v);
    else load8<PSK_BF16, false>(p, i, n, v);
  } else {
    if (vec) load8<PSK_F32, true>(p, i, n, v);
    else load8<PSK_F32, false>(p, i, n, v);
  }
}

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

__device__ __forceinline__ float act_rt(float z, int32_t act) {
  switch (act) {
    case ACT_RELU: return act_value<ACT_RELU>(z);
    case ACT_GELU: return act_value<ACT_GELU>(z);
    case ACT_SILU: return act_value<ACT_SILU>(z);
    default: return z;
  }
}

// Eight neighbouring columns of one row.
__device__ __forceinline__ void linear_row8(const MMEpilogue& E, int64_t r, int64_t c, int n, float* v) {
  float t[8];
  if (E.bias) {
    load8_rt(E.bias, E.bt, c, n, E.vec_bias, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += t[k];
  }
  if (E.z) store8_rt(E.z, E.zt, r * E.ldz + c, n, E.vec_z, v);
  if (E.act) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_rt(v[k], E.act);
  }
  if (E.res) {
    load8_rt(E.res, E.rt, r * E.ldr + c, n, E.vec_res, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += t[k];
  }
  store8_rt(E.y, E.yt, r * E.ldy + c, n, E.vec_y, v);
}

__device__ __forceinline__ float f16_to_f32(uint32_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)h));
  return f;
}
__device__ __forceinline__ uint32_t f32_to_f16(float f) {
  uint16_t h;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(f));
  return h;
}

// Eight columns of one row of an fp16 matrix in planes: v = alpha v + beta from.
__device__ __forceinline__ void ortho_mix8(const MMEpilogue& E, const uint16_t* from, float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= E.alpha;
  if (!from) return;
  for (int p = E.planes - 1; p >= 0; --p) {
    const uint4 u = *(const uint4*)(from + p * E.plane_stride);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = fmaf(E.beta, f16_to_f32(w[k] & 0xFFFF), v[2 * k]);
      v[2 * k + 1] = fmaf(E.beta, f16_to_f32(w[k] >> 16), v[2 * k + 1]);
    }
  }
}

// The epilogue of 32 neighbouring accumulators of row r, from column col on.
template <int KIND>
__device__ __forceinline__ void finish32(const MMParams& P, int32_t matrix, int64_t r, int64_t col, bool mirrored,
                                         float* v) {
  const MMEpilogue& E = P.e;
  if (r >= P.m) return;
  const int64_t at = (int64_t)matrix * E.planes * E.plane_stride;
#pragma unroll
  for (int g = 0; g < 32; g += 8) {
    const int64_t left = P.n - (col + g);
    if (left <= 0) break;
    const int have = left < 8 ? (int)left : 8;
    if constexpr (KIND == MM_LINEAR) {
      linear_row8(E, r, col + g, have, v + g);
    } else {
      ortho_mix8(E, E.from ? E.from + at + r * E.ld + col + g : nullptr, v + g);
      if (E.to) {
        uint16_t* q = E.to + at + r * E.ld + col + g;
        for (int p = 0; p < E.planes; ++p) {
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            h[k] = f32_to_f16(v[g + k]);
            v[g + k] -= f16_to_f32(h[k]);
          }
          *(uint4*)(q + p * E.plane_stride) = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                                         h[6] | h[7] << 16);
          if (mirrored) {
            uint16_t* o = E.to + at + p * E.plane_stride + (col + g) * E.ld + r;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < have) o[(int64_t)k * E.ld] = (uint16_t)h[k];
          }
        }
      } else {
        const MMLeaf L = E.leaves[matrix];
        if (E.transposed) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < have) store1_rt(L.y, E.yt, (col + g + k) * L.ld + r, v[g + k]);
        } else {
          store8_rt(L.y, E.yt, r * L.ld + col + g, have, L.vec != 0, v + g);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- kernel

template <int CG, int BN>
struct MMShape {
  static constexpr int BM = 128 * CG;
  static constexpr int B_ROWS = BN / CG;                        // of B's tile in one CTA
  static constexpr int STAGE = MM_A_BYTES + B_ROWS * MM_BK * 2;
  static constexpr int STAGES = (200 * 1024) / STAGE < 8 ? (200 * 1024) / STAGE : 8;
  static constexpr int SMEM = STAGES * STAGE + 1024;            // and what aligns the ring to 1024 bytes
  static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
};

template <int CG, int BN, int KIND, bool SUM>
__global__ void __launch_bounds__(MM_THREADS, 1) mm_kernel(const __grid_constant__ MMParams P) {
  using S = MMShape<CG, BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[S::STAGES], empty[S::STAGES], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int32_t first = blockIdx.x / CG, step = gridDim.x / CG;
  const int32_t total = P.tiles * P.matrices;

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], MM_EPI_WARPS * CG);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<CG>(&tmem_slot, S::TMEM_COLS);
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---- producer
    const long long drop = g_pipe_drop_row;
    long long issued = 0;
    bool ok = true;
    for (int32_t t = first; ok && t < total; t += step) {
      const Tile tile = tile_at<S::BM / BN>(P, t);
      const int32_t am = tile.tm * S::BM + (int32_t)rank * 128;
      const int32_t bn = tile.tn * BN + (int32_t)rank * S::B_ROWS;
      for (int32_t k = 0; ok && k < P.kblocks; k += P.chunk)
      for (int p = 0; ok && p < P.pairs; ++p) {
        const int32_t za = tile.matrix * P.planes_a + P.pa[p], zb = tile.matrix * P.planes_b + P.pb[p];
        const int32_t end = P.kblocks - k < P.chunk ? P.kblocks : k + P.chunk;
        for (int32_t kb = k; kb < end; ++kb) {
          const int s = (int)(issued % S::STAGES);
          const uint32_t round = (uint32_t)(issued / S::STAGES);
          if (!mbar_wait(&empty[s], (round & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (drop >= 0 && issued >= drop) {      // the lost copies of the test hook
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], S::STAGE * CG);
          const uint32_t a = ring + s * S::STAGE, b = a + MM_A_BYTES, bar = smem_addr(&full[s]);
          const int32_t k0 = kb * MM_BK;
          if (P.a_k) {
            tma_box<CG>(a, &P.ta, k0, am, za, bar);
          } else {
            tma_box<CG>(a, &P.ta, am, k0, za, bar);
            tma_box<CG>(a + MM_A_BYTES / 2, &P.ta, am + 64, k0, za, bar);
          }
          if (P.b_k) {
            tma_box<CG>(b, &P.tb, k0, bn, zb, bar);
          } else {
#pragma unroll
            for (int j = 0; j < S::B_ROWS / 64; ++j)
              tma_box<CG>(b + j * (64 * MM_BK * 2), &P.tb, bn + j * 64, k0, zb, bar);
          }
          ++issued;
        }
      }
    }
    if (!ok && rank == 0)        // copies in flight land before the kernel's memory is given up
      for (long long i = issued > S::STAGES ? issued - S::STAGES : 0; i < issued; ++i)
        mbar_wait(&full[i % S::STAGES], (uint32_t)(i / S::STAGES) & 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    const uint32_t idesc = (1u << 4) | (P.f16 ? 0u : (1u << 7) | (1u << 10)) | (P.a_k ? 0u : 1u << 15) |
                           (P.b_k ? 0u : 1u << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(S::BM >> 4) << 24);
    const uint32_t a_step = (P.a_k ? 32u : 2048u) >> 4, b_step = (P.b_k ? 32u : 2048u) >> 4;
    uint32_t n = 0, it = 0;
    bool ok = true;
    for (int32_t t = first; ok && t < total; t += step)
      for (int32_t k = 0; ok && k < P.kblocks; k += P.chunk, ++n) {
        const int buf = n & 1;
        if (!mbar_wait(&acc_empty[buf], ((n >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t d = tmem + buf * BN;
        const int32_t blocks = (P.kblocks - k < P.chunk ? P.kblocks - k : P.chunk) * P.pairs;
        for (int32_t i = 0; i < blocks; ++i, ++it) {
          const int s = it % S::STAGES;
          if (!mbar_wait(&full[s], (it / S::STAGES) & 1)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t a = ring + s * S::STAGE, b = a + MM_A_BYTES;
          const uint64_t da = operand_desc(a, MM_A_BYTES / 2), db = operand_desc(b, 64 * MM_BK * 2);
#pragma unroll
          for (int j = 0; j < MM_BK / 16; ++j)
            mma_16<CG>(d, da + (uint64_t)(j * a_step), db + (uint64_t)(j * b_step), idesc, (i | j) != 0);
          mma_commit<CG>(&empty[s]);
        }
        if (ok) mma_commit<CG>(&acc_full[buf]);
      }
    if (!ok) {                   // products in flight end before the memory is given up
      mma_commit<CG>(&drain);
      mbar_wait(&drain, 0);
    }
  } else if (warp >= 4) {
    // ---- epilogue: a warp's 32 accumulator rows (set by its number), half the columns
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * (BN / 2);
    constexpr int COLS = BN / 2;
    uint32_t n = 0;
    for (int32_t t = first; t < total; t += step) {
      const Tile tile = tile_at<S::BM / BN>(P, t);
      const int64_t r = (int64_t)tile.tm * S::BM + rank * 128 + quarter * 32 + lane;
      const int64_t col = (int64_t)tile.tn * BN + half * COLS;
      const bool mirrored = P.symmetric && (tile.tn + 1) * BN <= tile.tm * S::BM;
      bool ok = true;
      if constexpr (SUM) {
        float sum[COLS];
        for (int32_t k = 0; k < P.kblocks; k += P.chunk, ++n) {
          const int buf = n & 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], (n >> 1) & 1));
          if (!ok) break;
          fence_after();
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            float v[32];
            tmem_load32(mine + buf * BN + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] = k ? sum[c + i] + v[i] : v[i];
          }
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < COLS; c += 32) finish32<KIND>(P, tile.matrix, r, col + c, mirrored, sum + c);
      } else {
        const int buf = n & 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], (n >> 1) & 1));
        if (!ok) break;
        ++n;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < COLS; c += 32) {
          float v[32];
          __syncwarp();
          tmem_load32(mine + buf * BN + c, v);
          if (c + 32 >= COLS) {      // the accumulator is read: the next tile but one may have it
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
          }
          finish32<KIND>(P, tile.matrix, r, col + c, mirrored, v);
        }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  fence_after();
  if (warp == 2) tmem_free<CG>(tmem, S::TMEM_COLS);
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
  const CUresult r = fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<void*>(o.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PSK_E_CUDA, "tensor map encoding failed (CUresult %d)", (int)r);
  return PSK_OK;
}

// Blocks of the summed axis that one accumulator takes where the sum is an
// f32 operand's: the tensor core's additions truncate (an f32 result of 2048
// terms is off by 1e-5 of its size, of 65536 by 2e-4), so every 256 terms the
// accumulator is added to a register with one rounding instead.
constexpr int MM_SUM_BLOCKS = 4;

template <int CG, int BN, int KIND, bool SUM>
static int launch_shape(const MMCall& C, cudaStream_t stream) {
  using S = MMShape<CG, BN>;
  MMParams P{};
  int rc = encode_operand(&P.ta, C.a, C.matrices, C.f16, C.a.k_inner ? 128 : 64);
  if (!rc) rc = encode_operand(&P.tb, C.b, C.matrices, C.f16, C.b.k_inner ? S::B_ROWS : 64);
  if (rc) return rc;
  P.e = C.e;
  P.m = C.m, P.n = C.n;
  P.kblocks = (int32_t)((C.k + MM_BK - 1) / MM_BK), P.pairs = C.pairs, P.matrices = (int32_t)C.matrices;
  P.chunk = SUM ? MM_SUM_BLOCKS : P.kblocks;
  P.planes_a = C.a.planes, P.planes_b = C.b.planes;
  P.a_k = C.a.k_inner, P.b_k = C.b.k_inner, P.f16 = C.f16;
  const int64_t tm = (C.m + S::BM - 1) / S::BM, tn = (C.n + BN - 1) / BN;
  int64_t tiles = tm * tn;
  if (C.symmetric) {                 // the last row of tiles may end before the diagonal block does
    constexpr int Q = S::BM / BN;
    tiles = Q * (tm * (tm - 1) / 2) + (Q * tm < tn ? Q * tm : tn);
  }
  if (tiles * C.matrices > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many output tiles");
  P.tiles_m = (int32_t)tm, P.tiles_n = (int32_t)tn, P.tiles = (int32_t)tiles, P.symmetric = C.symmetric;
  for (int i = 0; i < 8; ++i) P.pa[i] = C.pa[i], P.pb[i] = C.pb[i];
  static bool limit[PSK_MAX_DEVICES] = {};
  smem_limit_once((const void*)mm_kernel<CG, BN, KIND, SUM>, S::SMEM, limit);
  const int64_t most = device_sm_count() / CG, want = tiles * C.matrices;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((want < most ? want : most) * CG));
  cfg.blockDim = dim3(MM_THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 1 : 0;
  cudaLaunchKernelEx(&cfg, mm_kernel<CG, BN, KIND, SUM>, P);
  return check_launch("matrix product kernel");
}

template <int KIND>
static int launch_kind(const MMCall& C, cudaStream_t stream) {
  return C.pairs > 1 ? launch_shape<1, 128, KIND, true>(C, stream) : launch_shape<1, 128, KIND, false>(C, stream);
}

int mm_launch(const MMCall& C, cudaStream_t stream) {
  return C.kind == MM_LINEAR ? launch_kind<MM_LINEAR>(C, stream) : launch_kind<MM_ORTHO>(C, stream);
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
