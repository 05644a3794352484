// Dropout with a mask that is never stored: element (r, c) is kept or dropped
// by one 32-bit word of a counter-based generator, so the backward pass draws
// the same mask again from the same seed and offset.
//
// The generator is Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror,
// D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): ten
// rounds over a 128-bit counter (c0, c1, c2, c3) with a 64-bit key,
//   (c0, c1, c2, c3) <- (hi(M1 c2) ^ c1 ^ k0, lo(M1 c2), hi(M0 c0) ^ c3 ^ k1, lo(M0 c0)),
// the key advancing by two Weyl constants between rounds.  One call gives
// the words of four neighbouring columns: counter (c / 4, r, offset), so a
// group of four never straddles a row whatever its length.
#include "vec8.cuh"

namespace psk {

struct DropoutParams {
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy, cols;
  uint32_t row0;               // first row of this launch
  uint32_t items;              // threads' worth of work in this launch
  FastDiv per_row;             // and in a row
  uint32_t key[20];            // the ten round keys
  uint64_t offset;
  const uint64_t* counter;     // added to offset when the kernel runs; NULL for none
  uint32_t least_kept;         // words below this drop their element
  int32_t drop_all;
  float scale;
};

constexpr uint32_t PHILOX_M0 = 0xD2511F53u, PHILOX_M1 = 0xCD9E8D57u;
constexpr uint32_t PHILOX_W0 = 0x9E3779B9u, PHILOX_W1 = 0xBB67AE85u;
constexpr int SHIFT_THREADS = 256;         // of the shifted kernel
constexpr int DROP_THREADS = 128;          // 121 us for [32768, 4096] bf16 with residual; 256: 126

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const uint32_t* key) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)PHILOX_M0 * c0, b = (uint64_t)PHILOX_M1 * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ key[2 * r];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ key[2 * r + 1];
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The words' test costs every element; p = 1, which no 32-bit threshold
// expresses, has zero words and the threshold 1 instead.
__device__ __forceinline__ float dropped(float x, uint32_t w, const DropoutParams& P) {
  return w >= P.least_kept ? __fmul_rn(x, P.scale) : 0.0f;
}

// Integer instructions bind as hard as HBM (wide products run at a quarter of
// the lanes' rate, logic at half: the generator alone needs about 75 us for
// [32768, 4096]; bf16 with residual, 805 MB: 121 us, 6.6 TB/s, without, 537 MB:
// 107 us), so a thread takes NO groups of eight columns of one row, 256 columns
// apart, and shares among them its row's addresses and what the first two
// rounds know of row and offset.
// RT < 0: no residual.  VEC: rows of whole groups, moved by 16-byte accesses;
// all loads are issued before the generator's instructions.
template <int XT, int RT, int YT, bool VEC, int NO>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const __grid_constant__ DropoutParams P) {
  const uint64_t t = (uint64_t)blockIdx.x * DROP_THREADS + threadIdx.x;
  if (t >= P.items) return;
  const uint32_t r = P.per_row.div((uint32_t)t);
  const uint32_t g = (uint32_t)t - r * P.per_row.d;
  const uint32_t row = P.row0 + r;
  constexpr int RES = RT >= 0 ? RT : 0;
  // NO > 1: g is a lane of a slice of 256 NO columns.
  const int64_t c = NO > 1 ? (int64_t)(g >> 5) * (256 * NO) + (g & 31) * 8 : (int64_t)g * 8;
  Piece<XT, VEC, 8> x[NO];
  Piece<RES, VEC, 8> res[NO];
#pragma unroll
  for (int j = 0; j < NO; ++j) {
    const Columns<VEC, 8> cols(c + 256 * j, 1, 0, P.cols);
    cols.load(P.x, (int64_t)row * P.ldx, x[j]);
    if (RT >= 0) cols.load(P.res, (int64_t)row * P.ldr, res[j]);
  }
  const uint64_t off = P.offset + (P.counter ? *P.counter : 0);
#pragma unroll
  for (int j = 0; j < NO; ++j) {
    const uint32_t q = (uint32_t)(c >> 2) + 64 * j;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (!P.drop_all) {
      w0 = philox(q, row, (uint32_t)off, (uint32_t)(off >> 32), P.key);
      w1 = philox(q + 1, row, (uint32_t)off, (uint32_t)(off >> 32), P.key);
    }
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] = dropped(x[j].get(k), w[k], P);
      if (RT >= 0) y[k] = __fadd_rn(res[j].get(k), y[k]);
    }
    Columns<VEC, 8>(c + 256 * j, 1, 0, P.cols).template store<YT>(P.y, (int64_t)row * P.ldy, y);
  }
}

// Rows that begin anywhere, x, y and the residual of one type and alike: a
// thread's eight elements begin at a 16-byte boundary of the row, `shift`
// columns past a multiple of four, and take their words from three groups of
// four columns.  The third group is the first of the lane above: a warp has 31
// lanes with elements, and a row a last group of no elements, for their words
// ([16384, 3001] bf16 with residual: 72 us; each lane drawing three 87).  A
// row's first and last elements go one by one.
template <int TY, bool RES>
__global__ void __launch_bounds__(SHIFT_THREADS) dropout_shifted_kernel(const __grid_constant__ DropoutParams P) {
  constexpr int ESZ = TY == PSK_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const uint64_t w = ((uint64_t)blockIdx.x * SHIFT_THREADS + threadIdx.x) >> 5;
  if (w * 31 >= P.items) return;
  const uint64_t t = min(w * 31 + lane, (uint64_t)P.items - 1);   // past the end: the last row's words again
  const uint32_t r = P.per_row.div((uint32_t)t);
  const uint32_t g = (uint32_t)t - r * P.per_row.d;
  const uint32_t row = P.row0 + r;
  const int64_t xo = (int64_t)row * P.ldx, ro = (int64_t)row * P.ldr, yo = (int64_t)row * P.ldy;
  const int before = (int)(((uintptr_t)P.x + (uintptr_t)xo * ESZ) & 15u) / ESZ;   // elements from the boundary to column 0
  const int64_t c = (int64_t)g * 8 - before;
  const bool mine = lane < 31 && c < P.cols;
  const bool whole = mine && c >= 0 && c + 8 <= P.cols;
  const Columns<true, 8> cols(c, 1, 0, P.cols);
  Piece<TY, true, 8> x, res;
  float xv[8], rv[8];
  if (whole) {
    cols.load(P.x, xo, x);
    if (RES) cols.load(P.res, ro, res);
  } else if (mine) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = c + k >= 0 && c + k < P.cols;
      auto at = [&](const void* p, int64_t i) {
        return TY == PSK_BF16 ? bf16_bits_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
      };
      xv[k] = in ? at(P.x, xo + c + k) : 0.0f;
      rv[k] = RES && in ? at(P.res, ro + c + k) : 0.0f;
    }
  }
  const uint64_t off = P.offset + (P.counter ? *P.counter : 0);
  const uint32_t lo = (uint32_t)off, hi = (uint32_t)(off >> 32);
  const int shift = (int)(c & 3);
  const uint32_t quad = (uint32_t)(c >> 2);        // of columns before the row's first: words that nothing takes
  const uint4 w0 = philox(quad, row, lo, hi, P.key), w1 = philox(quad + 1, row, lo, hi, P.key);
  const uint4 w2 = make_uint4(__shfl_down_sync(0xFFFFFFFFu, w0.x, 1), __shfl_down_sync(0xFFFFFFFFu, w0.y, 1),
                              __shfl_down_sync(0xFFFFFFFFu, w0.z, 1), __shfl_down_sync(0xFFFFFFFFu, w0.w, 1));
  if (!mine) return;
  uint32_t word[12] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w, w2.x, w2.y, w2.z, w2.w};
#pragma unroll
  for (int k = 0; k < 11; ++k) word[k] = shift & 1 ? word[k + 1] : word[k];
#pragma unroll
  for (int k = 0; k < 9; ++k) word[k] = shift & 2 ? word[k + 2] : word[k];
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    y[k] = dropped(whole ? x.get(k) : xv[k], word[k], P);
    if (RES) y[k] = __fadd_rn(whole ? res.get(k) : rv[k], y[k]);
  }
  if (whole) {
    cols.template store<TY>(P.y, yo, y);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k >= 0 && c + k < P.cols) {
        if constexpr (TY == PSK_BF16) ((uint16_t*)P.y)[yo + c + k] = f32_to_bf16_bits(y[k]);
        else ((float*)P.y)[yo + c + k] = y[k];
      }
  }
}

}  // namespace psk

using namespace psk;

extern "C" int psk_dropout(const void* x, int32_t xt, const void* residual, int32_t rt, void* y, int32_t yt,
                           int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, int64_t ldy, double p, uint64_t seed,
                           uint64_t offset, const uint64_t* counter, void* stream) {
  clear_error();
  if (!dtype_ok(xt)) return fail(PSK_E_DTYPE, "x dtype %d", xt);
  if (!dtype_ok(yt)) return fail(PSK_E_DTYPE, "y dtype %d", yt);
  if (residual && !dtype_ok(rt)) return fail(PSK_E_DTYPE, "residual dtype %d", rt);
  if (!(p >= 0.0 && p <= 1.0)) return fail(PSK_E_ARG, "p %g is not in [0, 1]", p);
  if (rows < 0 || cols < 0) return fail(PSK_E_SHAPE, "rows %lld, cols %lld", (long long)rows, (long long)cols);
  if (rows > (1LL << 32)) return fail(PSK_E_SHAPE, "rows %lld above 2^32", (long long)rows);
  if (cols > (1LL << 34)) return fail(PSK_E_SHAPE, "cols %lld above 2^34", (long long)cols);
  if (rows == 0 || cols == 0) return PSK_OK;
  if (!x || !y) return fail(PSK_E_NULL, "x or y is NULL");
  if ((uintptr_t)x % dtype_size(xt) || (uintptr_t)y % dtype_size(yt) || (residual && (uintptr_t)residual % dtype_size(rt)))
    return fail(PSK_E_ARG, "x, y or the residual is not aligned to its type");
  if (ldx < cols || ldy < cols || (residual && ldr < cols)) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(rows, ldx) || !rows_addressable(rows, ldy) || (residual && !rows_addressable(rows, ldr)))
    return fail(PSK_E_SHAPE, "rows x leading dimension too large");
  if ((uintptr_t)counter % 8 != 0) return fail(PSK_E_ARG, "counter is not 8-byte aligned");
  const uint64_t xb = rows_bytes(rows, cols, ldx, xt), yb = rows_bytes(rows, cols, ldy, yt);
  if (ranges_overlap(x, xb, y, yb) && !(x == y && xt == yt && ldx == ldy))
    return fail(PSK_E_ALIAS, "y overlaps x and is not the same buffer");
  if (residual && ranges_overlap(residual, rows_bytes(rows, cols, ldr, rt), y, yb) &&
      !(residual == y && rt == yt && ldr == ldy))
    return fail(PSK_E_ALIAS, "y overlaps the residual and is not the same buffer");
  if (counter && ranges_overlap(counter, 8, y, yb)) return fail(PSK_E_ALIAS, "y overlaps the counter");

  DropoutParams P{};
  P.x = x, P.res = residual, P.y = y;
  P.ldx = ldx, P.ldr = ldr, P.ldy = ldy, P.cols = cols;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int r = 0; r < 10; ++r, k0 += PHILOX_W0, k1 += PHILOX_W1) P.key[2 * r] = k0, P.key[2 * r + 1] = k1;
  P.offset = offset, P.counter = counter;
  const uint64_t dropped = (uint64_t)__builtin_llrint(p * 4294967296.0);   // words below this drop
  P.drop_all = dropped >> 32 != 0;
  P.least_kept = P.drop_all ? 1u : (uint32_t)dropped;
  P.scale = (float)(1.0 / (1.0 - p));
  const bool vec = cols % 8 == 0 && rows_vec8(x, xt, ldx, rows) && rows_vec8(y, yt, ldy, rows) &&
                   (!residual || rows_vec8(residual, rt, ldr, rows));
  // Unaligned rows that begin equally far from a 16-byte boundary: shifted
  // groups (16384 x 3001 bf16 with residual: 72 us, element by element 114);
  // others element by element.
  auto alike = [&](const void* p, int32_t dt, int64_t ld) {
    return dt == xt && ((uintptr_t)p - (uintptr_t)x) % 16 == 0 && (rows == 1 || ((ld - ldx) * dtype_size(xt)) % 16 == 0);
  };
  const bool shifted = !vec && !P.drop_all && alike(y, yt, ldy) && (!residual || alike(residual, rt, ldr));
  // Four groups a thread, or two, where no more than an eighth of the lanes
  // stays idle past the row's end and every SM still has its threads.
  int groups = 1;
  for (int n = 4; n > 1 && groups == 1; n /= 2) {
    const int64_t span = 256 * n, padded = (cols + span - 1) / span * span;
    if (vec && padded - cols <= padded / 8 && rows * (padded / (8 * n)) >= 2048 * (int64_t)device_sm_count()) groups = n;
  }
  const uint64_t per_row = shifted      ? (uint64_t)(cols + 7 + 7) / 8 + 1
                           : groups > 1 ? (uint64_t)(cols + 256 * groups - 1) / (256 * groups) * 32
                                        : (uint64_t)(cols + 7) / 8;
  P.per_row = FastDiv((uint32_t)per_row);
  cudaStream_t s = (cudaStream_t)stream;
  // Slices of rows whose groups are counted in 32 bits (one slice up to
  // 2^35 elements).
  const uint64_t slice = 0xFFFFFFFFull / per_row;
  for (uint64_t r0 = 0; r0 < (uint64_t)rows; r0 += slice) {
    const uint64_t nr = (uint64_t)rows - r0 < slice ? (uint64_t)rows - r0 : slice;
    P.row0 = (uint32_t)r0;
    P.items = (uint32_t)(nr * per_row);
    const int threads = shifted ? SHIFT_THREADS : DROP_THREADS;
    const uint64_t lanes = shifted ? ((uint64_t)P.items + 30) / 31 * 32 : P.items;
    const unsigned grid = (unsigned)((lanes + threads - 1) / threads);
    with_dtype(xt, [&](auto XT) {
      if (shifted) {
        return with_bool(residual != nullptr, [&](auto RES) {
          dropout_shifted_kernel<XT.value, RES.value><<<grid, threads, 0, s>>>(P);
          return 0;
        });
      }
      return with_dtype(yt, [&](auto YT) {
        auto launch = [&](auto VEC, auto NO) {
          if (!residual)
            dropout_kernel<XT.value, -1, YT.value, VEC.value, NO.value><<<grid, threads, 0, s>>>(P);
          else if (rt == PSK_BF16)
            dropout_kernel<XT.value, PSK_BF16, YT.value, VEC.value, NO.value><<<grid, threads, 0, s>>>(P);
          else
            dropout_kernel<XT.value, PSK_F32, YT.value, VEC.value, NO.value><<<grid, threads, 0, s>>>(P);
          return 0;
        };
        if (groups == 4) return launch(std::true_type{}, std::integral_constant<int, 4>{});
        if (groups == 2) return launch(std::true_type{}, std::integral_constant<int, 2>{});
        return with_bool(vec, [&](auto VEC) { return launch(VEC, std::integral_constant<int, 1>{}); });
      });
    });
    const int rc = check_launch("dropout kernel");
    if (rc) return rc;
  }
  return PSK_OK;
}
