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
  uint32_t items;              // groups of eight columns in this launch
  FastDiv per_row;             // groups per row
  uint32_t key[20];            // the ten round keys
  uint64_t offset;
  const uint64_t* counter;     // added to offset when the kernel runs; NULL for none
  uint32_t last_dropped;       // words <= this drop their element
  int32_t keep_all;
  float scale;
};

constexpr uint32_t PHILOX_M0 = 0xD2511F53u, PHILOX_M1 = 0xCD9E8D57u;
constexpr uint32_t PHILOX_W0 = 0x9E3779B9u, PHILOX_W1 = 0xBB67AE85u;
constexpr int DROP_THREADS = 256;

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

// One group of eight columns a thread; RT < 0: no residual.  VEC: rows of
// whole groups, moved by 16-byte accesses, all loads issued before the
// generator's instructions, which hide their latency.
template <int XT, int RT, int YT, bool VEC>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const __grid_constant__ DropoutParams P) {
  const uint64_t t = (uint64_t)blockIdx.x * DROP_THREADS + threadIdx.x;
  if (t >= P.items) return;
  const uint32_t r = P.per_row.div((uint32_t)t);
  const uint32_t g = (uint32_t)t - r * P.per_row.d;
  const uint32_t row = P.row0 + r;
  constexpr int RES = RT >= 0 ? RT : 0;
  const int64_t c = (int64_t)g * 8;
  const Columns<VEC, 8> cols(c, 1, 0, P.cols);
  Piece<XT, VEC, 8> x;
  Piece<RES, VEC, 8> res;
  cols.load(P.x, (int64_t)row * P.ldx, x);
  if (RT >= 0) cols.load(P.res, (int64_t)row * P.ldr, res);
  const uint64_t off = P.offset + (P.counter ? *P.counter : 0);
  const uint4 w0 = philox(2 * g, row, (uint32_t)off, (uint32_t)(off >> 32), P.key);
  const uint4 w1 = philox(2 * g + 1, row, (uint32_t)off, (uint32_t)(off >> 32), P.key);
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    y[k] = (w[k] > P.last_dropped || P.keep_all) ? __fmul_rn(x.get(k), P.scale) : 0.0f;
    if (RT >= 0) y[k] = __fadd_rn(res.get(k), y[k]);
  }
  cols.template store<YT>(P.y, (int64_t)row * P.ldy, y);
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
  const uint64_t per_row = (uint64_t)(cols + 7) / 8;
  P.per_row = FastDiv((uint32_t)per_row);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int r = 0; r < 10; ++r, k0 += PHILOX_W0, k1 += PHILOX_W1) P.key[2 * r] = k0, P.key[2 * r + 1] = k1;
  P.offset = offset, P.counter = counter;
  const uint64_t dropped = (uint64_t)__builtin_llrint(p * 4294967296.0);   // words below this drop
  P.keep_all = dropped == 0;
  P.last_dropped = (uint32_t)(dropped - 1);
  P.scale = (float)(1.0 / (1.0 - p));
  const bool vec = cols % 8 == 0 && rows_vec8(x, xt, ldx, rows) && rows_vec8(y, yt, ldy, rows) &&
                   (!residual || rows_vec8(residual, rt, ldr, rows));
  cudaStream_t s = (cudaStream_t)stream;
  // Slices of rows whose groups are counted in 32 bits (one slice up to
  // 2^35 elements).
  const uint64_t slice = 0xFFFFFFFFull / per_row;
  for (uint64_t r0 = 0; r0 < (uint64_t)rows; r0 += slice) {
    const uint64_t nr = (uint64_t)rows - r0 < slice ? (uint64_t)rows - r0 : slice;
    P.row0 = (uint32_t)r0;
    P.items = (uint32_t)(nr * per_row);
    const unsigned grid = (unsigned)(((uint64_t)P.items + DROP_THREADS - 1) / DROP_THREADS);
    with_dtype(xt, [&](auto XT) {
      return with_dtype(yt, [&](auto YT) {
        return with_bool(vec, [&](auto VEC) {
          if (!residual)
            dropout_kernel<XT.value, -1, YT.value, VEC.value><<<grid, DROP_THREADS, 0, s>>>(P);
          else if (rt == PSK_BF16)
            dropout_kernel<XT.value, PSK_BF16, YT.value, VEC.value><<<grid, DROP_THREADS, 0, s>>>(P);
          else
            dropout_kernel<XT.value, PSK_F32, YT.value, VEC.value><<<grid, DROP_THREADS, 0, s>>>(P);
          return 0;
        });
      });
    });
    const int rc = check_launch("dropout kernel");
    if (rc) return rc;
  }
  return PSK_OK;
}
