// psk_linear: y = act(x w + bias) + residual, and its backward.  The products
// run in matmul.cu; here are what prepares their operands and the host side.
//
// An operand stored in bf16 with 16-byte aligned rows goes to the tensor
// cores as it stands.  Any other is copied into the workspace first: rows
// padded to 16 bytes, and an f32 operand split into three bf16 parts, h =
// RN(x), m = RN(x - h), l = RN(x - h - m), whose sum is x to its last bit (24
// = 3 x 8 significant bits).  Of the nine products of parts the six above
// 2^-24 of the largest are added, from the smallest up; the three left out
// are below 2^-24 |x w| together.
#include "common.cuh"
#include "vec8.cuh"
#include "act.cuh"
#include "mm.h"
#include "views.h"

namespace psk {

constexpr int64_t LINEAR_MAX_SUM = 1LL << 25;      // of a product: a tile's time stays far below a wait's bound
constexpr int64_t LINEAR_MAX_SIDE = (1LL << 31) - 1024;
constexpr int PACK_THREADS = 256;

struct PackJob {
  const void *x, *z;            // z: the value is x slope(z)
  uint16_t* to;                 // planes of prows x pcols (NULL: column sums alone)
  float* sums;                  // column sums of `blocks` blocks of rows (NULL: not wanted)
  int64_t rows, cols, ldx, ldz, prows, pcols, plane_stride;
  int32_t planes, blocks, xt, vec;
};

// Up to three operands in one launch; job j has the CTAs from first[j] on.
struct PackParams {
  PackJob job[3];
  int32_t first[3], jobs;
};

// Eight columns a thread, 256 a CTA, its warps the rows of a block in turn,
// two rows on their way at once.  VEC: 16-byte accesses, the columns
// neighbours; else every 32nd, so that lanes read neighbours.
template <int XT, int ZT, int ACT, bool VEC>
__device__ __forceinline__ void pack_job(const PackJob& P, int64_t cta, float (&part)[8][256]) {
  constexpr int R = 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t groups = (P.pcols + 255) / 256;
  const int64_t cb = cta % groups, rb = cta / groups;
  // The span that is written, padding among it, and the part of it that is read.
  const Columns<VEC, 8> wide(cb * 256, 32, lane, P.pcols), cols(cb * 256, 32, lane, P.cols);
  const int64_t each = (P.prows + P.blocks - 1) / P.blocks;
  const int64_t end = (rb + 1) * each < P.prows ? (rb + 1) * each : P.prows;
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.0f;
  for (int64_t r0 = rb * each + warp; r0 < end; r0 += 8 * R) {
    Piece<XT, VEC, 8> x[R];
    Piece<ZT, VEC, 8> z[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = r0 + 8 * j;
      const bool there = r < end && r < P.rows;
      if (there) {
        cols.template load<XT>(P.x, r * P.ldx, x[j]);
      } else {
#pragma unroll
        for (int i = 0; i < Piece<XT, VEC, 8>::W; ++i) x[j].w[i] = 0;
      }
      if constexpr (ACT != ACT_NONE) {
        if (there) {
          cols.template load<ZT>(P.z, r * P.ldz, z[j]);
        } else {
#pragma unroll
          for (int i = 0; i < Piece<ZT, VEC, 8>::W; ++i) z[j].w[i] = 0;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = r0 + 8 * j;
      if (r >= end) break;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float2 t = make_float2(x[j].get(k), x[j].get(k + 1));
        if constexpr (ACT != ACT_NONE) t = __fmul2_rn(t, act_slope<ACT>(make_float2(z[j].get(k), z[j].get(k + 1))));
        v[k] = t.x, v[k + 1] = t.y;
        s[k] += t.x, s[k + 1] += t.y;
      }
      if (!P.to) continue;
      if (P.planes == 1) {
        wide.template store<PSK_BF16>(P.to, r * P.pcols, v);
      } else {
        // each part is what bf16 leaves of the value; an infinity or a NaN is the first part alone
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          float h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t b = f32_to_bf16_bits(v[k]);
            const bool finite = fabsf(v[k]) <= 3.4028234663852886e38f;
            if (finite && (b & 0x7FFF) == 0x7F80) b -= 1;      // rounded up to infinity: the largest bf16 instead
            h[k] = bf16_bits_to_f32(b);
            v[k] = finite ? v[k] - h[k] : 0.0f;
          }
          wide.template store<PSK_BF16>(P.to + p * P.plane_stride, r * P.pcols, h);
        }
      }
    }
  }
  if (!P.sums) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) part[warp][k * 32 + lane] = s[k];
  __syncthreads();
  const int t = threadIdx.x;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += part[w][t];
  const int64_t c = cb * 256 + (VEC ? (t & 31) * 8 + (t >> 5) : t);
  if (c < P.cols) P.sums[rb * P.cols + c] = sum;
}

// The first job's types are the kernel's; the others have no activation and
// no sums.
template <int XT, int ZT, int ACT, bool VEC>
__global__ void __launch_bounds__(PACK_THREADS, 3) linear_pack_kernel(const __grid_constant__ PackParams P) {
  __shared__ float part[8][256];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = (int)blockIdx.x;
  if (P.jobs == 1 || cta < P.first[1]) {
    pack_job<XT, ZT, ACT, VEC>(P.job[0], cta, part);
    return;
  }
  const int j = P.jobs == 3 && cta >= P.first[2] ? 2 : 1;
  const PackJob& J = P.job[j];
  if (J.xt == PSK_BF16) {
    if (J.vec) pack_job<PSK_BF16, PSK_BF16, ACT_NONE, true>(J, cta - P.first[j], part);
    else pack_job<PSK_BF16, PSK_BF16, ACT_NONE, false>(J, cta - P.first[j], part);
  } else {
    if (J.vec) pack_job<PSK_F32, PSK_BF16, ACT_NONE, true>(J, cta - P.first[j], part);
    else pack_job<PSK_F32, PSK_BF16, ACT_NONE, false>(J, cta - P.first[j], part);
  }
}

// dbias from the row blocks' sums where no product is launched: 32 columns a CTA, 8 warps the blocks in turn.
__global__ void __launch_bounds__(256) linear_bias_kernel(const float* sums, int blocks, int64_t cols, void* out,
                                                          int32_t dt, int32_t add) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int b = warp; b < blocks; b += 8) s += sums[(int64_t)b * cols + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp || c >= cols) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) s += part[w][lane];
  if (dt == PSK_BF16) {
    uint16_t* q = (uint16_t*)out + c;
    *q = f32_to_bf16_bits(add ? bf16_bits_to_f32(*q) + s : s);
  } else {
    float* q = (float*)out + c;
    *q = add ? *q + s : s;
  }
}

// ---------------------------------------------------------------------- host

static int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// A matrix of `rows` memory rows and where its tensor-core form stands.
struct Matrix {
  const void* p;
  int32_t dt;
  int64_t rows, cols, ld;
  bool packed;
  int planes;
  int64_t prows, pcols;
  uint64_t offset, bytes;       // in the workspace, when packed
};

static Matrix matrix(const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld, uint64_t* used) {
  Matrix m{p, dt, rows, cols, ld};
  m.planes = dt == PSK_F32 ? 3 : 1;
  m.packed = dt == PSK_F32 || rows == 0 || cols == 0 || !rows_vec8(p, dt, ld, rows);
  m.prows = rows ? rows : 1, m.pcols = cols ? up8(cols) : 8;
  m.offset = *used;
  m.bytes = m.packed ? ((uint64_t)m.planes * m.prows * m.pcols * 2 + 255) / 256 * 256 : 0;
  *used += m.bytes;
  return m;
}

static MMOperand operand(const Matrix& m, void* workspace, bool k_inner) {
  MMOperand o{};
  o.planes = m.planes, o.k_inner = k_inner;
  if (m.packed) {
    o.p = (char*)workspace + m.offset;
    o.inner = m.cols ? m.cols : 8, o.outer = m.prows, o.ld = m.pcols;
  } else {
    o.p = m.p, o.inner = m.cols, o.outer = m.rows, o.ld = m.rows > 1 ? m.ld : up8(m.cols);
  }
  o.plane_stride = o.ld * o.outer;
  return o;
}

// Blocks of rows of the pack kernel: six CTAs an SM (twice what it holds) of 32
// rows each at least, or of 16 where those are fewer than half the SMs (128 x
// 512 x 128 f32 10.0 us, 8.8; 2000 x 512 x 1024's gradients stay at 32: 22.7, 24.6).
static int pack_blocks(int64_t rows, int64_t cols) {
  const int64_t groups = (cols + 255) / 256;
  const int64_t each = (rows + 31) / 32 * groups < NOMINAL_SMS / 2 ? 16 : 32;
  int64_t b = NOMINAL_SMS * 6 / groups;
  if (b > (rows + each - 1) / each) b = (rows + each - 1) / each;
  return (int)(b < 1 ? 1 : b);
}

// The operands to be packed, in one launch.
struct Packing {
  PackParams P{};
  int64_t ctas = 0;
  int32_t act = ACT_NONE, zt = PSK_BF16;
  // The first one may have an activation's slope and column sums.
  void add(const Matrix& m, void* workspace, bool store = true, const void* z = nullptr, int32_t z_type = PSK_BF16,
           int64_t ldz = 0, int32_t slope = ACT_NONE, float* sums = nullptr) {
    PackJob& J = P.job[P.jobs];
    J.x = m.p, J.z = z;
    J.to = store ? (uint16_t*)((char*)workspace + m.offset) : nullptr;
    J.sums = sums;
    J.rows = m.rows, J.cols = m.cols, J.ldx = m.ld, J.ldz = ldz;
    J.prows = m.prows, J.pcols = m.pcols, J.plane_stride = m.prows * m.pcols;
    J.planes = m.planes, J.xt = m.dt;
    J.vec = m.cols % 8 == 0 && rows_vec8(m.p, m.dt, m.ld, m.rows) && (!slope || rows_vec8(z, z_type, ldz, m.rows));
    J.blocks = pack_blocks(m.prows, m.pcols);
    if (!P.jobs) act = slope, zt = z_type;
    P.first[P.jobs++] = (int32_t)(ctas < 0x7FFFFFFF ? ctas : 0x7FFFFFFF);
    ctas += (m.pcols + 255) / 256 * J.blocks;
  }
  int launch(cudaStream_t s) const {
    if (!P.jobs) return PSK_OK;
    if (ctas > 0x7FFFFFFF) return fail(PSK_E_SHAPE, "too many blocks");
    const unsigned grid = (unsigned)ctas;
    with_dtype(P.job[0].xt, [&](auto XT) {
      return with_bool(P.job[0].vec != 0, [&](auto VEC) {
        if (act == ACT_NONE) {
          linear_pack_kernel<XT.value, PSK_BF16, ACT_NONE, VEC.value><<<grid, PACK_THREADS, 0, s>>>(P);
          return 0;
        }
        return with_dtype(zt, [&](auto ZT) {
          if (act == ACT_RELU) linear_pack_kernel<XT.value, ZT.value, ACT_RELU, VEC.value><<<grid, PACK_THREADS, 0, s>>>(P);
          else if (act == ACT_GELU) linear_pack_kernel<XT.value, ZT.value, ACT_GELU, VEC.value><<<grid, PACK_THREADS, 0, s>>>(P);
          else linear_pack_kernel<XT.value, ZT.value, ACT_SILU, VEC.value><<<grid, PACK_THREADS, 0, s>>>(P);
          return 0;
        });
      });
    });
    return check_launch("linear pack kernel");
  }
};

// The products of the operands' planes, smallest first.
static void plane_pairs(MMCall& C) {
  C.pairs = 0;
  for (int sum = 2; sum >= 0; --sum)
    for (int a = 0; a <= sum; ++a)
      if (a < C.a.planes && sum - a < C.b.planes) C.pa[C.pairs] = a, C.pb[C.pairs] = sum - a, ++C.pairs;
}

static int check_side(const char* what, int64_t v, int64_t most) {
  if (v < 0 || v > most) return fail(PSK_E_SHAPE, "%s %lld is not in [0, %lld]", what, (long long)v, (long long)most);
  return PSK_OK;
}

static int check_rows(const char* what, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!dtype_ok(dt)) return fail(PSK_E_DTYPE, "%s dtype %d", what, dt);
  if (ld < cols) return fail(PSK_E_SHAPE, "%s: leading dimension %lld below %lld", what, (long long)ld, (long long)cols);
  if (!rows_addressable(rows, ld)) return fail(PSK_E_SHAPE, "%s: rows x leading dimension too large", what);
  if (rows && cols && !p) return fail(PSK_E_NULL, "%s is NULL", what);
  if ((uintptr_t)p % dtype_size(dt)) return fail(PSK_E_ARG, "%s is not aligned to its type", what);
  return PSK_OK;
}

struct Named {
  const char* name;
  View view;
};

static View mat_view(const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!p) return View{0, 0, 0, 0};
  return view_of(p, rows, cols, ld, dtype_size(dt));
}

static int check_apart(const Named& out, const Named* others, int n) {
  for (int i = 0; i < n; ++i)
    if (views_overlap(out.view, others[i].view)) return fail(PSK_E_ALIAS, "%s overlaps %s", out.name, others[i].name);
  return PSK_OK;
}

static int check_workspace(const void* workspace, uint64_t bytes, uint64_t need) {
  if (!need) return PSK_OK;
  if (!workspace) return fail(PSK_E_NULL, "workspace is NULL, %llu bytes needed", (unsigned long long)need);
  if ((uintptr_t)workspace % 16) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
  if (bytes < need)
    return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)bytes, (unsigned long long)need);
  return PSK_OK;
}

static int check_layout(int32_t layout) {
  if (layout != PSK_W_IN_OUT && layout != PSK_W_OUT_IN) return fail(PSK_E_ARG, "weight layout %d", layout);
  return PSK_OK;
}

static int check_act(int32_t act) {
  if (act < PSK_ACT_NONE || act > PSK_ACT_SILU) return fail(PSK_E_ARG, "activation %d", act);
  return PSK_OK;
}

// The checked operands of both directions.
static int check_operands(const void* x, int32_t xt, int64_t ldx, const void* w, int32_t wt, int64_t ldw,
                          int32_t layout, int64_t rows, int64_t in, int64_t out) {
  int rc = check_side("rows", rows, LINEAR_MAX_SIDE);
  if (!rc) rc = check_side("in", in, LINEAR_MAX_SUM);
  if (!rc) rc = check_side("out", out, LINEAR_MAX_SIDE);
  if (!rc) rc = check_layout(layout);
  if (!rc) rc = check_rows("x", x, xt, rows, in, ldx);
  if (!rc) rc = layout == PSK_W_IN_OUT ? check_rows("w", w, wt, in, out, ldw) : check_rows("w", w, wt, out, in, ldw);
  return rc;
}

static Matrix weight(const void* w, int32_t wt, int64_t ldw, int32_t layout, int64_t in, int64_t out, uint64_t* used) {
  return layout == PSK_W_IN_OUT ? matrix(w, wt, in, out, ldw, used) : matrix(w, wt, out, in, ldw, used);
}

}  // namespace psk

using namespace psk;

extern "C" int psk_linear_workspace(const void* x, int32_t xt, int64_t ldx, const void* w, int32_t wt, int64_t ldw,
                                    int32_t layout, int64_t rows, int64_t in, int64_t out, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = check_operands(x, xt, ldx, w, wt, ldw, layout, rows, in, out);
  if (rc) return rc;
  *bytes = 0;
  if (!rows || !out) return PSK_OK;
  matrix(x, xt, rows, in, ldx, bytes);
  weight(w, wt, ldw, layout, in, out, bytes);
  return PSK_OK;
}

extern "C" int psk_linear(const void* x, int32_t xt, int64_t ldx, const void* w, int32_t wt, int64_t ldw,
                          int32_t layout, int64_t rows, int64_t in, int64_t out, const void* bias, int32_t bt,
                          int32_t act, const void* residual, int32_t rt, int64_t ldr, void* z, int32_t zt, int64_t ldz,
                          void* y, int32_t yt, int64_t ldy, void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  int rc = check_operands(x, xt, ldx, w, wt, ldw, layout, rows, in, out);
  if (!rc) rc = check_act(act);
  if (!rc && bias) rc = check_rows("bias", bias, bt, 1, out, out);
  if (!rc && residual) rc = check_rows("residual", residual, rt, rows, out, ldr);
  if (!rc && z) rc = check_rows("z", z, zt, rows, out, ldz);
  if (!rc) rc = check_rows("y", y, yt, rows, out, ldy);
  if (rc || !rows || !out) return rc;
  uint64_t need = 0;
  const Matrix mx = matrix(x, xt, rows, in, ldx, &need), mw = weight(w, wt, ldw, layout, in, out, &need);
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc) return rc;
  const View vy = mat_view(y, yt, rows, out, ldy), vz = mat_view(z, zt, rows, out, ldz),
             vr = mat_view(residual, rt, rows, out, ldr);
  const View vws{(uintptr_t)workspace, need ? 1 : 0, need, need};
  const Named read[] = {{"x", mat_view(x, xt, mx.rows, mx.cols, ldx)},
                        {"w", mat_view(w, wt, mw.rows, mw.cols, ldw)},
                        {"the bias", mat_view(bias, bt, 1, out, out)},
                        {"the workspace", vws},
                        {"z", vz}};
  rc = check_apart({"y", vy}, read, 5);
  if (!rc && views_overlap(vy, vr) && !(same_view(vy, vr) && yt == rt))
    rc = fail(PSK_E_ALIAS, "y overlaps the residual and is not the same buffer");
  if (!rc && z) rc = check_apart({"z", vz}, read, 4);
  if (!rc && z && views_overlap(vz, vr)) rc = fail(PSK_E_ALIAS, "z overlaps the residual");
  if (!rc) rc = check_apart({"the workspace", vws}, read, 3);
  if (!rc && views_overlap(vws, vr)) rc = fail(PSK_E_ALIAS, "the workspace overlaps the residual");
  if (rc) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  Packing K;
  if (mx.packed) K.add(mx, workspace);
  if (mw.packed) K.add(mw, workspace);
  rc = K.launch(s);
  if (rc) return rc;
  MMCall C{};
  C.m = rows, C.n = out, C.k = in ? in : 1, C.matrices = 1;
  C.a = operand(mx, workspace, true);
  C.b = operand(mw, workspace, layout == PSK_W_OUT_IN);
  plane_pairs(C);
  MMEpilogue& E = C.e;
  E.bias = bias, E.bt = bt, E.act = act;
  E.res = residual, E.rt = rt, E.ldr = ldr;
  E.z = z, E.zt = zt, E.ldz = ldz;
  E.y = y, E.yt = yt, E.ldy = ldy;
  return mm_launch(&C, 1, nullptr, s);
}

namespace psk {

// The backward's operands and where they stand in the workspace.  dz carries
// three parts where a product stored in f32 reads it, or where it is f32.
struct LinearBackward {
  Matrix x, w, dz;
  bool want_dx, want_dw, want_db, direct;    // direct: dz is ct as it stands
  int dx_planes, dw_planes;                  // of dz, in each product
  int blocks;
  uint64_t sums, need;
};

static void plan_backward(LinearBackward& B, const void* ct, int32_t ct_t, int64_t ldc, const void* x, int32_t xt,
                          int64_t ldx, const void* w, int32_t wt, int64_t ldw, int32_t layout, int64_t rows,
                          int64_t in, int64_t out, int32_t act, const void* dx, int32_t dxt, const void* dw,
                          int32_t dwt, const void* db) {
  B.need = 0;
  B.want_dx = dx && rows && in, B.want_dw = dw && in && out, B.want_db = db && out;
  uint64_t none = 0;
  B.x = matrix(x, xt, rows, in, ldx, B.want_dw ? &B.need : &none);
  B.w = weight(w, wt, ldw, layout, in, out, B.want_dx ? &B.need : &none);
  // With an activation dz is rounded: to bf16 where that is the product's own
  // storage (a rounding beside ct's and the result's), else kept in three parts.
  const bool act_on = act != PSK_ACT_NONE;
  const auto planes = [&](int32_t result, int32_t other) {
    return ct_t == PSK_F32 || (act_on && (result == PSK_F32 || other == PSK_F32)) ? 3 : 1;
  };
  B.dx_planes = planes(dxt, wt), B.dw_planes = planes(dwt, xt);
  B.dz = Matrix{ct, ct_t, rows, out, ldc};
  B.dz.planes = (B.want_dx && B.dx_planes == 3) || (B.want_dw && B.dw_planes == 3) ? 3 : 1;
  B.direct = !act_on && ct_t == PSK_BF16 && rows && out && rows_vec8(ct, ct_t, ldc, rows);
  B.dz.packed = !B.direct;
  B.dz.prows = rows ? rows : 1, B.dz.pcols = out ? up8(out) : 8;
  B.dz.offset = B.need;
  if (!B.direct && (B.want_dx || B.want_dw))
    B.need += ((uint64_t)B.dz.planes * B.dz.prows * B.dz.pcols * 2 + 255) / 256 * 256;
  B.blocks = pack_blocks(B.dz.prows, B.dz.pcols);
  B.sums = B.need;
  if (B.want_db) B.need += ((uint64_t)B.blocks * out * 4 + 255) / 256 * 256;
}

static int check_backward(const void* ct, int32_t ct_t, int64_t ldc, const void* x, int32_t xt, int64_t ldx,
                          const void* w, int32_t wt, int64_t ldw, int32_t layout, int64_t rows, int64_t in,
                          int64_t out, int32_t act, const void* dx, int32_t dxt, const void* dw, int32_t dwt,
                          const void* db, int32_t dbt) {
  int rc = check_side("rows", rows, LINEAR_MAX_SUM);
  if (!rc) rc = check_side("in", in, LINEAR_MAX_SIDE);
  if (!rc) rc = check_side("out", out, LINEAR_MAX_SUM);
  if (!rc) rc = check_layout(layout);
  if (!rc) rc = check_act(act);
  if (!rc) rc = check_rows("ct", ct, ct_t, rows, out, ldc);
  if (!rc && dw) rc = check_rows("x", x, xt, rows, in, ldx);
  if (!rc && dx)
    rc = layout == PSK_W_IN_OUT ? check_rows("w", w, wt, in, out, ldw) : check_rows("w", w, wt, out, in, ldw);
  if (!rc && dx && !dtype_ok(dxt)) rc = fail(PSK_E_DTYPE, "dx dtype %d", dxt);
  if (!rc && dw && !dtype_ok(dwt)) rc = fail(PSK_E_DTYPE, "dw dtype %d", dwt);
  if (!rc && db && !dtype_ok(dbt)) rc = fail(PSK_E_DTYPE, "dbias dtype %d", dbt);
  return rc;
}

}  // namespace psk

extern "C" int psk_linear_backward_workspace(const void* ct, int32_t ct_t, int64_t ldc, const void* x, int32_t xt,
                                             int64_t ldx, const void* w, int32_t wt, int64_t ldw, int32_t layout,
                                             int64_t rows, int64_t in, int64_t out, int32_t act, const void* dx,
                                             int32_t dxt, const void* dw, int32_t dwt, const void* dbias, int32_t dbt,
                                             uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = check_backward(ct, ct_t, ldc, x, xt, ldx, w, wt, ldw, layout, rows, in, out, act, dx, dxt, dw, dwt,
                                dbias, dbt);
  if (rc) return rc;
  LinearBackward B{};
  plan_backward(B, ct, ct_t, ldc, x, xt, ldx, w, wt, ldw, layout, rows, in, out, act, dx, dxt, dw, dwt, dbias);
  *bytes = B.need;
  return PSK_OK;
}

extern "C" int psk_linear_backward(const void* ct, int32_t ct_t, int64_t ldc, const void* x, int32_t xt, int64_t ldx,
                                   const void* w, int32_t wt, int64_t ldw, int32_t layout, int64_t rows, int64_t in,
                                   int64_t out, int32_t act, const void* z, int32_t zt, int64_t ldz, void* dx,
                                   int32_t dxt, int64_t lddx, void* dw, int32_t dwt, int64_t lddw, void* dbias,
                                   int32_t dbt, int32_t accumulate, void* workspace, uint64_t workspace_bytes,
                                   void* stream) {
  clear_error();
  int rc = check_backward(ct, ct_t, ldc, x, xt, ldx, w, wt, ldw, layout, rows, in, out, act, dx, dxt, dw, dwt, dbias,
                          dbt);
  if (!rc && act != PSK_ACT_NONE) rc = check_rows("z", z, zt, rows, out, ldz);
  if (!rc && dx) rc = check_rows("dx", dx, dxt, rows, in, lddx);
  const int64_t wrows = layout == PSK_W_IN_OUT ? in : out, wcols = layout == PSK_W_IN_OUT ? out : in;
  if (!rc && dw) rc = check_rows("dw", dw, dwt, wrows, wcols, lddw);
  if (!rc && dbias) rc = check_rows("dbias", dbias, dbt, 1, out, out);
  if (rc) return rc;
  LinearBackward B{};
  plan_backward(B, ct, ct_t, ldc, x, xt, ldx, w, wt, ldw, layout, rows, in, out, act, dx, dxt, dw, dwt, dbias);
  rc = check_workspace(workspace, workspace_bytes, B.need);
  if (rc) return rc;
  const View vws{(uintptr_t)workspace, B.need ? 1 : 0, B.need, B.need};
  const Named read[] = {{"ct", mat_view(ct, ct_t, rows, out, ldc)},
                        {"z", act != PSK_ACT_NONE ? mat_view(z, zt, rows, out, ldz) : View{0, 0, 0, 0}},
                        {"x", dw ? mat_view(x, xt, rows, in, ldx) : View{0, 0, 0, 0}},
                        {"w", dx ? mat_view(w, wt, wrows, wcols, ldw) : View{0, 0, 0, 0}},
                        {"the workspace", vws}};
  const Named wrote[] = {{"dx", mat_view(dx, dxt, rows, in, lddx)},
                         {"dw", mat_view(dw, dwt, wrows, wcols, lddw)},
                         {"dbias", mat_view(dbias, dbt, 1, out, out)}};
  for (int i = 0; !rc && i < 3; ++i) {
    rc = check_apart(wrote[i], read, 5);
    if (!rc) rc = check_apart(wrote[i], wrote + i + 1, 2 - i);
  }
  if (!rc) rc = check_apart({"the workspace", vws}, read, 4);
  if (rc) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  const bool products = B.want_dx || B.want_dw;
  float* sums = B.want_db ? (float*)((char*)workspace + B.sums) : nullptr;
  Packing K;
  if (B.want_db || (products && !B.direct)) K.add(B.dz, workspace, products && !B.direct, z, zt, ldz, act, sums);
  if (B.want_dx && B.w.packed) K.add(B.w, workspace);
  if (B.want_dw && B.x.packed) K.add(B.x, workspace);
  rc = K.launch(s);
  if (rc) return rc;
  if (B.want_db && !products) {
    linear_bias_kernel<<<(unsigned)((out + 31) / 32), 256, 0, s>>>(sums, B.blocks, out, dbias, dbt, accumulate != 0);
    return check_launch("linear bias kernel");
  }
  if (!products) return PSK_OK;
  MMCall C[2] = {};
  int count = 0;
  if (B.want_dx) {
    MMCall& D = C[count++];
    D.m = rows, D.n = in, D.k = out ? out : 1, D.matrices = 1;
    D.a = operand(B.dz, workspace, true);
    D.a.planes = B.dx_planes;
    D.b = operand(B.w, workspace, layout == PSK_W_IN_OUT);
    plane_pairs(D);
    D.e.y = dx, D.e.yt = dxt, D.e.ldy = lddx;
  }
  if (B.want_dw) {
    MMCall& D = C[count++];
    MMOperand ox = operand(B.x, workspace, false), oz = operand(B.dz, workspace, false);
    oz.planes = B.dw_planes;
    D.m = wrows, D.n = wcols, D.k = rows ? rows : 1, D.matrices = 1;
    D.a = layout == PSK_W_IN_OUT ? ox : oz;
    D.b = layout == PSK_W_IN_OUT ? oz : ox;
    plane_pairs(D);
    D.e.y = dw, D.e.yt = dwt, D.e.ldy = lddw;
    if (accumulate) D.e.res = dw, D.e.rt = dwt, D.e.ldr = lddw;
  }
  const MMColumnSums J{sums, dbias, out, B.blocks, dbt, accumulate != 0};
  return mm_launch(C, count, B.want_db ? &J : nullptr, s);
}
