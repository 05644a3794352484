// The token embedding and its gradient.
//
// Forward: a gather of table rows, scaled.  Backward: the leaf's gradient
//   dtable[v, :] = scale * sum of ct[i, :] over the positions i with id v,
// without atomics: positions are sorted by id (a stable radix sort, so each
// id's positions stay in increasing order), the sorted list is cut into runs
// of EMB_RUN entries, each run is summed left to right by its own warps, and
// an id whose entries span several runs has its run sums joined left to
// right.  The order of every sum is fixed by the ids alone.
#include "vec8.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace psk {

constexpr int EMB_THREADS = 256;
constexpr int EMB_RUN = 32;               // sorted entries a warp sums (one id per lane)
constexpr int SORT_CTAS = 8;              // one cluster
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BITS = 8;              // digit of a pass
constexpr int SORT_BINS = 1 << SORT_BITS;
constexpr int SORT_PER_LANE = 8;          // entries a lane ranks in one tile
constexpr int SORT_TILE = SORT_THREADS * SORT_PER_LANE;

// ------------------------------------------------------------------ forward

struct EmbedParams {
  const void* ids;
  const void* table;
  void* y;
  int64_t vocab, cols, ldt, ldy;
  int64_t row0;
  uint32_t items;
  FastDiv per_row;
  float scale;
};

template <bool I64>
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i) {
  return I64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

template <int TT, int YT, bool I64, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) embed_kernel(const __grid_constant__ EmbedParams P) {
  const uint64_t t = (uint64_t)blockIdx.x * EMB_THREADS + threadIdx.x;
  if (t >= P.items) return;
  const uint32_t r = P.per_row.div((uint32_t)t);
  const int64_t c = (int64_t)((uint32_t)t - r * P.per_row.d) * 8;
  const int64_t left = P.cols - c;
  const int n = left < 8 ? (int)left : 8;
  const int64_t row = P.row0 + r;
  const int64_t id = load_id<I64>(P.ids, row);
  float v[8] = {};
  if (id >= 0 && id < P.vocab) {
    load8<TT, VEC>(P.table, id * P.ldt + c, n, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], P.scale);
  }
  store8<YT, VEC>(P.y, row * P.ldy + c, n, v);
}

// ----------------------------------------------------------------- backward

struct EmbedGradParams {
  const void* ids;
  const void* ct;
  void* d;
  int64_t vocab, cols, ldc, ldd;
  int64_t tokens;
  uint32_t* key[2];      // sort buffers: ids (vocab for a position without one) ...
  uint32_t* pos[2];      // ... and their positions
  float* head;           // per run: the sum of its leading entries whose id the run before ends with
  float* tail;           // per run: the sum of its trailing entries whose id the next run goes on with
  int64_t pcols;         // row length of head and tail
  int32_t passes, out;   // radix passes and the buffer the last one writes
  int32_t bits;          // digit bits of each pass
  int32_t accumulate;
  int32_t slices;        // column slices of 256 of a row
  float scale;
};

// Zero the rows of the gradient (8 columns a step).
template <int DT, bool VEC>
__device__ void zero_rows(const EmbedGradParams& P, int64_t first, int64_t step) {
  const float z[8] = {};
  const uint32_t per_row = (uint32_t)((P.cols + 7) / 8);
  const int64_t total = P.vocab * per_row;
  for (int64_t t = first; t < total; t += step) {
    const int64_t r = t / per_row;
    const int64_t c = (t - r * per_row) * 8;
    store8<DT, VEC>(P.d, r * P.ldd + c, (int)(P.cols - c < 8 ? P.cols - c : 8), z);
  }
}

// Cluster 0 sorts the positions by id; the other clusters meanwhile zero the
// gradient (when it is not accumulated into), so the sort's latency hides
// behind the store of the rows that no position has.
//
// One radix pass: every CTA counts the digits of its own range of entries;
// the counts of all CTAs, read through distributed shared memory, give each
// digit's first place for this CTA's entries; then tile by tile each warp
// ranks its entries among equal digits in order (match_any), and the entries
// move to their places.  Entries live in global memory (L2); the cluster
// barrier orders the passes.
template <bool I64, int DT, bool VEC>
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS)
    embed_sort_kernel(const __grid_constant__ EmbedGradParams P) {
  if (blockIdx.x >= SORT_CTAS) {
    zero_rows<DT, VEC>(P, (int64_t)(blockIdx.x - SORT_CTAS) * SORT_THREADS + threadIdx.x,
                       (int64_t)(gridDim.x - SORT_CTAS) * SORT_THREADS);
    return;
  }
  __shared__ uint32_t count[SORT_BINS];               // this CTA's digit counts (read by the cluster)
  __shared__ uint32_t place[SORT_BINS];               // next place of each digit
  __shared__ uint32_t warp_count[SORT_WARPS][SORT_BINS];
  __shared__ uint32_t scan[SORT_BINS];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)blockIdx.x;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per = (((P.tokens + SORT_CTAS - 1) / SORT_CTAS) + 31) / 32 * 32;
  const int64_t begin = rank * per < P.tokens ? rank * per : P.tokens;
  const int64_t end = begin + per < P.tokens ? begin + per : P.tokens;

  auto read_key = [&](int pass, int64_t i) -> uint32_t {
    if (pass > 0) return __ldcg(P.key[(pass - 1) & 1] + i);
    const int64_t id = load_id<I64>(P.ids, i);
    return id >= 0 && id < P.vocab ? (uint32_t)id : (uint32_t)P.vocab;
  };
  const uint32_t mask = (1u << P.bits) - 1;
  for (int pass = 0; pass < P.passes; ++pass) {
    const int shift = pass * P.bits;
    for (int b = tid; b < SORT_BINS; b += SORT_THREADS) count[b] = 0;
    __syncthreads();
    for (int64_t i = begin + tid; i < end; i += SORT_THREADS)
      atomicAdd(&count[(read_key(pass, i) >> shift) & mask], 1u);
    cluster.sync();
    // place[b] = entries with a smaller digit anywhere + with digit b in the CTAs before.
    uint32_t before = 0, total = 0;
    if (tid < SORT_BINS) {
      for (int q = 0; q < SORT_CTAS; ++q) {
        const uint32_t n = *cluster.map_shared_rank(&count[tid], q);
        if (q < rank) before += n;
        total += n;
      }
      scan[tid] = total;
    }
    __syncthreads();
    for (int step = 1; step < SORT_BINS; step <<= 1) {
      uint32_t v = 0;
      if (tid < SORT_BINS && tid >= step) v = scan[tid - step];
      __syncthreads();
      if (tid < SORT_BINS) scan[tid] += v;
      __syncthreads();
    }
    if (tid < SORT_BINS) place[tid] = scan[tid] - total + before;
    __syncthreads();
    for (int64_t t0 = begin; t0 < end; t0 += SORT_TILE) {
      for (int b = tid; b < SORT_WARPS * SORT_BINS; b += SORT_THREADS) (&warp_count[0][0])[b] = 0;
      __syncthreads();
      uint32_t key[SORT_PER_LANE], p[SORT_PER_LANE], rnk[SORT_PER_LANE];
      const int64_t w0 = t0 + (int64_t)warp * (32 * SORT_PER_LANE) + lane;
#pragma unroll
      for (int k = 0; k < SORT_PER_LANE; ++k) {
        const int64_t i = w0 + 32 * k;
        key[k] = i < end ? read_key(pass, i) : 0u;
        p[k] = i < end ? (pass > 0 ? __ldcg(P.pos[(pass - 1) & 1] + i) : (uint32_t)i) : 0u;
      }
#pragma unroll
      for (int k = 0; k < SORT_PER_LANE; ++k) {
        const bool in = w0 + 32 * k < end;
        const uint32_t digit = in ? (key[k] >> shift) & mask : SORT_BINS;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
        const uint32_t below = __popc(peers & ((1u << lane) - 1));
        rnk[k] = 0;
        if (in) rnk[k] = warp_count[warp][digit] + below;
        __syncwarp();
        if (in && below == 0) warp_count[warp][digit] += __popc(peers);
        __syncwarp();
      }
      __syncthreads();
      // The warps' counts of each digit become their first places.
      if (tid < SORT_BINS) {
        uint32_t at = place[tid];
        for (int w = 0; w < SORT_WARPS; ++w) {
          const uint32_t n = warp_count[w][tid];
          warp_count[w][tid] = at;
          at += n;
        }
        place[tid] = at;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < SORT_PER_LANE; ++k) {
        if (w0 + 32 * k < end) {
          const uint32_t at = warp_count[warp][(key[k] >> shift) & mask] + rnk[k];
          __stcg(P.key[pass & 1] + at, key[k]);
          __stcg(P.pos[pass & 1] + at, p[k]);
        }
      }
      __syncthreads();
    }
    __threadfence();
    cluster.sync();
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void write_row(const EmbedGradParams& P, const SliceCols<VEC>& sc, uint32_t id, const float* sum) {
  float o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = __fmul_rn(sum[k], P.scale);
  const int64_t row = (int64_t)id * P.ldd;
  if (P.accumulate) {
    float old[8];
    sc.template load<DT>(P.d, row, old);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = __fadd_rn(old[k], o[k]);
  }
  sc.template store<DT>(P.d, row, o);
}

// One run and one slice of 256 columns a warp.
template <int CT, int DT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) embed_runs_kernel(const __grid_constant__ EmbedGradParams P) {
  const int64_t w = ((int64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t run = w / P.slices;
  const int64_t i0 = run * EMB_RUN;
  if (i0 >= P.tokens) return;
  const SliceCols<VEC> sc((int)(w - run * P.slices), lane, P.cols);
  const uint32_t* key = P.key[P.out];
  const uint32_t none = (uint32_t)P.vocab;
  const int n = P.tokens - i0 < EMB_RUN ? (int)(P.tokens - i0) : EMB_RUN;
  const uint32_t my_key = lane < n ? key[i0 + lane] : none;
  const uint32_t my_pos = lane < n ? P.pos[P.out][i0 + lane] : 0;
  const uint32_t next_key = __shfl_down_sync(0xFFFFFFFFu, my_key, 1);
  const uint32_t after = i0 + n < P.tokens ? key[i0 + n] : none;
  const bool first_continues = i0 > 0 && key[i0 - 1] == __shfl_sync(0xFFFFFFFFu, my_key, 0);
  const int valid = __popc(__ballot_sync(0xFFFFFFFFu, my_key != none));   // ids come before the positions without one
  // Entries after which the sum ends: the id's last of this run.
  const uint32_t ends = __ballot_sync(0xFFFFFFFFu, lane < valid && (lane == valid - 1 || next_key != my_key));
  float acc[8] = {};
  bool head = first_continues;
  constexpr int GROUP = 8;
  for (int e0 = 0; e0 < valid; e0 += GROUP) {
    float v[GROUP][8];
#pragma unroll
    for (int j = 0; j < GROUP; ++j) {
      const uint32_t p = __shfl_sync(0xFFFFFFFFu, my_pos, (e0 + j) & 31);
      if (e0 + j < valid) sc.template load<CT>(P.ct, (int64_t)p * P.ldc, v[j]);
    }
#pragma unroll
    for (int j = 0; j < GROUP; ++j) {
      const int e = e0 + j;
      if (e < valid) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = __fadd_rn(acc[k], v[j][k]);
        if ((ends >> e) & 1) {
          const uint32_t id = __shfl_sync(0xFFFFFFFFu, my_key, e);
          const bool goes_on = e == n - 1 && after == id;
          if (head) {
            sc.template store<PSK_F32>(P.head, run * P.pcols, acc);
          } else if (goes_on) {
            sc.template store<PSK_F32>(P.tail, run * P.pcols, acc);
          } else {
            write_row<DT, VEC>(P, sc, id, acc);
          }
          head = false;
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
        }
      }
    }
  }
}

// Join the run sums of each id whose entries span several runs: the warps of
// the run it begins in.
template <int DT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) embed_join_kernel(const __grid_constant__ EmbedGradParams P) {
  const int64_t w = ((int64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t run = w / P.slices;
  const int64_t i0 = run * EMB_RUN, i1 = i0 + EMB_RUN;
  if (i1 >= P.tokens) return;                       // the last run goes on nowhere
  const uint32_t* key = P.key[P.out];
  const uint32_t id = key[i1 - 1];
  if (id == (uint32_t)P.vocab || key[i1] != id) return;
  if (key[i0] == id && i0 > 0 && key[i0 - 1] == id) return;   // begun in an earlier run
  // The first entry past the id's own (entries are sorted).
  int64_t lo = i1, hi = P.tokens;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key[mid] > id) hi = mid;
    else lo = mid + 1;
  }
  const int64_t last = (lo - 1) / EMB_RUN;
  const SliceCols<VEC> sc((int)(w - run * P.slices), lane, P.cols);
  float acc[8];
  sc.template load<PSK_F32>(P.tail, run * P.pcols, acc);
  constexpr int GROUP = 8;
  for (int64_t r = run + 1; r <= last; r += GROUP) {
    float v[GROUP][8];
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
      if (r + j <= last) sc.template load<PSK_F32>(P.head, (r + j) * P.pcols, v[j]);
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
      if (r + j <= last) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = __fadd_rn(acc[k], v[j][k]);
      }
  }
  write_row<DT, VEC>(P, sc, id, acc);
}

static uint64_t align256(uint64_t n) { return (n + 255) / 256 * 256; }

// Workspace layout: key and pos buffers, then the head and tail run sums.
static uint64_t embed_ws_layout(int64_t tokens, int64_t cols, uint64_t* list, uint64_t* part) {
  const uint64_t runs = (uint64_t)(tokens + EMB_RUN - 1) / EMB_RUN;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  *list = align256((uint64_t)tokens * 4);
  *part = align256(runs * pcols * 4);
  return 4 * *list + 2 * *part;
}

static int embed_check_sizes(int64_t tokens, int64_t vocab, int64_t cols) {
  if (tokens < 0 || vocab < 0 || cols < 0)
    return fail(PSK_E_SHAPE, "tokens %lld, vocab %lld, cols %lld", (long long)tokens, (long long)vocab, (long long)cols);
  if (tokens > 0x7FFFFFFFll || vocab > 0x7FFFFFFFll || cols > (1LL << 31))
    return fail(PSK_E_SHAPE, "tokens %lld or vocab %lld above 2^31 - 1, or cols %lld above 2^31", (long long)tokens,
                (long long)vocab, (long long)cols);
  return PSK_OK;
}

static bool id_type_ok(int32_t t) { return t == PSK_I32 || t == PSK_I64; }

}  // namespace psk

using namespace psk;

extern "C" int psk_embed(const void* ids, int32_t idt, int64_t tokens, const void* table, int32_t tt, int64_t vocab,
                         int64_t cols, int64_t ldt, double scale, void* y, int32_t yt, int64_t ldy, void* stream) {
  clear_error();
  if (!id_type_ok(idt)) return fail(PSK_E_DTYPE, "id dtype %d", idt);
  if (!dtype_ok(tt)) return fail(PSK_E_DTYPE, "table dtype %d", tt);
  if (!dtype_ok(yt)) return fail(PSK_E_DTYPE, "y dtype %d", yt);
  int rc = embed_check_sizes(tokens, vocab, cols);
  if (rc) return rc;
  if (!(scale >= -3.4e38 && scale <= 3.4e38)) return fail(PSK_E_ARG, "scale is not a finite f32 value");
  if (tokens == 0 || cols == 0) return PSK_OK;
  if (!ids || !y || (!table && vocab > 0)) return fail(PSK_E_NULL, "ids, table or y is NULL");
  if ((uintptr_t)table % dtype_size(tt) || (uintptr_t)y % dtype_size(yt))
    return fail(PSK_E_ARG, "table or y is not aligned to its type");
  if (ldt < cols || ldy < cols) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(tokens, ldy) || !rows_addressable(vocab, ldt))
    return fail(PSK_E_SHAPE, "rows x leading dimension too large");
  const uint64_t isz = idt == PSK_I64 ? 8 : 4;
  if ((uintptr_t)ids % isz != 0) return fail(PSK_E_ARG, "ids are not aligned to their type");
  const uint64_t yb = rows_bytes(tokens, cols, ldy, yt);
  if (vocab > 0 && ranges_overlap(table, rows_bytes(vocab, cols, ldt, tt), y, yb))
    return fail(PSK_E_ALIAS, "y overlaps the table");
  if (ranges_overlap(ids, (uint64_t)tokens * isz, y, yb)) return fail(PSK_E_ALIAS, "y overlaps the ids");
  EmbedParams P{ids, table, y, vocab, cols, ldt, ldy, 0, 0, FastDiv((uint32_t)((cols + 7) / 8)), (float)scale};
  const bool vec = rows_vec8(table, tt, ldt, vocab) && rows_vec8(y, yt, ldy, tokens);
  const uint64_t slice = 0xFFFFFFFFull / P.per_row.d;
  cudaStream_t s = (cudaStream_t)stream;
  for (uint64_t r0 = 0; r0 < (uint64_t)tokens; r0 += slice) {
    const uint64_t nr = (uint64_t)tokens - r0 < slice ? (uint64_t)tokens - r0 : slice;
    P.row0 = (int64_t)r0;
    P.items = (uint32_t)(nr * P.per_row.d);
    const unsigned grid = (unsigned)(((uint64_t)P.items + EMB_THREADS - 1) / EMB_THREADS);
    with_dtype(tt, [&](auto TT) {
      return with_dtype(yt, [&](auto YT) {
        return with_bool(idt == PSK_I64, [&](auto I64) {
          return with_bool(vec, [&](auto VEC) {
            embed_kernel<TT.value, YT.value, I64.value, VEC.value><<<grid, EMB_THREADS, 0, s>>>(P);
            return 0;
          });
        });
      });
    });
    rc = check_launch("embedding kernel");
    if (rc) return rc;
  }
  return PSK_OK;
}

extern "C" int psk_embed_workspace(int64_t tokens, int64_t vocab, int64_t cols, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(PSK_E_NULL, "bytes is NULL");
  const int rc = embed_check_sizes(tokens, vocab, cols);
  if (rc) return rc;
  uint64_t list, part;
  *bytes = tokens && vocab && cols ? embed_ws_layout(tokens, cols, &list, &part) : 0;
  return PSK_OK;
}

extern "C" int psk_embed_backward(const void* ids, int32_t idt, int64_t tokens, const void* ct, int32_t ct_t, int64_t ldc,
                                  double scale, void* dtable, int32_t dt, int64_t vocab, int64_t cols, int64_t ldd,
                                  int32_t accumulate, void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  if (!id_type_ok(idt)) return fail(PSK_E_DTYPE, "id dtype %d", idt);
  if (!dtype_ok(ct_t)) return fail(PSK_E_DTYPE, "ct dtype %d", ct_t);
  if (!dtype_ok(dt)) return fail(PSK_E_DTYPE, "gradient dtype %d", dt);
  int rc = embed_check_sizes(tokens, vocab, cols);
  if (rc) return rc;
  if (!(scale >= -3.4e38 && scale <= 3.4e38)) return fail(PSK_E_ARG, "scale is not a finite f32 value");
  if (vocab == 0 || cols == 0 || (tokens == 0 && accumulate)) return PSK_OK;
  if (!dtable || (tokens > 0 && (!ids || !ct))) return fail(PSK_E_NULL, "ids, ct or the gradient is NULL");
  if ((uintptr_t)dtable % dtype_size(dt) || (tokens > 0 && (uintptr_t)ct % dtype_size(ct_t)))
    return fail(PSK_E_ARG, "ct or the gradient is not aligned to its type");
  if (ldd < cols || (tokens > 0 && ldc < cols)) return fail(PSK_E_SHAPE, "leading dimension below cols");
  if (!rows_addressable(tokens, ldc) || !rows_addressable(vocab, ldd))
    return fail(PSK_E_SHAPE, "rows x leading dimension too large");
  EmbedGradParams P{};
  uint64_t list = 0, part = 0;
  const uint64_t db = rows_bytes(vocab, cols, ldd, dt);
  if (tokens > 0) {
    const uint64_t isz = idt == PSK_I64 ? 8 : 4;
    if ((uintptr_t)ids % isz != 0) return fail(PSK_E_ARG, "ids are not aligned to their type");
    const uint64_t need = embed_ws_layout(tokens, cols, &list, &part);
    if (!workspace) return fail(PSK_E_NULL, "workspace is NULL");
    if ((uintptr_t)workspace % 16 != 0) return fail(PSK_E_ARG, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(PSK_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                  (unsigned long long)need);
    const uint64_t cb = rows_bytes(tokens, cols, ldc, ct_t);
    const uint64_t ib = (uint64_t)tokens * isz;
    if (ranges_overlap(dtable, db, ct, cb) || ranges_overlap(dtable, db, ids, ib) ||
        ranges_overlap(dtable, db, workspace, need))
      return fail(PSK_E_ALIAS, "the gradient overlaps ct, the ids or the workspace");
    if (ranges_overlap(workspace, need, ct, cb) || ranges_overlap(workspace, need, ids, ib))
      return fail(PSK_E_ALIAS, "the workspace overlaps ct or the ids");
  }
  P.ids = ids, P.ct = ct, P.d = dtable;
  P.vocab = vocab, P.cols = cols, P.ldc = ldc, P.ldd = ldd, P.tokens = tokens;
  char* w = (char*)workspace;
  for (int k = 0; k < 2; ++k) {
    P.key[k] = (uint32_t*)(w + (uint64_t)k * list);
    P.pos[k] = (uint32_t*)(w + (uint64_t)(2 + k) * list);
  }
  P.head = (float*)(w + 4 * list);
  P.tail = (float*)(w + 4 * list + part);
  P.pcols = (cols + 7) / 8 * 8;
  int bits = 0;                                     // bits of the largest key, vocab
  while (bits < 32 && ((uint64_t)vocab >> bits) != 0) ++bits;
  P.passes = (bits + SORT_BITS - 1) / SORT_BITS;
  P.bits = (bits + P.passes - 1) / P.passes;
  P.out = (P.passes - 1) & 1;
  P.accumulate = accumulate != 0;
  P.slices = (int32_t)((cols + 255) / 256);
  P.scale = (float)scale;
  const int64_t runs = (tokens + EMB_RUN - 1) / EMB_RUN;
  const uint64_t ctas = ((uint64_t)runs * P.slices + EMB_THREADS / 32 - 1) / (EMB_THREADS / 32);
  if (ctas > 0x7FFFFFFFull) return fail(PSK_E_SHAPE, "tokens x cols too large");
  const bool vec = (tokens == 0 || rows_vec8(ct, ct_t, ldc, tokens)) && rows_vec8(dtable, dt, ldd, vocab);
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t zero_groups = accumulate ? 0 : vocab * ((cols + 7) / 8);
  int64_t zero_ctas = (zero_groups + SORT_THREADS * 4 - 1) / (SORT_THREADS * 4);
  const int64_t most = (int64_t)device_sm_count() * 4;
  if (zero_ctas > most) zero_ctas = most;
  const unsigned grid = (unsigned)((zero_ctas + SORT_CTAS - 1) / SORT_CTAS + 1) * SORT_CTAS;
  with_dtype(dt, [&](auto DT) {
    return with_bool(idt == PSK_I64, [&](auto I64) {
      return with_bool(vec, [&](auto VEC) {
        embed_sort_kernel<I64.value, DT.value, VEC.value><<<grid, SORT_THREADS, 0, s>>>(P);
        return 0;
      });
    });
  });
  rc = check_launch("embedding sort kernel");
  if (rc || tokens == 0) return rc;
  with_dtype(ct_t, [&](auto CT) {
    return with_dtype(dt, [&](auto DT) {
      return with_bool(vec, [&](auto VEC) {
        embed_runs_kernel<CT.value, DT.value, VEC.value><<<(unsigned)ctas, EMB_THREADS, 0, s>>>(P);
        return 0;
      });
    });
  });
  rc = check_launch("embedding run sums kernel");
  if (rc) return rc;
  with_dtype(dt, [&](auto DT) {
    return with_bool(vec, [&](auto VEC) {
      embed_join_kernel<DT.value, VEC.value><<<(unsigned)ctas, EMB_THREADS, 0, s>>>(P);
      return 0;
    });
  });
  return check_launch("embedding join kernel");
}
