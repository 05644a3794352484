// The token embedding and its gradient.
//
// Forward: a gather of table rows, scaled.  Backward: the leaf's gradient
//   dtable[v, :] = scale * sum of ct[i, :] over the positions i with id v,
// without atomics on it: positions are sorted by id (a stable sort, so each
// id's positions stay in increasing order), the sorted list is cut into runs
// of EMB_RUN entries, each run is summed left to right by its own warps, and
// an id whose entries span several runs has its run sums joined left to
// right, by whichever of the runs' warps finishes last.  The order of every sum
// is fixed by the ids alone.
#include "vec8.cuh"
#include "pair.cuh"

namespace psk {

constexpr int EMB_THREADS = 256;
constexpr int EMB_RUN = 32;               // sorted entries a warp sums (one id per lane)

// ------------------------------------------------------------------ forward

struct EmbedParams {
  const void* ids;
  const void* table;
  void* y;
  int64_t vocab, cols, ldt, ldy;
  int64_t row0;
  uint32_t warps;        // of this launch: one for each slice of 256 NO columns of each row
  FastDiv slices;        // of a row
  float scale;
};

template <bool I64>
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i) {
  return I64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

// A warp's slice of a row: NO groups of eight columns a lane, 256 columns apart,
// all of their loads in flight.  (A thread for each group spent more integer
// instructions, at half of the lanes' rate, on its row's addresses than the
// 33 million values of a 16384 x 2048 lookup could hide.)
template <int TT, int YT, bool I64, bool VEC, int NO>
__global__ void __launch_bounds__(EMB_THREADS) embed_kernel(const __grid_constant__ EmbedParams P) {
  const uint32_t w = (uint32_t)(((uint64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5);
  if (w >= P.warps) return;
  const uint32_t r = P.slices.div(w);
  const int64_t c = (int64_t)(w - r * P.slices.d) * (256 * NO);
  const int lane = threadIdx.x & 31;
  const int64_t row = P.row0 + r, id = load_id<I64>(P.ids, row);
  if (id >= 0 && id < P.vocab) {
    Piece<TT, VEC, 8> v[NO];
#pragma unroll
    for (int j = 0; j < NO; ++j) Columns<VEC, 8>(c + 256 * j, 32, lane, P.cols).load(P.table, id * P.ldt, v[j]);
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(v[j].get(k), P.scale);
      Columns<VEC, 8>(c + 256 * j, 32, lane, P.cols).template store<YT>(P.y, row * P.ldy, y);
    }
  } else {
    const float z[8] = {};
#pragma unroll
    for (int j = 0; j < NO; ++j) Columns<VEC, 8>(c + 256 * j, 32, lane, P.cols).template store<YT>(P.y, row * P.ldy, z);
  }
}

// ----------------------------------------------------------------- backward

constexpr int SORT_THREADS = 512;                         // of the sort; as many again zero rows beside it
constexpr int SORT_FILL_BYTES = 384 * 1024;               // of a slice's rows zeroed beside the sort
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_PER_LANE = 16;
constexpr int SORT_TILE = SORT_THREADS * SORT_PER_LANE;   // ids scanned at a time
constexpr int SORT_BINS = 2048;                           // most ids of a slice
constexpr int SORT_LIST = SORT_TILE;                      // entries ranked at a time

constexpr uint32_t NO_ID = 0xFFFFFFFFu;
constexpr int SMALL_TOKENS = 128;                         // longest list that needs no sort

struct EmbedGradParams {
  const void* ids;
  const void* ct;
  void* d;
  int64_t vocab, cols;
  int64_t tokens;
  uint32_t ct_row, d_row;   // bytes from a row to the next: an address is one wide multiply-add
  uint32_t* key;         // the sorted ids of the positions that have one, NO_ID after them ...
  uint32_t* pos;         // ... and the positions
  uint2* places;         // per id: its first place in the sorted list, its number of places
  uint32_t* arrived;     // per run and column slice: run sums in of the id that begins there and goes on
  float* head;           // per run: the sum of its leading entries whose id the run before ends with
  float* tail;           // per run: the sum of its trailing entries whose id the next run goes on with
  int64_t pcols;         // row length of head and tail
  int32_t slice_ids;     // ids of a sorting CTA's slice of the vocabulary
  int32_t fill_ids;      // of them, first, whose rows the sort kernel zeroes unasked
  FastDiv per_slice;     // by slice_ids
  int32_t accumulate;
  int32_t slices;        // column slices of a row in the run sums
  int32_t run_ctas;      // CTAs of the run sums; the others zero the rows that do not occur
  float scale;
};

// The stable sort, without exchange between CTAs: each takes a slice of the
// vocabulary, reads all ids (from L2: 8 bytes a token), counts those below
// its slice -- its entries' first place in the list -- and collects its own
// positions in order; the few collected entries are then counting-sorted by
// id, warp by warp in order.  More entries than the collecting list holds
// (a slice with very frequent ids in a long batch) are collected and ranked
// a list at a time in a second scan.
struct SortShared {
  uint32_t pos[SORT_LIST];
  uint16_t key[SORT_LIST];
  uint32_t place[SORT_BINS];                 // counts, then each id's next place
  uint16_t before[SORT_WARPS][SORT_BINS];    // a warp's entries of an id; then those of the warps before, growing
  uint32_t warp_total[SORT_WARPS];
  uint32_t below;
};

// A row of zeros, by one warp: whole 16-byte blocks, and where rows begin
// anywhere the few elements before and after them one a lane.
template <int DT, bool VEC>
__device__ __forceinline__ void zero_row(const EmbedGradParams& P, int64_t row, int lane) {
  char* q = (char*)P.d + (uint64_t)row * P.d_row;
  constexpr int ESZ = DT == PSK_BF16 ? 2 : 4;
  int64_t bytes = P.cols * ESZ;
  if constexpr (!VEC) {
    auto element = [&](int64_t at, int n) {        // of n < 16 / ESZ
      if (lane < n) {
        if constexpr (DT == PSK_BF16) *(uint16_t*)(q + at + lane * ESZ) = 0;
        else *(uint32_t*)(q + at + lane * ESZ) = 0;
      }
    };
    const int64_t head = min((int64_t)(-(uintptr_t)q & 15u), bytes);
    element(0, (int)head / ESZ);
    q += head, bytes -= head;
    element(bytes & ~15ll, (int)(bytes & 15) / ESZ);
    bytes &= ~15ll;
  }
#pragma unroll 1
  for (int64_t c = lane * 16; c < bytes; c += 512) *(uint4*)(q + c) = make_uint4(0, 0, 0, 0);
}

// Barrier of the sorting threads.
__device__ __forceinline__ void sort_sync() { asm volatile("bar.sync 1, %0;" ::"n"(SORT_THREADS) : "memory"); }

// The sort's few microseconds of latency leave memory idle, so the other
// half of the CTA's threads zero the first rows of the slice meanwhile (all of
// them in a small table), whether they occur or not; the run sums' kernel,
// which knows, zeroes the rest.
template <bool I64, int DT, bool VEC>
__global__ void __launch_bounds__(2 * SORT_THREADS) embed_sort_kernel(const __grid_constant__ EmbedGradParams P) {
  extern __shared__ __align__(16) unsigned char sort_smem[];
  SortShared& S = *reinterpret_cast<SortShared*>(sort_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t lt = (1u << lane) - 1;
  const int64_t first = (int64_t)blockIdx.x * P.slice_ids;
  const int bins = (int)(P.vocab - first < P.slice_ids ? P.vocab - first : P.slice_ids);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid >= SORT_THREADS) {
    for (int v = warp - SORT_WARPS; v < P.fill_ids && v < bins; v += SORT_WARPS) zero_row<DT, VEC>(P, first + v, lane);
    return;
  }
  for (int b = tid; b < bins; b += SORT_THREADS) S.place[b] = 0;
  if (tid == 0) S.below = 0;
  sort_sync();

  // Scan the ids of one tile: the slice's entries go to the list from `at` on,
  // in order, where it has room; their number is returned.
  uint32_t below = 0;
  auto scan_tile = [&](int64_t t0, uint32_t at, bool count) -> uint32_t {
    uint32_t key[SORT_PER_LANE];
    uint32_t mine = 0;
    const int64_t w0 = t0 + (int64_t)warp * 32 * SORT_PER_LANE + lane;
#pragma unroll
    for (int k = 0; k < SORT_PER_LANE; ++k) {
      const int64_t i = w0 + 32 * k;
      const int64_t id = i < P.tokens ? load_id<I64>(P.ids, i) : -1;
      key[k] = id >= 0 && id < P.vocab ? (uint32_t)id : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int k = 0; k < SORT_PER_LANE; ++k) {
      if (count) below += key[k] < (uint32_t)first;
      const uint32_t local = key[k] - (uint32_t)first;     // an id below the slice, or none, wraps past it
      key[k] = local < (uint32_t)bins ? local : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int k = 0; k < SORT_PER_LANE; ++k) mine += __popc(__ballot_sync(0xFFFFFFFFu, key[k] != 0xFFFFFFFFu));
    sort_sync();                         // the list's and warp_total's last readers are done
    if (lane == 0) S.warp_total[warp] = mine;
    sort_sync();
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      const uint32_t n = S.warp_total[w];
      if (w < warp) at += n;
      sum += n;
    }
#pragma unroll
    for (int k = 0; k < SORT_PER_LANE; ++k) {
      const bool in = key[k] != 0xFFFFFFFFu;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
      if (in) {
        if (count) atomicAdd(&S.place[key[k]], 1u);
        const uint32_t q = at + __popc(m & lt);
        if (q < SORT_LIST) {
          S.key[q] = (uint16_t)key[k];
          S.pos[q] = (uint32_t)(w0 + 32 * k);
        }
      }
      at += __popc(m);
    }
    return sum;
  };

  // Write the list's n entries to their places.
  auto rank_list = [&](uint32_t n) {
    const uint32_t per = ((n + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32;
    const uint32_t a = warp * per, e = a + per < n ? a + per : n;
    for (int b = lane; b < bins; b += 32) S.before[warp][b] = 0;
    sort_sync();
    for (uint32_t i = a; i < e; i += 32) {
      const bool in = i + lane < e;
      const uint32_t key = in ? S.key[i + lane] : 0xFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
      if (in && (peers & lt) == 0) S.before[warp][key] += (uint16_t)__popc(peers);
      __syncwarp();
    }
    sort_sync();
    for (int b = tid; b < bins; b += SORT_THREADS) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        const uint32_t c = S.before[w][b];
        S.before[w][b] = (uint16_t)sum;
        sum += c;
      }
    }
    sort_sync();
    for (uint32_t i = a; i < e; i += 32) {
      const bool in = i + lane < e;
      const uint32_t key = in ? S.key[i + lane] : 0xFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
      const uint32_t under = __popc(peers & lt);
      uint32_t at = 0;
      if (in) at = S.before[warp][key] + under;
      __syncwarp();
      if (in && under == 0) S.before[warp][key] += (uint16_t)__popc(peers);
      __syncwarp();
      if (in) {
        const uint32_t q = S.place[key] + at;
        P.key[q] = (uint32_t)first + key;
        P.pos[q] = S.pos[i + lane];
      }
    }
    sort_sync();
    // The last warp's counters have grown to the list's counts.
    for (int b = tid; b < bins; b += SORT_THREADS) S.place[b] += S.before[SORT_WARPS - 1][b];
    sort_sync();
  };

  uint32_t n = 0;
  for (int64_t t0 = 0; t0 < P.tokens; t0 += SORT_TILE) n += scan_tile(t0, n, true);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
  if (lane == 0) atomicAdd(&S.below, below);
  sort_sync();
  const int64_t runs = (P.tokens + EMB_RUN - 1) / EMB_RUN;
  for (int64_t i = (int64_t)blockIdx.x * SORT_THREADS + tid; i < runs * P.slices; i += (int64_t)gridDim.x * SORT_THREADS)
    P.arrived[i] = 0;
  if (blockIdx.x + 1 == gridDim.x)
    for (int64_t i = (int64_t)S.below + n + tid; i < P.tokens; i += SORT_THREADS) P.key[i] = NO_ID;
  // Counts to first places: four neighbouring ids a thread.
  static_assert(SORT_BINS == 4 * SORT_THREADS, "four ids a thread");
  uint32_t c[4], sum = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = 4 * tid + k < bins ? S.place[4 * tid + k] : 0;
    sum += c[k];
  }
  uint32_t scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) S.warp_total[warp] = scan;
  sort_sync();
  uint32_t at = S.below + scan - sum;
#pragma unroll
  for (int w = 0; w < SORT_WARPS; ++w)
    if (w < warp) at += S.warp_total[w];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (4 * tid + k < bins) {
      S.place[4 * tid + k] = at;
      P.places[first + 4 * tid + k] = make_uint2(at, c[k]);
    }
    at += c[k];
  }
  sort_sync();
  if (n <= SORT_LIST) {
    rank_list(n);
    return;
  }
  uint32_t held = 0;
  for (int64_t t0 = 0; t0 < P.tokens; t0 += SORT_TILE) {
    uint32_t more = scan_tile(t0, held, false);
    if (held + more > SORT_LIST) {           // the tile's entries do not fit behind the held ones:
      sort_sync();
      rank_list(held);                       // rank those, and collect the tile again
      more = scan_tile(t0, 0, false);
      held = 0;
    }
    held += more;
    sort_sync();
  }
  rank_list(held);
}

template <int DT, bool VEC, int NC, bool ACC>
__device__ __forceinline__ void write_row(const EmbedGradParams& P, const Columns<VEC, NC>& cols, uint32_t id, const f2* sum,
                                          const Piece<DT, VEC, NC>* before = nullptr) {
  float o[NC];
#pragma unroll
  for (int k = 0; k < NC / 2; ++k) {
    const f2 v = f2_mul(sum[k], f2_splat(P.scale));
    o[2 * k] = v.x, o[2 * k + 1] = v.y;
  }
  char* q = (char*)cols.template at<DT>(P.d) + (uint64_t)id * P.d_row;
  if (ACC) {
    Piece<DT, VEC, NC> old;
    if (before) old = *before;
    else cols.load_at(q, old);
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = __fadd_rn(old.get(k), o[k]);
  }
  cols.template store_at<DT>(q, o);
}

// A run sum of an id whose entries span several runs: kept, and by the warp
// that brings the last of them all joined in order and written.
template <int DT, bool VEC, int NC, bool ACC>
__device__ __forceinline__ void join_runs(const EmbedGradParams& P, const Columns<VEC, NC>& cols, int64_t run, int slice,
                                          uint32_t id, bool head, const f2* sum) {
  float o[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) o[k] = k & 1 ? sum[k / 2].y : sum[k / 2].x;
  cols.template store<PSK_F32>(head ? P.head : P.tail, run * P.pcols, o);
  const uint2 place = P.places[id];
  const int64_t begin = place.x / EMB_RUN, last = (place.x + place.y - 1) / EMB_RUN;
  __threadfence();
  __syncwarp();
  uint32_t before = 0;
  if ((threadIdx.x & 31) == 0) before = atomicAdd(&P.arrived[begin * P.slices + slice], 1u);
  before = __shfl_sync(0xFFFFFFFFu, before, 0);
  if (before != (uint32_t)(last - begin)) return;
  __threadfence();
  f2 acc[NC / 2];
  Piece<PSK_F32, VEC, NC> t;
  cols.load_l2(P.tail, begin * P.pcols, t);
#pragma unroll
  for (int k = 0; k < NC / 2; ++k) acc[k] = f2{t.get(2 * k), t.get(2 * k + 1)};
  constexpr int GROUP = 64 / NC;
  for (int64_t r = begin + 1; r <= last; r += GROUP) {
    Piece<PSK_F32, VEC, NC> v[GROUP];
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
      if (r + j <= last) cols.load_l2(P.head, (r + j) * P.pcols, v[j]);
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
      if (r + j <= last) {
#pragma unroll
        for (int k = 0; k < NC / 2; ++k) acc[k] = f2_add(acc[k], f2{v[j].get(2 * k), v[j].get(2 * k + 1)});
      }
  }
  write_row<DT, VEC, NC, ACC>(P, cols, id, acc);
}

// The first run_ctas CTAs: one slice of 32 NC columns of one run a warp, or of
// a quarter of it (PARTS = 4: the ids that begin there, each to its end in the
// run).  The others zero the rows of ids that do not occur.
//
// 16384 tokens x 2048 bf16 into 32000 rows (198 MB): 48 us with the sort, 4.1
// TB/s; 30000 x 1000 f32 into 60000: 73 us, 4.9 TB/s; rows beginning anywhere,
// 4000 x 8001 bf16 into 8000: 50 us, 3.9 TB/s.  What is left is latency: a
// warp's chain of sorted list, four groups of rows, stores.  More rows in
// flight (copied asynchronously into shared memory), more warps, smaller or
// rolled loops all took as long or longer, as did zeroing elsewhere.
template <int CT, int DT, bool VEC, int NC, bool ACC, int PARTS>
__global__ void __launch_bounds__(EMB_THREADS, 2) embed_runs_kernel(const __grid_constant__ EmbedGradParams P) {
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x >= P.run_ctas) {
    // A warp's rows are a grid's warps apart; it looks 32 of them up at once.
    const int64_t warps = (int64_t)(gridDim.x - P.run_ctas) * (EMB_THREADS / 32);
    for (int64_t v0 = ((int64_t)(blockIdx.x - P.run_ctas) * EMB_THREADS + threadIdx.x) >> 5; v0 < P.vocab; v0 += 32 * warps) {
      const int64_t v = v0 + lane * warps;
      const bool zero = v < P.vocab && P.places[v].y == 0 &&
                        (int)((uint32_t)v - P.per_slice.div((uint32_t)v) * P.slice_ids) >= P.fill_ids;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, zero); m; m &= m - 1)
        zero_row<DT, VEC>(P, v0 + (__ffs(m) - 1) * warps, lane);
    }
    return;
  }
  const int64_t w = ((int64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5;
  const int64_t unit = w / P.slices, run = unit / PARTS;
  const int slice = (int)(w - unit * P.slices), part = (int)(unit % PARTS);
  const int64_t i0 = run * EMB_RUN;
  if (i0 >= P.tokens) return;
  const Columns<VEC, NC> cols((int64_t)slice * (32 * NC), 32, lane, P.cols);
  const uint32_t my_key = i0 + lane < P.tokens ? P.key[i0 + lane] : NO_ID;
  const uint32_t my_pos = i0 + lane < P.tokens ? P.pos[i0 + lane] : 0;
  const uint32_t after = i0 + EMB_RUN < P.tokens ? P.key[i0 + EMB_RUN] : NO_ID;
  const uint32_t prior = i0 > 0 ? P.key[i0 - 1] : NO_ID;
  const int n = __popc(__ballot_sync(0xFFFFFFFFu, my_key != NO_ID));
  if (n == 0) return;
  const uint32_t next_key = __shfl_down_sync(0xFFFFFFFFu, my_key, 1);
  // The first id of the run may have begun in an earlier one, the last may go
  // on in the next: their sums are joined, the others written as they end.
  bool leads = prior == __shfl_sync(0xFFFFFFFFu, my_key, 0);
  bool goes_on = n == EMB_RUN && after == __shfl_sync(0xFFFFFFFFu, my_key, EMB_RUN - 1);
  // Entries after which a sum ends.
  const uint32_t ends = __ballot_sync(0xFFFFFFFFu, lane < n && (lane == n - 1 ? !goes_on : next_key != my_key));
  // The warp's entries.
  int begin = 0, stop = n;
  if constexpr (PARTS > 1) {
    const uint32_t last_key = __shfl_up_sync(0xFFFFFFFFu, my_key, 1);
    const uint32_t starts = __ballot_sync(0xFFFFFFFFu, lane < n && (lane == 0 || last_key != my_key));
    auto first_from = [&](int at) {          // the first entry from `at` on with which an id begins
      const uint32_t m = at < 32 ? starts >> at : 0;
      return m ? at + __ffs(m) - 1 : n;
    };
    begin = first_from(part * (EMB_RUN / PARTS)), stop = first_from((part + 1) * (EMB_RUN / PARTS));
    if (begin >= stop) return;
    leads = leads && begin == 0, goes_on = goes_on && stop == n;
  }
  f2 acc[NC / 2], lead[NC / 2];
#pragma unroll
  for (int k = 0; k < NC / 2; ++k) acc[k] = lead[k] = f2{0.0f, 0.0f};
  bool head = leads;
  const char* ct = cols.template at<CT>(P.ct);
  // Rows in flight: eight of eight columns (sixteen of bf16 took the gradient of
  // 16384 x 2048 from 48 to 52 us, in registers that then spill), sixteen of
  // four, or eight with the rows that they are added to, or of a part.
  constexpr int GROUP = ACC || PARTS > 1 ? 8 : 64 / NC;
  for (int e0 = begin; e0 < stop; e0 += GROUP) {
    Piece<CT, VEC, NC> v[GROUP];
    Piece<DT, VEC, NC> old[ACC ? GROUP : 1];
    const uint32_t now = ends >> e0;
#pragma unroll
    for (int j = 0; j < GROUP; ++j) {
      const uint32_t p = __shfl_sync(0xFFFFFFFFu, my_pos, (e0 + j) & 31);
      if (e0 + j < stop) cols.load_at(ct + (uint64_t)p * P.ct_row, v[j]);
      if constexpr (ACC) {
        const uint32_t id = __shfl_sync(0xFFFFFFFFu, my_key, (e0 + j) & 31);
        if (e0 + j < stop && ((now >> j) & 1)) cols.load_at(cols.template at<DT>(P.d) + (uint64_t)id * P.d_row, old[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < GROUP; ++j) {
      if (e0 + j < stop) {
#pragma unroll
        for (int k = 0; k < NC / 2; ++k) acc[k] = f2_add(acc[k], f2{v[j].get(2 * k), v[j].get(2 * k + 1)});
        if ((now >> j) & 1) {
          if (head) {
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) lead[k] = acc[k];
            head = false;
          } else {
            write_row<DT, VEC, NC, ACC>(P, cols, __shfl_sync(0xFFFFFFFFu, my_key, e0 + j), acc, ACC ? &old[ACC ? j : 0] : nullptr);
          }
#pragma unroll
          for (int k = 0; k < NC / 2; ++k) acc[k] = f2{0.0f, 0.0f};
        }
      }
    }
  }
  // A run all of one id that began before is one leading sum.
  const uint32_t first_id = __shfl_sync(0xFFFFFFFFu, my_key, 0), last_id = __shfl_sync(0xFFFFFFFFu, my_key, EMB_RUN - 1);
  if (head && goes_on) {
#pragma unroll
    for (int k = 0; k < NC / 2; ++k) lead[k] = acc[k];
  }
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !leads : !goes_on || head) continue;
    f2 v[NC / 2];
#pragma unroll
    for (int k = 0; k < NC / 2; ++k) v[k] = which == 0 ? lead[k] : acc[k];
    join_runs<DT, VEC, NC, ACC>(P, cols, run, slice, which == 0 ? first_id : last_id, which == 0, v);
  }
}

// The gradient of up to SMALL_TOKENS tokens in one launch, with the same order
// of every sum: the warps of an id's first position find its others by
// comparing all ids (four a lane), and where the sorted list's runs would cut
// its entries by counting the smaller ids; other CTAs zero the rows of ids that
// do not occur.
template <int CT, int DT, bool I64, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) embed_small_kernel(const __grid_constant__ EmbedGradParams P) {
  constexpr int PER = SMALL_TOKENS / 32, NC = 8, GROUP = 8;
  const int lane = threadIdx.x & 31;
  uint32_t ids[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int64_t id = lane + 32 * k < P.tokens ? load_id<I64>(P.ids, lane + 32 * k) : -1;
    ids[k] = id >= 0 && id < P.vocab ? (uint32_t)id : NO_ID;
  }
  if ((int)blockIdx.x >= P.run_ctas) {
    const int64_t warps = (int64_t)(gridDim.x - P.run_ctas) * (EMB_THREADS / 32);
    for (int64_t v = ((int64_t)(blockIdx.x - P.run_ctas) * EMB_THREADS + threadIdx.x) >> 5; v < P.vocab; v += warps) {
      bool mine = false;
#pragma unroll
      for (int k = 0; k < PER; ++k) mine = mine || ids[k] == (uint32_t)v;
      if (!__any_sync(0xFFFFFFFFu, mine)) zero_row<DT, VEC>(P, v, lane);
    }
    return;
  }
  const int w = (int)(((int64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5);
  const int p = w / P.slices;
  if (p >= P.tokens) return;
  const Columns<VEC, NC> cols((int64_t)(w - p * P.slices) * (32 * NC), 32, lane, P.cols);
  uint32_t id = NO_ID;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const uint32_t u = __shfl_sync(0xFFFFFFFFu, ids[k], p & 31);
    if (k == p >> 5) id = u;
  }
  uint32_t at[PER];
  int place = 0;                                  // of the id's next entry in the sorted list
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    at[k] = __ballot_sync(0xFFFFFFFFu, ids[k] == id);
    place += __popc(__ballot_sync(0xFFFFFFFFu, ids[k] < id));
  }
  if (id == NO_ID) return;
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if ((k < p >> 5 && at[k]) || (k == p >> 5 && (at[k] & ((1u << (p & 31)) - 1)))) return;   // not the first
  f2 acc[NC / 2], total[NC / 2];
#pragma unroll
  for (int k = 0; k < NC / 2; ++k) acc[k] = f2{0.0f, 0.0f};
  bool first_run = true;
  auto end_run = [&]() {
#pragma unroll
    for (int k = 0; k < NC / 2; ++k) {
      total[k] = first_run ? acc[k] : f2_add(total[k], acc[k]);
      acc[k] = f2{0.0f, 0.0f};
    }
    first_run = false;
  };
  bool any = false;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    for (uint32_t m = at[k]; m;) {
      Piece<CT, VEC, NC> v[GROUP];
      int got = 0;
#pragma unroll
      for (int j = 0; j < GROUP; ++j)
        if (m) {
          cols.load_at(cols.template at<CT>(P.ct) + (uint64_t)(32 * k + __ffs(m) - 1) * P.ct_row, v[j]);
          m &= m - 1;
          ++got;
        }
#pragma unroll
      for (int j = 0; j < GROUP; ++j)
        if (j < got) {
          if (any && place % EMB_RUN == 0) end_run();
          any = true;
          ++place;
#pragma unroll
          for (int q = 0; q < NC / 2; ++q) acc[q] = f2_add(acc[q], f2{v[j].get(2 * q), v[j].get(2 * q + 1)});
        }
    }
  }
  end_run();
  if (P.accumulate) write_row<DT, VEC, NC, true>(P, cols, id, total);
  else write_row<DT, VEC, NC, false>(P, cols, id, total);
}

// The gradient of no tokens.
template <int DT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) embed_zero_kernel(const __grid_constant__ EmbedGradParams P) {
  const int64_t warps = (int64_t)gridDim.x * (EMB_THREADS / 32);
  for (int64_t v = ((int64_t)blockIdx.x * EMB_THREADS + threadIdx.x) >> 5; v < P.vocab; v += warps)
    zero_row<DT, VEC>(P, v, threadIdx.x & 31);
}

// Launch a kernel whose set-up may overlap the one before it (it waits for
// that one's results itself).
template <typename K>
static void launch_after(K kernel, unsigned grid, int threads, cudaStream_t s, const EmbedGradParams& P) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, P);
}

static uint64_t align256(uint64_t n) { return (n + 255) / 256 * 256; }

// How the run sums are cut: eight columns a lane where that leaves 16 warps an
// SM; four, into a gradient that is added to too (latency then counts
// more than the instructions for each row); and quarters of a run where four
// columns leave fewer than 4 warps an SM, each of which would pass its 32
// entries alone on its scheduler (500 tokens x 1001 bf16: 14.9 us, whole runs
// 17.9; 10000 x 501 f32, above the limit: 20.9 us whole, 23.1 in quarters).
struct EmbedCut {
  int columns, parts;
};
static EmbedCut embed_cut(int64_t tokens, int64_t cols, bool accumulate) {
  const int64_t runs = (tokens + EMB_RUN - 1) / EMB_RUN;
  if (!accumulate && runs * ((cols + 255) / 256) >= 16 * NOMINAL_SMS) return {8, 1};
  return {4, runs * ((cols + 127) / 128) >= 4 * NOMINAL_SMS ? 1 : 4};
}

// Workspace layout: the sorted list, each id's places in it, the head and tail
// run sums, their arrivals.
struct EmbedWorkspace {
  uint64_t key, pos, places, head, tail, arrived, bytes;
};
static EmbedWorkspace embed_ws_layout(int64_t tokens, int64_t vocab, int64_t cols) {
  const uint64_t runs = (uint64_t)(tokens + EMB_RUN - 1) / EMB_RUN;
  const uint64_t pcols = (uint64_t)(cols + 7) / 8 * 8;
  EmbedWorkspace w;
  w.key = 0;
  w.pos = align256((uint64_t)tokens * 4);
  w.places = 2 * w.pos;
  w.head = w.places + align256((uint64_t)vocab * 8);
  w.tail = w.head + align256(runs * pcols * 4);
  w.arrived = w.tail + align256(runs * pcols * 4);
  w.bytes = w.arrived + align256(runs * (uint64_t)((cols + 127) / 128) * 4);
  return w;
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
  const bool vec = cols % 8 == 0 && rows_vec8(table, tt, ldt, vocab) && rows_vec8(y, yt, ldy, tokens);
  // Four groups a lane (bf16 rows of 1024 columns and more: 16384 x 2048 18.8
  // us, one 24.7) where that leaves every SM its warps, else one (f32, whose
  // groups are two loads: 8000 x 4096 33 us, four 37; and decoding, where more
  // warps mean less latency).
  const int64_t wide = (cols + 1023) / 1024, narrow = (cols + 255) / 256;
  const bool four = tt == PSK_BF16 && cols >= 1024 && tokens * wide >= 32 * (int64_t)device_sm_count();
  EmbedParams P{ids, table, y, vocab, cols, ldt, ldy, 0, 0, FastDiv((uint32_t)(four ? wide : narrow)), (float)scale};
  const uint64_t slice = 0xFFFFFFFFull / P.slices.d;
  cudaStream_t s = (cudaStream_t)stream;
  for (uint64_t r0 = 0; r0 < (uint64_t)tokens; r0 += slice) {
    const uint64_t nr = (uint64_t)tokens - r0 < slice ? (uint64_t)tokens - r0 : slice;
    P.row0 = (int64_t)r0;
    P.warps = (uint32_t)(nr * P.slices.d);
    const unsigned grid = (unsigned)(((uint64_t)P.warps + EMB_THREADS / 32 - 1) / (EMB_THREADS / 32));
    with_dtype(tt, [&](auto TT) {
      return with_dtype(yt, [&](auto YT) {
        return with_bool(idt == PSK_I64, [&](auto I64) {
          return with_bool(vec, [&](auto VEC) {
            if constexpr (TT.value == PSK_BF16) {
              if (four) {
                embed_kernel<TT.value, YT.value, I64.value, VEC.value, 4><<<grid, EMB_THREADS, 0, s>>>(P);
                return 0;
              }
            }
            embed_kernel<TT.value, YT.value, I64.value, VEC.value, 1><<<grid, EMB_THREADS, 0, s>>>(P);
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
  *bytes = tokens && vocab && cols ? embed_ws_layout(tokens, vocab, cols).bytes : 0;
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
  if ((vocab > 1 && ldd > (1LL << 29)) || (tokens > 1 && ldc > (1LL << 29))) return fail(PSK_E_SHAPE, "leading dimension above 2^29");
  EmbedGradParams P{};
  EmbedWorkspace at{};
  const uint64_t db = rows_bytes(vocab, cols, ldd, dt);
  if (tokens > 0) {
    const uint64_t isz = idt == PSK_I64 ? 8 : 4;
    if ((uintptr_t)ids % isz != 0) return fail(PSK_E_ARG, "ids are not aligned to their type");
    at = embed_ws_layout(tokens, vocab, cols);
    const uint64_t need = at.bytes;
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
  P.vocab = vocab, P.cols = cols, P.tokens = tokens;
  P.ct_row = (uint32_t)(ldc * dtype_size(ct_t)), P.d_row = (uint32_t)(ldd * dtype_size(dt));
  P.pcols = (cols + 7) / 8 * 8;
  P.accumulate = accumulate != 0;
  P.scale = (float)scale;
  const bool vec = cols % 8 == 0 && (tokens == 0 || rows_vec8(ct, ct_t, ldc, tokens)) && rows_vec8(dtable, dt, ldd, vocab);
  cudaStream_t s = (cudaStream_t)stream;
  const int sms = device_sm_count();
  // Zeroing CTAs: four an SM beside the run sums, a row a warp at least.
  int64_t zero_ctas = accumulate ? 0 : (vocab + EMB_THREADS / 32 - 1) / (EMB_THREADS / 32);
  if (zero_ctas > 4 * sms) zero_ctas = 4 * sms;
  if (tokens == 0) {
    with_dtype(dt, [&](auto DT) {
      return with_bool(vec, [&](auto VEC) {
        embed_zero_kernel<DT.value, VEC.value><<<(unsigned)zero_ctas, EMB_THREADS, 0, s>>>(P);
        return 0;
      });
    });
    return check_launch("embedding gradient kernel");
  }
  if (tokens <= SMALL_TOKENS) {
    P.slices = (int32_t)((cols + 255) / 256);
    P.run_ctas = (int32_t)((tokens * P.slices + EMB_THREADS / 32 - 1) / (EMB_THREADS / 32));
    with_dtype(ct_t, [&](auto CT) {
      return with_dtype(dt, [&](auto DT) {
        return with_bool(idt == PSK_I64, [&](auto I64) {
          return with_bool(vec, [&](auto VEC) {
            embed_small_kernel<CT.value, DT.value, I64.value, VEC.value>
                <<<(unsigned)(P.run_ctas + zero_ctas), EMB_THREADS, 0, s>>>(P);
            return 0;
          });
        });
      });
    });
    return check_launch("embedding gradient kernel");
  }
  char* w = (char*)workspace;
  P.key = (uint32_t*)(w + at.key), P.pos = (uint32_t*)(w + at.pos);
  P.places = (uint2*)(w + at.places), P.arrived = (uint32_t*)(w + at.arrived);
  P.head = (float*)(w + at.head), P.tail = (float*)(w + at.tail);
  // A sorting CTA an SM, or more where a slice would pass SORT_BINS ids.
  int64_t slice = (vocab + sms - 1) / sms;
  if (slice > SORT_BINS) slice = SORT_BINS;
  P.slice_ids = (int32_t)slice;
  P.per_slice = FastDiv((uint32_t)slice);
  // Unaligned rows' zeros would outlast the sort (4099 x 771 f32: 20.9 us with
  // them, 18.9 without).
  const int64_t row_bytes = cols * dtype_size(dt), fill = SORT_FILL_BYTES / row_bytes;
  P.fill_ids = accumulate || !vec ? 0 : (int32_t)(fill < slice ? fill : slice);
  if (P.fill_ids == slice) zero_ctas = 0;
  const unsigned sort_ctas = (unsigned)((vocab + slice - 1) / slice);
  const int64_t runs = (tokens + EMB_RUN - 1) / EMB_RUN;
  const EmbedCut cut = embed_cut(tokens, cols, accumulate);
  P.slices = (int32_t)((cols + 32 * cut.columns - 1) / (32 * cut.columns));
  const uint64_t ctas = ((uint64_t)runs * cut.parts * P.slices + EMB_THREADS / 32 - 1) / (EMB_THREADS / 32);
  if (ctas + 4 * sms > 0x7FFFFFFFull) return fail(PSK_E_SHAPE, "tokens x cols too large");
  P.run_ctas = (int32_t)ctas;
  with_bool(idt == PSK_I64, [&](auto I64) {
    return with_dtype(dt, [&](auto DT) {
      return with_bool(vec, [&](auto VEC) {
        static bool limit[PSK_MAX_DEVICES] = {};
        smem_limit_once((const void*)embed_sort_kernel<I64.value, DT.value, VEC.value>, (int)sizeof(SortShared), limit);
        embed_sort_kernel<I64.value, DT.value, VEC.value>
            <<<sort_ctas, 2 * SORT_THREADS, sizeof(SortShared), s>>>(P);
        return 0;
      });
    });
  });
  rc = check_launch("embedding sort kernel");
  if (rc) return rc;
  with_dtype(ct_t, [&](auto CT) {
    return with_dtype(dt, [&](auto DT) {
      return with_bool(vec, [&](auto VEC) {
        const unsigned grid = (unsigned)(ctas + zero_ctas);
        auto launch = [&](auto NC, auto ACC, auto PARTS) {
          launch_after(embed_runs_kernel<CT.value, DT.value, VEC.value, NC.value, ACC.value, PARTS.value>, grid, EMB_THREADS, s, P);
        };
        using std::integral_constant;
        using Four = integral_constant<int, 4>;
        using One = integral_constant<int, 1>;
        if (cut.columns == 8) launch(integral_constant<int, 8>{}, std::false_type{}, One{});
        else with_bool(accumulate != 0, [&](auto ACC) {
          if (cut.parts == 4) launch(Four{}, ACC, Four{});
          else launch(Four{}, ACC, One{});
          return 0;
        });
        return 0;
      });
    });
  });
  return check_launch("embedding run sums kernel");
}
