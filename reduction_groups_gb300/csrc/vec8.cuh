// Groups of eight neighbouring elements of a row, the unit of the training
// operators' kernels: 16 bytes of bf16 or 32 of f32, moved with 16-byte
// accesses where the rows allow it (VEC: 16-byte aligned bases and leading
// dimensions) and element by element at a row's ragged end and in other rows.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace psk {

// SMs that the rules of cutting work count on where the answer must not vary
// with the device, or be known without one (workspace sizes): a GB300's.
constexpr int NOMINAL_SMS = 152;

// bf16 or f32 elements [i, i + n) of p as f32; lanes from n on are 0.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float* v) {
  if constexpr (DT == PSK_BF16) {
    const uint16_t* q = (const uint16_t*)p + i;
    if (VEC && n >= 8) {
      const uint4 u = *(const uint4*)q;
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? bf16_bits_to_f32(q[k]) : 0.0f;
    }
  } else {
    const float* q = (const float*)p + i;
    if (VEC && n >= 8) {
      const float4 a = *(const float4*)q, b = *(const float4*)(q + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? q[k] : 0.0f;
    }
  }
}

// NC of a thread's columns as loaded, so that a batch of loads can be in
// flight before the first is widened.
template <int TY, bool VEC, int NC>
struct Piece {
  static constexpr int W = VEC && TY == PSK_BF16 ? NC / 2 : NC;
  uint32_t w[W];
  __device__ __forceinline__ float get(int k) const {
    if constexpr (VEC && TY == PSK_BF16)
      return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
    else
      return __uint_as_float(TY == PSK_BF16 ? w[k] << 16 : w[k]);
  }
};

// A thread's NC columns of the (T NC)-wide span that begins at column `base`,
// for thread t of T: neighbouring ones when rows move by 16-byte accesses
// (cols is then a multiple of 8), else every T-th, so that a warp's accesses
// coalesce.  Columns from cols on are read as zeros and not written.
template <bool VEC, int NC>
struct Columns {
  int64_t first;
  int stride, present;       // of the thread's columns, those below cols
  __device__ __forceinline__ Columns(int64_t base, int T, int t, int64_t cols)
      : first(base + (VEC ? (int64_t)t * NC : t)), stride(VEC ? 1 : T) {
    const int64_t left = cols - first;
    present = VEC ? (left > 0 ? NC : 0) : left <= 0 ? 0 : left > (int64_t)(NC - 1) * T ? NC : (int)((left + T - 1) / T);
  }
  __device__ __forceinline__ int64_t col(int k) const { return first + (int64_t)k * stride; }
  __device__ __forceinline__ bool has(int k) const { return k < present; }
  // Where the thread's columns of the row at element `row` begin.
  template <int TY>
  __device__ __forceinline__ const char* at(const void* p, int64_t row = 0) const {
    return (const char*)p + (row + first) * (TY == PSK_BF16 ? 2 : 4);
  }
  template <int TY>
  __device__ __forceinline__ void load(const void* p, int64_t row, Piece<TY, VEC, NC>& o) const {
    load_at(at<TY>(p, row), o);
  }
  template <int TY>
  __device__ __forceinline__ void load_at(const char* q, Piece<TY, VEC, NC>& o) const {
    if constexpr (VEC) {
      constexpr int W = Piece<TY, VEC, NC>::W;
#pragma unroll
      for (int i = 0; i < W; ++i) o.w[i] = 0;
      if (has(0)) {
        if constexpr (W == 2) {
          const uint2 u = *(const uint2*)q;
          o.w[0] = u.x, o.w[1] = u.y;
        } else {
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const uint4 u = *(const uint4*)(q + 4 * i);
            o.w[i] = u.x, o.w[i + 1] = u.y, o.w[i + 2] = u.z, o.w[i + 3] = u.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        o.w[k] = 0;
        if (has(k)) {
          if constexpr (TY == PSK_BF16) o.w[k] = ((const uint16_t*)q)[k * stride];
          else o.w[k] = ((const uint32_t*)q)[k * stride];
        }
      }
    }
  }
  // The same of f32 that other SMs have just written (from L2).
  __device__ __forceinline__ void load_l2(const float* p, int64_t row, Piece<PSK_F32, VEC, NC>& o) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NC; i += 4) {
        const uint4 u = has(0) ? __ldcg((const uint4*)(p + row + first + i)) : make_uint4(0, 0, 0, 0);
        o.w[i] = u.x, o.w[i + 1] = u.y, o.w[i + 2] = u.z, o.w[i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NC; ++k) o.w[k] = has(k) ? __ldcg((const uint32_t*)p + row + col(k)) : 0u;
    }
  }
  template <int TY>
  __device__ __forceinline__ void store(void* p, int64_t row, const float* v) const {
    store_at<TY>((char*)at<TY>(p, row), v);
  }
  template <int TY>
  __device__ __forceinline__ void store_at(char* q, const float* v) const {
    if constexpr (VEC) {
      if (has(0)) {
        if constexpr (TY == PSK_BF16) {
          if constexpr (NC == 4) *(uint2*)q = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
          else
            *(uint4*)q = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                    f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
        } else {
#pragma unroll
          for (int i = 0; i < NC; i += 4) *(float4*)(q + 4 * i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (has(k)) {
          if constexpr (TY == PSK_BF16) ((uint16_t*)q)[k * stride] = f32_to_bf16_bits(v[k]);
          else ((float*)q)[k * stride] = v[k];
        }
    }
  }
};

// Whether a row tensor's groups of eight can move by 16-byte accesses.
inline bool rows_vec8(const void* p, int32_t dt, int64_t ld, int64_t rows) {
  return (uintptr_t)p % 16 == 0 && (rows <= 1 || (ld * dtype_size(dt)) % 16 == 0);
}

// Bytes from the first to the last element of `rows` rows (rows, cols >= 1).
inline uint64_t rows_bytes(int64_t rows, int64_t cols, int64_t ld, int32_t dt) {
  return ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)dtype_size(dt);
}

// Whether rows * ld elements stay far inside 64-bit byte offsets.
inline bool rows_addressable(int64_t rows, int64_t ld) { return rows == 0 || ld <= (int64_t)((1LL << 56) / rows); }

inline bool ranges_overlap(const void* a, uint64_t abytes, const void* b, uint64_t bbytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + bbytes && b0 < a0 + abytes;
}

// Run F with compile-time storage types for run-time ones (each PSK_F32 or
// PSK_BF16, checked by the caller).
template <typename F>
inline int with_dtype(int32_t dt, F&& f) {
  return dt == PSK_BF16 ? f(std::integral_constant<int, PSK_BF16>{}) : f(std::integral_constant<int, PSK_F32>{});
}
template <typename F>
inline int with_bool(bool b, F&& f) {
  return b ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace psk
