// Groups of eight neighbouring elements of a row, the unit of the training
// operators' kernels: 16 bytes of bf16 or 32 of f32, moved with 16-byte
// accesses where the rows allow it (VEC: 16-byte aligned bases and leading
// dimensions) and element by element at a row's ragged end and in other rows.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace psk {

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

// v[0, n) rounded to DT into elements [i, i + n) of p.
template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float* v) {
  if constexpr (DT == PSK_BF16) {
    uint16_t* q = (uint16_t*)p + i;
    if (VEC && n >= 8) {
      *(uint4*)q = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                              f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = f32_to_bf16_bits(v[k]);
    }
  } else {
    float* q = (float*)p + i;
    if (VEC && n >= 8) {
      *(float4*)q = make_float4(v[0], v[1], v[2], v[3]);
      *(float4*)(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = v[k];
    }
  }
}

// A lane's eight columns of slice s: neighbouring ones when rows move by
// 16-byte accesses, else every 32nd (so that a warp's loads coalesce).
template <bool VEC>
struct SliceCols {
  int64_t c0;
  int n;
  __device__ __forceinline__ SliceCols(int slice, int lane, int64_t cols) {
    if (VEC) {
      c0 = (int64_t)slice * 256 + lane * 8;
      const int64_t left = cols - c0;
      n = left < 0 ? 0 : left < 8 ? (int)left : 8;
    } else {
      c0 = (int64_t)slice * 256 + lane;
      const int64_t left = cols - c0;
      n = left <= 0 ? 0 : left > 224 ? 8 : (int)((left + 31) / 32);
    }
  }
  template <int DT>
  __device__ __forceinline__ void load(const void* p, int64_t row, float* v) const {
    if (VEC) {
      load8<DT, true>(p, row + c0, n, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = 0.0f;
        if (k < n) {
          if (DT == PSK_BF16) v[k] = bf16_bits_to_f32(((const uint16_t*)p)[row + c0 + 32 * k]);
          else v[k] = ((const float*)p)[row + c0 + 32 * k];
        }
      }
    }
  }
  template <int DT>
  __device__ __forceinline__ void store(void* p, int64_t row, const float* v) const {
    if (VEC) {
      store8<DT, true>(p, row + c0, n, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < n) {
          if (DT == PSK_BF16) ((uint16_t*)p)[row + c0 + 32 * k] = f32_to_bf16_bits(v[k]);
          else ((float*)p)[row + c0 + 32 * k] = v[k];
        }
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
