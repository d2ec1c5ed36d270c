// Element access shared by the 8-bit operators: eight adjacent entries of a row
// of float32, bfloat16 or float16 as floats, and back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace ecasq {

enum : int { kF32 = 0, kBF16 = 1, kF16 = 2 };  // mirrors ECASQ_F32, ECASQ_BF16, ECASQ_F16

__host__ __device__ constexpr int type_bytes(int type) { return type == kF32 ? 4 : 2; }

template <int kType>
struct Elem;
template <>
struct Elem<kF32> {
  using T = float;
  __device__ __forceinline__ static float get(T v) { return v; }
  __device__ __forceinline__ static T put(float v) { return v; }
};
template <>
struct Elem<kBF16> {
  using T = __nv_bfloat16;
  __device__ __forceinline__ static float get(T v) { return __bfloat162float(v); }
  __device__ __forceinline__ static T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<kF16> {
  using T = __half;
  __device__ __forceinline__ static float get(T v) { return __half2float(v); }
  __device__ __forceinline__ static T put(float v) { return __float2half_rn(v); }
};

// Entries j .. j+7 of a row of k entries, zeros beyond k. `wide`: the row starts
// on a 16-byte boundary (j is a multiple of 8).
template <int kType>
__device__ __forceinline__ void load8(const typename Elem<kType>::T* __restrict__ row, int64_t j, int64_t k, bool wide,
                                      float (&v)[8]) {
  using T = typename Elem<kType>::T;
  if (wide && j + 8 <= k) {
    T e[8];
    const uint4* p = reinterpret_cast<const uint4*>(row + j);
    constexpr int n = sizeof(T) * 8 / 16;
#pragma unroll
    for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(e)[i] = __ldg(p + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<kType>::get(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j + i < k ? Elem<kType>::get(row[j + i]) : 0.0f;
  }
}

template <int kType>
__device__ __forceinline__ void store8(typename Elem<kType>::T* __restrict__ row, int64_t j, int64_t k, bool wide,
                                       const float (&v)[8]) {
  using T = typename Elem<kType>::T;
  if (wide && j + 8 <= k) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = Elem<kType>::put(v[i]);
    uint4* p = reinterpret_cast<uint4*>(row + j);
    constexpr int n = sizeof(T) * 8 / 16;
#pragma unroll
    for (int i = 0; i < n; ++i) p[i] = reinterpret_cast<const uint4*>(e)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < k) row[j + i] = Elem<kType>::put(v[i]);
  }
}

// Whether every row of a matrix starts on a 16-byte boundary.
inline bool rows_aligned16(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * bytes) % 16 == 0;
}

}  // namespace ecasq
