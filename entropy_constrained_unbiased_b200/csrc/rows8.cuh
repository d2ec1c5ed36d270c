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
  using Bits = uint32_t;
  __device__ __forceinline__ static T put(float v) { return v; }
};
template <>
struct Elem<kBF16> {
  using T = __nv_bfloat16;
  using Bits = uint16_t;
  __device__ __forceinline__ static T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<kF16> {
  using T = __half;
  using Bits = uint16_t;
  __device__ __forceinline__ static T put(float v) { return __float2half_rn(v); }
};

// Eight adjacent entries as they lie in memory.
template <int kType>
struct Eight {
  uint4 w[type_bytes(kType) * 8 / 16];
};

// Entries j .. j+7 of a row of k entries, zeros beyond k. `wide`: the row starts
// on a 16-byte boundary (j is a multiple of 8).
template <int kType>
__device__ __forceinline__ Eight<kType> load8(const typename Elem<kType>::T* __restrict__ row, int64_t j, int64_t k,
                                              bool wide) {
  constexpr int n = sizeof(Eight<kType>) / 16;
  Eight<kType> v;
  if (wide && j + 8 <= k) {
    const uint4* p = reinterpret_cast<const uint4*>(row + j);
#pragma unroll
    for (int i = 0; i < n; ++i) v.w[i] = __ldg(p + i);
  } else {
    using Bits = typename Elem<kType>::Bits;
    const Bits* p = reinterpret_cast<const Bits*>(row);
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = j + i < k ? __ldg(p + j + i) : 0;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4 * n; ++i) w[i] = kType == kF32 ? e[i] : e[(2 * i) & 7] | e[(2 * i + 1) & 7] << 16;
  }
  return v;
}
template <int kType>
__device__ __forceinline__ void floats8(const Eight<kType>& e, float (&v)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kType == kF32)
      v[i] = __uint_as_float(w[i]);
    else if constexpr (kType == kBF16)
      v[i] = __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else
      v[i] = __half2float(__ushort_as_half(static_cast<unsigned short>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu)));
  }
}

// The largest magnitude of entries, kept as the type's own bits (sign cleared): their
// order is that of the magnitudes, with infinity and NaN above every finite value.
template <int kType>
struct Largest {
  uint32_t m = 0;  // 16-bit types: two running maxima
  __device__ __forceinline__ void add(const Eight<kType>& e) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&e);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(e) / 4); ++i) {
      if constexpr (kType == kF32)
        m = max(m, w[i] & 0x7fffffffu);
      else
        m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
  }
  // As the bits of a float.
  __device__ __forceinline__ uint32_t bits() const {
    if constexpr (kType == kF32) return m;
    const uint32_t one = max(m >> 16, m & 0xffffu);
    if constexpr (kType == kBF16) return one << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(one)))) & 0x7fffffffu;
  }
};

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
