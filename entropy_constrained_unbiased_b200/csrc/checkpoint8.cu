// Activation checkpoints in 8 bits and the weight gradient read from them
// (include/ecasq.h, "8-bit operators").
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.cuh"
#include "rows8.cuh"

namespace ecasq {

namespace {

constexpr uint32_t kStreamCheckpoint = 2;  // third counter word (ecasq_encode uses 0 and 1)
constexpr uint32_t kScaleNaN = 255;        // scale byte of a block without finite values

// The byte b of the smallest power of two 2^(b - 127) >= a / 127, from the bits of
// a >= 0: with a = c 2^E, 1 <= c < 2, and 127 = 1.984375 * 2^6, the exponent is
// E - 6 if c <= 1.984375, else E - 5; at least 2^-126.
__device__ __forceinline__ uint32_t scale_byte(uint32_t a_bits) {
  const int b = static_cast<int>(a_bits >> 23) - 6 + ((a_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return b > 248 ? kScaleNaN : static_cast<uint32_t>(b < 1 ? 1 : b);
}

// One thread per 8 entries (one Philox block), four threads per block of 32; a CTA
// covers blockDim.y rows by 8 * blockDim.x columns.
template <int kType>
__global__ void __launch_bounds__(256)
    k_checkpoint8(const typename Elem<kType>::T* __restrict__ X, int64_t t, int64_t k, int64_t ldx, bool wide,
                  uint64_t seed, const uint64_t* __restrict__ seed_add, int8_t* __restrict__ Q, int64_t ldq,
                  uint8_t* __restrict__ S, int64_t lds) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t pieces = (k + 31) / 32 * 4;
  if (seed_add) seed += *seed_add;
  float v[8];
  const bool live = r < t && c < pieces;
  if (live)
    load8<kType>(X + r * ldx, c * 8, k, wide, v);
  else
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (!live) return;
  const uint32_t b = scale_byte(m);
  uint32_t word[2] = {0, 0};
  if (b != kScaleNaN && m != 0) {
    const uint4 u = Philox4x32::block(
        make_uint4(static_cast<uint32_t>(c), static_cast<uint32_t>(r), kStreamCheckpoint, 0),
        static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
    const uint32_t rnd[4] = {u.x, u.y, u.z, u.w};
    const float inv = __uint_as_float((254u - b) << 23);  // 1 / s, exact
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float z = fabsf(v[e]) * inv;
      const float low = floorf(z);
      const int up = __float2int_rn((z - low) * 65536.0f);
      const int u16 = static_cast<int>((e & 1) ? rnd[e >> 1] >> 16 : rnd[e >> 1] & 0xffffu);
      int q = static_cast<int>(low) + (u16 < up ? 1 : 0);
      q = v[e] < 0.0f ? -q : q;
      word[e >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (e & 3));
    }
  }
  *reinterpret_cast<uint2*>(Q + r * ldq + c * 8) = make_uint2(word[0], word[1]);
  if ((c & 3) == 0) S[r * lds + (c >> 2)] = static_cast<uint8_t>(b);
}

__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == kScaleNaN ? 0x7fc00000u : b << 23);
}

template <int kType>
__global__ void __launch_bounds__(256)
    k_checkpoint8_restore(const int8_t* __restrict__ Q, int64_t ldq, const uint8_t* __restrict__ S, int64_t lds,
                          int64_t t, int64_t k, typename Elem<kType>::T* __restrict__ X, int64_t ldx, bool wide) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  if (r >= t || c * 8 >= k) return;
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(Q + r * ldq + c * 8));
  const float s = scale_value(S[r * lds + (c >> 2)]);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t x = e < 4 ? w.x : w.y;
    v[e] = static_cast<float>(static_cast<int8_t>(x >> (8 * (e & 3)))) * s;
    if (kType == kF16 && fabsf(v[e]) > 65504.0f) v[e] = copysignf(65504.0f, v[e]);
  }
  store8<kType>(X + r * ldx, c * 8, k, wide, v);
}

// Threads along a row and rows per CTA (256 threads), and the grid, for `pieces`
// pieces of 8 entries per row.
void piece_grid(int64_t t, int64_t pieces, dim3* grid, dim3* block) {
  unsigned x = 4;
  while (x < 256 && x < pieces) x *= 2;
  *block = dim3(x, 256 / x);
  *grid = dim3(static_cast<unsigned>((t + block->y - 1) / block->y), static_cast<unsigned>((pieces + x - 1) / x));
}

template <int kIn, int kOut>
__global__ void __launch_bounds__(256)
    k_wgrad_plain(const typename Elem<kIn>::T* __restrict__ dY, int64_t ldy, const int8_t* __restrict__ Q, int64_t ldq,
                  const uint8_t* __restrict__ S, int64_t lds, int64_t t, int64_t o, int64_t k,
                  typename Elem<kOut>::T* __restrict__ dW, int64_t ldw) {
  __shared__ float ta[16][65], tb[16][65];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 64, j0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t r0 = 0; r0 < t; r0 += 16) {
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int64_t r = r0 + (e >> 6), i = i0 + (e & 63), j = j0 + (e & 63);
      ta[e >> 6][e & 63] = r < t && i < o ? Elem<kIn>::get(dY[r * ldy + i]) : 0.0f;
      tb[e >> 6][e & 63] =
          r < t && j < k ? static_cast<float>(Q[r * ldq + j]) * scale_value(S[r * lds + j / 32]) : 0.0f;
    }
    __syncthreads();
    for (int w = 0; w < 16; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += ta[w][ty + 16 * i] * tb[w][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
      if (r < o && c < k) dW[r * ldw + c] = Elem<kOut>::put(acc[i][j]);
    }
}

template <int kIn>
cudaError_t wgrad_plain(const void* dY, int64_t ldy, const int8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds,
                        int64_t t, int64_t o, int64_t k, void* dW, int out, int64_t ldw, cudaStream_t st) {
  const auto* y = static_cast<const typename Elem<kIn>::T*>(dY);
  const dim3 grid(static_cast<unsigned>((o + 63) / 64), static_cast<unsigned>((k + 63) / 64));
  if (out == kF32)
    k_wgrad_plain<kIn, kF32><<<grid, 256, 0, st>>>(y, ldy, q, ldq, scale, lds, t, o, k, static_cast<float*>(dW), ldw);
  else if (out == kBF16)
    k_wgrad_plain<kIn, kBF16>
        <<<grid, 256, 0, st>>>(y, ldy, q, ldq, scale, lds, t, o, k, static_cast<__nv_bfloat16*>(dW), ldw);
  else
    k_wgrad_plain<kIn, kF16><<<grid, 256, 0, st>>>(y, ldy, q, ldq, scale, lds, t, o, k, static_cast<__half*>(dW), ldw);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_checkpoint8(const void* X, int type, int64_t t, int64_t k, int64_t ldx, uint64_t seed,
                               const uint64_t* seed_add, int8_t* q, int64_t ldq, uint8_t* scale, int64_t lds,
                               cudaStream_t st) {
  dim3 grid, block;
  piece_grid(t, (k + 31) / 32 * 4, &grid, &block);
  const bool wide = rows_aligned16(X, ldx, type_bytes(type));
  if (type == kF32)
    k_checkpoint8<kF32><<<grid, block, 0, st>>>(static_cast<const float*>(X), t, k, ldx, wide, seed, seed_add, q, ldq,
                                                scale, lds);
  else if (type == kBF16)
    k_checkpoint8<kBF16><<<grid, block, 0, st>>>(static_cast<const __nv_bfloat16*>(X), t, k, ldx, wide, seed, seed_add,
                                                 q, ldq, scale, lds);
  else
    k_checkpoint8<kF16><<<grid, block, 0, st>>>(static_cast<const __half*>(X), t, k, ldx, wide, seed, seed_add, q, ldq,
                                                scale, lds);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_checkpoint8_restore(const int8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds, int64_t t,
                                       int64_t k, void* X, int type, int64_t ldx, cudaStream_t st) {
  dim3 grid, block;
  piece_grid(t, (k + 7) / 8, &grid, &block);
  const bool wide = rows_aligned16(X, ldx, type_bytes(type));
  if (type == kF32)
    k_checkpoint8_restore<kF32><<<grid, block, 0, st>>>(q, ldq, scale, lds, t, k, static_cast<float*>(X), ldx, wide);
  else if (type == kBF16)
    k_checkpoint8_restore<kBF16>
        <<<grid, block, 0, st>>>(q, ldq, scale, lds, t, k, static_cast<__nv_bfloat16*>(X), ldx, wide);
  else
    k_checkpoint8_restore<kF16><<<grid, block, 0, st>>>(q, ldq, scale, lds, t, k, static_cast<__half*>(X), ldx, wide);
  note_launch();
  return cudaGetLastError();
}

size_t checkpoint8_wgrad_workspace(int64_t, int64_t, int64_t, int, int64_t) { return 0; }

cudaError_t launch_checkpoint8_wgrad(const void* dY, int dy_type, int64_t ldy, const int8_t* q, int64_t ldq,
                                     const uint8_t* scale, int64_t lds, int64_t t, int64_t o, int64_t k, void* dW,
                                     int dw_type, int64_t ldw, void*, cudaStream_t st) {
  if (dy_type == kF32) return wgrad_plain<kF32>(dY, ldy, q, ldq, scale, lds, t, o, k, dW, dw_type, ldw, st);
  if (dy_type == kBF16) return wgrad_plain<kBF16>(dY, ldy, q, ldq, scale, lds, t, o, k, dW, dw_type, ldw, st);
  return wgrad_plain<kF16>(dY, ldy, q, ldq, scale, lds, t, o, k, dW, dw_type, ldw, st);
}

}  // namespace ecasq
