// Linear layer in 8-bit integers: the rows' quantiser and the product with a
// scale per token and per output channel (include/ecasq.h, "8-bit operators").
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.cuh"
#include "rows8.cuh"

namespace ecasq {

namespace {

// ---- quantiser -------------------------------------------------------------------
//
// Two steps per row, a = max |x| and q = nearest(127 x / a). A row's kTPR threads
// keep it in registers between the two (kKeep pieces of 8 entries each), so X is
// read once; longer rows read the rest again, from L2.

// nearest(127 x / a) with ties to even, decided by the exact quotient: the float32
// product t is within 127 * 2^-22 of it, so only a t that close to a half needs
// the fp64 quotient (127 x is exact there, and a quotient of a 31-bit by a 24-bit
// integer that is not a half differs from it by more than an fp64 rounding).
__device__ __forceinline__ int nearest127(float x, float xs, float r, float a) {
  const float t = xs * r;
  int q = __float2int_rn(t);
  if (fabsf(t - static_cast<float>(q)) > 0.5f - 0x1p-14f)
    q = __double2int_rn(__ddiv_rn(static_cast<double>(x) * 127.0, static_cast<double>(a)));
  return q;
}

template <int kType, int kTPR, int kKeep, bool kLong>
__global__ void __launch_bounds__(kTPR < 128 ? 128 : kTPR)
    k_int8_rows(const typename Elem<kType>::T* __restrict__ X, int64_t n, int64_t k, int64_t ldx, bool wide,
                int8_t* __restrict__ Q, int64_t ldq, float* __restrict__ scale, int32_t* __restrict__ status) {
  constexpr int kThreads = kTPR < 128 ? 128 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  __shared__ uint32_t part[kThreads / 32];
  const int lane = threadIdx.x % kTPR;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  const bool live = r < n;
  const auto* row = X + (live ? r : 0) * ldx;
  float v[kKeep][8];
  uint32_t m = 0;  // max |x| as bits: NaN and infinity order above every finite value
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    load8<kType>(row, static_cast<int64_t>(lane + i * kTPR) * 8, k, wide, v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[i][e]) & 0x7fffffffu);
  }
  if (kLong) {
    for (int64_t j = static_cast<int64_t>(lane + kKeep * kTPR) * 8; j < k; j += kTPR * 8) {
      float w[8];
      load8<kType>(row, j, k, wide, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(w[e]) & 0x7fffffffu);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (kTPR > 32) {
    if (lane_id() == 0) part[warp_id()] = m;
    __syncthreads();
    m = part[lane_id() % (kTPR / 32)];
    m = __reduce_max_sync(0xffffffffu, m);
  }
  if (!live) return;
  const bool bad = m >= 0x7f800000u;
  const float a = __uint_as_float(m);
  // tiny rows are lifted by 2^80 (exact) so that 127 / a stays finite
  const float lift = a < 0x1p-60f ? 0x1p80f : 1.0f;
  const float inv = (bad || m == 0) ? 0.0f : __fdiv_rn(127.0f, a * lift);
  if (lane == 0) {
    scale[r] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(a, 127.0f);
    status[r] = bad ? kStatusRange : kStatusOk;
  }
  int8_t* out = Q + r * ldq;
  const auto put = [&](int64_t j, const float(&w)[8]) {
    if (j >= k) return;
    uint32_t word[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = bad || m == 0 ? 0 : nearest127(w[e], w[e] * lift, inv, a);
      word[e >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (e & 3));
    }
    if (j + 8 <= k) {
      *reinterpret_cast<uint2*>(out + j) = make_uint2(word[0], word[1]);
    } else {
      for (int e = 0; j + e < k; ++e) out[j + e] = static_cast<int8_t>(word[e >> 2] >> (8 * (e & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) put(static_cast<int64_t>(lane + i * kTPR) * 8, v[i]);
  if (kLong) {
    for (int64_t j = static_cast<int64_t>(lane + kKeep * kTPR) * 8; j < k; j += kTPR * 8) {
      float w[8];
      load8<kType>(row, j, k, wide, w);
      put(j, w);
    }
  }
}

template <int kType>
cudaError_t int8_rows(const void* X, int64_t n, int64_t k, int64_t ldx, int8_t* Q, int64_t ldq, float* scale,
                      int32_t* status, cudaStream_t st) {
  const auto* x = static_cast<const typename Elem<kType>::T*>(X);
  const bool wide = rows_aligned16(X, ldx, type_bytes(kType));
  if (k <= 1024 && n > 148) {
    k_int8_rows<kType, 32, 4, false>
        <<<static_cast<unsigned>((n + 3) / 4), 128, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  } else if (k <= 4096) {
    k_int8_rows<kType, 128, 4, false><<<static_cast<unsigned>(n), 128, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  } else {
    k_int8_rows<kType, 512, 4, true><<<static_cast<unsigned>(n), 512, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  }
  note_launch();
  return cudaGetLastError();
}

// ---- product ---------------------------------------------------------------------

template <int kType>
__global__ void __launch_bounds__(256)
    k_int8_matmul_plain(const int8_t* __restrict__ A, int64_t lda, const float* __restrict__ sa,
                        const int8_t* __restrict__ B, int64_t ldb, const float* __restrict__ sb,
                        const float* __restrict__ bias, int64_t m, int64_t n, int64_t k,
                        typename Elem<kType>::T* __restrict__ Y, int64_t ldy) {
  __shared__ int ta[64][17], tb[64][17];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 64, j0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int64_t l0 = 0; l0 < k; l0 += 64) {
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      const int r = e >> 4, w = e & 15;
      int a = 0, b = 0;
      for (int t = 0; t < 4; ++t) {
        const int64_t l = l0 + 4 * w + t;
        if (l < k && i0 + r < m) a |= (A[(i0 + r) * lda + l] & 0xff) << (8 * t);
        if (l < k && j0 + r < n) b |= (B[(j0 + r) * ldb + l] & 0xff) << (8 * t);
      }
      ta[r][w] = a;
      tb[r][w] = b;
    }
    __syncthreads();
    for (int w = 0; w < 16; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(ta[ty + 16 * i][w], tb[tx + 16 * j][w], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
      if (r < m && c < n) {
        const float y = static_cast<float>(acc[i][j]) * sa[r] * sb[c];
        Y[r * ldy + c] = Elem<kType>::put(bias ? y + bias[c] : y);
      }
    }
}

}  // namespace

cudaError_t launch_int8_quantize(const void* X, int type, int64_t n, int64_t k, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, int32_t* status, cudaStream_t st) {
  switch (type) {
    case kF32: return int8_rows<kF32>(X, n, k, ldx, q, ldq, scale, status, st);
    case kBF16: return int8_rows<kBF16>(X, n, k, ldx, q, ldq, scale, status, st);
    default: return int8_rows<kF16>(X, n, k, ldx, q, ldq, scale, status, st);
  }
}

cudaError_t launch_int8_matmul(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb,
                               const float* sb, const float* bias, int64_t m, int64_t n, int64_t k, void* Y, int type,
                               int64_t ldy, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((m + 63) / 64), static_cast<unsigned>((n + 63) / 64));
  if (type == kF32)
    k_int8_matmul_plain<kF32><<<grid, 256, 0, st>>>(A, lda, sa, B, ldb, sb, bias, m, n, k, static_cast<float*>(Y), ldy);
  else if (type == kBF16)
    k_int8_matmul_plain<kBF16>
        <<<grid, 256, 0, st>>>(A, lda, sa, B, ldb, sb, bias, m, n, k, static_cast<__nv_bfloat16*>(Y), ldy);
  else
    k_int8_matmul_plain<kF16><<<grid, 256, 0, st>>>(A, lda, sa, B, ldb, sb, bias, m, n, k, static_cast<__half*>(Y), ldy);
  note_launch();
  return cudaGetLastError();
}

}  // namespace ecasq
