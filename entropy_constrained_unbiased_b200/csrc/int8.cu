// Linear layer in 8-bit integers: the rows' quantiser and the product with a
// scale per token and per output channel (include/ecasq.h, "8-bit operators").
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kernels.cuh"
#include "rows8.cuh"
#include "tensor.cuh"

namespace ecasq {

namespace {

// ---- quantiser -------------------------------------------------------------------
//
// Two steps per row, a = max |x| and q = nearest(127 x / a). A row's kTPR threads
// keep it in registers between the two (kKeep pieces of 8 entries each, as they lie in
// memory), so X is read once; longer rows read the rest again, from L2. Between memory
// and instruction issue: 3 bytes for a bfloat16 entry leave 16 instructions for it at
// full bandwidth, and it takes 14 (16384 x 16384 bfloat16 activations with outliers: 170
// us, 4.7 TB/s, issue 64%). Entries that are exactly half the largest are ties, which the
// fp64 quotient decides: plain normal entries, of which one in 600 is, take 266 us.

// A row's quantisation from its largest magnitude, given as the bits of a float.
struct RowScale {
  float a, lift, inv, scale;
  bool bad;
};
__device__ __forceinline__ RowScale row_scale(uint32_t a_bits) {
  RowScale s;
  s.bad = a_bits >= 0x7f800000u;
  s.a = __uint_as_float(a_bits);
  // tiny rows are lifted by 2^80 (exact) so that 127 / a stays finite
  s.lift = s.a < 0x1p-60f ? 0x1p80f : 1.0f;
  s.inv = (s.bad || a_bits == 0) ? 0.0f : __fdiv_rn(127.0f, s.a * s.lift);
  s.scale = s.bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(s.a, 127.0f);
  return s;
}
// Eight integers of a row, in order: nearest(127 x / a) with ties to even, decided by
// the exact quotient. The float32 product t is within 127 * 2^-23 < 2^-16 of it, so
// only a t that close to a half needs the fp64 quotient (127 x is exact there, and a
// quotient of a 31-bit by a 24-bit integer that is not a half differs from it by more
// than an fp64 rounding). Adding 1.5 * 2^23 leaves the nearest integer in the low
// bits, two's complement.
__device__ __forceinline__ uint2 quantize8(float (&v)[8], const RowScale& s) {
  if (s.inv == 0.0f) return make_uint2(0, 0);
  constexpr float kInt = 12582912.0f;
  constexpr float kClear = 0.5f - 0x1p-16f;
  if (s.lift != 1.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s.lift;
  }
  uint32_t b[8];
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __fmul_rn(v[e], s.inv), m = __fadd_rn(t, kInt);
    far = fmaxf(far, fabsf(t - __fadd_rn(m, -kInt)));
    b[e] = __float_as_uint(m);
  }
  if (far > kClear) {
    const double a = static_cast<double>(s.a) * static_cast<double>(s.lift);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = __fmul_rn(v[e], s.inv);
      if (fabsf(t - rintf(t)) > kClear)
        b[e] = static_cast<uint32_t>(__double2int_rn(__ddiv_rn(static_cast<double>(v[e]) * 127.0, a)));
    }
  }
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

template <int kType, int kTPR, int kKeep, bool kLong>
__global__ void __launch_bounds__(kTPR < 128 ? 128 : kTPR, kTPR > 128 ? 3 : 1)
    k_int8_rows(const typename Elem<kType>::T* __restrict__ X, int64_t n, int64_t k, int64_t ldx, bool wide,
                int8_t* __restrict__ Q, int64_t ldq, float* __restrict__ scale, int32_t* __restrict__ status) {
  constexpr int kThreads = kTPR < 128 ? 128 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  __shared__ uint32_t part[kThreads / 32];
  next_may_begin();
  const int lane = threadIdx.x % kTPR;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  const bool live = r < n;
  const auto* row = X + (live ? r : 0) * ldx;
  Eight<kType> v[kKeep];
  Largest<kType> top;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) v[i] = load8<kType>(row, static_cast<int64_t>(lane + i * kTPR) * 8, k, wide);
#pragma unroll
  for (int i = 0; i < kKeep; ++i) top.add(v[i]);
  if (kLong) {
#pragma unroll 4
    for (int64_t j = static_cast<int64_t>(lane + kKeep * kTPR) * 8; j < k; j += kTPR * 8)
      top.add(load8<kType>(row, j, k, wide));
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, top.bits());
  if (kTPR > 32) {
    if (lane_id() == 0) part[warp_id()] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, part[lane_id() % (kTPR / 32)]);
  }
  if (!live) return;
  const RowScale a = row_scale(m);
  if (lane == 0) {
    scale[r] = a.scale;
    status[r] = a.bad ? kStatusRange : kStatusOk;
  }
  int8_t* out = Q + r * ldq;
  const auto put = [&](int64_t j, const Eight<kType>& e) {
    if (j >= k) return;
    float w[8];
    floats8<kType>(e, w);
    const uint2 q = quantize8(w, a);
    if (j + 8 <= k) {
      *reinterpret_cast<uint2*>(out + j) = q;
    } else {
      for (int i = 0; j + i < k; ++i) out[j + i] = static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) put(static_cast<int64_t>(lane + i * kTPR) * 8, v[i]);
  if (kLong) {
    for (int64_t j = static_cast<int64_t>(lane + kKeep * kTPR) * 8; j < k; j += kTPR * 8)
      put(j, load8<kType>(row, j, k, wide));
  }
}

template <int kType>
cudaError_t int8_rows(const void* X, int64_t n, int64_t k, int64_t ldx, int8_t* Q, int64_t ldq, float* scale,
                      int32_t* status, cudaStream_t st) {
  const auto* x = static_cast<const typename Elem<kType>::T*>(X);
  const bool wide = rows_aligned16(X, ldx, type_bytes(kType));
  constexpr int kMost = kType == kF32 ? 4 : 8;  // 16384 16-bit or 8192 32-bit entries in registers
  // A warp, four or eight of them per row: few rows take the most threads (latency),
  // many rows the fewest. bfloat16, us with 1 / 4 / 8 warps: 100 x 1024 5.6 / - / 3.2,
  // 1000 x 1024 5.8 / 4.5 / 8.7, 16384 x 1024 19 / 35 / 99, 1000 x 4096 - / 8.5 / 10.4,
  // 16384 x 4096 175 (spills) / 70 / 118.
  if (k <= 1024 && n > 2048) {
    k_int8_rows<kType, 32, 4, false>
        <<<static_cast<unsigned>((n + 3) / 4), 128, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  } else if (k <= 4096 && n > 148) {
    k_int8_rows<kType, 128, 4, false><<<static_cast<unsigned>(n), 128, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  } else {
    k_int8_rows<kType, 256, kMost, true><<<static_cast<unsigned>(n), 256, 0, st>>>(x, n, k, ldx, wide, Q, ldq, scale, status);
  }
  note_launch();
  return cudaGetLastError();
}

// ---- product ---------------------------------------------------------------------
//
// tcgen05.mma kind::i8 (int32 accumulators in TMEM: the sum is exact). The output
// channels are the M side of the MMA and the tokens its N side, so one token costs a
// 16-column tile instead of a 128-row one, and a thread of the epilogue owns one
// channel: its scale and bias are read once, the 32 lanes of a warp write 32
// adjacent outputs of a token, and outputs of any pitch or alignment are served by
// the same stores. Operand rows come through TMA in 128-byte pieces of k (zeros
// beyond the sizes).

__device__ int g_stalled_int8;  // set when a bounded wait gave up

constexpr int kPieceK = 128;  // bytes of k per stage
constexpr int kStepK = 32;    // k of one MMA
constexpr int kMostPieces = 1024;  // of the longest sum, the only one that may wrap

struct Product {
  const float* sa;
  const float* sb;
  const float* bias;
  void* Y;
  int64_t m, n, ldy;
  int pieces;  // ceil(k / 128)
  bool early;  // launched behind the quantiser of the tokens
};

// The exact sum behind a 32-bit accumulator that wraps around. The least sum of 131072
// products, of -128 by 127, is above -2^31, so that value stands for the one sum that
// wraps: 2^31, all products being -128 by -128.
__device__ __forceinline__ float sum_value(int acc) { return acc == INT32_MIN ? 0x1p31f : static_cast<float>(acc); }

// Whether any sum times the token scale a lies inside float32's normal range.
__device__ __forceinline__ bool plain_scale(float a) {
  const float size = fabsf(a);
  return (size >= 0x1p-95f || size == 0.0f) && size <= 0x1p96f;
}

// One output: the exact integer sum, scaled. kPlain: the sum has not wrapped and the scale
// is a plain one. Other scales multiply in fp64, so that nothing overflows or is lost
// before the channel's scale. (Both looked at for each output, 16384 x 4096 x 16384 with
// the quantiser took 888 instead of 811 us; for 32 tokens at once, 812.)
template <int kType, bool kPlain = false>
__device__ __forceinline__ void put_output(const Product& p, int64_t token, int64_t channel, int acc, float a, float s,
                                           float bias) {
  const float sum = kPlain ? static_cast<float>(acc) : sum_value(acc);
  float y;
  if (kPlain || plain_scale(a))
    y = fmaf(sum * a, s, bias);
  else
    y = static_cast<float>(
        fma(static_cast<double>(sum) * static_cast<double>(a), static_cast<double>(s), static_cast<double>(bias)));
  static_cast<typename Elem<kType>::T*>(p.Y)[token * p.ldy + channel] = Elem<kType>::put(y);
}

// -- up to 128 tokens: a tile of 128 channels by all of them per cluster, k split over the
// cluster's CTAs and joined through distributed shared memory (integers: the order
// does not matter). Bound by the loads into shared memory: 64 tokens by 16384 x 4096
// weights take 11.2 us from L2 (67 MB, 6.0 TB/s). --

template <int kTok>
struct TileCfg {
  static constexpr int kA = 128 * kPieceK, kB = kTok * kPieceK;
  static constexpr int kStages = kTok <= 64 ? 4 : 3;
  static constexpr int kJoin = kTok * 128 * 4;  // partial sums, over the stages
  static constexpr int kTiles = kStages * (kA + kB) > kJoin ? kStages * (kA + kB) : kJoin;
  static constexpr int kSmem = kTiles + 1024;
  static constexpr int kColumns = kTok < 32 ? 32 : kTok;
};

template <int kType, int kTok>
__global__ void __launch_bounds__(192, 2)
    k_int8_tile(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Product p,
                int split) {
  using Cfg = TileCfg<kTok>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[2 * Cfg::kStages + 1];
  __shared__ uint32_t tmem_slot;
  const uint32_t tiles = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * Cfg::kStages, done = empty + 8 * Cfg::kStages;
  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
  const int channel0 = static_cast<int>(blockIdx.x) / split * 128;
  const int part = static_cast<int>(blockIdx.x) % split;
  const int tokens = static_cast<int>(p.m);  // at most kTok
  const int per = (p.pieces + split - 1) / split;
  const int first = part * per;
  const int count = min(p.pieces, first + per) - first;  // at least 1 (the host's choice of split)

  if (warp == 4) tmem_alloc<1>(smem_addr(&tmem_slot), Cfg::kColumns);
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t acc = __shfl_sync(0xffffffffu, tmem_slot, 0);
  bool ok = true;

  if (warp == 4) {
    const bool elected = elect_one();
    // the first stages' weights do not wait for the quantiser
    const int begun = min(count, Cfg::kStages);
    if (elected)
      for (int i = 0; i < begun; ++i) {
        mbar_expect_tx(full + 8 * i, Cfg::kA + Cfg::kB);
        tma_2d(tiles + i * (Cfg::kA + Cfg::kB), &map_w, (first + i) * kPieceK, channel0, full + 8 * i);
      }
    after_previous();
    Ring<Cfg::kStages> at;
    for (int i = 0; i < count; ++i, at.next()) {
      ok = __all_sync(0xffffffffu, at.wait_empty(empty, kWaitLimit));
      if (!ok) break;
      const uint32_t a = tiles + at.stage * (Cfg::kA + Cfg::kB), bar = full + 8 * at.stage;
      if (elected) {
        if (i >= begun) {
          mbar_expect_tx(bar, Cfg::kA + Cfg::kB);
          tma_2d(a, &map_w, (first + i) * kPieceK, channel0, bar);
        }
        tma_2d(a + Cfg::kA, &map_x, (first + i) * kPieceK, 0, bar);
      }
    }
    if (!ok) at.drain(full, kWaitLimit);  // before the memory is given back
  } else if (warp == 5) {
    const bool elected = elect_one();
    Ring<Cfg::kStages> at;
    for (int i = 0; i < count; ++i, at.next()) {
      ok = __all_sync(0xffffffffu, at.wait_full(full, kWaitLimit));
      if (!ok) break;
      tcgen05_after_sync();
      const uint32_t a = tiles + at.stage * (Cfg::kA + Cfg::kB);
      const uint64_t da = smem_desc(a, 16, 1024), db = smem_desc(a + Cfg::kA, 16, 1024);
      if (elected) {
#pragma unroll
        for (int j = 0; j < kPieceK / kStepK; ++j)
          mma_i8<1>(acc, da + j * (kStepK >> 4), db + j * (kStepK >> 4), idesc_i8(128, kTok), i > 0 || j > 0);
        mma_commit<1>(empty + 8 * at.stage);
      }
    }
    if (elected) mma_commit<1>(done);
  } else {
    after_previous();
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(done, 0, kWaitLimit));
    tcgen05_after_sync();
    const int64_t channel = channel0 + warp * 32 + lane;
    const bool live = ok && channel < p.n;
    const float s = live && split == 1 ? p.sb[channel] : 0.0f;
    const float bias = live && split == 1 && p.bias ? p.bias[channel] : 0.0f;
    constexpr int kCols = kTok < 32 ? 16 : 32;
    for (int j0 = 0; j0 < tokens; j0 += kCols) {
      uint32_t v[kCols];
      const uint32_t at = acc + (static_cast<uint32_t>(warp) << 21) + j0;  // lane 32 * warp in bits 16 and up
      if constexpr (kCols == 16)
        tmem_ld16(at, v);
      else
        tmem_ld32(at, v);
      tcgen05_wait_ld();
      if (split == 1) {
        const float mine = j0 + lane < tokens ? p.sa[j0 + lane] : 0.0f;
        if (!__any_sync(0xffffffffu, !plain_scale(mine)) && p.pieces < kMostPieces) {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (live && j0 + j < tokens)
              put_output<kType, true>(p, j0 + j, channel, static_cast<int>(v[j]), p.sa[j0 + j], s, bias);
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (live && j0 + j < tokens)
              put_output<kType>(p, j0 + j, channel, static_cast<int>(v[j]), p.sa[j0 + j], s, bias);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (j0 + j < tokens)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(tiles + 4 * ((j0 + j) * 128 + warp * 32 + lane)), "r"(v[j])
                         : "memory");
      }
    }
    tcgen05_before_sync();
  }
  if (!ok) g_stalled_int8 = 1;
  __syncwarp();
  if (split > 1) {
    cluster_sync_all();
    if (warp < 4) {
      const int64_t channel = channel0 + warp * 32 + lane;
      if (channel < p.n) {
        const float s = p.sb[channel], bias = p.bias ? p.bias[channel] : 0.0f;
        constexpr int kAtOnce = 8;  // tokens of this CTA's share whose partial sums are in flight
        for (int j0 = part; j0 < tokens; j0 += split * kAtOnce) {
          uint32_t sum[kAtOnce] = {};
          for (int r = 0; r < split; ++r) {
            const uint32_t from = map_shared(tiles + 4 * (warp * 32 + lane), r);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
              if (j0 + u * split < tokens) sum[u] += static_cast<uint32_t>(ld_shared_cluster(from + 512 * (j0 + u * split)));
          }
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            const int j = j0 + u * split;
            if (j < tokens) put_output<kType>(p, j, channel, static_cast<int>(sum[u]), p.sa[j], s, bias);
          }
        }
      }
    }
    cluster_sync_all();  // the partial sums stay until every CTA has read them
  } else {
    __syncthreads();
  }
  if (warp == 4) {
    tcgen05_after_sync();
    tmem_free<1>(acc, Cfg::kColumns);
  }
}

template <int kType, int kTok>
cudaError_t int8_tile(const CUtensorMap& map_w, const CUtensorMap& map_x, const Product& p, int split, cudaStream_t st) {
  using Cfg = TileCfg<kTok>;
  const cudaError_t e = cudaFuncSetAttribute(k_int8_tile<kType, kTok>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((p.n + 127) / 128 * split));
  note_launch();
  return launch_kernel(k_int8_tile<kType, kTok>, grid, 192, Cfg::kSmem, st, static_cast<unsigned>(split), p.early, map_w,
                       map_x, p, split);
}

// -- many tokens: a pair of CTAs (cta_group::2) per 256 channels by 256 tokens,
// persistent over the tiles, the accumulators of one tile written out while the next
// one is computed. Against the tiles above, with 4096 of k: 128 tokens by 4096 channels
// 16.6 (tiles: 13.8) us, 256 by 4096 17.0 (19.5), 256 by 16384 18.7 (24.2), 512 by 4096
// 17.4 (29.3). Bound by the tensor cores: 16384 tokens by 4096 channels by 16384 take
// 597 to 638 us by the clock that the power limit leaves, 3.4 to 3.7 POP/s, with the tensor
// pipe busy 96% of the time. --

constexpr int kPairStages = 6;
constexpr int kPairThreads = 320;  // eight epilogue warps, the producer, the MMA issuer
constexpr int kPairStage = 2 * 128 * kPieceK;  // each CTA: 128 rows of either operand
constexpr int kPairSmem = kPairStages * kPairStage + 1024;

// The tile order: blocks of up to 16 channel tiles, token tiles within a block, so
// that the operand rows that CTAs share at one time stay in L2.
struct TileAt {
  int channel, token;
};
__device__ __forceinline__ TileAt tile_at(int t, int channel_tiles, int token_tiles) {
  const int block = t / (16 * token_tiles), in = t - block * 16 * token_tiles;
  const int width = min(16, channel_tiles - 16 * block);
  return {16 * block + in % width, in / width};
}

template <int kType>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_int8_pair(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Product p,
                int channel_tiles, int token_tiles) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[2 * kPairStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ float token_scale[2][256];
  const uint32_t tiles = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kPairStages;
  const uint32_t done = empty + 8 * kPairStages, freed = done + 16;  // per accumulator buffer
  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
  const int rank = static_cast<int>(cluster_rank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  const int all = channel_tiles * token_tiles;

  if (warp == 8) tmem_alloc<2>(smem_addr(&tmem_slot), 512);
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(freed + 8 * i, 16);  // eight warps of either CTA
    }
    fence_mbar_init();
  }
  tcgen05_before_sync();
  cluster_sync_all();
  tcgen05_after_sync();
  const uint32_t acc = __shfl_sync(0xffffffffu, tmem_slot, 0);
  bool ok = true;

  if (warp == 8) {
    const bool elected = elect_one();
    const uint32_t full0 = map_shared(full, 0);
    after_previous();
    Ring<kPairStages> at;
    for (int t = pair; t < all && ok; t += pairs) {
      const TileAt tile = tile_at(t, channel_tiles, token_tiles);
      const int c0 = tile.channel * 256 + rank * 128, t0 = tile.token * 256 + rank * 128;
      for (int i = 0; i < p.pieces; ++i, at.next()) {
        ok = __all_sync(0xffffffffu, at.wait_empty(empty, kWaitLimit));
        if (!ok) break;
        const uint32_t a = tiles + at.stage * kPairStage, bar = full0 + 8 * at.stage;
        if (elected) {
          if (rank == 0) mbar_expect_tx(full + 8 * at.stage, 2 * kPairStage);
          tma_2d_pair(a, &map_w, i * kPieceK, c0, bar);
          tma_2d_pair(a + 128 * kPieceK, &map_x, i * kPieceK, t0, bar);
        }
      }
    }
    if (!ok && rank == 0) at.drain(full, kWaitLimit);
  } else if (warp == 9) {
    if (rank == 0) {
      const bool elected = elect_one();
      Ring<kPairStages> at;
      Ring<2> out;
      for (int t = pair; t < all && ok; t += pairs, out.next()) {
        ok = __all_sync(0xffffffffu, out.wait_empty(freed, kWaitLimit));
        if (!ok) break;
        tcgen05_after_sync();
        for (int i = 0; i < p.pieces; ++i, at.next()) {
          ok = __all_sync(0xffffffffu, at.wait_full(full, kWaitLimit));
          if (!ok) break;
          tcgen05_after_sync();
          const uint32_t a = tiles + at.stage * kPairStage;
          const uint64_t da = smem_desc(a, 16, 1024), db = smem_desc(a + 128 * kPieceK, 16, 1024);
          if (elected) {
#pragma unroll
            for (int j = 0; j < kPieceK / kStepK; ++j)
              mma_i8<2>(acc + out.stage * 256, da + j * (kStepK >> 4), db + j * (kStepK >> 4), idesc_i8(256, 256),
                        i > 0 || j > 0);
            mma_commit<2>(empty + 8 * at.stage);
          }
        }
        if (elected) mma_commit<2>(done + 8 * out.stage);
      }
    }
  } else {
    after_previous();
    int n = 0;
    for (int t = pair; t < all; t += pairs, ++n) {
      const int buf = n & 1;
      const TileAt at = tile_at(t, channel_tiles, token_tiles);
      const int64_t channel = static_cast<int64_t>(at.channel) * 256 + rank * 128 + (warp & 3) * 32 + lane;
      const int64_t token0 = static_cast<int64_t>(at.token) * 256;
      const int tokens = static_cast<int>(min(static_cast<int64_t>(256), p.m - token0));
      for (int j = threadIdx.x; j < tokens; j += 256) token_scale[buf][j] = p.sa[token0 + j];
      const bool live = channel < p.n;
      const float s = live ? p.sb[channel] : 0.0f;
      const float bias = live && p.bias ? p.bias[channel] : 0.0f;
      // the eight warps leave together: none waits here for one whose last wait ran out
      ok = barrier_and(1, 256, ok);
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(done + 8 * buf, (n >> 1) & 1, kWaitLimit));
      if (!ok) continue;
      tcgen05_after_sync();
      const int half = (warp >> 2) * 128, end = min(tokens, half + 128);  // this warp's tokens
      for (int j0 = half; j0 < end; j0 += 32) {
        uint32_t v[32];
        tmem_ld32(acc + (static_cast<uint32_t>(warp & 3) << 21) + buf * 256 + j0, v);
        tcgen05_wait_ld();
        const float mine = j0 + lane < tokens ? token_scale[buf][j0 + lane] : 0.0f;
        const bool plain = !__any_sync(0xffffffffu, !plain_scale(mine)) && p.pieces < kMostPieces;
        if (live && plain) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j0 + j < tokens)
              put_output<kType, true>(p, token0 + j0 + j, channel, static_cast<int>(v[j]), token_scale[buf][j0 + j], s, bias);
        } else if (live) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j0 + j < tokens)
              put_output<kType>(p, token0 + j0 + j, channel, static_cast<int>(v[j]), token_scale[buf][j0 + j], s, bias);
        }
      }
      tcgen05_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_shared(freed + 8 * buf, 0));
    }
  }
  if (!ok) g_stalled_int8 = 1;
  __syncwarp();
  tcgen05_before_sync();
  cluster_sync_all();  // neither CTA leaves while the other's MMAs or copies use its memory
  if (warp == 8) {
    tcgen05_after_sync();
    tmem_free<2>(acc, 512);
  }
}

template <int kType>
cudaError_t int8_pair(const CUtensorMap& map_w, const CUtensorMap& map_x, const Product& p, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(k_int8_pair<kType>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  const int64_t channel_tiles = (p.n + 255) / 256, token_tiles = (p.m + 255) / 256;
  if (channel_tiles * token_tiles > INT32_MAX / 32) return cudaErrorInvalidValue;
  const int pairs = static_cast<int>(std::min<int64_t>(sm_count() / 2, channel_tiles * token_tiles));
  note_launch();
  return launch_kernel(k_int8_pair<kType>, dim3(2 * pairs), kPairThreads, kPairSmem, st, 1, p.early, map_w, map_x, p,
                       static_cast<int>(channel_tiles), static_cast<int>(token_tiles));
}

// -- one or two tokens: the weights' bytes are the cost, and set-up time. Each CTA holds
// the tokens in shared memory (quantising them itself when they come as floats) and its
// warps take output channels in turn, a lane 16 bytes of k at a time (dp4a). The first
// channels' weights are on their way while the tokens are. Without barriers, TMEM and a
// join it beats the tensor-core tiles below for 4096 x 4096 weights in L2: 3.9 against
// 6.2 us for one token, 4.9 against 6.3 for two; at four (9.0 against 6.4) each token's
// reads of shared memory cost more than they. Bound by latency: 16.8 MB in 3.9 us. --

constexpr int kFewTokens = 2;
constexpr int64_t kFewBytes = 64 << 10;  // shared memory of the tokens
constexpr int kFewThreads = 256;

// kIn: the tokens' type, or -1 for rows that are quantised already (A, sa). kM tokens.
template <int kIn, int kType, int kM>
__global__ void __launch_bounds__(kFewThreads)
    k_int8_few(const void* X, int64_t ldx, bool wide, const int8_t* __restrict__ B, int64_t ldb,
               const Product p, int64_t k) {
  extern __shared__ int4 tokens[];  // [kM][ceil(k / 16)]
  __shared__ uint32_t part[kFewThreads / 32];
  __shared__ float token_scale[kM];
  constexpr int kAhead = 8;  // pieces of 16 bytes in flight per lane
  const int warp = warp_id(), lane = lane_id();
  const int kp = static_cast<int>((k + 15) / 16);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kFewThreads / 32);
  int64_t channel = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + warp;
  const int whole = static_cast<int>(k / 16);  // pieces that end inside the row
  const int tail = static_cast<int>(k) - whole * 16;  // bytes of the last, short piece: one per lane
  int4 w[kAhead];
  int last = 0;
  const auto load = [&](int64_t c, int at) {
    const int8_t* row = B + min(c, p.n - 1) * ldb;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int piece = at + lane + 32 * i;
      w[i] = piece < whole ? __ldg(reinterpret_cast<const int4*>(row) + piece) : make_int4(0, 0, 0, 0);
    }
    if (at == 0 && lane < tail) last = __ldg(row + whole * 16 + lane);
  };
  load(channel, 0);

  if constexpr (kIn >= 0) {
    using T = typename Elem<kIn < 0 ? 0 : kIn>::T;
    const T* x = static_cast<const T*>(X);
    // the warps share the tokens out: 8 / kM of them to each
    constexpr int kType1 = kIn < 0 ? 0 : kIn, kWarps = kFewThreads / 32 / kM;
    const int j = warp / kWarps, first = warp % kWarps * 32 + lane;
    const T* row = x + j * ldx;
    Largest<kType1> top;
#pragma unroll 4
    for (int64_t c = first; c < 2 * kp; c += kWarps * 32) top.add(load8<kType1>(row, c * 8, k, wide));
    const uint32_t mine = __reduce_max_sync(0xffffffffu, top.bits());
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    const RowScale a = row_scale(__reduce_max_sync(0xffffffffu, part[j * kWarps + lane % kWarps]));
    if (first == 0) token_scale[j] = a.scale;
#pragma unroll 4
    for (int64_t c = first; c < 2 * kp; c += kWarps * 32) {
      float v[8];
      floats8<kType1>(load8<kType1>(row, c * 8, k, wide), v);
      reinterpret_cast<uint2*>(tokens)[static_cast<int64_t>(j) * kp * 2 + c] = quantize8(v, a);
    }
  } else {
    after_previous();
    const int8_t* x = static_cast<const int8_t*>(X);
#pragma unroll 8
    for (int i = threadIdx.x; i < kM * kp; i += kFewThreads) {
      const int j = i / kp, c = i - j * kp;
      if (c < whole) tokens[i] = reinterpret_cast<const int4*>(x + j * ldx)[c];
    }
    for (int i = threadIdx.x; i < kM * tail; i += kFewThreads) {
      const int j = i / tail, c = whole * 16 + i - j * tail;
      reinterpret_cast<int8_t*>(tokens)[static_cast<int64_t>(j) * kp * 16 + c] = x[j * ldx + c];
    }
    if (threadIdx.x < kM) token_scale[threadIdx.x] = p.sa[threadIdx.x];
  }
  __syncthreads();

  for (; channel < p.n; channel += step) {
    int acc[kM] = {};
    if (lane < tail) {
#pragma unroll
      for (int j = 0; j < kM; ++j)
        acc[j] = last * reinterpret_cast<const int8_t*>(tokens)[(j * kp + whole) * 16 + lane];
    }
    for (int at = 0; at < whole; at += 32 * kAhead) {
      if (at > 0) load(channel, at);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int piece = at + lane + 32 * i;
        if (piece < whole) {
#pragma unroll
          for (int j = 0; j < kM; ++j) {
            const int4 x = tokens[j * kp + piece];
            acc[j] = __dp4a(w[i].w, x.w, __dp4a(w[i].z, x.z, __dp4a(w[i].y, x.y, __dp4a(w[i].x, x.x, acc[j]))));
          }
        }
      }
    }
    const float s = p.sb[channel], bias = p.bias ? p.bias[channel] : 0.0f;
    if (channel + step < p.n) load(channel + step, 0);
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kM; ++j) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[j]);
      if (lane == j) mine = sum;
    }
    if (lane < kM) put_output<kType>(p, lane, channel, mine, token_scale[lane], s, bias);
  }
}

template <int kIn, int kType>
cudaError_t int8_few_tokens(const void* X, int64_t ldx, const int8_t* B, int64_t ldb, const Product& p, int64_t k,
                            cudaStream_t st) {
  const size_t smem = static_cast<size_t>(p.m) * ((k + 15) / 16 * 16);
  const bool wide = kIn >= 0 && rows_aligned16(X, ldx, type_bytes(kIn));
  const auto run = [&](auto kernel) {
    // the 48 KB that need no opt-in are for this and the kernel's own shared variables
    if (smem > (48 << 10) - 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFewBytes));
      if (e != cudaSuccess) return e;
    }
    const int64_t per = kFewThreads / 32, most = static_cast<int64_t>(sm_count()) * 4;
    note_launch();
    return launch_kernel(kernel, dim3(static_cast<unsigned>(std::min((p.n + per - 1) / per, most))), kFewThreads, smem, st,
                         1, p.early, X, ldx, wide, B, ldb, p, k);
  };
  return p.m == 1 ? run(k_int8_few<kIn, kType, 1>) : run(k_int8_few<kIn, kType, 2>);
}

bool few_tokens(int64_t m, int64_t k) { return m <= kFewTokens && m * ((k + 15) / 16 * 16) <= kFewBytes; }
// Whether each CTA quantises the tokens itself. That repeats the work in every CTA, but
// spares a caller the second launch and its workspace. bfloat16, 4096 channels, us in a
// graph and from Python, so / as two launches: one token of 1024 entries 5.0 / 5.2 and 11.2
// / 15.6, of 2048 5.3 / 5.1, of 4096 7.5 / 6.4 and 11.1 / 15.5, of 8192 10.6 / 8.5 and 12.3 /
// 15.6, two of 2048 6.4 / 5.6, two of 4096 9.4 / 7.3; 16384 channels, one of 4096 12.2 / 10.0
// and 14.4 / 15.5. So up to 4096 entries, where a graph loses no more than a launch gains.
bool few_entries(int64_t m, int64_t k) { return few_tokens(m, k) && m * k <= 4096; }

// A map of 8-bit rows in boxes of 128 bytes by `rows`.
bool map_rows8(CUtensorMap* map, const int8_t* p, int64_t n, int64_t k, int64_t ld, int rows) {
  const uint64_t sizes[2] = {static_cast<uint64_t>(k), static_cast<uint64_t>(n)}, strides[1] = {static_cast<uint64_t>(ld)};
  const uint32_t box[2] = {kPieceK, static_cast<uint32_t>(rows)};
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, sizes, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kType, int kTok>
cudaError_t int8_split(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const Product& p, int64_t k,
                       cudaStream_t st) {
  CUtensorMap map_w, map_x;
  if (!map_rows8(&map_w, B, p.n, k, ldb, 128) || !map_rows8(&map_x, A, p.m, k, lda, kTok)) return cudaErrorInvalidValue;
  const int64_t tiles = (p.n + 127) / 128;
  // Split k while the CTAs leave SMs idle, with at least two pieces each. us with 1 / 2 / 4
  // / 8 parts: 16 tokens by 4096 x 4096 8.4 / 7.2 / 6.4 / 8.0, 128 by 4096 x 4096 17.3 / 16.8
  // / 13.8 / 15.1; 64 by 16384 x 4096 12.5 / 13.9 (a second CTA per SM shares its loads).
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sm_count() && p.pieces >= 4 * split) split *= 2;
  while (split > 1 && (split - 1) * ((p.pieces + split - 1) / split) >= p.pieces) split /= 2;
  return int8_tile<kType, kTok>(map_w, map_x, p, split, st);
}

template <int kType>
cudaError_t int8_product(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const Product& p, int64_t k,
                         cudaStream_t st) {
  if (few_tokens(p.m, k)) return int8_few_tokens<-1, kType>(A, lda, B, ldb, p, k, st);
  if (p.m <= 16) return int8_split<kType, 16>(A, lda, B, ldb, p, k, st);
  if (p.m <= 32) return int8_split<kType, 32>(A, lda, B, ldb, p, k, st);
  if (p.m <= 64) return int8_split<kType, 64>(A, lda, B, ldb, p, k, st);
  if (p.m <= 128) return int8_split<kType, 128>(A, lda, B, ldb, p, k, st);
  CUtensorMap map_w, map_x;
  if (!map_rows8(&map_w, B, p.n, k, ldb, 128) || !map_rows8(&map_x, A, p.m, k, lda, 128)) return cudaErrorInvalidValue;
  return int8_pair<kType>(map_w, map_x, p, st);
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

namespace {
cudaError_t int8_matmul(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb, const float* sb,
                        const float* bias, int64_t m, int64_t n, int64_t k, void* Y, int type, int64_t ldy, bool early,
                        cudaStream_t st) {
  const Product p = {sa, sb, bias, Y, m, n, ldy, static_cast<int>((k + kPieceK - 1) / kPieceK), early};
  switch (type) {
    case kF32: return int8_product<kF32>(A, lda, B, ldb, p, k, st);
    case kBF16: return int8_product<kBF16>(A, lda, B, ldb, p, k, st);
    default: return int8_product<kF16>(A, lda, B, ldb, p, k, st);
  }
}
}  // namespace

cudaError_t launch_int8_matmul(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb,
                               const float* sb, const float* bias, int64_t m, int64_t n, int64_t k, void* Y, int type,
                               int64_t ldy, cudaStream_t st) {
  return int8_matmul(A, lda, sa, B, ldb, sb, bias, m, n, k, Y, type, ldy, false, st);
}

size_t int8_linear_workspace(int64_t m, int64_t k) {
  if (m == 0 || few_entries(m, k)) return 0;
  return static_cast<size_t>(m) * ((k + 31) / 32 * 32 + 8);  // integers, scales, status
}

cudaError_t launch_int8_linear(const void* X, int x_type, int64_t ldx, const int8_t* B, int64_t ldb, const float* sb,
                               const float* bias, int64_t m, int64_t n, int64_t k, void* Y, int64_t ldy, void* ws,
                               cudaStream_t st) {
  if (few_entries(m, k)) {
    const Product p = {nullptr, sb, bias, Y, m, n, ldy, 0, false};
    switch (x_type) {
      case kF32: return int8_few_tokens<kF32, kF32>(X, ldx, B, ldb, p, k, st);
      case kBF16: return int8_few_tokens<kBF16, kBF16>(X, ldx, B, ldb, p, k, st);
      default: return int8_few_tokens<kF16, kF16>(X, ldx, B, ldb, p, k, st);
    }
  }
  const int64_t ldq = (k + 31) / 32 * 32;
  auto* q = static_cast<int8_t*>(ws);
  auto* scale = reinterpret_cast<float*>(q + m * ldq);
  const cudaError_t e =
      launch_int8_quantize(X, x_type, m, k, ldx, q, ldq, scale, reinterpret_cast<int32_t*>(scale + m), st);
  if (e != cudaSuccess) return e;
  return int8_matmul(q, ldq, scale, B, ldb, sb, bias, m, n, k, Y, x_type, ldy, true, st);
}

cudaError_t int8_stalled(bool* stalled) {
  int v = 0;
  cudaError_t e = cudaDeviceSynchronize();  // the copy alone does not wait for non-blocking streams
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_stalled_int8, sizeof(v));
  *stalled = v != 0;
  if (e == cudaSuccess && v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_stalled_int8, &v, sizeof(v));
  }
  return e;
}

}  // namespace ecasq
