// Activation checkpoints in 8 bits and the weight gradient read from them
// (include/ecasq.h, "8-bit operators").
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kernels.cuh"
#include "rows8.cuh"
#include "tensor.cuh"

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

// Four bytes, each filled with the sign bit of the byte that its selector nibble (8 plus
// the byte's number) names.
__device__ __forceinline__ uint32_t byte_signs(uint32_t a, uint32_t b, uint32_t selector) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(selector));
  return r;
}

// One thread per 8 entries (one Philox block), four threads per block of 32; a CTA
// covers blockDim.y rows by 8 * blockDim.x columns. Bound by instruction issue: 26
// instructions per entry, half of them the ten Philox rounds and what feeds them
// (16384 x 4096 bfloat16: 72 us, 2.8 TB/s, issue 70%).
//
// With Z = nearest(2^16 |x| / s), the magnitude floor(|x| / s) plus one if 16 random
// bits u are below the fraction's nearest(65536 f) is (Z + 65535 - u) >> 16. Adding
// 2^23 in a fused multiply-add leaves Z in the low 23 bits (the scaling is exact, so
// there is one rounding, ties to even), and the magnitude in bits 16 to 22 of the sum.
template <int kType, bool kSeedWord>
__global__ void __launch_bounds__(256)
    k_checkpoint8(const typename Elem<kType>::T* __restrict__ X, int64_t t, int64_t k, int64_t ldx, bool wide,
                  const Philox4x32::RoundKeys keys, uint64_t seed, const uint64_t* __restrict__ seed_add,
                  int8_t* __restrict__ Q, int64_t ldq, uint8_t* __restrict__ S, int64_t lds) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t pieces = (k + 31) / 32 * 4;
  const bool live = r < t && c < pieces;
  Eight<kType> in = {};
  if (live) in = load8<kType>(X + r * ldx, c * 8, k, wide);
  Largest<kType> top;
  top.add(in);
  uint32_t m = top.bits();
  // the random bits do not wait for the load
  const uint4 counter = make_uint4(static_cast<uint32_t>(c), static_cast<uint32_t>(r), kStreamCheckpoint, 0);
  uint4 u;
  if constexpr (kSeedWord) {
    const uint64_t key = seed + *seed_add;
    u = Philox4x32::block(counter, static_cast<uint32_t>(key), static_cast<uint32_t>(key >> 32));
  } else {
    u = Philox4x32::block(counter, keys);
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (!live) return;
  const uint32_t b = scale_byte(m);
  uint32_t word[2] = {0, 0};
  if (b != kScaleNaN) {
    const uint32_t rnd[4] = {~u.x, ~u.y, ~u.z, ~u.w};  // 65535 - u in either half
    float v[8];
    floats8<kType>(in, v);
    uint32_t up_bits = (254u + 16u - b) << 23;  // 2^16 / s, a power of two
    if (b < 17) {                               // beyond float32: in two exact steps
      up_bits -= 64u << 23;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= 0x1p64f;
    }
    const float up = __uint_as_float(up_bits);
    const uint32_t* raw = reinterpret_cast<const uint32_t*>(&in);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = fmaf(fabsf(v[4 * h + e]), up, 8388608.0f);
        const uint32_t w = rnd[2 * h + (e >> 1)];
        q[e] = __float_as_uint(z) + ((e & 1) ? w >> 16 : w & 0xffffu);
      }
      // the magnitudes (byte 2 of each sum), negated where the sign byte is all ones; the
      // addition of one stays inside its byte
      const uint32_t mag = __byte_perm(__byte_perm(q[0], q[1], 0x0062), __byte_perm(q[2], q[3], 0x0062), 0x5410);
      uint32_t neg;
      if constexpr (kType == kF32)
        neg = __byte_perm(byte_signs(raw[4 * h], raw[4 * h + 1], 0x00FB),
                          byte_signs(raw[4 * h + 2], raw[4 * h + 3], 0x00FB), 0x5410);
      else
        neg = byte_signs(raw[2 * h], raw[2 * h + 1], 0xFDB9);
      const uint32_t flip = mag ^ neg, one = neg & 0x01010101u;
      word[h] = ((flip & 0x7f7f7f7fu) + one) ^ (flip & 0x80808080u);
    }
  }
  *reinterpret_cast<uint2*>(Q + r * ldq + c * 8) = make_uint2(word[0], word[1]);
  if ((c & 3) == 0) S[r * lds + (c >> 2)] = static_cast<uint8_t>(b);
}

__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == kScaleNaN ? 0x7fc00000u : b << 23);
}

// One thread per 8 entries; bound by memory (16384 x 4096 bfloat16: 40 us, 5.1 TB/s).
// Rows off the 16-byte boundary go through shared memory, so
// that a warp's stores of single entries are adjacent (a thread's own eight at a time
// took 10.3 instead of 5 us for 3001 x 777 float32).
template <int kType>
__global__ void __launch_bounds__(256)
    k_checkpoint8_restore(const int8_t* __restrict__ Q, int64_t ldq, const uint8_t* __restrict__ S, int64_t lds,
                          int64_t t, int64_t k, typename Elem<kType>::T* __restrict__ X, int64_t ldx, bool wide) {
  __shared__ float lines[8][8 * 33];
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  const bool live = r < t && c * 8 < k;
  float v[8] = {};
  if (live) {
    const int8_t* from = Q + r * ldq + c * 8;
    uint2 w = make_uint2(0, 0);
    if (c * 8 + 8 <= k) {
      w = __ldg(reinterpret_cast<const uint2*>(from));
    } else {  // the memory of the last row may end with its entries
      for (int e = 0; c * 8 + e < k; ++e) (e < 4 ? w.x : w.y) |= static_cast<uint32_t>(static_cast<uint8_t>(from[e])) << (8 * (e & 3));
    }
    const float s = scale_value(S[r * lds + (c >> 2)]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = e < 4 ? w.x : w.y;
      v[e] = static_cast<float>(static_cast<int8_t>(x >> (8 * (e & 3)))) * s;
      if (kType == kF16 && fabsf(v[e]) > 65504.0f) v[e] = copysignf(65504.0f, v[e]);
    }
  }
  if (wide || blockDim.x < 32) {
    if (live) store8<kType>(X + r * ldx, c * 8, k, wide, v);
    return;
  }
  const int lane = lane_id();  // a warp's pieces are adjacent pieces of one row
  float* line = lines[(threadIdx.y * blockDim.x + threadIdx.x) >> 5];
#pragma unroll
  for (int e = 0; e < 8; ++e) line[lane * 8 + e + (lane >> 2)] = v[e];
  __syncwarp();
  const int64_t c0 = (c - lane) * 8;
  if (r < t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t j = c0 + e * 32 + lane;
      if (j < k) X[r * ldx + j] = Elem<kType>::put(line[e * 32 + lane + e]);
    }
  }
}

// Threads along a row and rows per CTA (256 threads), and the grid, for `pieces`
// pieces of 8 entries per row.
void piece_grid(int64_t t, int64_t pieces, dim3* grid, dim3* block) {
  unsigned x = 4;
  while (x < 256 && x < pieces) x *= 2;
  *block = dim3(x, 256 / x);
  *grid = dim3(static_cast<unsigned>((t + block->y - 1) / block->y), static_cast<unsigned>((pieces + x - 1) / x));
}

// ---- weight gradient -------------------------------------------------------------
//
// dW = dY^T X^ with tcgen05.mma kind::f16 (bf16 operands, float32 accumulators in
// TMEM). X^ = q s is exact in bf16 (8 bits times a power of two) and is made from
// the checkpoint on its way to the tensor cores: warps read the integers from the
// stage that TMA filled and write bf16 into the operand's shared memory, once for
// all terms of dY. Both operands lie token by token, so both are M- or N-contiguous
// ("MN-major") and nothing is transposed. The features of X are the M side: a
// thread of the epilogue owns one feature and the 32 lanes of a warp write 32
// adjacent entries of a row of dW. A pair of CTAs (cta_group::2) takes 256 features
// by 256 outputs; each CTA converts its own 128 features only.
//
// Bound by the tensor cores and their clock, with instruction issue close behind (16384
// tokens, 4096 x 4096, bfloat16: 420 to 450 us by the clock that the power limit leaves, 1.22
// to 1.31 PFLOP/s; in 449 us at 1.57 GHz tensor pipe 64%, issue 72%; the 256 tiles are 3.46
// rounds of 74 pairs). float32 dY, 4096 tokens, 4096 x 1024: 70 us behind 30 us for its terms.
//
// The tensor core adds to its float32 accumulator by cutting, not rounding: a step of
// 16 tokens loses up to 2^-23 of the running sum, always towards zero (measured: 2.2e-6
// after 96 steps of random signs, 7.1e-4 after 8192 steps of positive products). So an accumulator takes a few steps only and
// the epilogue warps add it, rounding to nearest, to sums that they hold in registers:
// 16 steps (24 for the three terms of a float32 dY) for float32 and float16 results, 64
// for bfloat16 results (at most 2^-17 of the sum, against 2^-8 for their own rounding).

__device__ int g_stalled_checkpoint8;  // set when a bounded wait gave up

constexpr int kTok = 64;                  // tokens per stage
constexpr int kOperand = kTok * 128 * 2;  // bf16 operand of one CTA: 128 features, or 128 outputs
constexpr int kHalf = kTok * 64 * 2;      // its 64-wide half (one swizzle atom across)
constexpr int kInts = kTok * 128;         // integers of 128 features
constexpr int kScales = kTok * 16;        // scale bytes of 512 features
constexpr int kQStage = kInts + kScales;
// Stages of integers, of converted X^ and of dY. A stage of 64 tokens keeps the tensor
// cores busy for 512 clocks and its loads take two to four times as long.
constexpr int kQStages = 7, kXStages = 4, kYStages = 6;
constexpr int kGradSmem = kQStages * kQStage + kXStages * kOperand + kYStages * kOperand + 1024;

// Warps: the epilogue's, the producers of dY and of the integers, the MMA issuer, an
// idle one, the converters. The converters
// come in kXStages groups that take the stages in turn, so that the latencies of one
// stage's conversion (its wait, its loads, the fence, the arrival at the other CTA)
// are covered by three others'. The epilogue's threads hold 128 sums each, so the warps
// come in groups of four that trade registers (setmaxnreg): of the launch's 896 * 72 =
// 64512 they take 256 * 168 + 640 * 32 = 63488. 16384 x 4096 x 4096, us, with 4 / 8 / 16
// converters: 538 / 441 / 420.
constexpr int kEpilogue = 8;
constexpr int kLoad = 8, kIssue = 9, kLoadInts = 10;
constexpr int kConvert0 = 12, kConvert = 16;
constexpr int kGradThreads = 32 * (kConvert0 + kConvert);
constexpr int kLaunchRegisters = 72;  // 65536 / 896 in steps of 8: what __launch_bounds__ gives a thread
constexpr int kMostRegisters = 168, kFewRegisters = 32;
static_assert(32 * kEpilogue * kMostRegisters + (kGradThreads - 32 * kEpilogue) * kFewRegisters <=
                  kGradThreads * kLaunchRegisters,
              "the warps wait for ever for registers that the block was not launched with");

struct Gradient {
  void* out;          // dW, or the partial sums when the tokens are split
  int64_t o, k, ld;   // size and pitch of one output matrix
  int feature_tiles, output_tiles;
  int pieces;         // ceil(t / 64)
  int terms;          // bf16 terms of dY, the smallest first
  int split, per;     // parts of the token axis, pieces of one
  int chunk;          // pieces that one accumulator takes
  bool early;         // launched behind the copy of dY's terms
};

// Two bytes of x as two's complement integers times s, in bf16. 0x4300 | b is the bf16
// number 128 + (b & 127) with bit 7 cleared, and 128 or 256 with the low bits
// cleared; their difference is the integer, exactly.
__device__ __forceinline__ uint32_t two_values(uint32_t x, uint32_t selector, __nv_bfloat162 s) {
  const uint32_t h = __byte_perm(x, 0x43434343u, selector);
  const uint32_t low = h & 0xFF7FFF7Fu, high = h & 0xFF80FF80u;
  const __nv_bfloat162 v = __hmul2(
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&low), *reinterpret_cast<const __nv_bfloat162*>(&high)), s);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    k_wgrad(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_s,
            const __grid_constant__ CUtensorMap map_y, const Gradient g) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[2 * kQStages + 2 * kXStages + 2 * kYStages + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t xs = (smem_addr(smem_raw) + 1023) & ~1023u, ys = xs + kXStages * kOperand, qs = ys + kYStages * kOperand;
  // integers and scales here, and read (own CTA); X^ converted (both CTAs, on the even
  // one), X^ read by the MMAs; dY here (both CTAs, on the even one), dY read; per
  // accumulator: done, freed
  const uint32_t ints = smem_addr(bars), q_empty = ints + 8 * kQStages, ready = q_empty + 8 * kQStages,
                 x_empty = ready + 8 * kXStages, full = x_empty + 8 * kXStages, y_empty = full + 8 * kYStages,
                 done = y_empty + 8 * kYStages, freed = done + 16;
  constexpr int kGroup = kConvert / kXStages;  // warps that convert one stage
  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
  const int rank = static_cast<int>(cluster_rank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  const int tiles = g.feature_tiles * g.output_tiles;
  const int all = tiles * g.split;
  next_may_begin();

  if (warp == kLoad) tmem_alloc<2>(smem_addr(&tmem_slot), 512);
  if (threadIdx.x == 0) {
    prefetch_map(&map_q);
    prefetch_map(&map_s);
    prefetch_map(&map_y);
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(ints + 8 * i, 1);
      mbar_init(q_empty + 8 * i, kGroup);
    }
    for (int i = 0; i < kXStages; ++i) {
      mbar_init(ready + 8 * i, 2 * kGroup);
      mbar_init(x_empty + 8 * i, 1);
    }
    for (int i = 0; i < kYStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(y_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(freed + 8 * i, 2 * kEpilogue);
    }
    fence_mbar_init();
  }
  tcgen05_before_sync();
  cluster_sync_all();
  tcgen05_after_sync();
  const uint32_t acc = __shfl_sync(0xffffffffu, tmem_slot, 0);
  bool ok = true;

  if (warp >= kEpilogue) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegisters));
    if (warp == kLoad) {
      const bool elected = elect_one();
      const uint32_t full0 = map_shared(full, 0);
      after_previous();  // dY's terms; the integers do not wait for them
      Ring<kYStages> y;
      for (int w = pair; w < all && ok; w += pairs) {
        const int tile = w % tiles, part = w / tiles;
        const int o0 = (tile / g.feature_tiles) * 256 + rank * 128;
        const int last = min(g.pieces, (part + 1) * g.per);
        for (int i = part * g.per; i < last && ok; ++i)
          for (int term = 0; term < g.terms; ++term, y.next()) {
            ok = __all_sync(0xffffffffu, y.wait_empty(y_empty, kWaitLimit));
            if (!ok) break;
            const uint32_t to = ys + y.stage * kOperand, bar = full0 + 8 * y.stage;
            if (elected) {
              if (rank == 0) mbar_expect_tx(full + 8 * y.stage, 2 * kOperand);
              tma_3d_pair(to, &map_y, o0, i * kTok, term, bar);
              tma_3d_pair(to + kHalf, &map_y, o0 + 64, i * kTok, term, bar);
            }
          }
      }
      if (!ok && rank == 0) y.drain(full, kWaitLimit);  // before the memory is given back
    } else if (warp == kLoadInts) {
      const bool elected = elect_one();
      Ring<kQStages> q;
      for (int w = pair; w < all && ok; w += pairs) {
        const int tile = w % tiles, part = w / tiles;
        const int f0 = (tile % g.feature_tiles) * 256 + rank * 128;
        const int last = min(g.pieces, (part + 1) * g.per);
        for (int i = part * g.per; i < last; ++i, q.next()) {
          ok = __all_sync(0xffffffffu, q.wait_empty(q_empty, kWaitLimit));
          if (!ok) break;
          const uint32_t to = qs + q.stage * kQStage, bar = ints + 8 * q.stage;
          if (elected) {
            mbar_expect_tx(bar, kInts + kScales);
            tma_2d(to, &map_q, f0, i * kTok, bar);
            tma_2d(to + kInts, &map_s, (f0 / 32) & ~15, i * kTok, bar);
          }
        }
      }
      if (!ok) q.drain(ints, kWaitLimit);
    } else if (warp == kIssue && rank == 0) {
      const bool elected = elect_one();
      Ring<kXStages> x;
      Ring<kYStages> y;
      Ring<2> out;
      for (int w = pair; w < all && ok; w += pairs) {
        const int part = w / tiles;
        const int count = min(g.pieces, (part + 1) * g.per) - part * g.per;
        for (int i = 0; i < count && ok; out.next()) {
          ok = __all_sync(0xffffffffu, out.wait_empty(freed, kWaitLimit));
          if (!ok) break;
          tcgen05_after_sync();
          const int end = min(count, i + g.chunk);
          for (bool add = false; i < end && ok; ++i, x.next()) {
            ok = __all_sync(0xffffffffu, x.wait_full(ready, kWaitLimit));
            const uint64_t da = smem_desc(xs + x.stage * kOperand, kHalf, 1024);
            for (int term = 0; term < g.terms && ok; ++term, y.next()) {
              ok = __all_sync(0xffffffffu, y.wait_full(full, kWaitLimit));
              if (!ok) break;
              tcgen05_after_sync();
              const uint64_t db = smem_desc(ys + y.stage * kOperand, kHalf, 1024);
              if (elected) {
#pragma unroll
                for (int j = 0; j < kTok / 16; ++j)  // 16 tokens per MMA: 16 rows of 128 bytes
                  mma_bf16_pair(acc + out.stage * 256, da + j * (2048 >> 4), db + j * (2048 >> 4),
                                idesc_bf16_mn(256, 256), add || j > 0);
                mma_commit<2>(y_empty + 8 * y.stage);
              }
              add = true;
            }
            if (elected) mma_commit<2>(x_empty + 8 * x.stage);
          }
          if (elected) mma_commit<2>(done + 8 * out.stage);
        }
      }
    } else if (warp >= kConvert0) {
      constexpr int kRows = kTok / kGroup;  // tokens of one warp
      const uint32_t ready0 = map_shared(ready, 0);
      const uint32_t group = (warp - kConvert0) / kGroup;  // and the X^ stage that it fills
      const int row = (warp - kConvert0) % kGroup * kRows + (lane >> 3), chunk = lane & 7;
      // 16-byte pieces 2c and 2c + 1 of a 128-byte row, swizzled by the row; the upper 64
      // features write theirs in the other order, so that the eight threads of a row
      // hit different banks
      const int half = chunk >> 2, c = (chunk & 3) * 2;
      const uint32_t to = xs + group * kOperand + half * kHalf + row * 128;
      Ring<kQStages> q;
      Ring<kXStages> x;
      for (int w = pair; w < all && ok; w += pairs) {
        const int tile = w % tiles, part = w / tiles;
        const int f0 = (tile % g.feature_tiles) * 256 + rank * 128;
        const uint32_t block = ((f0 / 32) & 15) + (chunk >> 1);
        const int count = min(g.pieces, (part + 1) * g.per) - part * g.per;
        for (int i = 0; i < count; ++i, q.next(), x.next()) {
          if (x.stage != group) continue;
          ok = __all_sync(0xffffffffu, q.wait_full(ints, kWaitLimit) && x.wait_empty(x_empty, kWaitLimit));
          if (!ok) break;
          const uint32_t from = qs + q.stage * kQStage + row * 128 + chunk * 16;
          const uint32_t scales = qs + q.stage * kQStage + kInts + row * 16 + block;
#pragma unroll 2
          for (int r = 0; r < kRows; r += 4) {
            const uint4 x = ld_shared16(from + r * 128);
            const uint32_t b = ld_shared1(scales + r * 16);
            const uint32_t bits = (b == kScaleNaN ? 0x7FFFu : b << 7) * 0x10001u;
            const __nv_bfloat162 sc = *reinterpret_cast<const __nv_bfloat162*>(&bits);
            const uint4 v0 = make_uint4(two_values(x.x, 0x4140, sc), two_values(x.x, 0x4342, sc),
                                        two_values(x.y, 0x4140, sc), two_values(x.y, 0x4342, sc));
            const uint4 v1 = make_uint4(two_values(x.z, 0x4140, sc), two_values(x.z, 0x4342, sc),
                                        two_values(x.w, 0x4140, sc), two_values(x.w, 0x4342, sc));
            const int swizzle = (row + r) & 7;
            st_shared16(to + r * 128 + (((c + half) ^ swizzle) << 4), half ? v1 : v0);
            st_shared16(to + r * 128 + (((c + 1 - half) ^ swizzle) << 4), half ? v0 : v1);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_cluster(ready0 + 8 * group);
            mbar_arrive(q_empty + 8 * q.stage);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMostRegisters));
    constexpr int kCols = 128;  // columns of this warp
    const int col0 = (warp >> 2) * 128;
    const uint32_t lanes = acc + (static_cast<uint32_t>(warp & 3) << 21) + col0;
    const uint32_t freed0 = map_shared(freed, 0);
    int n = 0;
    for (int w = pair; w < all && ok; w += pairs) {
      const int tile = w % tiles, part = w / tiles;
      const int64_t feature = static_cast<int64_t>(tile % g.feature_tiles) * 256 + rank * 128 + (warp & 3) * 32 + lane;
      const int64_t o0 = static_cast<int64_t>(tile / g.feature_tiles) * 256 + col0;
      const int rows = static_cast<int>(min(static_cast<int64_t>(kCols), g.o - o0));  // may be 0 or less
      auto* out = static_cast<typename Elem<kOut>::T*>(g.out) + (part * g.o + o0) * g.ld + feature;
      const int count = min(g.pieces, (part + 1) * g.per) - part * g.per;
      float sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j] = 0.0f;
      for (int i = 0; i < count; i += g.chunk, ++n) {
        const int buf = n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(done + 8 * buf, (n >> 1) & 1, kWaitLimit));
        if (!ok) break;
        tcgen05_after_sync();
#pragma unroll
        for (int j0 = 0; j0 < kCols; j0 += 16) {
          uint32_t v[16];
          tmem_ld16(lanes + buf * 256 + j0, v);
          tcgen05_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[j0 + j] += __uint_as_float(v[j]);
        }
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(freed0 + 8 * buf);
      }
      if (ok && feature < g.k) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (j < rows) out[j * g.ld] = Elem<kOut>::put(sum[j]);
      }
    }
  }
  if (!ok) g_stalled_checkpoint8 = 1;
  __syncwarp();
  tcgen05_before_sync();
  cluster_sync_all();  // neither CTA leaves while the other's MMAs or copies use its memory
  if (warp == kLoad) {
    tcgen05_after_sync();
    tmem_free<2>(acc, 512);
  }
}

// dY [t][o] as bf16 terms [kTerms][t][ld], whose sum is dY exactly: each term is the rest
// so far cut (not rounded: no overflow) to its upper 8 bits; the largest term is the
// last one. (Of a float32 entry below 2^-110 the third term cuts what is under 2^-133,
// bfloat16's smallest value.) What is not finite is the last term, with zeros before it.
template <int kIn, int kTerms>
__global__ void __launch_bounds__(256)
    k_terms(const typename Elem<kIn>::T* __restrict__ dY, int64_t ldy, bool wide, int64_t t, int64_t o,
            __nv_bfloat16* __restrict__ out, int64_t ld) {
  next_may_begin();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  if (r >= t || c * 8 >= o) return;
  float v[8];
  floats8<kIn>(load8<kIn>(dY + r * ldy, c * 8, o, wide), v);
#pragma unroll
  for (int term = 0; term < kTerms; ++term) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t bits = __float_as_uint(v[e]);
      const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
      if (!finite && (bits & 0x7fffffu)) bits |= 0x400000u;  // a NaN stays one
      w[e] = bits >> 16;
      v[e] = finite ? v[e] - __uint_as_float(bits & 0xffff0000u) : 0.0f;
    }
    *reinterpret_cast<uint4*>(out + ((kTerms - 1 - term) * t + r) * ld + c * 8) =
        make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
}

// dW = the sum of `split` partial matrices [o][k], in their order.
template <int kOut>
__global__ void __launch_bounds__(256)
    k_join(const float* part, int split, int64_t o, int64_t k, typename Elem<kOut>::T* dW, int64_t ldw) {
  after_previous();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= k) return;
  for (int64_t r = blockIdx.y; r < o; r += gridDim.y) {
    float sum = 0.0f;
    const float* from = part + r * k + c;
#pragma unroll 16
    for (int i = 0; i < split; ++i) sum += from[i * (o * k)];
    dW[r * ldw + c] = Elem<kOut>::put(sum);
  }
}

// The grid of kernels with 256 columns per CTA that walk the rows.
dim3 column_grid(int64_t o, int64_t k) {
  return dim3(static_cast<unsigned>((k + 255) / 256), static_cast<unsigned>(std::min<int64_t>(o, 65535)));
}

template <int kOut>
__global__ void __launch_bounds__(256)
    k_zero(int64_t o, int64_t k, typename Elem<kOut>::T* __restrict__ dW, int64_t ldw) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t r = blockIdx.y; r < o && c < k; r += gridDim.y) dW[r * ldw + c] = Elem<kOut>::put(0.0f);
}

// How a gradient is cut: the token axis into as many parts as leave pairs idle otherwise, of
// at least 4 pieces (512 x 512, us in one part and split: 65536 tokens 350 and 41, 4096
// tokens 32 and 17.2, where parts of at least 8 pieces took 18.6; 1024 tokens 15.5 and 15.0);
// bf16 terms and whether dY is copied into them; the workspace.
struct GradientPlan {
  int terms, split, per;
  bool copy;
  int64_t ld;  // pitch of the copied terms
  size_t terms_bytes, bytes;
};
GradientPlan gradient_plan(const void* dY, int64_t t, int64_t o, int64_t k, int type, int64_t ldy) {
  GradientPlan p = {};
  p.terms = type == kF32 ? 3 : (type == kF16 ? 2 : 1);
  // TMA reads bf16 rows in place when they start on 16-byte boundaries
  p.copy = type != kBF16 || (t > 1 && ldy % 8 != 0) || (reinterpret_cast<uintptr_t>(dY) & 15) != 0;
  p.ld = (o + 7) / 8 * 8;
  const int64_t pieces = (t + kTok - 1) / kTok, tiles = ((o + 255) / 256) * ((k + 255) / 256);
  const int64_t pairs = sm_count() / 2;
  int64_t split = tiles < pairs ? pairs / tiles : 1;
  split = std::max<int64_t>(1, std::min(split, pieces / 4));
  p.per = static_cast<int>((pieces + split - 1) / split);
  p.split = static_cast<int>((pieces + p.per - 1) / p.per);
  p.terms_bytes = p.copy ? (static_cast<size_t>(p.terms) * t * p.ld * 2 + 255) / 256 * 256 : 0;
  p.bytes = p.terms_bytes + (p.split > 1 ? static_cast<size_t>(p.split) * o * k * 4 : 0);
  return p;
}

template <int kIn, int kTerms>
void split_terms(const void* dY, int64_t ldy, int64_t t, int64_t o, __nv_bfloat16* out, int64_t ld, cudaStream_t st) {
  dim3 grid, block;
  piece_grid(t, (o + 7) / 8, &grid, &block);
  k_terms<kIn, kTerms><<<grid, block, 0, st>>>(static_cast<const typename Elem<kIn>::T*>(dY), ldy,
                                               rows_aligned16(dY, ldy, type_bytes(kIn)), t, o, out, ld);
  note_launch();
}

template <int kOut>
cudaError_t wgrad(const CUtensorMap& map_q, const CUtensorMap& map_s, const CUtensorMap& map_y, const Gradient& g,
                  cudaStream_t st) {
  // setmaxnreg waits for ever if the compiler gave the launch fewer registers than its split hands out
  static const bool enough = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, k_wgrad<kOut>) == cudaSuccess && a.numRegs == kLaunchRegisters;
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(k_wgrad<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
  if (e != cudaSuccess) return e;
  const int64_t all = static_cast<int64_t>(g.feature_tiles) * g.output_tiles * g.split;
  const int pairs = static_cast<int>(std::min<int64_t>(sm_count() / 2, all));
  note_launch();
  return launch_kernel(k_wgrad<kOut>, dim3(2 * pairs), kGradThreads, kGradSmem, st, 1, g.early,
                       map_q, map_s, map_y, g);
}

template <int kOut>
cudaError_t wgrad_all(const CUtensorMap& map_q, const CUtensorMap& map_s, const CUtensorMap& map_y, Gradient g,
                      float* part, void* dW, int64_t ldw, cudaStream_t st) {
  // Pieces of four steps for each term of dY. bfloat16 results of 16384 x 4096 x 4096 take
  // 449 / 431 / 420 / 416 us with 4 / 8 / 16 / 32 pieces (398 with one accumulator for all).
  g.chunk = kOut == kBF16 ? 16 / g.terms : (g.terms == 1 ? 4 : 2);
  if (g.split == 1) {
    g.out = dW;
    g.ld = ldw;
    return wgrad<kOut>(map_q, map_s, map_y, g, st);
  }
  g.out = part;
  g.ld = g.k;
  const cudaError_t e = wgrad<kF32>(map_q, map_s, map_y, g, st);
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_kernel(k_join<kOut>, column_grid(g.o, g.k), 256, 0, st, 1, true, part, g.split, g.o, g.k, static_cast<typename Elem<kOut>::T*>(dW), ldw);
}

}  // namespace

cudaError_t launch_checkpoint8(const void* X, int type, int64_t t, int64_t k, int64_t ldx, uint64_t seed,
                               const uint64_t* seed_add, int8_t* q, int64_t ldq, uint8_t* scale, int64_t lds,
                               cudaStream_t st) {
  dim3 grid, block;
  piece_grid(t, (k + 31) / 32 * 4, &grid, &block);
  const bool wide = rows_aligned16(X, ldx, type_bytes(type));
  const Philox4x32::RoundKeys keys = Philox4x32::round_keys(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
  const auto run = [&](auto kernel, const auto* x) {
    kernel<<<grid, block, 0, st>>>(x, t, k, ldx, wide, keys, seed, seed_add, q, ldq, scale, lds);
  };
  if (type == kF32) {
    const auto* x = static_cast<const float*>(X);
    seed_add ? run(k_checkpoint8<kF32, true>, x) : run(k_checkpoint8<kF32, false>, x);
  } else if (type == kBF16) {
    const auto* x = static_cast<const __nv_bfloat16*>(X);
    seed_add ? run(k_checkpoint8<kBF16, true>, x) : run(k_checkpoint8<kBF16, false>, x);
  } else {
    const auto* x = static_cast<const __half*>(X);
    seed_add ? run(k_checkpoint8<kF16, true>, x) : run(k_checkpoint8<kF16, false>, x);
  }
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

size_t checkpoint8_wgrad_workspace(const void* dY, int dy_type, int64_t ldy, int64_t t, int64_t o, int64_t k) {
  return t == 0 ? 0 : gradient_plan(dY, t, o, k, dy_type, ldy).bytes;
}

cudaError_t launch_checkpoint8_wgrad(const void* dY, int dy_type, int64_t ldy, const int8_t* q, int64_t ldq,
                                     const uint8_t* scale, int64_t lds, int64_t t, int64_t o, int64_t k, void* dW,
                                     int dw_type, int64_t ldw, void* ws, cudaStream_t st) {
  if (t == 0) {
    const dim3 grid = column_grid(o, k);
    if (dw_type == kF32)
      k_zero<kF32><<<grid, 256, 0, st>>>(o, k, static_cast<float*>(dW), ldw);
    else if (dw_type == kBF16)
      k_zero<kBF16><<<grid, 256, 0, st>>>(o, k, static_cast<__nv_bfloat16*>(dW), ldw);
    else
      k_zero<kF16><<<grid, 256, 0, st>>>(o, k, static_cast<__half*>(dW), ldw);
    note_launch();
    return cudaGetLastError();
  }
  const GradientPlan p = gradient_plan(dY, t, o, k, dy_type, ldy);
  auto* terms = static_cast<__nv_bfloat16*>(ws);
  if (p.copy) {
    if (dy_type == kF32)
      split_terms<kF32, 3>(dY, ldy, t, o, terms, p.ld, st);
    else if (dy_type == kF16)
      split_terms<kF16, 2>(dY, ldy, t, o, terms, p.ld, st);
    else
      split_terms<kBF16, 1>(dY, ldy, t, o, terms, p.ld, st);
    dY = terms;
    ldy = p.ld;
  }
  if (t == 1) ldy = (o + 7) / 8 * 8;  // one row: its pitch is never used
  CUtensorMap map_q, map_s, map_y;
  const uint64_t rows = static_cast<uint64_t>(t);
  const uint64_t sizes_q[2] = {static_cast<uint64_t>(k), rows}, strides_q[1] = {static_cast<uint64_t>(ldq)};
  const uint64_t sizes_s[2] = {static_cast<uint64_t>((k + 31) / 32), rows}, strides_s[1] = {static_cast<uint64_t>(lds)};
  const uint64_t sizes_y[3] = {static_cast<uint64_t>(o), rows, static_cast<uint64_t>(p.terms)};
  const uint64_t strides_y[2] = {static_cast<uint64_t>(ldy) * 2, static_cast<uint64_t>(ldy) * 2 * rows};
  const uint32_t box_q[2] = {128, kTok}, box_s[2] = {16, kTok}, box_y[3] = {64, kTok, 1};
  if (!make_map(&map_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, sizes_q, strides_q, box_q, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&map_s, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, scale, sizes_s, strides_s, box_s, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&map_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dY, sizes_y, strides_y, box_y, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Gradient g = {};
  g.o = o;
  g.k = k;
  g.feature_tiles = static_cast<int>((k + 255) / 256);
  g.output_tiles = static_cast<int>((o + 255) / 256);
  g.pieces = static_cast<int>((t + kTok - 1) / kTok);
  g.terms = p.terms;
  g.split = p.split;
  g.per = p.per;
  g.early = p.copy;
  if (static_cast<int64_t>(g.feature_tiles) * g.output_tiles > INT32_MAX / 256) return cudaErrorInvalidValue;
  auto* part = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + p.terms_bytes);
  switch (dw_type) {
    case kF32: return wgrad_all<kF32>(map_q, map_s, map_y, g, part, dW, ldw, st);
    case kBF16: return wgrad_all<kBF16>(map_q, map_s, map_y, g, part, dW, ldw, st);
    default: return wgrad_all<kF16>(map_q, map_s, map_y, g, part, dW, ldw, st);
  }
}

cudaError_t checkpoint8_stalled(bool* stalled) {
  int v = 0;
  cudaError_t e = cudaDeviceSynchronize();  // the copy alone does not wait for non-blocking streams
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_stalled_checkpoint8, sizeof(v));
  *stalled = v != 0;
  if (e == cudaSuccess && v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_stalled_checkpoint8, &v, sizeof(v));
  }
  return e;
}

}  // namespace ecasq
