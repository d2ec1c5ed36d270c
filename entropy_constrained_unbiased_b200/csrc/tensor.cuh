// sm_100a tensor-core plumbing of the 8-bit operators: tensor maps and TMA tile
// loads, mbarriers across a pair of CTAs, tcgen05.mma with accumulators in TMEM.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace ecasq {

// Attempts of one bounded wait; each may suspend the thread for a while, so that
// giving up takes seconds, against microseconds of a wait that ends.
constexpr int kWaitLimit = 1 << 21;

// ---- host ------------------------------------------------------------------------

// Multiprocessors of the current device (asked once per device).
inline int sm_count() {
  static int counts[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (counts[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
    counts[dev] = n;
  }
  return counts[dev];
}

// Launches a kernel that may begin before the previous kernel of the stream, this
// library's own and launched just before, has ended (`early`): its set-up and its
// reads of what that kernel does not write overlap it; what it does write is read
// after after_previous(), by plain loads (the read-only path is for what nobody writes
// while the kernel lives). That kernel calls next_may_begin().
template <typename... Params, typename... Args>
cudaError_t launch_kernel(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                          unsigned cluster, bool early, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits for the previous kernel's end where this one was launched early; else nothing.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- host: tensor maps -----------------------------------------------------------

// A two- or three-dimensional map: sizes and box from the innermost dimension, the
// strides of the outer ones in bytes. Entries outside the sizes read as zero.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const uint64_t* sizes,
                     const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  const uint32_t ones[3] = {1, 1, 1};
  return encode && encode(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), sizes, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- device: clusters and barriers -----------------------------------------------

// One thread of a converged warp. Roles of one thread run as whole warps in which only
// the copies, MMAs and commits are the elected thread's: their operands then stay in
// uniform registers. (With the loop itself inside a branch of one lane, issuing the
// four MMAs of a stage took about 450 clocks, of the 512 that they run.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The address of `addr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int ld_shared_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mbar_arrive(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mbar) : "memory");
}
// On a barrier of either CTA of the cluster, with the instruction's default release, which
// orders for threads of this CTA. No thread of the other CTA reads what is handed over: it
// lies in this CTA's shared or tensor memory, and the thread that waits only issues MMAs,
// of which this CTA's own tensor core reads, or overwrites, this CTA's part. Write and read
// so meet inside one SM, where the proxy fence (shared memory) or tcgen05.wait::ld and the
// tcgen05 fence (tensor memory) before the arrival have finished the former. That is the
// hardware's working, not a promise of the PTX memory model, which knows no order between
// the CTAs without cluster scope; release and acquire at cluster scope cost a third of the
// gradient's speed (16384 x 4096 x 4096: 584 instead of 438 us, and 896 through a warp that
// relays them), and the tests compare every tile's results with 64 bits.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mbar) : "memory");
}

// Named barrier of `threads` threads: whether all of them brought true.
__device__ __forceinline__ bool barrier_and(int id, int threads, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbarrier.cta.red.and.aligned.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return all != 0;
}

// A place in a ring of kStages stages, walked in order: the stage, the parity of the
// current round, and whether it is the first one. (Divisions of a running count cost
// a single-threaded role hundreds of clocks per stage.)
template <int kStages>
struct Ring {
  uint32_t stage = 0, parity = 0;
  bool first = true;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1;
      first = false;
    }
  }
  // Waits until the stage's last use is over (nothing to wait for in the first round).
  __device__ __forceinline__ bool wait_empty(uint32_t bars, int limit) const {
    return first || mbar_wait_bounded(bars + 8 * stage, parity ^ 1, limit);
  }
  __device__ __forceinline__ bool wait_full(uint32_t bars, int limit) const {
    return mbar_wait_bounded(bars + 8 * stage, parity, limit);
  }
  // After a wait gave up: waits for the loads of every stage begun before this place.
  __device__ __forceinline__ void drain(uint32_t bars, int limit) const {
    if (!first)
      for (uint32_t i = stage; i < kStages; ++i) mbar_wait_bounded(bars + 8 * i, parity ^ 1, limit);
    for (uint32_t i = 0; i < stage; ++i) mbar_wait_bounded(bars + 8 * i, parity, limit);
  }
};

// ---- device: TMA tile loads ------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
// The same into this CTA's memory, counted on a barrier of either CTA of the pair
// (a shared::cluster address, see map_shared).
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}

// ---- device: tcgen05 -------------------------------------------------------------

template <int kGroup>
__device__ __forceinline__ void tmem_alloc(uint32_t out_shared, uint32_t columns) {
  if constexpr (kGroup == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(out_shared), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(out_shared), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int kGroup>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  if constexpr (kGroup == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tcgen05_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor with the 128-byte swizzle. Along the operand's
// contiguous axis a row of 128 bytes is one atom, eight rows 1024 bytes; `sbo`
// is the distance of the next eight rows, `lbo` that of the next 128-byte column
// (used only when the M or N axis is the contiguous one).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (static_cast<uint64_t>(addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptors: accumulator format, operand formats, major axes, sizes.
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n) {  // int32 += int8 x int8, both with K contiguous
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_bf16_mn(int m, int n) {  // float32 += bf16 x bf16, M and N contiguous
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

#define ECASQ_MMA(kind, group)                                                                                   \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::" group ".kind::" kind    \
               " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)) \
               : "memory")
template <int kGroup>
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (kGroup == 1)
    ECASQ_MMA("i8", "1");
  else
    ECASQ_MMA("i8", "2");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  ECASQ_MMA("f16", "2");
}
#undef ECASQ_MMA

// Arrives on the barrier (of both CTAs of a pair) when this thread's MMAs so far are done.
template <int kGroup>
__device__ __forceinline__ void mma_commit(uint32_t mbar) {
  if constexpr (kGroup == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            mbar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// 32 columns of this warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}

}  // namespace ecasq
