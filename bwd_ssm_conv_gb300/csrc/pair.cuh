// pair.cuh -- tcgen05 products of one CTA or of a pair of CTAs (CG = 1, 2): the bf16 MMA with both
// operands in shared memory and fp32 accumulators in tensor memory, its completion, the tensor memory of
// both CTAs, barriers of the first CTA that the second arrives on, and the kernel's place in a call.
#pragma once

#include "tma.cuh"
#include "tmem.cuh"

namespace ssm {

// Instruction descriptor: D fp32, A and B bf16, M x N; *_mn: that operand's tile lies MN-major.
__host__ __device__ __forceinline__ constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N, bool a_mn,
                                                                  bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <int CG> struct Mma {
  static __device__ __forceinline__ void mma(uint32_t idesc, uint32_t d, uint64_t a, uint64_t b,
                                             bool accumulate) {
    if constexpr (CG == 1)
      asm volatile(
          "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
          "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
          "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
          : "memory");
    else
      asm volatile(
          "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
          "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
          "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
          : "memory");
  }
  // Arrives on `bar` (of both CTAs) once the MMAs issued before have completed.
  static __device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (CG == 1)
      tc::mma_commit(bar);
    else
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
          "[%0], %1;" ::"r"(smem_u32(bar)),
          "h"((uint16_t)3)
          : "memory");
  }
  static __device__ __forceinline__ void commit_here(uint64_t* bar) {  // of this CTA only
    if constexpr (CG == 1)
      tc::mma_commit(bar);
    else
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              smem_u32(bar))
          : "memory");
  }
  static __device__ __forceinline__ void alloc(uint32_t* dst, uint32_t cols) {
    if constexpr (CG == 1) {
      tmem_alloc(dst, cols);
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(dst)),
                   "r"(cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  static __device__ __forceinline__ void dealloc(uint32_t t, uint32_t cols) {
    if constexpr (CG == 1)
      tmem_dealloc(t, cols);
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols)
                   : "memory");
  }
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(smem_u32(bar))
               : "memory");
}
// The first CTA's barrier at the same place, and an arrival there.
template <int CG> __device__ __forceinline__ uint32_t bar_of_first(uint64_t* bar) {
  uint32_t a = smem_u32(bar);
  if constexpr (CG > 1) asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(a));
  return a;
}
template <int CG> __device__ __forceinline__ void mbar_arrive_first(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One lane of a converged warp, in a form that the compiler knows to be a single one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
// Where an agent stands in the ring of stages: the slot, and the parity of its current use.
template <int S> struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == S) s = 0, phase ^= 1;
  }
};
// This kernel may start while the one before it in the call runs (wgrad8.cu): here its results are
// complete, also for TMA.
__device__ __forceinline__ void wait_for_copies() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
template <int CG> __device__ __forceinline__ void sync_tile() {  // every thread of the tile's CTAs
  if constexpr (CG == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
}

}  // namespace ssm
