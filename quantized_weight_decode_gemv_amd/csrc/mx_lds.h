// LDS DMA of the cache and product kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qwg {

// Asynchronous 16-byte global -> LDS copy of every active lane, lane l to LDS byte
// lds + 16 l (lds wavefront-uniform). The compiler does not count these copies:
// wait_vmcnt does, and its LDS reads of them must follow it. Neither does it look
// for hazards inside: the leading s_nop gives the five wait states that a vector
// memory instruction needs after a vector instruction (v_readfirstlane) wrote one
// of its scalar operands, M0 among them; with fewer the base address can be stale.
__device__ __forceinline__ void dma16(const void *g, uint32_t lds) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds), "v"(g) : "memory");
}

// The same for lines that no other workgroup reads: the non-temporal hint keeps
// them out of the way of what is read again.
__device__ __forceinline__ void dma16_once(const void *g, uint32_t lds) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, off nt" ::"{m0}"(lds), "v"(g) : "memory");
}

// The same as dma16 from a wavefront-uniform base and a byte offset per lane.
__device__ __forceinline__ void dma16(const void *base, uint32_t offset, uint32_t lds) {
    // (readfirstlane returns int: widen through uint32_t, never by sign extension)
    const uint64_t p = (uint64_t)(uintptr_t)base;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    const uint64_t u = (uint64_t)lo | (uint64_t)hi << 32;
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(offset),
                 "s"((const void *)(uintptr_t)u)
                 : "memory");
}

// Wait until at most N vector-memory operations of this wavefront are
// outstanding (they complete in issue order).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace qwg
