// LDS DMA of the cache and product kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qwg {

// Asynchronous 16-byte global -> LDS copy of every active lane, lane l to LDS byte
// lds + 16 l (lds wavefront-uniform). The compiler does not count these copies:
// wait_vmcnt does, and its LDS reads of them must follow it. The leading s_nop
// covers the hazard from the write of M0.
__device__ __forceinline__ void dma16(const void *g, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds), "v"(g) : "memory");
}

// Wait until at most N vector-memory operations of this wavefront are
// outstanding (they complete in issue order).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace qwg
