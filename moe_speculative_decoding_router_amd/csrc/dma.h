// Loads from global memory straight into LDS whose waits are written by hand.
//
// The compiler waits for every load into LDS that it knows of before it reads
// LDS at all, so a loop that fills one buffer while it reads another would stop
// for the loads it has just started.  Written as assembly, they are unknown to
// it; the kernel waits for them itself (dma_wait) before the barrier that hands a
// buffer over.  They have no register outputs, so nothing the compiler moves
// can be overwritten; its own waits for other loads become longer, never
// shorter, by those that are under way.
#pragma once

#include "common.h"

namespace moe {

// Byte address in LDS, the same in every lane.
__device__ __forceinline__ unsigned lds_address(const void *p) {
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}

// 16 bytes a lane from base + offset (a byte offset below 2^32 of each lane's
// own) to LDS address at + 16 lane.
__device__ __forceinline__ void dma16(const void *base, unsigned offset, unsigned at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(offset), "s"(base) : "memory");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void dma16v(const void *from, unsigned at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory");
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void dma_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// Barrier that orders LDS: this wave's reads are done, its loads go on.
__device__ __forceinline__ void dma_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

}  // namespace moe
