// fsdp_waits.h -- a wave's waits for its own accesses, by count, and its workgroup's
// barrier without the wait for all of them that __syncthreads has.  A file of their own,
// so that a build for the CPU can stand in for them.  Not installed.
#pragma once

namespace fsdp {

// Until at most N of the wave's accesses to memory (loads, loads into LDS and stores alike,
// which end in the order in which they were issued) are on their way.
template <int N>
__device__ __forceinline__ void wait_memory() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Until at most MANY are where n >= MANY_FROM, at most SOME where n >= SOME_FROM, else at
// most FEW: one instruction to the compiler, which else would end a block here.
template <int MANY_FROM, int SOME_FROM, int FEW, int SOME, int MANY>
__device__ __forceinline__ void wait_memory_by(int n) {
    asm volatile("s_cmp_ge_i32 %0, %1\n\ts_cbranch_scc1 2f\n\ts_cmp_ge_i32 %0, %2\n\ts_cbranch_scc1 1f\n\t"
                 "s_waitcnt vmcnt(%3)\n1:\n\ts_waitcnt vmcnt(%4)\n2:\n\ts_waitcnt vmcnt(%5)"
                 ::"s"(__builtin_amdgcn_readfirstlane(n)), "n"(MANY_FROM), "n"(SOME_FROM), "n"(FEW), "n"(SOME), "n"(MANY)
                 : "memory", "scc");
}
// Every wave of the workgroup is here, and its accesses to LDS are over.
__device__ __forceinline__ void meet_in_lds() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// x as a value that the compiler cannot tell anything about.
__device__ __forceinline__ void unknown(int& x) { asm volatile("" : "+v"(x)); }
// x is needed here.
__device__ __forceinline__ void needed(uint32_t x) { asm volatile("" ::"v"(x)); }

}  // namespace fsdp
