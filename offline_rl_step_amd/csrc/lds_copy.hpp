// Asynchronous copies from global memory to LDS and the waits they need.
#pragma once
#include "common.hpp"

namespace iqlh {

// source of copies that lie outside of a matrix
__device__ __align__(16) const uint4 kZeroChunk[1] = {};

template <int N>
IQLH_DEV void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Asynchronous copy of 16 (4) bytes per lane, global -> LDS, to lds_at + 16 (4)
// lane.  As an instruction of its own and not the compiler's builtin: behind
// the builtin the compiler waits for every copy in flight before each LDS
// read that may alias one, which is all of them, and the ring runs empty.  It
// has no output registers; wait_vm orders it against the reads.  (One wait
// state between writing M0 and its use by the copy.)
IQLH_DEV void copy16(const void* src, uint32_t lds_at) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds_at), "v"(src) : "memory");
}
IQLH_DEV void copy4(const void* src, uint32_t lds_at) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(lds_at), "v"(src) : "memory");
}
// Workgroup barrier after this wave's LDS reads, leaving the asynchronous
// copies it has in flight
IQLH_DEV void bar() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace iqlh
