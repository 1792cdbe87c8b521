// Buffer loads that write LDS directly.
#pragma once

#include "kernels.hpp"

namespace skg {

// A buffer load of 16 bytes per lane into LDS, lane i at lds + 16 i. Written as one
// instruction block because the compiler makes every later LDS read wait for all loads
// into LDS it knows of; it has no output register, and stage_wait() waits for it. M0
// holds the LDS address; nothing else in these kernels uses M0 (the compiler reserves it
// and sets it right before its own uses).
template <bool NT = false>
__device__ __forceinline__ void load_to_lds(const u32x4 &rsrc, unsigned offset, unsigned lds)
{
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                     :
                     : "s"(lds), "v"(offset), "s"(rsrc)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(lds), "v"(offset), "s"(rsrc)
                     : "memory");
}

// The same with 4 bytes per lane, lane i at lds + 4 i.
__device__ __forceinline__ void load4_to_lds(const u32x4 &rsrc, unsigned offset, unsigned lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(rsrc)
                 : "memory");
}

// All but this wave's YOUNGER latest memory operations are done: loads retire in order, so
// a stage has landed once only those of the stages behind it are left.
template <int YOUNGER = 0>
__device__ __forceinline__ void stage_wait()
{
    static_assert(YOUNGER >= 0 && YOUNGER < 64, "the counter has six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(YOUNGER) : "memory");
}

// All but this wave's YOUNGER latest reads of LDS, which return in order, are there.
template <int YOUNGER = 0>
__device__ __forceinline__ void lds_read_wait()
{
    asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(YOUNGER) : "memory");
}

__device__ __forceinline__ u32x4 rsrc_words(const void *base, unsigned bytes)
{
    const unsigned long long p = (unsigned long long)base;
    u32x4 r;
    r[0] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)p);
    r[1] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(p >> 32)) & 0xFFFFu;
    r[2] = (unsigned)__builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = kBufferFlags;
    return r;
}

}  // namespace skg
