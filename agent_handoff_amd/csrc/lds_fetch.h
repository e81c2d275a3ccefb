// lds_fetch.h - loads from memory to LDS (device side). Written out: behind the builtin the compiler waits for all of
// them before the next read of LDS, of whichever buffer. Here it knows of none, and the kernels wait themselves, with
// wait_loads() (loads that the compiler knows of only make its own waits, and these, longer than they need be). No
// register is written but M0, which nothing else in these kernels uses (the compiler keeps it for itself and takes no note
// of it); what reads it comes a wait state behind its write. The compiler does not look into the text for hazards: a scalar
// address that a vector instruction wrote (v_readfirstlane) may be read five wait states later at the earliest, and the
// instruction before the text may be that write, so the text begins with them.
#pragma once

#include "kernels_common.h"

#define KVC_LDS __attribute__((address_space(3)))

namespace kvc {
namespace {

__device__ __forceinline__ uint32_t lds_place(uint8_t* lds) { return wave_uniform((uint32_t)(uint64_t)(KVC_LDS uint8_t*)lds); }

// N times 16 bytes of each lane: from base (the same in all lanes) + off[u] + 1024 u to lds + 1024 u + 16 * lane.
template <int N>
__device__ __forceinline__ void fetch16(const uint8_t* base, const uint32_t (&off)[N], uint8_t* lds) {
    const uint64_t from = (uint64_t)base;
    const uint64_t at = (uint64_t)wave_uniform((uint32_t)(from >> 32)) << 32 | wave_uniform((uint32_t)from);
    const uint32_t to = lds_place(lds);
    static_assert(N == 1 || N == 2 || N == 4);
    if constexpr (N == 4)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\t"
                     "global_load_lds_dwordx4 %2, %1\n\t"
                     "global_load_lds_dwordx4 %3, %1 offset:0x400\n\t"
                     "global_load_lds_dwordx4 %4, %1 offset:0x800\n\t"
                     "global_load_lds_dwordx4 %5, %1 offset:0xc00"
                     :
                     : "s"(to), "s"(at), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3])
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\t"
                     "global_load_lds_dwordx4 %2, %1\n\t"
                     "global_load_lds_dwordx4 %3, %1 offset:0x400"
                     :
                     : "s"(to), "s"(at), "v"(off[0]), "v"(off[1])
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\t"
                     "global_load_lds_dwordx4 %2, %1"
                     :
                     : "s"(to), "s"(at), "v"(off[0])
                     : "memory");
}

// 4 bytes of each lane, from an address of its own, to lds + 4 * lane.
__device__ __forceinline__ void fetch_lane4(const uint8_t* from, uint8_t* lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t"
                 "global_load_lds_dword %1, off"
                 :
                 : "s"(lds_place(lds)), "v"((uint64_t)from)
                 : "memory");
}

// Waits until no more than the loads of the last `behind` groups of EACH, MOST of them at most, are on their way.
template <int EACH, int MOST>
__device__ __forceinline__ void wait_loads(uint32_t behind) {
    if constexpr (MOST > 0) {
        if (behind >= (uint32_t)MOST) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(EACH * MOST) : "memory");
            return;
        }
        wait_loads<EACH, MOST - 1>(behind);
    } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
}

}  // namespace
}  // namespace kvc
