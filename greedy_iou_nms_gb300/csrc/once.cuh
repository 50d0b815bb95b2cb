// Accesses of what a call touches once: where its operands are larger than L2
// they leave it first, so that they do not push out of it what is read again or
// still has to be written.
#pragma once

#include <cstdint>

#include "head.cuh"

namespace gbnms {

// Whether so many bytes are more than L2 keeps (three quarters of its 129 MB).
inline bool beyond_l2(int64_t bytes) { return bytes > (int64_t(96) << 20); }

// The L2 policy of such accesses, or one that leaves L2's order as it is: a register, so that neither
// way has a branch at each access (which took 173 us for a layer norm's 125).
__device__ __forceinline__ uint64_t once_policy(bool once)
{
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_unchanged.b64 %0, 1.0;" : "=l"(normal));
    return once ? first : normal;
}

template <typename P>
__device__ __forceinline__ P load_once(const P* p, uint64_t policy)
{
    if constexpr (sizeof(P) == 16) {
        uint4 v;
        asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p), "l"(policy)
                     : "memory");
        return *reinterpret_cast<const P*>(&v);
    } else {
        return *p;
    }
}

template <typename P>
__device__ __forceinline__ void store_once(P* p, const P& q, uint64_t policy)
{
    if constexpr (sizeof(P) == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(&q);
        asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                     "r"(v.w), "l"(policy)
                     : "memory");
    } else {
        *p = q;
    }
}

}  // namespace gbnms
