// What the kernels on the tensor cores (tcgen05) share: barriers, copies by TMA,
// matrix instructions, tensor memory, and the order of tiles.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int TC_M = 128, TC_K = 64;        // of a tile, of a stage
constexpr int TC_WRITERS = 256;             // threads of the epilogue: warps 2 to 9
constexpr int TC_THREADS = TC_WRITERS + 64;
constexpr int A_BYTES = TC_M * TC_K * 2;
constexpr int HALF_BYTES = 64 * TC_K * 2;   // a box of an operand that lies across: 64 of m or n, 64 of k

// ------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void barrier_init(uint32_t bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t peer_address(uint32_t at, int rank)
{
    uint32_t peer;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(rank));
    return peer;
}

// Arrives at a barrier of another block of the cluster.
__device__ __forceinline__ void barrier_arrive_at(uint32_t peer)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer) : "memory");
}

// Sleeps until the phase of this parity is complete, so many ns at most; the
// warps that wait for a tile's sums would else take issue slots and power from
// those that feed the tensor cores.
__device__ __forceinline__ bool barrier_done(uint32_t bar, int parity, uint32_t most)
{
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(most)
        : "memory");
    return done;
}

// How long a wait lasts before it gives up, and how long it sleeps at a time, ns.
struct Patience {
    uint64_t all;
    uint32_t nap;
};

// Waits for the phase of this parity, `times` its patience; false when it gave up.
// (The last look is for a wait that was itself kept waiting, as by another process's
// turn.)
__device__ __forceinline__ bool barrier_wait(uint32_t bar, int parity, const Patience& p, int times = 1)
{
    if (barrier_done(bar, parity, p.nap)) return true;
    uint64_t start, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(start));
    do {
        if (barrier_done(bar, parity, p.nap)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    } while (now - start < times * p.all);
    return barrier_done(bar, parity, p.nap);
}

// PAIR: the barrier is the pair's first block's (an address without the rank's bit).
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
            "[%2];" ::"r"(dst),
            "l"(map), "r"(bar & 0xfeffffffu), "r"(x), "r"(y)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t form, bool add)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(form), "r"(static_cast<uint32_t>(add))
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(form), "r"(static_cast<uint32_t>(add))
            : "memory");
}

// The barrier (PAIR: each block's) completes when all matrix instructions
// issued so far have.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// After a wait that gave up, when the block's threads have met and start nothing
// more: says so, and what is in flight, copies and matrix instructions, ends long
// before this does.
static __device__ __noinline__ void settle(int32_t* status)
{
    uint64_t start, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(start));
    do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    while (now - start < 1000000);
    if (status) set_status(status, NMS_ERR_TIMEOUT);
}

// N columns of this thread's lane of tensor memory.
template <int N>
__device__ __forceinline__ void tensor_load(float (&v)[N], uint32_t at)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    if constexpr (N == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
              "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
              "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(at));
    } else {
        static_assert(N == 8, "8 or 32 columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(at));
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of an operand with 128-byte swizzle, at address 0:
// 16-byte units; version 1 in bits 46 on, swizzle code 2 in bits 61 on.  Along
// k: groups of eight rows 1024 bytes apart.  Across: groups of eight k 1024
// bytes apart, the next 64 of m or n a box further.
__device__ __forceinline__ uint64_t operand_form(int across)
{
    const uint64_t leading = across ? HALF_BYTES / 16 : 1, stride = 1024 / 16;
    return (leading << 16) | (stride << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: binary32 accumulators, both operands of T, rows x bn.
template <typename T>
__device__ __forceinline__ uint32_t instruction_form(int a_across, int b_across, int rows, int bn)
{
    const uint32_t kind = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return (1u << 4) | (kind << 7) | (kind << 10) | (static_cast<uint32_t>(a_across) << 15) |
           (static_cast<uint32_t>(b_across) << 16) | (static_cast<uint32_t>(bn / 8) << 17) |
           (static_cast<uint32_t>(rows / 16) << 24);
}

// -------------------------------------------------------------------- tiles

struct Place {
    int64_t m, n;
};

// Tile t of tiles_m x tiles_n: strips of 16 tiles along n, within a strip n
// first, so that the tiles that run together share rows of both operands in L2.
__device__ __forceinline__ Place tile_place(int64_t t, int64_t tiles_m, int64_t tiles_n, int rows, int bn)
{
    const int64_t strip = t / (16 * tiles_m), left = t - strip * 16 * tiles_m;
    const int64_t width = min(static_cast<int64_t>(16), tiles_n - strip * 16);
    const int64_t m = left / width;
    return {m * rows, (strip * 16 + left - m * width) * bn};
}

// --------------------------------------------------------------------- host

inline Patience patience()
{
    const uint64_t all = product_patience();
    return {all, static_cast<uint32_t>(all < 1000000 ? all : 1000000)};
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encoder()
{
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

}  // namespace gbnms
