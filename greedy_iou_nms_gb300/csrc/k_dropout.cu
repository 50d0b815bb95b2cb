// Dropout from a counter-based generator: y = x * mask / keep (+ residual),
// the mask a function of (seed, offset, element index) and never stored; the
// gradient is the same map of the incoming gradient.
//
// HBM bounds it where the generator's some fifty integer instructions for
// eight elements hide behind the loads; so a thread loads several blocks of
// eight before it draws for the first, and three blocks share an SM (24 warps;
// two took 110 us).  128 M bf16: 92 us, 5.6 TB/s of the 6.7 that a copy reaches; fp16 83,
// 64 M fp32 94.
#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int DR_THREADS = 256;

// One block of eight elements: V of them an access (all, or 1 where a
// pointer is not aligned).
template <typename T, int V>
struct Eight {
    Pack<T, V> q[8 / V];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int k = 0; k < 8 / V; ++k) q[k] = *reinterpret_cast<const Pack<T, V>*>(p + k * V);
    }
    __device__ __forceinline__ float operator[](int i) const { return to_f32(q[i / V].v[i % V]); }
};

// RES: with a residual.  DROP: some element may be dropped.
template <typename T, int V, bool RES, bool DROP>
__global__ void __launch_bounds__(DR_THREADS, 3)
dropout_kernel(const T* x, const T* residual, T* y, int64_t n, DropArgs d)
{
    constexpr int DR_BATCH = RES ? 2 : 4;  // blocks of eight elements a thread has in flight
    const int64_t whole = n / 8, step = static_cast<int64_t>(gridDim.x) * DR_THREADS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * DR_THREADS + threadIdx.x;
    for (int64_t b = first; b < whole; b += DR_BATCH * step) {
        Eight<T, V> q[DR_BATCH], r[RES ? DR_BATCH : 1];
#pragma unroll
        for (int k = 0; k < DR_BATCH; ++k)
            if (b + k * step < whole) {
                q[k].load(x + 8 * (b + k * step));
                if (RES) r[k].load(residual + 8 * (b + k * step));
            }
#pragma unroll
        for (int k = 0; k < DR_BATCH; ++k) {
            const int64_t at = 8 * (b + k * step);
            if (at >= 8 * whole) break;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = q[k][i];
            if (DROP) drop<8>(v, static_cast<uint64_t>(at), d);
            if (RES) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += r[k][i];
            }
#pragma unroll
            for (int i = 0; i < 8; i += V) {
                float part[V];
#pragma unroll
                for (int j = 0; j < V; ++j) part[j] = v[i + j];
                *reinterpret_cast<Pack<T, V>*>(y + at + i) = pack_results<T, V>(part);
            }
        }
    }
    // The last n mod 8 elements.
    if (first == 0 && n % 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 8 * whole + i < n ? to_f32(x[8 * whole + i]) : 0.0f;
        if (DROP) drop<8>(v, static_cast<uint64_t>(8 * whole), d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (8 * whole + i < n)
                y[8 * whole + i] = from_f32<T>(RES ? v[i] + to_f32(residual[8 * whole + i]) : v[i]);
    }
}

template <typename T>
static void launch(const void* x, const void* residual, void* y, int64_t n, const DropArgs& d, cudaStream_t st)
{
    constexpr int MOST = 16 / sizeof(T);
    auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool wide = aligned(x) && aligned(residual) && aligned(y), res = residual != nullptr, drop = d.limit < 65536u;
    // Short tensors: a block a thread.  Long ones: full SMs, each thread many.
    const int64_t want = (n / 8 + DR_THREADS - 1) / DR_THREADS, most = SMS * 3;
    const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most);
    auto run = [&](auto kernel) {
        kernel<<<grid, DR_THREADS, 0, st>>>(static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<T*>(y),
                                            n, d);
    };
    if (wide) {
        if (res) drop ? run(dropout_kernel<T, MOST, true, true>) : run(dropout_kernel<T, MOST, true, false>);
        else drop ? run(dropout_kernel<T, MOST, false, true>) : run(dropout_kernel<T, MOST, false, false>);
    } else {
        if (res) drop ? run(dropout_kernel<T, 1, true, true>) : run(dropout_kernel<T, 1, true, false>);
        else drop ? run(dropout_kernel<T, 1, false, true>) : run(dropout_kernel<T, 1, false, false>);
    }
}

void launch_dropout(const void* x, const void* residual, void* y, int type, int64_t n, const DropArgs& d,
                    cudaStream_t st)
{
    if (type == NMS_TYPE_F32) launch<float>(x, residual, y, n, d, st);
    else if (type == NMS_TYPE_F16) launch<__half>(x, residual, y, n, d, st);
    else launch<__nv_bfloat16>(x, residual, y, n, d, st);
}

}  // namespace gbnms
