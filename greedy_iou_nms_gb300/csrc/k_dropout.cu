// Dropout from a counter-based generator: y = x * mask / keep (+ residual),
// the mask a function of (seed, offset, element index) and never stored; the
// gradient is the same map of the incoming gradient.
#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int DR_THREADS = 256;

// One thread per block of eight elements.
template <typename T>
__global__ void __launch_bounds__(DR_THREADS)
dropout_kernel(const T* __restrict__ x, const T* __restrict__ residual, T* __restrict__ y, int64_t n, DropArgs d,
               int wide)
{
    const int64_t blocks = (n + 7) / 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * DR_THREADS;
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * DR_THREADS + threadIdx.x; b < blocks; b += step) {
        const int64_t at = 8 * b;
        const int m = static_cast<int>(n - at < 8 ? n - at : 8);
        float v[8];
        for (int i = 0; i < 8; ++i) v[i] = i < m ? to_f32(x[at + i]) : 0.0f;
        drop<8>(v, static_cast<uint64_t>(at), d);
        for (int i = 0; i < m; ++i) y[at + i] = from_f32<T>(residual ? v[i] + to_f32(residual[at + i]) : v[i]);
    }
}

template <typename T>
static void launch(const void* x, const void* residual, void* y, int64_t n, const DropArgs& d, cudaStream_t st)
{
    const int64_t want = ((n + 7) / 8 + DR_THREADS - 1) / DR_THREADS;
    dropout_kernel<T><<<static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64), DR_THREADS, 0, st>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<T*>(y), n, d, 0);
}

void launch_dropout(const void* x, const void* residual, void* y, int type, int64_t n, const DropArgs& d,
                    cudaStream_t st)
{
    if (type == NMS_TYPE_F32) launch<float>(x, residual, y, n, d, st);
    else if (type == NMS_TYPE_F16) launch<__half>(x, residual, y, n, d, st);
    else launch<__nv_bfloat16>(x, residual, y, n, d, st);
}

}  // namespace gbnms
