// dz = dy * act'(pre) and the sums of its columns: what a linear layer's
// gradient has to do before its two products.
//
// HBM bounds it (dy and pre read once, dz written once).  A block has a strip
// of columns and a run of rows; each of its SL_SLOTS warps goes through every
// SL_SLOTS-th row, a lane V columns of it, and keeps their sums in registers.
// The warps' sums are added in order, the runs' by one short kernel.
#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

namespace {

constexpr int SL_SLOTS = 8;

template <typename T, int V>
__global__ void __launch_bounds__(32 * SL_SLOTS, 5)
slope_kernel(const SlopeArgs s, int64_t run, float* parts)
{
    __shared__ float sums[SL_SLOTS][32 * V];
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x) * V;
    const int64_t first = blockIdx.y * run, last = min(s.rows, first + run);
    float sum[V] = {};
    if (e < s.width) {
        const T* dy = static_cast<const T*>(s.dy) + e;
        const T* pre = static_cast<const T*>(s.pre) + e;
        T* dz = static_cast<T*>(s.dz) + e;
        for (int64_t row = first + threadIdx.y; row < last; row += SL_SLOTS) {
            const Pack<T, V> g = *reinterpret_cast<const Pack<T, V>*>(dy + row * s.dy_row);
            Pack<T, V> z{};
            if (s.pre) z = *reinterpret_cast<const Pack<T, V>*>(pre + row * s.width);
            float d[V], v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                d[i] = to_f32(g.v[i]);
                v[i] = to_f32(z.v[i]);
            }
            if (s.pre) act_slopes<T, V>(d, v, s.act);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += d[i];
            // Rounded here to the type that the products take: half a step of a factor, no more than the factors
            // themselves came with.
            if (s.dz) *reinterpret_cast<Pack<T, V>*>(dz + row * s.dz_row) = pack_results<T, V>(d);
        }
    }
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < V; ++i) sums[threadIdx.y][i * 32 + threadIdx.x] = sum[i];
    __syncthreads();
    if (threadIdx.y == 0 && e < s.width) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            for (int k = 1; k < SL_SLOTS; ++k) sum[i] += sums[k][i * 32 + threadIdx.x];
            parts[blockIdx.y * s.width + e + i] = sum[i];
        }
    }
}

// Runs of rows: as many blocks as fill the SMs, and a warp's sums over 256
// rows at most (while the grid's second axis has room).
int64_t slope_runs(int64_t rows, int64_t width)
{
    const int64_t strips = (width + 255) / 256, full = (SMS * 8 + strips - 1) / strips;
    const int64_t want = (rows + 8 * SL_SLOTS - 1) / (8 * SL_SLOTS), least = (rows + 256 * SL_SLOTS - 1) / (256 * SL_SLOTS);
    return want < full ? want : least > full ? (least < 65535 ? least : 65535) : full;
}

template <typename T>
void launch(const SlopeArgs& s, float* parts, cudaStream_t st)
{
    constexpr int MOST = 16 / sizeof(T);
    auto even = [&](int v) {
        auto starts = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (v * sizeof(T)) == 0; };
        return s.width % v == 0 && s.dy_row % v == 0 && s.dz_row % v == 0 && starts(s.dy) && starts(s.pre) && starts(s.dz);
    };
    const int v = even(MOST) ? MOST : even(2) ? 2 : 1;
    int64_t runs = slope_runs(s.rows, s.width);
    const int64_t run = (s.rows + runs - 1) / runs;
    runs = (s.rows + run - 1) / run;
    if (runs == 1 && parts) parts = s.dbias;
    const dim3 grid(static_cast<unsigned>((s.width + 32 * v - 1) / (32 * v)), static_cast<unsigned>(runs));
    if (v == MOST) slope_kernel<T, MOST><<<grid, dim3(32, SL_SLOTS), 0, st>>>(s, run, parts);
    else if (v == 2) slope_kernel<T, 2><<<grid, dim3(32, SL_SLOTS), 0, st>>>(s, run, parts);
    else slope_kernel<T, 1><<<grid, dim3(32, SL_SLOTS), 0, st>>>(s, run, parts);
    if (runs > 1 && parts) launch_column_join(parts, runs, s.width, s.width, s.dbias, nullptr, st);
}

}  // namespace

size_t slope_workspace_bytes(int64_t rows, int64_t width)
{
    return rows == 0 ? 0 : static_cast<size_t>(slope_runs(rows, width)) * width * sizeof(float);
}

void launch_slope(const SlopeArgs& s, void* workspace, cudaStream_t st)
{
    float* parts = s.dbias ? static_cast<float*>(workspace) : nullptr;
    if (s.type == NMS_TYPE_F32) launch<float>(s, parts, st);
    else if (s.type == NMS_TYPE_F16) launch<__half>(s, parts, st);
    else launch<__nv_bfloat16>(s, parts, st);
}

}  // namespace gbnms
