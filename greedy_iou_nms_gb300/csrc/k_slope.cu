// dz = dy * act'(pre) and the sums of its columns: what a linear layer's
// gradient has to do before its two products.
//
// HBM bounds it (dy and pre read once, dz written once, where the products go by
// planes as those: a pass of its own over dz for them was 8 bytes an element
// more; of 16 bits, what rounding dz leaves out goes to a second array).  A
// block has a strip of columns and a run of rows; each of its SL_SLOTS warps
// goes through every SL_SLOTS-th row, a lane V columns of it, and keeps their
// sums in registers.  The warps' sums are added in order, the runs' by one short
// kernel.
#include "block.h"
#include "head.cuh"
#include "internal.h"
#include "once.cuh"
#include "planes.cuh"

namespace gbnms {

namespace {

constexpr int SL_SLOTS = 8;

// joined: the runs of a strip are a cluster, whose first block adds up their sums.
template <typename T, int V>
__global__ void __launch_bounds__(32 * SL_SLOTS, 5)
slope_kernel(const SlopeArgs s, int64_t run, float* parts, bool joined)
{
    __shared__ float sums[SL_SLOTS][32 * V];
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x) * V;
    const int64_t first = blockIdx.y * run, last = min(s.rows, first + run);
    float sum[V] = {};
    const uint64_t once = once_policy(s.dz || s.planes);  // the products read dz in place of dy: L2 is for that
    if (e < s.width) {
        const T* dy = static_cast<const T*>(s.dy) + e;
        const T* pre = static_cast<const T*>(s.pre) + e;
        T* dz = static_cast<T*>(s.dz) + e;
        for (int64_t row = first + threadIdx.y; row < last; row += SL_SLOTS) {
            const Pack<T, V> g = load_once(reinterpret_cast<const Pack<T, V>*>(dy + row * s.dy_row), once);
            Pack<T, V> z{};
            if (s.pre) z = load_once(reinterpret_cast<const Pack<T, V>*>(pre + row * s.width), once);
            float d[V], v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                d[i] = to_f32(g.v[i]);
                v[i] = to_f32(z.v[i]);
            }
            if (s.pre) act_slopes<T, V>(d, v, s.act);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += d[i];
            // The type that the products take; without `low` dz is rounded to it, half a step of a factor.
            if constexpr (sizeof(T) == 2) {
                if (s.low) {
                    Pack<T, V> h, l;
                    split_two(d, h, l);
                    *reinterpret_cast<Pack<T, V>*>(dz + row * s.dz_row) = h;
                    *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(s.low) + row * s.dz_row + e) = l;
                } else if (s.dz) {
                    *reinterpret_cast<Pack<T, V>*>(dz + row * s.dz_row) = pack_results<T, V>(d);
                }
            } else {
                if (s.dz) *reinterpret_cast<Pack<T, V>*>(dz + row * s.dz_row) = pack_results<T, V>(d);
                if (s.planes) {
                    Pack<__nv_bfloat16, V> h, m, l;
                    split_parts(d, h, m, l);
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(s.planes) + row * s.dz_row + e;
                    *reinterpret_cast<Pack<__nv_bfloat16, V>*>(to) = h;
                    *reinterpret_cast<Pack<__nv_bfloat16, V>*>(to + s.rows * s.dz_row) = m;
                    *reinterpret_cast<Pack<__nv_bfloat16, V>*>(to + 2 * s.rows * s.dz_row) = l;
                }
            }
        }
    }
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < V; ++i) sums[threadIdx.y][i * 32 + threadIdx.x] = sum[i];
    __syncthreads();
    if (threadIdx.y == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            for (int k = 1; k < SL_SLOTS; ++k) sum[i] += sums[k][i * 32 + threadIdx.x];
            if (gridDim.y == 1 || !joined) {
                if (e < s.width) parts[blockIdx.y * s.width + e + i] = sum[i];
            } else {
                sums[0][i * 32 + threadIdx.x] = sum[i];
            }
        }
    }
    if (gridDim.y == 1 || !joined) return;
    cluster_barrier();
    if (blockIdx.y == 0 && threadIdx.y == 0 && e < s.width) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t own = static_cast<uint32_t>(__cvta_generic_to_shared(&sums[0][i * 32 + threadIdx.x]));
            for (unsigned k = 1; k < gridDim.y; ++k) {
                uint32_t peer;
                float v;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(own), "r"(k));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer));
                sum[i] += v;
            }
            s.dbias[e + i] = sum[i];
        }
    }
    __syncwarp();
    cluster_barrier();  // no block leaves while the first reads its sums
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
    const bool joined = parts && runs > 1 && runs <= 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((s.width + 32 * v - 1) / (32 * v)), static_cast<unsigned>(runs));
    cfg.blockDim = dim3(32, SL_SLOTS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.z = 1;
    attr[0].val.clusterDim.y = joined ? static_cast<unsigned>(runs) : 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) { cudaLaunchKernelEx(&cfg, kernel, s, run, parts, joined); };
    if (v == MOST) go(slope_kernel<T, MOST>);
    else if (v == 2) go(slope_kernel<T, 2>);
    else go(slope_kernel<T, 1>);
    if (runs > 1 && parts && !joined) launch_column_join(parts, runs, s.width, s.width, s.dbias, nullptr, st);
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
