// Layer normalisation of rows and its gradient.
//
//   s = x + residual (rounded to the rows' type),  u = (s - mean) * rstd,
//   y = u * weight + bias; mean and the biased variance over the row.
//   du = dy * weight,  dx = rstd * (du - avg(du) - u * avg(du * u)) + dsum,
//   dweight = sum dy * u, dbias = sum dy over the rows.
//
// HBM bounds both: a row is read once and stays in the registers of a team of
// threads (a warp up to 1024 elements, 128 threads up to 4096, 512 up to 16384)
// from its moments to its results.  The gradient's teams go through many rows
// and keep the parameters' sums of their own columns in registers too; blocks
// leave theirs in the workspace and one short kernel joins them in order.
#pragma once

#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

// Two sums over a team of TEAM threads; with more than a warp, TEAM is the
// block and `shared` holds two values a warp (two sets, used in turn).
template <int TEAM>
__device__ __forceinline__ void team_sums(float& a, float& b, float (*shared)[2])
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(FULL, a, o);
        b += __shfl_xor_sync(FULL, b, o);
    }
    if constexpr (TEAM > 32) {
        constexpr int WARPS = TEAM / 32;
        if (threadIdx.x % 32 == 0) {
            shared[threadIdx.x / 32][0] = a;
            shared[threadIdx.x / 32][1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            a += shared[w][0];
            b += shared[w][1];
        }
    }
}

// V consecutive parameters from element e on (the caller keeps e below the width).
template <typename T, int V>
__device__ __forceinline__ void load_params(float (&v)[V], const void* p, int is_f32, int e, float absent)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = absent;
    } else if (is_f32 || sizeof(T) == 4) {
        constexpr int W = V > 4 ? 4 : V;
#pragma unroll
        for (int i = 0; i < V; i += W) {
            const Pack<float, W> q = *reinterpret_cast<const Pack<float, W>*>(static_cast<const float*>(p) + e + i);
#pragma unroll
            for (int j = 0; j < W; ++j) v[i + j] = q.v[j];
        }
    } else {
        const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p) + e);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = to_f32(q.v[i]);
    }
}

// V: elements an access, NV: accesses of a thread.
template <typename T, int V, int NV, int TEAM, int THREADS>
__global__ void __launch_bounds__(THREADS)
layer_kernel(const LayerArgs a)
{
    static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the block");
    __shared__ float shared[2][THREADS / 32][2];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / TEAM) + threadIdx.x / TEAM;
    const int t = threadIdx.x % TEAM;
    if (row >= a.rows) return;  // a whole team, and with TEAM == THREADS no block
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    Pack<T, V> q[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TEAM + t) * V;
        if (e < a.width) q[k] = *reinterpret_cast<const Pack<T, V>*>(x + e);
    }
    if (a.second) {
        const T* r = static_cast<const T*>(a.second) + row * a.second_row;
        T* sum = static_cast<T*>(a.sum) + row * a.width;
        Pack<T, V> p[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e < a.width) p[k] = *reinterpret_cast<const Pack<T, V>*>(r + e);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e >= a.width) break;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(q[k].v[i]) + to_f32(p[k].v[i]);
            q[k] = pack_results<T, V>(v);
            *reinterpret_cast<Pack<T, V>*>(sum + e) = q[k];
        }
    }
    const float share = 1.0f / static_cast<float>(a.width);
    float total = 0.0f, none = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if ((k * TEAM + t) * V < a.width) {
#pragma unroll
            for (int i = 0; i < V; ++i) total += to_f32(q[k].v[i]);
        }
    team_sums<TEAM>(total, none, shared[0]);
    const float mean = total * share;
    // Deviations from the rounded mean: their own mean is what its rounding left out.
    float off = 0.0f, squares = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if ((k * TEAM + t) * V < a.width) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(q[k].v[i]) - mean;
                off += d;
                squares = fmaf(d, d, squares);
            }
        }
    team_sums<TEAM>(off, squares, shared[1]);
    off *= share;
    squares *= share;
    // The deviations' own roundings leave up to some 2^-22 of their size in it: below that the first mean is nearer.
    if (off * off < 0x1p-42f * squares) off = 0.0f;
    const float variance = fmaf(-off, off, squares);  // a NaN stays one
    const float rstd = 1.0f / sqrtf((variance < 0.0f ? 0.0f : variance) + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean + off;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.out) + row * a.width;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TEAM + t) * V;
        if (e >= a.width) break;
        float w[V], b[V], v[V];
        load_params<T, V>(w, a.weight, a.param_f32, e, 1.0f);
        load_params<T, V>(b, a.bias, a.param_f32, e, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(((to_f32(q[k].v[i]) - mean) - off) * rstd, w[i], b[i]);
        *reinterpret_cast<Pack<T, V>*>(y + e) = pack_results<T, V>(v);
    }
}

// Each block's sums of dy * u and of dy go to parts[block][2][width].
template <typename T, int V, int NV, int TEAM, int THREADS>
__global__ void __launch_bounds__(THREADS, TEAM == 32 ? 3 : 1)
layer_grad_kernel(const LayerArgs a, float* parts)
{
    static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the block");
    __shared__ float shared[2][THREADS / 32][2];
    extern __shared__ float columns[];  // [2][width], with a team a warp
    constexpr int TEAMS = THREADS / TEAM;
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float share = 1.0f / static_cast<float>(a.width);
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_row;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_row;
        Pack<T, V> q[NV], g[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e < a.width) {
                q[k] = *reinterpret_cast<const Pack<T, V>*>(x + e);
                g[k] = *reinterpret_cast<const Pack<T, V>*>(dy + e);
            }
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        float first = 0.0f, along = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e >= a.width) break;
            float w[V];
            load_params<T, V>(w, a.weight, a.param_f32, e, 1.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u = (to_f32(q[k].v[i]) - mean) * rstd, d = to_f32(g[k].v[i]), du = d * w[i];
                dw[k][i] = fmaf(d, u, dw[k][i]);
                db[k][i] += d;
                first += du;
                along = fmaf(du, u, along);
            }
        }
        team_sums<TEAM>(first, along, shared[turn]);
        turn ^= 1;
        first *= share;
        along *= share;
        T* dx = static_cast<T*>(a.out) + row * a.width;
        const T* more = static_cast<const T*>(a.second) + (a.second ? row * a.second_row : 0);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e >= a.width) break;
            float w[V], v[V];
            load_params<T, V>(w, a.weight, a.param_f32, e, 1.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u = (to_f32(q[k].v[i]) - mean) * rstd, du = to_f32(g[k].v[i]) * w[i];
                v[i] = rstd * fmaf(-u, along, du - first);
            }
            if (a.second) {
                const Pack<T, V> p = *reinterpret_cast<const Pack<T, V>*>(more + e);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += to_f32(p.v[i]);
            }
            *reinterpret_cast<Pack<T, V>*>(dx + e) = pack_results<T, V>(v);
        }
    }
    if (!parts) return;
    float* part = parts + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
    if constexpr (TEAMS > 1) {
        // The block's teams one after another: a fixed order.
        for (int turn_of = 0; turn_of < TEAMS; ++turn_of) {
            if (team == turn_of) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int e = (k * TEAM + t) * V + i;
                        if (e >= a.width) break;
                        columns[e] = (turn_of ? columns[e] : 0.0f) + dw[k][i];
                        columns[a.width + e] = (turn_of ? columns[a.width + e] : 0.0f) + db[k][i];
                    }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < 2 * a.width; e += THREADS) part[e] = columns[e];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (k * TEAM + t) * V + i;
                if (e >= a.width) break;
                part[e] = dw[k][i];
                part[a.width + e] = db[k][i];
            }
    }
}

// Threads of a team and the values that one holds.
struct LayerShape {
    int team, values;
};
inline LayerShape layer_shape(int width)
{
    if (width <= 1024) return {32, width <= 256 ? 8 : width <= 512 ? 16 : 32};
    if (width <= 4096) return {128, width <= 2048 ? 16 : 32};
    return {512, width <= 8192 ? 16 : 32};
}
constexpr int LAYER_GRAD_THREADS = 128;  // of a block whose teams are warps

// Blocks of the gradient: all that the SMs hold, and more where a team's sums
// would run over more than 256 rows.
inline int64_t layer_grad_blocks(int64_t rows, int width)
{
    const LayerShape s = layer_shape(width);
    const int64_t teams = s.team == 32 ? LAYER_GRAD_THREADS / 32 : 1;
    const int64_t want = (rows + teams - 1) / teams, full = SMS * (s.team == 32 ? 3 : s.team == 128 ? 3 : 1);
    const int64_t least = (rows + 256 * teams - 1) / (256 * teams);
    return want < full ? want : least > full ? least : full;
}

template <typename T, int V, int TEAM, int VALUES>
void launch_layer_rows(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    if (grad) {
        constexpr int THREADS = TEAM == 32 ? LAYER_GRAD_THREADS : TEAM;
        const unsigned grid = static_cast<unsigned>(layer_grad_blocks(a.rows, a.width));
        const size_t smem = TEAM == 32 ? 2 * a.width * sizeof(float) : 0;
        layer_grad_kernel<T, V, VALUES / V, TEAM, THREADS><<<grid, THREADS, smem, st>>>(a, parts);
    } else {
        constexpr int THREADS = TEAM == 32 ? 256 : TEAM;
        const int64_t teams = THREADS / TEAM;
        const unsigned grid = static_cast<unsigned>((a.rows + teams - 1) / teams);
        layer_kernel<T, V, VALUES / V, TEAM, THREADS><<<grid, THREADS, 0, st>>>(a);
    }
}

template <typename T, int V>
void launch_layer_width(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    const LayerShape s = layer_shape(a.width);
    if (s.team == 32) {
        if (s.values == 8) launch_layer_rows<T, V, 32, 8>(a, parts, grad, st);
        else if (s.values == 16) launch_layer_rows<T, V, 32, 16>(a, parts, grad, st);
        else launch_layer_rows<T, V, 32, 32>(a, parts, grad, st);
    } else if (s.team == 128) {
        if (s.values == 16) launch_layer_rows<T, V, 128, 16>(a, parts, grad, st);
        else launch_layer_rows<T, V, 128, 32>(a, parts, grad, st);
    } else {
        if (s.values == 16) launch_layer_rows<T, V, 512, 16>(a, parts, grad, st);
        else launch_layer_rows<T, V, 512, 32>(a, parts, grad, st);
    }
}

// Accesses of 16 bytes where every row starts at a multiple of them, else of
// one element.
template <typename T>
void launch_layer_type(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    constexpr int MOST = 16 / sizeof(T);
    auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool wide = a.width % MOST == 0 && a.x_row % MOST == 0 && a.second_row % MOST == 0 && a.dy_row % MOST == 0 &&
                      aligned(a.x) && aligned(a.second) && aligned(a.dy) && aligned(a.out) && aligned(a.sum) &&
                      aligned(a.weight) && aligned(a.bias);
    if (wide) launch_layer_width<T, MOST>(a, parts, grad, st);
    else launch_layer_width<T, 1>(a, parts, grad, st);
}

void launch_layer_f32(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);
void launch_layer_f16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);
void launch_layer_bf16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);

}  // namespace gbnms
