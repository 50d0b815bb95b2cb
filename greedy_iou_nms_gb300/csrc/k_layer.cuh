// Layer normalisation of rows and its gradient.
//
//   s = x + residual (rounded to the rows' type),  u = (s - mean) * rstd,
//   y = u * weight + bias; mean and the biased variance over the row.
//   du = dy * weight,  dx = rstd * (du - avg(du) - u * avg(du * u)) + dsum,
//   dweight = sum dy * u, dbias = sum dy over the rows.
//
// HBM bounds both: a row is read once and stays in the registers of a team of
// threads (8 up to 64 elements, 16 up to 128, a warp up to 1024, 128 threads up
// to 4096, 512 up to 8192, 1024 up to 16384) from its moments to its results.
// The gradient's teams go through many rows and keep the parameters' sums of
// their own columns in registers too; blocks leave theirs in the workspace and
// one short kernel joins them in order.  102400 x 1024 bf16: 124 us with residual
// and statistics (141 without the streaming accesses of once.cuh), 131 the
// gradient: 6.8 and 6.4 of 6.8 TB/s.  A warp a row for 50 elements took 39 us for
// the gradient of 100000, four rows a warp 20.
#pragma once

#include "block.h"
#include "head.cuh"
#include "internal.h"
#include "once.cuh"

namespace gbnms {

// Two sums over a team of TEAM threads, all of whose warp's lanes take part; with
// more than a warp, TEAM is the block and `shared` holds two values a warp (two
// sets, used in turn).
template <int TEAM>
__device__ __forceinline__ void team_sums(float& a, float& b, float (*shared)[2])
{
#pragma unroll
    for (int o = (TEAM < 32 ? TEAM : 32) / 2; o; o >>= 1) {
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

// V consecutive parameters from element e on (the caller keeps e below the
// width), by the read-only path, so that they are fetched ahead of the stores.
template <typename T, int V>
__device__ __forceinline__ void load_params(float (&v)[V], const void* p, int is_f32, int e, float absent)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = absent;
    } else if (is_f32 || sizeof(T) == 4) {
        const float* q = static_cast<const float*>(p) + e;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(q + i));
                v[i] = f.x;
                v[i + 1] = f.y;
                v[i + 2] = f.z;
                v[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __ldg(q + i);
        }
    } else if constexpr (sizeof(T) == 2) {
        const T* q = static_cast<const T*>(p) + e;
        if constexpr (V == 2) {
            const uint32_t f = __ldg(reinterpret_cast<const uint32_t*>(q));
            const Pack<T, 2> h = *reinterpret_cast<const Pack<T, 2>*>(&f);
            v[0] = to_f32(h.v[0]);
            v[1] = to_f32(h.v[1]);
        } else if constexpr (V == 8) {
            const uint4 f = __ldg(reinterpret_cast<const uint4*>(q));
            const Pack<T, 8> h = *reinterpret_cast<const Pack<T, 8>*>(&f);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(h.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(__ldg(q + i));
        }
    }
}

// V: elements an access, NV: accesses of a thread.
template <typename T, int V, int NV, int TEAM, int THREADS>
__global__ void __launch_bounds__(THREADS)
layer_kernel(const LayerArgs a)
{
    static_assert(TEAM <= 32 || TEAM == THREADS, "a team lies in a warp or is the block");
    __shared__ float shared[2][THREADS / 32][2];
    int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / TEAM) + threadIdx.x / TEAM;
    const int t = threadIdx.x % TEAM;
    if (TEAM == 32 && row >= a.rows) return;
    const bool here = row < a.rows;  // teams that share a warp go on together, the last ones with the last row again
    if (!here) row = a.rows - 1;
    const uint64_t policy = once_policy(a.once);
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    Pack<T, V> q[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TEAM + t) * V;
        if (e < a.width) q[k] = load_once(reinterpret_cast<const Pack<T, V>*>(x + e), policy);
    }
    if (a.second) {
        const T* r = static_cast<const T*>(a.second) + row * a.second_row;
        T* sum = static_cast<T*>(a.sum) + row * a.width;
        Pack<T, V> p[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e < a.width) p[k] = load_once(reinterpret_cast<const Pack<T, V>*>(r + e), policy);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(q[k].v[i]) + to_f32(p[k].v[i]);
            q[k] = pack_results<T, V>(v);
            if (here && e < a.width) store_once(reinterpret_cast<Pack<T, V>*>(sum + e), q[k], policy);
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
    if (here && t == 0) {
        if (a.mean) a.mean[row] = mean + off;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.out) + row * a.width;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TEAM + t) * V;
        if (here && e < a.width) {
            float w[V], b[V], v[V];
            load_params<T, V>(w, a.weight, a.param_f32, e, 1.0f);
            load_params<T, V>(b, a.bias, a.param_f32, e, 0.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = fmaf(((to_f32(q[k].v[i]) - mean) - off) * rstd, w[i], b[i]);
            store_once(reinterpret_cast<Pack<T, V>*>(y + e), pack_results<T, V>(v), policy);
        }
    }
}

// The gradient's rows on their way: each thread copies its own elements of x,
// dy and dsum to its own places in shared memory (cp.async), a row ahead of the
// one that is worked on, so nothing but the thread itself waits for them.
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void* to, const void* from)
{
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// Operands that a block copies ahead: all three, x and dy, or none, as rows and
// weights fit.
template <typename T, int V, int NV, int TEAM, int THREADS>
constexpr bool layer_fits(int operands)
{
    return 2 * operands * THREADS * NV * V * sizeof(T) + TEAM * NV * V * 4 <= (TEAM >= 512 ? 220 : 112) * 1024;
}
template <typename T, int V, int NV, int TEAM, int THREADS>
constexpr int LAYER_AHEAD = sizeof(T) * V < 4                            ? 0
                            : layer_fits<T, V, NV, TEAM, THREADS>(3)     ? 3
                            : layer_fits<T, V, NV, TEAM, THREADS>(2)     ? 2
                                                                         : 0;

template <typename T, int V, int NV, int TEAM, int THREADS>
constexpr int LAYER_GRAD_SMEM = TEAM * NV * V * 4 + (TEAM < THREADS ? TEAM * NV * V * 8 : 0) +
                                2 * LAYER_AHEAD<T, V, NV, TEAM, THREADS> * THREADS * NV * V * static_cast<int>(sizeof(T));

constexpr int LAYER_GRAD_THREADS = 128;  // of a block whose teams are warps

// Each block's sums of dy * u and of dy go to parts[block][2][width].
template <typename T, int V, int NV, int TEAM, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
layer_grad_kernel(const LayerArgs a, float* parts)
{
    static_assert(TEAM <= 32 || TEAM == THREADS, "a team lies in a warp or is the block");
    using Vec = Pack<T, V>;
    constexpr int AHEAD = LAYER_AHEAD<T, V, NV, TEAM, THREADS>;
    constexpr int TEAMS = THREADS / TEAM, SPAN = TEAM * NV * V;
    __shared__ float shared[2][THREADS / 32][2];
    extern __shared__ __align__(16) char dynamic[];
    float* weights = reinterpret_cast<float*>(dynamic);   // [SPAN], 0 behind the width
    float* columns = weights + SPAN;                      // [2][SPAN] where teams are warps
    Vec* rows = reinterpret_cast<Vec*>(columns + (TEAMS > 1 ? 2 * SPAN : 0));  // [2][AHEAD][NV][THREADS]
    const uint64_t policy = once_policy(a.once);
    const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
    // Teams that share a warp go on together, by the row of its first one; rows that are not there count as nothing.
    const int behind = TEAM < 32 ? team % (32 / TEAM) : 0;
    auto fetch = [&](int64_t r, int set) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_row;
        const T* dy = static_cast<const T*>(a.dy) + r * a.dy_row;
        const T* more = a.second ? static_cast<const T*>(a.second) + r * a.second_row : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (e < a.width) {
                Vec* to = rows + (set * AHEAD * NV + k) * THREADS + threadIdx.x;
                copy_ahead<sizeof(Vec)>(to, x + e);
                copy_ahead<sizeof(Vec)>(to + NV * THREADS, dy + e);
                if (AHEAD == 3 && more) copy_ahead<sizeof(Vec)>(to + 2 * NV * THREADS, more + e);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (AHEAD > 0) {
        if (row < a.rows) fetch(row, 0);
    }
    float mean = 0.0f, rstd = 0.0f;  // 0 where there is no row, so that 0 * u is 0
    if (row < a.rows) {
        mean = a.mean[row];
        rstd = a.rstd[row];
    }
    for (int e = threadIdx.x * V; e < SPAN; e += THREADS * V) {
        float w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = 0.0f;
        if (e < a.width) load_params<T, V>(w, a.weight, a.param_f32, e, 1.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) weights[e + i] = w[i];
    }
    __syncthreads();
    const float share = 1.0f / static_cast<float>(a.width);
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
    const Vec none{};
    for (int set = 0; row - behind < a.rows; row += step, set ^= 1) {
        const float m = mean, r = rstd;
        const bool there = TEAM >= 32 || row < a.rows;
        Vec q[AHEAD ? 1 : NV], g[AHEAD ? 1 : NV];
        const Vec* here = rows + set * AHEAD * NV * THREADS + threadIdx.x;
        const bool next = row + step < a.rows;
        mean = next ? a.mean[row + step] : 0.0f;
        rstd = next ? a.rstd[row + step] : 0.0f;
        if constexpr (AHEAD > 0) {
            if (row + step < a.rows) {
                fetch(row + step, set ^ 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncwarp();
        } else {
            const T* x = static_cast<const T*>(a.x) + row * a.x_row;
            const T* dy = static_cast<const T*>(a.dy) + row * a.dy_row;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int e = (k * TEAM + t) * V;
                q[k] = there && e < a.width ? *reinterpret_cast<const Vec*>(x + e) : none;
                g[k] = there && e < a.width ? *reinterpret_cast<const Vec*>(dy + e) : none;
            }
        }
        float first = 0.0f, along = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            const bool in = there && e < a.width;
            const Vec xk = AHEAD ? (in ? here[k * THREADS] : none) : q[AHEAD ? 0 : k];
            const Vec gk = AHEAD ? (in ? here[(NV + k) * THREADS] : none) : g[AHEAD ? 0 : k];
            const Pack<float, V> w = *reinterpret_cast<const Pack<float, V>*>(weights + e);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u = (to_f32(xk.v[i]) - m) * r, d = to_f32(gk.v[i]), du = d * w.v[i];
                dw[k][i] = fmaf(d, u, dw[k][i]);
                db[k][i] += d;
                first += du;
                along = fmaf(du, u, along);
            }
        }
        team_sums<TEAM>(first, along, shared[set]);
        first *= share;
        along *= share;
        T* dx = static_cast<T*>(a.out) + row * a.width;
        const T* more = a.second ? static_cast<const T*>(a.second) + row * a.second_row : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TEAM + t) * V;
            if (there && e < a.width) {
                const Vec xk = AHEAD ? here[k * THREADS] : q[AHEAD ? 0 : k], gk = AHEAD ? here[(NV + k) * THREADS] : g[AHEAD ? 0 : k];
                const Pack<float, V> w = *reinterpret_cast<const Pack<float, V>*>(weights + e);
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u = (to_f32(xk.v[i]) - m) * r, du = to_f32(gk.v[i]) * w.v[i];
                    v[i] = r * fmaf(-u, along, du - first);
                }
                if (more) {
                    const Vec p = AHEAD == 3 ? here[(2 * NV + k) * THREADS] : *reinterpret_cast<const Vec*>(more + e);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] += to_f32(p.v[i]);
                }
                store_once(reinterpret_cast<Vec*>(dx + e), pack_results<T, V>(v), policy);
            }
        }
    }
    if (!parts) return;
    float* part = parts + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
    if constexpr (TEAMS > 1) {
        // The teams of a warp in a tree, the block's warps one after another: a fixed order.
#pragma unroll
        for (int o = TEAM; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dw[k][i] += __shfl_xor_sync(FULL, dw[k][i], o);
                    db[k][i] += __shfl_xor_sync(FULL, db[k][i], o);
                }
        for (int now = 0; now < THREADS / 32; ++now) {
            if (threadIdx.x / 32 == now && threadIdx.x % 32 < TEAM) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int e = (k * TEAM + t) * V + i;
                        columns[e] = (now ? columns[e] : 0.0f) + dw[k][i];
                        columns[SPAN + e] = (now ? columns[SPAN + e] : 0.0f) + db[k][i];
                    }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < a.width; e += THREADS) {
            part[e] = columns[e];
            part[a.width + e] = columns[SPAN + e];
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (k * TEAM + t) * V + i;
                if (e < a.width) {
                    part[e] = dw[k][i];
                    part[a.width + e] = db[k][i];
                }
            }
    }
}

// Threads of a team and the values that one holds.  Rows that move element by
// element have more threads with fewer values, each a register and an access of
// its own (gradient of 40000 x 999 bf16: 187 us, by warps with 32 values 284).
struct LayerShape {
    int team, values;
};
inline LayerShape layer_shape(int width, bool single)
{
    if (width > 4096) return width <= 8192 ? LayerShape{512, 16} : LayerShape{1024, 16};
    if (width <= 128) return {width <= 64 ? 8 : 16, 8};
    if (single) return width <= 256 ? LayerShape{32, 8} : width <= 1024 ? LayerShape{128, 8} : LayerShape{512, 8};
    if (width <= 1024) return {32, width <= 256 ? 8 : width <= 512 ? 16 : 32};
    return {128, width <= 2048 ? 16 : 32};
}

// Blocks of the gradient that an SM holds by their registers: two sums a value,
// and some fifty.
constexpr int layer_grad_resident(int team, int values)
{
    return team == 1024 ? 1 : team == 512 ? (values == 8 ? 2 : 1) : values == 32 ? 4 : values == 16 ? 5 : team <= 32 ? 6 : 8;
}

// Blocks of the gradient: one wave of `resident`, and more where a team's sums
// would run over more than 256 rows.
inline int64_t layer_grad_blocks(int64_t rows, int team, int resident)
{
    const int64_t teams = team <= 32 ? LAYER_GRAD_THREADS / team : 1, want = (rows + teams - 1) / teams, full = SMS * resident;
    const int64_t least = (rows + 256 * teams - 1) / (256 * teams);
    return want < full ? want : least > full ? least : full;
}

template <typename T, int V, int TEAM, int VALUES>
int64_t launch_layer_rows(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    if (grad) {
        constexpr int THREADS = TEAM <= 32 ? LAYER_GRAD_THREADS : TEAM, BLOCKS = layer_grad_resident(TEAM, VALUES);
        constexpr int SMEM = LAYER_GRAD_SMEM<T, V, VALUES / V, TEAM, THREADS>;
        constexpr int FIT = SMEM * BLOCKS <= 220 * 1024 ? BLOCKS : 220 * 1024 / SMEM;
        auto kernel = layer_grad_kernel<T, V, VALUES / V, TEAM, THREADS, FIT>;
        if (SMEM > 40 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        const int64_t grid = layer_grad_blocks(a.rows, TEAM, FIT);
        kernel<<<static_cast<unsigned>(grid), THREADS, SMEM, st>>>(a, parts);
        return grid;
    }
    constexpr int THREADS = TEAM <= 32 ? 256 : TEAM;
    const int64_t teams = THREADS / TEAM;
    const unsigned grid = static_cast<unsigned>((a.rows + teams - 1) / teams);
    layer_kernel<T, V, VALUES / V, TEAM, THREADS><<<grid, THREADS, 0, st>>>(a);
    return 0;
}

// Returns the blocks that left parts.
template <typename T, int V>
int64_t launch_layer_width(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    const LayerShape s = layer_shape(a.width, V == 1);
    if (s.team == 8) return launch_layer_rows<T, V, 8, 8>(a, parts, grad, st);
    if (s.team == 16) return launch_layer_rows<T, V, 16, 8>(a, parts, grad, st);
    if constexpr (V == 1) {
        if (s.team == 32) return launch_layer_rows<T, V, 32, 8>(a, parts, grad, st);
        if (s.team == 128) return launch_layer_rows<T, V, 128, 8>(a, parts, grad, st);
        if (s.values == 8) return launch_layer_rows<T, V, 512, 8>(a, parts, grad, st);
    } else {
        if (s.team == 32) {
            if (s.values == 8) return launch_layer_rows<T, V, 32, 8>(a, parts, grad, st);
            if (s.values == 16) return launch_layer_rows<T, V, 32, 16>(a, parts, grad, st);
            return launch_layer_rows<T, V, 32, 32>(a, parts, grad, st);
        }
        if (s.team == 128) {
            if (s.values == 16) return launch_layer_rows<T, V, 128, 16>(a, parts, grad, st);
            return launch_layer_rows<T, V, 128, 32>(a, parts, grad, st);
        }
    }
    if (s.team == 512) return launch_layer_rows<T, V, 512, 16>(a, parts, grad, st);
    return launch_layer_rows<T, V, 1024, 16>(a, parts, grad, st);
}

// Accesses of 16 bytes where every row starts at a multiple of them, else of two
// elements or of one.
template <typename T>
int64_t launch_layer_type(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    constexpr int MOST = 16 / sizeof(T);
    const uintptr_t pe = a.param_f32 ? 4 : sizeof(T);
    auto even = [&](int v) {
        auto starts = [&](const void* p, uintptr_t e) { return reinterpret_cast<uintptr_t>(p) % (v * e < 16 ? v * e : 16) == 0; };
        return a.width % v == 0 && a.x_row % v == 0 && a.second_row % v == 0 && a.dy_row % v == 0 &&
               starts(a.x, sizeof(T)) && starts(a.second, sizeof(T)) && starts(a.dy, sizeof(T)) && starts(a.out, sizeof(T)) &&
               starts(a.sum, sizeof(T)) && starts(a.weight, pe) && starts(a.bias, pe);
    };
    if (even(MOST)) return launch_layer_width<T, MOST>(a, parts, grad, st);
    return even(2) ? launch_layer_width<T, 2>(a, parts, grad, st) : launch_layer_width<T, 1>(a, parts, grad, st);
}

int64_t launch_layer_f32(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);
int64_t launch_layer_f16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);
int64_t launch_layer_bf16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st);

}  // namespace gbnms
