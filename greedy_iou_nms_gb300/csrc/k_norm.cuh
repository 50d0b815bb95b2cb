// Group normalisation of channels-last maps with the affine map, the
// activation and dropout fused into its epilogue, and its gradient.
//
//   u = (x - mean) * rstd, z = u * weight + bias, y = drop(act(z)), the
//   statistics over the pixels and channels of one group of one image;
//   dz = drop(dy) * act'(z), dbias = sum dz, dweight = sum dz * u,
//   dx = rstd * (du - avg(du) - u * avg(du * u)) with du = dz * weight.
//
// Statistics are pieces (count, mean, sum of squared deviations).  A thread
// sums deviations from the first value it sees of a channel, so nothing is
// lost to a mean far above the spread (an outlier as that first value costs
// at most count * 2^-24 of the variance that it brings itself).  Pieces are
// joined in a fixed order, in two steps: the mean m of their means, then the
// deviations d of their means from m, M2 = sum of M2_i + n_i d_i^2 - n (avg
// d)^2.  A piece's mean is a pair (high + low), so that d is right to its own
// size and not to the mean's.
#pragma once

#include <type_traits>

#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int NT = 256;           // threads of a block
constexpr int NORM_CTAS = 1216;   // blocks that a call aims at: eight for each of 152 SMs

// Row pieces of an image (a function of the shape alone: the workspace's size
// depends on it).
inline int64_t norm_pieces(int64_t batch, int64_t pixels)
{
    const int64_t by_rows = (pixels + 63) / 64, by_ctas = (NORM_CTAS + batch - 1) / batch;
    const int64_t p = by_rows < by_ctas ? by_rows : by_ctas;
    return p < 1 ? 1 : p;
}

// Scratch: three partial planes [batch][pieces][channels] (mean high, M2, mean
// low; the gradient's two sums), two of [batch][groups].
struct NormScratch {
    float *pa, *pb, *pc, *ga, *gb;
};

inline NormScratch scratch(const NormArgs& a, void* ws)
{
    NormScratch s;
    const size_t plane = static_cast<size_t>(a.batch) * norm_pieces(a.batch, a.pixels) * a.channels;
    s.pa = static_cast<float*>(ws);
    s.pb = s.pa + plane;
    s.pc = s.pb + plane;
    s.ga = s.pc + plane;
    s.gb = s.ga + static_cast<size_t>(a.batch) * a.groups;
    return s;
}

// Tile of a block: `wide` vectors of V channels by NT / wide rows at a time.
struct NormTile {
    int wide;       // vectors a row of the tile
    int tiles;      // tiles a row of the map
    int64_t pieces;
};

template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float (&v)[V])
{
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(q.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&v)[V])
{
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(v[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = q;
}

// Where a thread stands: image, row range of the piece, first channel.
struct Spot {
    int64_t image, piece, row, row_end;
    int channel, ty, rows;
    bool in;
};

template <int V>
__device__ __forceinline__ Spot spot(const NormArgs& a, const NormTile& t)
{
    Spot s;
    s.image = blockIdx.x / t.pieces;
    s.piece = blockIdx.x % t.pieces;
    s.rows = NT / t.wide;
    s.ty = static_cast<int>(threadIdx.x) / t.wide;
    const int vec = static_cast<int>(blockIdx.y) * t.wide + static_cast<int>(threadIdx.x) % t.wide;
    s.channel = vec * V;
    s.in = s.ty < s.rows && s.channel < a.channels;
    const int64_t per = (a.pixels + t.pieces - 1) / t.pieces;
    s.row = s.piece * per;
    s.row_end = s.row + per < a.pixels ? s.row + per : a.pixels;
    return s;
}

// Per-channel (mean, squared deviations) of each row piece.
template <typename T, int V>
__global__ void __launch_bounds__(NT)
norm_partial_kernel(NormArgs a, NormTile t, NormScratch w)
{
    __shared__ float s_high[NT * V], s_low[NT * V], s_m2[NT * V];
    __shared__ int s_count[NT];
    const Spot p = spot<V>(a, t);
    float first[V], s[V], q[V];
    int count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) first[i] = s[i] = q[i] = 0.0f;
    if (p.in) {
        const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
        for (int64_t r = p.row + p.ty; r < p.row_end; r += p.rows, ++count) {
            float v[V];
            load_row<T, V>(x + r * a.x_pixel, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (count == 0) first[i] = v[i];
                const float d = v[i] - first[i];
                s[i] += d;
                q[i] = fmaf(d, d, q[i]);
            }
        }
    }
    s_count[threadIdx.x] = count;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float m = count ? s[i] / count : 0.0f;
        s_high[threadIdx.x * V + i] = first[i];
        s_low[threadIdx.x * V + i] = m;
        s_m2[threadIdx.x * V + i] = fmaxf(q[i] - s[i] * m, 0.0f);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.wide * V; c += NT) {
        const int channel = static_cast<int>(blockIdx.y) * t.wide * V + c;
        if (channel >= a.channels) continue;
        float n = 0.0f, mean = 0.0f, low = 0.0f, m2 = 0.0f;
        for (int y = 0; y < p.rows; ++y) n += static_cast<float>(s_count[y * t.wide + c / V]);
        if (n == 0.0f) n = 1.0f;
        const float origin = s_high[c];  // equal values give exactly that mean
        for (int y = 0; y < p.rows; ++y) {
            const int at = y * t.wide * V + c;
            mean += static_cast<float>(s_count[y * t.wide + c / V]) / n * (s_high[at] + s_low[at] - origin);
        }
        mean += origin;
        for (int y = 0; y < p.rows; ++y) {
            const int at = y * t.wide * V + c;
            const float k = static_cast<float>(s_count[y * t.wide + c / V]), d = (s_high[at] - mean) + s_low[at];
            low = fmaf(k, d, low);
            m2 += fmaf(k * d, d, s_m2[at]);
        }
        low /= n;
        const int64_t at = (p.image * t.pieces + p.piece) * a.channels + channel;
        w.pa[at] = mean;
        w.pb[at] = fmaxf(m2 - n * low * low, 0.0f);
        w.pc[at] = low;
    }
}

// mean and rstd of each (image, group) from the pieces; one warp each.
static __global__ void __launch_bounds__(NT)
norm_finish_kernel(NormArgs a, NormTile t, NormScratch w)
{
    const int64_t which = (static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x) / 32;
    if (which >= a.batch * a.groups) return;
    const int64_t image = which / a.groups;
    const int D = a.channels / a.groups, c0 = static_cast<int>(which % a.groups) * D;
    const int64_t per = (a.pixels + t.pieces - 1) / t.pieces, items = t.pieces * D;
    const float all = static_cast<float>(a.pixels) * static_cast<float>(D);
    const float origin = w.pa[image * t.pieces * a.channels + c0];
    float mean = 0.0f, low = 0.0f, m2 = 0.0f;
    for (int64_t i = lane_id(); i < items; i += 32) {
        const int64_t piece = i / D, left = a.pixels - piece * per;
        const float k = static_cast<float>(left < per ? (left > 0 ? left : 0) : per);
        if (k > 0.0f) mean += (w.pa[(image * t.pieces + piece) * a.channels + c0 + i % D] - origin) * (k / all);
    }
    mean = origin + warp_sum(mean);
    for (int64_t i = lane_id(); i < items; i += 32) {
        const int64_t piece = i / D, left = a.pixels - piece * per;
        const float k = static_cast<float>(left < per ? (left > 0 ? left : 0) : per);
        const int64_t at = (image * t.pieces + piece) * a.channels + c0 + i % D;
        const float d = (w.pa[at] - mean) + w.pc[at];
        if (k > 0.0f) {
            low = fmaf(d, k / all, low);
            m2 += fmaf(d * k, d, w.pb[at]);
        }
    }
    low = warp_sum(low);
    m2 = warp_sum(m2);
    if (lane_id() == 0) {
        a.mean[which] = mean + low;
        a.rstd[which] = 1.0f / sqrtf(fmaxf(m2 / all - low * low, 0.0f) + a.eps);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(NT)
norm_apply_kernel(NormArgs a, NormTile t)
{
    const Spot p = spot<V>(a, t);
    if (!p.in) return;
    const int D = a.channels / a.groups;
    float mean[V], scale[V], shift[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = p.image * a.groups + (p.channel + i) / D;
        mean[i] = a.mean[g];
        scale[i] = a.rstd[g] * (a.weight ? load_param<T>(a.weight, a.param_f32, p.channel + i) : 1.0f);
        shift[i] = a.bias ? load_param<T>(a.bias, a.param_f32, p.channel + i) : 0.0f;
    }
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
    T* y = static_cast<T*>(a.out);
    for (int64_t r = p.row + p.ty; r < p.row_end; r += p.rows) {
        float v[V];
        load_row<T, V>(x + r * a.x_pixel, v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(v[i] - mean[i], scale[i], shift[i]);
        act_values<V>(v, a.act);
        const int64_t at = (p.image * a.pixels + r) * a.channels + p.channel;
        if (a.drop.limit < 65536u) drop<V>(v, static_cast<uint64_t>(at), a.drop);
        store_row<T, V>(y + at, v);
    }
}

// dz and u of one vector.
template <typename T, int V>
__device__ __forceinline__ void slope_row(const NormArgs& a, const float (&mean)[V], const float (&rstd)[V],
                                          const float (&weight)[V], const float (&bias)[V], const T* x, const T* dy,
                                          uint64_t at, float (&u)[V], float (&dz)[V])
{
    float z[V];
    load_row<T, V>(x, u);
    load_row<T, V>(dy, dz);
    if (a.drop.limit < 65536u) drop<V>(dz, at, a.drop);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = (u[i] - mean[i]) * rstd[i];
        z[i] = fmaf(u[i], weight[i], bias[i]);
    }
    act_slopes<V>(dz, z, a.act);
}

template <typename T, int V>
__device__ __forceinline__ void load_channels(const NormArgs& a, const Spot& p, float (&mean)[V], float (&rstd)[V],
                                              float (&weight)[V], float (&bias)[V])
{
    const int D = a.channels / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = p.image * a.groups + (p.channel + i) / D;
        mean[i] = a.mean[g];
        rstd[i] = a.rstd[g];
        weight[i] = a.weight ? load_param<T>(a.weight, a.param_f32, p.channel + i) : 1.0f;
        bias[i] = a.bias ? load_param<T>(a.bias, a.param_f32, p.channel + i) : 0.0f;
    }
}

// Per-channel sums of dz and dz * u of each row piece.
template <typename T, int V>
__global__ void __launch_bounds__(NT)
norm_grad_partial_kernel(NormArgs a, NormTile t, NormScratch w)
{
    __shared__ float s_a[NT * V], s_b[NT * V];
    const Spot p = spot<V>(a, t);
    float sa[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sa[i] = sb[i] = 0.0f;
    if (p.in) {
        float mean[V], rstd[V], weight[V], bias[V];
        load_channels<T, V>(a, p, mean, rstd, weight, bias);
        const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
        const T* dy = static_cast<const T*>(a.dy) + p.image * a.dy_image + p.channel;
        for (int64_t r = p.row + p.ty; r < p.row_end; r += p.rows) {
            float u[V], dz[V];
            slope_row<T, V>(a, mean, rstd, weight, bias, x + r * a.x_pixel, dy + r * a.dy_pixel,
                                 static_cast<uint64_t>((p.image * a.pixels + r) * a.channels + p.channel), u, dz);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sa[i] += dz[i];
                sb[i] = fmaf(dz[i], u[i], sb[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s_a[threadIdx.x * V + i] = sa[i];
        s_b[threadIdx.x * V + i] = sb[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.wide * V; c += NT) {
        const int channel = static_cast<int>(blockIdx.y) * t.wide * V + c;
        if (channel >= a.channels) continue;
        float va = 0.0f, vb = 0.0f;
        for (int y = 0; y < p.rows; ++y) {
            va += s_a[y * t.wide * V + c];
            vb += s_b[y * t.wide * V + c];
        }
        const int64_t at = (p.image * t.pieces + p.piece) * a.channels + channel;
        w.pa[at] = va;
        w.pb[at] = vb;
    }
}

// avg(du) and avg(du * u) of each (image, group); one warp each.
template <typename T>
__global__ void __launch_bounds__(NT)
norm_grad_finish_kernel(NormArgs a, NormTile t, NormScratch w)
{
    const int64_t which = (static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x) / 32;
    if (which >= a.batch * a.groups) return;
    const int64_t image = which / a.groups;
    const int D = a.channels / a.groups, c0 = static_cast<int>(which % a.groups) * D;
    const float all = static_cast<float>(a.pixels) * static_cast<float>(D);
    float va = 0.0f, vb = 0.0f;
    for (int64_t i = lane_id(); i < t.pieces * D; i += 32) {
        const int c = c0 + static_cast<int>(i % D);
        const float k = a.weight ? load_param<T>(a.weight, a.param_f32, c) : 1.0f;
        const int64_t at = (image * t.pieces + i / D) * a.channels + c;
        va = fmaf(k, w.pa[at], va);
        vb = fmaf(k, w.pb[at], vb);
    }
    va = warp_sum(va);
    vb = warp_sum(vb);
    if (lane_id() == 0) {
        w.ga[which] = va / all;
        w.gb[which] = vb / all;
    }
}

// dweight and dbias: sums over `items` partial rows, 32 channels a block.
static __global__ void __launch_bounds__(NT)
norm_grad_param_kernel(NormArgs a, int64_t items, const float* pa, const float* pb)
{
    __shared__ float s_a[NT], s_b[NT];
    const int c = static_cast<int>(blockIdx.x) * 32 + static_cast<int>(lane_id());
    float va = 0.0f, vb = 0.0f;
    if (c < a.channels)
        for (int64_t i = threadIdx.x / 32; i < items; i += NT / 32) {
            va += pa[i * a.channels + c];
            vb += pb[i * a.channels + c];
        }
    s_a[threadIdx.x] = va;
    s_b[threadIdx.x] = vb;
    __syncthreads();
    if (threadIdx.x < 32 && c < a.channels) {
        for (int k = 1; k < NT / 32; ++k) {
            va += s_a[threadIdx.x + 32 * k];
            vb += s_b[threadIdx.x + 32 * k];
        }
        if (a.dbias) a.dbias[c] = va;
        if (a.dweight) a.dweight[c] = vb;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(NT)
norm_grad_apply_kernel(NormArgs a, NormTile t, NormScratch w)
{
    const Spot p = spot<V>(a, t);
    if (!p.in) return;
    const int D = a.channels / a.groups;
    float mean[V], rstd[V], weight[V], bias[V], m1[V], m2[V];
    load_channels<T, V>(a, p, mean, rstd, weight, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = p.image * a.groups + (p.channel + i) / D;
        m1[i] = w.ga[g];
        m2[i] = w.gb[g];
    }
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
    const T* dy = static_cast<const T*>(a.dy) + p.image * a.dy_image + p.channel;
    for (int64_t r = p.row + p.ty; r < p.row_end; r += p.rows) {
        float u[V], dz[V];
        const int64_t at = (p.image * a.pixels + r) * a.channels + p.channel;
        slope_row<T, V>(a, mean, rstd, weight, bias, x + r * a.x_pixel, dy + r * a.dy_pixel,
                             static_cast<uint64_t>(at), u, dz);
#pragma unroll
        for (int i = 0; i < V; ++i) dz[i] = rstd[i] * (fmaf(dz[i], weight[i], -m1[i]) - u[i] * m2[i]);
        store_row<T, V>(static_cast<T*>(a.out) + at, dz);
    }
}

// ------------------------------------------------------------------- clusters
//
// Where one image's slab of whole groups (a few dozen channels of every
// pixel) fits the registers of a cluster, it is read once: each block keeps
// its rows, the blocks exchange their sums through distributed shared memory,
// and the results are written from the registers.

// Tile of a cluster: `wide` vectors of V channels (whole groups), the rows
// split over `ctas` blocks of `rows` each.
struct NormCluster {
    int wide, tiles, ctas;
    int rows;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// *p of the block `rank` of the cluster.
__device__ __forceinline__ float peer_load(const float* p, int rank)
{
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// Where a thread of a cluster's block stands.
struct ClusterSpot {
    int64_t image;
    int rank, first_channel, channel, tx, ty, step, row0, row_end, groups;
    bool in;
};

template <int V>
__device__ __forceinline__ ClusterSpot cluster_spot(const NormArgs& a, const NormCluster& t, int D)
{
    ClusterSpot p;
    const unsigned id = blockIdx.x / t.ctas;
    p.rank = static_cast<int>(blockIdx.x % t.ctas);
    p.image = id / t.tiles;
    p.first_channel = static_cast<int>(id % t.tiles) * t.wide * V;
    p.tx = static_cast<int>(threadIdx.x) % t.wide;
    p.ty = static_cast<int>(threadIdx.x) / t.wide;
    p.step = NT / t.wide;
    p.channel = p.first_channel + p.tx * V;
    p.in = p.ty < p.step && p.channel < a.channels;
    const int64_t r0 = static_cast<int64_t>(p.rank) * t.rows, r1 = r0 + t.rows;
    p.row0 = static_cast<int>(r0 < a.pixels ? r0 : a.pixels);
    p.row_end = static_cast<int>(r1 < a.pixels ? r1 : a.pixels);
    const int left = a.channels - p.first_channel, channels = t.wide * V < left ? t.wide * V : left;
    p.groups = channels / D;
    return p;
}

// out[q][g] = sum of the threads' partials part[q][ty][...] of group g: `each`
// entries of a row of `width` belong to a group.  One warp a group.
template <int N>
__device__ __forceinline__ void sum_groups(const float* part, int plane, int width, int each, int steps, int groups,
                                           float* out, int out_plane)
{
    __syncthreads();
    for (int g = static_cast<int>(threadIdx.x) / 32; g < groups; g += NT / 32) {
        float v[N];
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = 0.0f;
        for (int k = static_cast<int>(lane_id()); k < steps * each; k += 32) {
            const int at = k / each * width + g * each + k % each;
#pragma unroll
            for (int q = 0; q < N; ++q) v[q] += part[q * plane + at];
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
            v[q] = warp_sum(v[q]);
            if (lane_id() == 0) out[q * out_plane + g] = v[q];
        }
    }
    __syncthreads();
}

// ONE: a vector lies in one group (its channels' sums are one).
template <typename T, int V, int NV, bool ONE>
__global__ void __launch_bounds__(NT)
norm_cluster_kernel(NormArgs a, NormCluster t)
{
    constexpr int P = ONE ? 1 : V;  // partial sums of a thread
    extern __shared__ float smem[];
    const int CW = t.wide * V, D = a.channels / a.groups;
    float* part = smem;                  // [2][NT * P]
    float* s_weight = part + 2 * NT * P; // [CW]
    float* s_bias = s_weight + CW;       // [CW]
    float* s_sum = s_bias + CW;          // [2][CW]: sums by group
    float* s_piece = s_sum + 2 * CW;     // [3][CW]: this block's mean (high, low) and squares by group
    float* s_mean = s_piece + 3 * CW;    // [CW]: the image's, by group
    float* s_rstd = s_mean + CW;
    const ClusterSpot p = cluster_spot<V>(a, t, D);
    Pack<T, V> q[NV];
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int r = p.row0 + p.ty + k * p.step;
        if (p.in && r < p.row_end) q[k] = *reinterpret_cast<const Pack<T, V>*>(x + r * a.x_pixel);
    }
    for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
        s_weight[c] = a.weight ? load_param<T>(a.weight, a.param_f32, p.first_channel + c) : 1.0f;
        s_bias[c] = a.bias ? load_param<T>(a.bias, a.param_f32, p.first_channel + c) : 0.0f;
    }
    const int width = ONE ? t.wide : CW, each = ONE ? D / V : D;
    auto put = [&](int plane, const float (&s)[P]) {
        if (p.ty < p.step) {
#pragma unroll
            for (int i = 0; i < P; ++i) part[plane * NT * P + (p.ty * t.wide + p.tx) * P + i] = s[i];
        }
    };
    // The block's mean by group, then the deviations from it.
    {
        float s[P];
#pragma unroll
        for (int i = 0; i < P; ++i) s[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (p.in && p.row0 + p.ty + k * p.step < p.row_end) {
#pragma unroll
                for (int i = 0; i < V; ++i) s[ONE ? 0 : i] += to_f32(q[k].v[i]);
            }
        put(0, s);
    }
    sum_groups<1>(part, 0, width, each, p.step, p.groups, s_sum, 0);
    const float n = static_cast<float>(p.row_end - p.row0) * static_cast<float>(D);
    const float each_n = n > 0.0f ? 1.0f / n : 0.0f;
    {
        float mean[P], s1[P], s2[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            mean[i] = p.in ? s_sum[(p.tx * V + i) / D] * each_n : 0.0f;
            s1[i] = s2[i] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (p.in && p.row0 + p.ty + k * p.step < p.row_end) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = to_f32(q[k].v[i]) - mean[ONE ? 0 : i];
                    s1[ONE ? 0 : i] += d;
                    s2[ONE ? 0 : i] = fmaf(d, d, s2[ONE ? 0 : i]);
                }
            }
        put(0, s1);
        put(1, s2);
        for (int g = threadIdx.x; g < p.groups; g += NT) s_piece[g] = s_sum[g] * each_n;
    }
    sum_groups<2>(part, NT * P, width, each, p.step, p.groups, s_sum, CW);
    for (int g = threadIdx.x; g < p.groups; g += NT) {
        const float low = s_sum[g] * each_n;
        s_piece[CW + g] = low;
        s_piece[2 * CW + g] = fmaxf(s_sum[CW + g] - s_sum[g] * low, 0.0f);
    }
    // The blocks' pieces, joined by every block in the same order.
    if (t.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const float all = static_cast<float>(a.pixels) * static_cast<float>(D);
    for (int g = threadIdx.x; g < p.groups; g += NT) {
        float mean, low = 0.0f, m2 = 0.0f;
        if (t.ctas == 1) {
            mean = s_piece[g];
            low = s_piece[CW + g];
            m2 = s_piece[2 * CW + g];
        } else {
            const float origin = peer_load(s_piece + g, 0);
            mean = 0.0f;
            for (int k = 0; k < t.ctas; ++k) {
                const int64_t left = a.pixels - static_cast<int64_t>(k) * t.rows;
                const float share = static_cast<float>(left < t.rows ? (left > 0 ? left : 0) : t.rows) * D / all;
                mean = fmaf(share, peer_load(s_piece + g, k) - origin, mean);
            }
            mean += origin;
            for (int k = 0; k < t.ctas; ++k) {
                const int64_t left = a.pixels - static_cast<int64_t>(k) * t.rows;
                const float m = static_cast<float>(left < t.rows ? (left > 0 ? left : 0) : t.rows) * D;
                if (m == 0.0f) break;
                const float d = (peer_load(s_piece + g, k) - mean) + peer_load(s_piece + CW + g, k);
                low = fmaf(d, m / all, low);
                m2 += fmaf(d * m, d, peer_load(s_piece + 2 * CW + g, k));
            }
            m2 -= all * low * low;
        }
        const float var = fmaxf(m2 / all, 0.0f), m = mean + low, r = 1.0f / sqrtf(var + a.eps);
        s_mean[g] = m;
        s_rstd[g] = r;
        if (p.rank == 0) {
            const int64_t at = p.image * a.groups + p.first_channel / D + g;
            if (a.mean) a.mean[at] = m;
            if (a.rstd) a.rstd[at] = r;
        }
    }
    if (t.ctas > 1) cluster_arrive();  // done with the peers' memory; waited for at the end
    __syncthreads();
    if (p.in) {
        float mean[P], scale[V], shift[V];
#pragma unroll
        for (int i = 0; i < P; ++i) mean[i] = s_mean[(p.tx * V + i) / D];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            scale[i] = s_rstd[ONE ? p.tx * V / D : (p.tx * V + i) / D] * s_weight[p.tx * V + i];
            shift[i] = s_bias[p.tx * V + i];
        }
        T* y = static_cast<T*>(a.out);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int r = p.row0 + p.ty + k * p.step;
            if (r >= p.row_end) break;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = fmaf(to_f32(q[k].v[i]) - mean[ONE ? 0 : i], scale[i], shift[i]);
            act_values<V>(v, a.act);
            const int64_t at = (p.image * a.pixels + r) * a.channels + p.channel;
            if (a.drop.limit < 65536u) drop<V>(v, static_cast<uint64_t>(at), a.drop);
            store_row<T, V>(y + at, v);
        }
    }
    if (t.ctas > 1) cluster_wait();
}

// The gradient: x stays packed and dz in binary32 (its activation is worked
// out once).  Rank 0 writes the image's channel sums for dweight and dbias.
template <typename T, int V, int NV, bool ONE>
__global__ void __launch_bounds__(NT)
norm_grad_cluster_kernel(NormArgs a, NormCluster t, NormScratch w)
{
    constexpr int P = ONE ? 1 : V;
    extern __shared__ float smem[];
    const int CW = t.wide * V, D = a.channels / a.groups;
    float* part = smem;                   // [2][NT * V]
    float* s_weight = part + 2 * NT * V;  // [CW]
    float* s_bias = s_weight + CW;        // [CW]
    float* s_mine = s_bias + CW;          // [2][CW]: this block's sums by channel
    float* s_all = s_mine + 2 * CW;       // [2][CW]: the image's
    float* s_avg = s_all + 2 * CW;        // [2][CW]: averages by group
    const ClusterSpot p = cluster_spot<V>(a, t, D);
    Pack<T, V> q[NV];
    Pack<T, V> dq[NV];
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + p.channel;
    const T* dy = static_cast<const T*>(a.dy) + p.image * a.dy_image + p.channel;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int r = p.row0 + p.ty + k * p.step;
        if (p.in && r < p.row_end) {
            q[k] = *reinterpret_cast<const Pack<T, V>*>(x + r * a.x_pixel);
            dq[k] = *reinterpret_cast<const Pack<T, V>*>(dy + r * a.dy_pixel);
        }
    }
    for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
        s_weight[c] = a.weight ? load_param<T>(a.weight, a.param_f32, p.first_channel + c) : 1.0f;
        s_bias[c] = a.bias ? load_param<T>(a.bias, a.param_f32, p.first_channel + c) : 0.0f;
    }
    float mean[P], rstd[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int64_t g = p.image * a.groups + (p.channel + i) / D;
        mean[i] = p.in ? a.mean[g] : 0.0f;
        rstd[i] = p.in ? a.rstd[g] : 0.0f;
    }
    __syncthreads();
    float dz[NV][V], sa[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sa[i] = sb[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int r = p.row0 + p.ty + k * p.step;
        if (!p.in || r >= p.row_end) continue;
        float z[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dz[k][i] = to_f32(dq[k].v[i]);
            z[i] = fmaf((to_f32(q[k].v[i]) - mean[ONE ? 0 : i]) * rstd[ONE ? 0 : i], s_weight[p.tx * V + i],
                        s_bias[p.tx * V + i]);
        }
        if (a.drop.limit < 65536u)
            drop<V>(dz[k], static_cast<uint64_t>((p.image * a.pixels + r) * a.channels + p.channel), a.drop);
        act_slopes<V>(dz[k], z, a.act);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sa[i] += dz[k][i];
            sb[i] = fmaf(dz[k][i], (to_f32(q[k].v[i]) - mean[ONE ? 0 : i]) * rstd[ONE ? 0 : i], sb[i]);
        }
    }
    if (p.ty < p.step) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            part[(p.ty * t.wide + p.tx) * V + i] = sa[i];
            part[NT * V + (p.ty * t.wide + p.tx) * V + i] = sb[i];
        }
    }
    // Sums by channel over the block's rows, in two steps: `lists` threads a channel, then one.
    const int lists = CW < NT ? NT / CW : 1;
    __syncthreads();
    for (int k = threadIdx.x; k < lists * CW; k += NT) {
        const int c = k % CW;
        float va = 0.0f, vb = 0.0f;
        for (int y = k / CW; y < p.step; y += lists) {
            va += part[y * CW + c];
            vb += part[NT * V + y * CW + c];
        }
        // Each entry (k / CW, c) was read by this thread alone.
        part[k] = va;
        part[NT * V + k] = vb;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < CW; c += NT) {
        float va = 0.0f, vb = 0.0f;
        for (int y = 0; y < lists; ++y) {
            va += part[y * CW + c];
            vb += part[NT * V + y * CW + c];
        }
        s_mine[c] = va;
        s_mine[CW + c] = vb;
    }
    if (t.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
        float va = 0.0f, vb = 0.0f;
        if (t.ctas == 1) {
            va = s_mine[c];
            vb = s_mine[CW + c];
        } else {
            for (int k = 0; k < t.ctas; ++k) {
                va += peer_load(s_mine + c, k);
                vb += peer_load(s_mine + CW + c, k);
            }
        }
        s_all[c] = va * s_weight[c];
        s_all[CW + c] = vb * s_weight[c];
        if (p.rank == 0) {
            w.pa[p.image * a.channels + p.first_channel + c] = va;
            w.pb[p.image * a.channels + p.first_channel + c] = vb;
        }
    }
    if (t.ctas > 1) cluster_arrive();
    sum_groups<2>(s_all, CW, CW, D, 1, p.groups, s_avg, CW);
    if (p.in) {
        const float each_n = 1.0f / (static_cast<float>(a.pixels) * static_cast<float>(D));
        float m1[P], m2[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int g = (p.tx * V + i) / D;
            m1[i] = s_avg[g] * each_n;
            m2[i] = s_avg[CW + g] * each_n;
        }
        T* dx = static_cast<T*>(a.out);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int r = p.row0 + p.ty + k * p.step;
            if (r >= p.row_end) break;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u = (to_f32(q[k].v[i]) - mean[ONE ? 0 : i]) * rstd[ONE ? 0 : i];
                v[i] = rstd[ONE ? 0 : i] * (fmaf(dz[k][i], s_weight[p.tx * V + i], -m1[ONE ? 0 : i]) - u * m2[ONE ? 0 : i]);
            }
            store_row<T, V>(dx + (p.image * a.pixels + r) * a.channels + p.channel, v);
        }
    }
    if (t.ctas > 1) cluster_wait();
}

// ------------------------------------------------------------------- launches

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Widest vector that every row of the operands can be moved by.
inline int vector_width(const NormArgs& a)
{
    const int e = a.type == NMS_TYPE_F32 ? 4 : 2;
    for (int v = 16 / e; v > 1; v /= 2)
        if (a.channels % v == 0 && a.x_image % v == 0 && a.x_pixel % v == 0 && a.dy_image % v == 0 &&
            a.dy_pixel % v == 0 && aligned_to(a.x, static_cast<size_t>(v) * e) &&
            aligned_to(a.dy, static_cast<size_t>(v) * e) && aligned_to(a.out, static_cast<size_t>(v) * e))
            return v;
    return 1;
}

inline NormTile tile(const NormArgs& a, int v)
{
    NormTile t;
    const int vecs = a.channels / v;
    t.wide = vecs <= 64 ? vecs : 32;
    t.tiles = (vecs + t.wide - 1) / t.wide;
    t.pieces = norm_pieces(a.batch, a.pixels);
    return t;
}

// Launches kernel k over clusters of t.ctas blocks.
template <typename K, typename... Args>
static void launch_clusters(K k, const NormArgs& a, const NormCluster& t, size_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch * t.tiles * t.ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = t.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k, a, t, args...);
}

// f(NV) with the first of the counts that holds n vectors.
template <int NV, int... MORE, typename F>
static void pick_held(int n, F f)
{
    if constexpr (sizeof...(MORE) == 0) {
        f(std::integral_constant<int, NV>{});
    } else {
        if (n <= NV) f(std::integral_constant<int, NV>{});
        else pick_held<MORE...>(n, f);
    }
}

// The cluster kernels, where a slab fits (else false).  A thread holds up to
// 64 elements forward, 32 of x and dz each backward; row segments are of 64
// bytes, or of 32 where that makes the slab fit.
template <typename T, int V>
static bool norm_in_clusters(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    const int e = sizeof(T), D = a.channels / a.groups, vecs = a.channels / V;
    const int most = (grad ? 32 : 64) / V;
    int whole = 1;  // vectors that hold whole groups: lcm(D, V) / V
    while (whole * V % D != 0) ++whole;
    for (int bytes = 64; bytes >= 32; bytes /= 2) {
        NormCluster t{};
        const int want = bytes / (V * e) > 0 ? bytes / (V * e) : 1;
        t.wide = (want + whole - 1) / whole * whole;
        if (t.wide > vecs) t.wide = vecs;
        if (t.wide > 64) return false;
        t.tiles = (vecs + t.wide - 1) / t.wide;
        const int step = NT / t.wide;
        const int64_t passes = (a.pixels + step - 1) / step;
        for (t.ctas = 1; t.ctas < 8 && passes > static_cast<int64_t>(t.ctas) * most; t.ctas *= 2) {}
        if (passes > static_cast<int64_t>(t.ctas) * most || a.batch * t.tiles * t.ctas > INT32_MAX) continue;
        const int held = static_cast<int>((passes + t.ctas - 1) / t.ctas), CW = t.wide * V;
        t.rows = held * step;
        const bool one = D % V == 0;
        if (!grad) {
            const size_t smem = 4 * (2 * NT * (one ? 1 : V) + 9 * static_cast<size_t>(CW));
            pick_held<16 / V, 32 / V, 64 / V>(held, [&](auto count) {
                constexpr int NV = decltype(count)::value;
                launch_clusters(one ? norm_cluster_kernel<T, V, NV, true> : norm_cluster_kernel<T, V, NV, false>, a, t,
                                smem, st);
            });
        } else {
            const size_t smem = 4 * (2 * NT * V + 8 * static_cast<size_t>(CW));
            const NormScratch w = scratch(a, ws);
            pick_held<8 / V, 16 / V, 32 / V>(held, [&](auto count) {
                constexpr int NV = decltype(count)::value;
                launch_clusters(one ? norm_grad_cluster_kernel<T, V, NV, true> : norm_grad_cluster_kernel<T, V, NV, false>,
                                a, t, smem, st, w);
            });
            if (a.dweight || a.dbias)
                norm_grad_param_kernel<<<(a.channels + 31) / 32, NT, 0, st>>>(a, a.batch, w.pa, w.pb);
        }
        return true;
    }
    return false;
}

template <typename T, int V>
static void norm_width(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    if constexpr (V > 1)
        if (norm_in_clusters<T, V>(a, ws, st, grad)) return;
    const NormTile t = tile(a, V);
    const NormScratch w = scratch(a, ws);
    const dim3 grid(static_cast<unsigned>(a.batch * t.pieces), t.tiles);
    const unsigned finish = static_cast<unsigned>((a.batch * a.groups + NT / 32 - 1) / (NT / 32));
    if (!grad) {
        NormArgs b = a;
        if (!b.mean) b.mean = w.ga;
        if (!b.rstd) b.rstd = w.gb;
        norm_partial_kernel<T, V><<<grid, NT, 0, st>>>(b, t, w);
        norm_finish_kernel<<<finish, NT, 0, st>>>(b, t, w);
        norm_apply_kernel<T, V><<<grid, NT, 0, st>>>(b, t);
    } else {
        norm_grad_partial_kernel<T, V><<<grid, NT, 0, st>>>(a, t, w);
        norm_grad_finish_kernel<T><<<finish, NT, 0, st>>>(a, t, w);
        norm_grad_apply_kernel<T, V><<<grid, NT, 0, st>>>(a, t, w);
        if (a.dweight || a.dbias)
            norm_grad_param_kernel<<<(a.channels + 31) / 32, NT, 0, st>>>(a, a.batch * t.pieces, w.pa, w.pb);
    }
}

template <typename T>
static void norm_type(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    const int v = vector_width(a);
    if constexpr (sizeof(T) == 2)
        if (v == 8) return norm_width<T, 8>(a, ws, st, grad);
    if (v == 4) return norm_width<T, 4>(a, ws, st, grad);
    if (v == 2) return norm_width<T, 2>(a, ws, st, grad);
    norm_width<T, 1>(a, ws, st, grad);
}

}  // namespace gbnms
