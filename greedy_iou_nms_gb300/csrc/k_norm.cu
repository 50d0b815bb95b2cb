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
#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int NT = 256;           // threads of a block
constexpr int NORM_CTAS = 1216;   // blocks that a call aims at: eight for each of 152 SMs

// Row pieces of an image (a function of the shape alone: the workspace's size
// depends on it).
static int64_t norm_pieces(int64_t batch, int64_t pixels)
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

size_t norm_workspace_bytes(int64_t batch, int64_t pixels, int channels, int groups)
{
    return 12 * static_cast<size_t>(batch) * norm_pieces(batch, pixels) * channels +
           8 * static_cast<size_t>(batch) * groups + 256;
}

static NormScratch scratch(const NormArgs& a, void* ws)
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
__global__ void __launch_bounds__(NT)
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

template <typename T, int V, int ACT>
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
        for (int i = 0; i < V; ++i) v[i] = act_value<ACT>(fmaf(v[i] - mean[i], scale[i], shift[i]));
        const int64_t at = (p.image * a.pixels + r) * a.channels + p.channel;
        if (a.drop.limit < 65536u) drop<V>(v, static_cast<uint64_t>(at), a.drop);
        store_row<T, V>(y + at, v);
    }
}

// dz and u of one vector.
template <typename T, int V, int ACT>
__device__ __forceinline__ void slope_row(const NormArgs& a, const float (&mean)[V], const float (&rstd)[V],
                                          const float (&weight)[V], const float (&bias)[V], const T* x, const T* dy,
                                          uint64_t at, float (&u)[V], float (&dz)[V])
{
    load_row<T, V>(x, u);
    load_row<T, V>(dy, dz);
    if (a.drop.limit < 65536u) drop<V>(dz, at, a.drop);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = (u[i] - mean[i]) * rstd[i];
        dz[i] *= act_slope<ACT>(fmaf(u[i], weight[i], bias[i]));
    }
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
template <typename T, int V, int ACT>
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
            slope_row<T, V, ACT>(a, mean, rstd, weight, bias, x + r * a.x_pixel, dy + r * a.dy_pixel,
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

// dweight and dbias: sums over the images and pieces, 32 channels a block.
__global__ void __launch_bounds__(NT)
norm_grad_param_kernel(NormArgs a, NormTile t, NormScratch w)
{
    __shared__ float s_a[NT], s_b[NT];
    const int c = static_cast<int>(blockIdx.x) * 32 + static_cast<int>(lane_id());
    float va = 0.0f, vb = 0.0f;
    if (c < a.channels)
        for (int64_t i = threadIdx.x / 32; i < a.batch * t.pieces; i += NT / 32) {
            va += w.pa[i * a.channels + c];
            vb += w.pb[i * a.channels + c];
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

template <typename T, int V, int ACT>
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
        slope_row<T, V, ACT>(a, mean, rstd, weight, bias, x + r * a.x_pixel, dy + r * a.dy_pixel,
                             static_cast<uint64_t>(at), u, dz);
#pragma unroll
        for (int i = 0; i < V; ++i) dz[i] = rstd[i] * (fmaf(dz[i], weight[i], -m1[i]) - u[i] * m2[i]);
        store_row<T, V>(static_cast<T*>(a.out) + at, dz);
    }
}

// ------------------------------------------------------------------- launches

static bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Widest vector that every row of the operands can be moved by.
static int vector_width(const NormArgs& a)
{
    const int e = a.type == NMS_TYPE_F32 ? 4 : 2;
    for (int v = 16 / e; v > 1; v /= 2)
        if (a.channels % v == 0 && a.x_image % v == 0 && a.x_pixel % v == 0 && a.dy_image % v == 0 &&
            a.dy_pixel % v == 0 && aligned_to(a.x, static_cast<size_t>(v) * e) &&
            aligned_to(a.dy, static_cast<size_t>(v) * e) && aligned_to(a.out, static_cast<size_t>(v) * e))
            return v;
    return 1;
}

static NormTile tile(const NormArgs& a, int v)
{
    NormTile t;
    const int vecs = a.channels / v;
    t.wide = vecs <= 64 ? vecs : 32;
    t.tiles = (vecs + t.wide - 1) / t.wide;
    t.pieces = norm_pieces(a.batch, a.pixels);
    return t;
}

template <typename T, int V, int ACT>
static void norm_act(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
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
        norm_apply_kernel<T, V, ACT><<<grid, NT, 0, st>>>(b, t);
    } else {
        norm_grad_partial_kernel<T, V, ACT><<<grid, NT, 0, st>>>(a, t, w);
        norm_grad_finish_kernel<T><<<finish, NT, 0, st>>>(a, t, w);
        norm_grad_apply_kernel<T, V, ACT><<<grid, NT, 0, st>>>(a, t, w);
        if (a.dweight || a.dbias) norm_grad_param_kernel<<<(a.channels + 31) / 32, NT, 0, st>>>(a, t, w);
    }
}

template <typename T, int V>
static void norm_width(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    switch (a.act) {
    case NMS_ACT_RELU: return norm_act<T, V, NMS_ACT_RELU>(a, ws, st, grad);
    case NMS_ACT_SILU: return norm_act<T, V, NMS_ACT_SILU>(a, ws, st, grad);
    case NMS_ACT_GELU: return norm_act<T, V, NMS_ACT_GELU>(a, ws, st, grad);
    default: return norm_act<T, V, NMS_ACT_NONE>(a, ws, st, grad);
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

static void norm_any(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    if (a.type == NMS_TYPE_F32) norm_type<float>(a, ws, st, grad);
    else if (a.type == NMS_TYPE_F16) norm_type<__half>(a, ws, st, grad);
    else norm_type<__nv_bfloat16>(a, ws, st, grad);
}

void launch_norm(const NormArgs& a, void* workspace, cudaStream_t st) { norm_any(a, workspace, st, false); }
void launch_norm_grad(const NormArgs& a, void* workspace, cudaStream_t st) { norm_any(a, workspace, st, true); }

}  // namespace gbnms
