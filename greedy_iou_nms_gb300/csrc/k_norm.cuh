// Group normalisation of channels-last maps with the affine map, the
// activation and dropout fused into its epilogue, and its gradient.
//
//   u = (x - mean) * rstd, z = u * weight + bias, y = drop(act(z)), the
//   statistics over the pixels and channels of one group of one image;
//   dz = drop(dy) * act'(z), dbias = sum dz, dweight = sum dz * u,
//   dx = rstd * (du - avg(du) - u * avg(du * u)) with du = dz * weight.
//
// Statistics are pieces (count, mean, sum of squared deviations).  A thread
// sums deviations from an origin: the mean of the first row that it sees, moved
// to the mean of all that it has seen after 1, 2, 4, ... batches of rows.  So
// nothing is lost to a mean far above the spread, and an outlier among the
// first values costs a few roundings of its own square (as a fixed origin it
// would add that square for every later value, to be taken off again: up to
// 1 % of rstd over 2048 values).  Pieces are joined in a fixed order, in two
// steps: the mean m of their means, then the deviations d of their means from
// m, M2 = sum of M2_i + n_i d_i^2 - n (avg d)^2.  A piece's mean is a pair
// (high + low), so that d is right to its own size and not to the mean's.
#pragma once

#include <type_traits>

#include "head.cuh"
#include "internal.h"

namespace gbnms {

constexpr int NT = 256;  // threads of a block

// ---------------------------------------------------------------- streaming
//
// Large maps in two launches: sums by rows' pieces; then their join (every
// block for its own groups: some kilobytes from L2 and a launch less; images
// of many pieces in a launch of its own) and the results.  The second reading
// comes from L2 as far as that holds the map: the last launch goes through the
// pieces backwards.

// Rows of a piece, at most: 256 of a thread, whose sums by channel are chains
// of so many additions (sums by group: 64 batches of 32 values, each added up
// on its own).
constexpr int MOST_ROWS = 1024;

// Row pieces of an image, at most: 32 rows each at least, and one wave of
// four blocks on every SM, more where MOST_ROWS asks for it (a function of
// the shape alone: the workspace's size depends on it).
inline int64_t norm_pieces(int64_t batch, int64_t pixels, int channels)
{
    const int64_t tiles = channels > 256 ? channels / 256 : 1, ctas = SMS * 4;
    const int64_t by_rows = (pixels + 31) / 32, by_ctas = ctas / (batch * tiles);
    const int64_t p = by_rows < by_ctas ? by_rows : by_ctas, least = (pixels + MOST_ROWS - 1) / MOST_ROWS;
    return p < least ? least : p;
}

// Scratch: four partial planes [batch][pieces][channels] (forward: mean high,
// M2, mean low; gradient: two sums by channel, two by column), two of
// [batch][channels] (the cluster gradient's sums of an image) and two of
// [batch][groups] (joined values).
struct NormScratch {
    float *pa, *pb, *pc, *pd, *ca, *cb, *ga, *gb;
};

// Columns of an image's pieces, for one group, that each block may join
// itself; more are joined in a launch of their own (with 608 pieces of one
// image the blocks' own joins took 40 us).
constexpr int OWN_JOIN = 96;

inline NormScratch scratch(const NormArgs& a, void* ws)
{
    NormScratch s;
    const size_t image = static_cast<size_t>(a.batch) * a.channels;
    const size_t plane = image * norm_pieces(a.batch, a.pixels, a.channels);
    s.pa = static_cast<float*>(ws);
    s.pb = s.pa + plane;
    s.pc = s.pb + plane;
    s.pd = s.pc + plane;
    s.ca = s.pd + plane;
    s.cb = s.ca + image;
    s.ga = s.cb + image;
    s.gb = s.ga + static_cast<size_t>(a.batch) * a.groups;
    return s;
}

// Tile of a block: `wide` vectors of V channels by NT / wide rows at a time.
struct NormTile {
    int wide;    // vectors a row of the tile
    int tiles;   // tiles a row of the map
    int pieces;  // of an image
    int per;     // rows a piece
    int values;  // channels of a column of the partial planes: a vector's (of one group), one, or a group's
};

// A sum of squares that rounding took below 0 is 0; a NaN (an infinity in the
// group) stays one.
__device__ __forceinline__ float not_below_0(float x) { return x < 0.0f ? 0.0f : x; }

template <typename T, int V>
__device__ __forceinline__ void widen(float (&v)[V], const Pack<T, V>& q)
{
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(q.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&v)[V])
{
    *reinterpret_cast<Pack<T, V>*>(p) = pack_results<T, V>(v);
}

// Where a thread stands: image, row range of the piece, first channel.
struct Spot {
    int64_t image;
    int piece, row, row_end;
    int channel, tx, ty, rows;
    bool in;
};

template <int V>
__device__ __forceinline__ Spot spot(const NormArgs& a, const NormTile& t, unsigned block)
{
    Spot s;
    s.image = block / static_cast<unsigned>(t.pieces);
    s.piece = static_cast<int>(block % static_cast<unsigned>(t.pieces));
    s.rows = NT / t.wide;
    s.tx = static_cast<int>(threadIdx.x) % t.wide;
    s.ty = static_cast<int>(threadIdx.x) / t.wide;
    s.channel = (static_cast<int>(blockIdx.y) * t.wide + s.tx) * V;
    s.in = s.ty < s.rows && s.channel < a.channels;
    const int pixels = static_cast<int>(a.pixels);
    s.row = s.piece * t.per < pixels ? s.piece * t.per : pixels;
    s.row_end = s.row + t.per < pixels ? s.row + t.per : pixels;
    return s;
}

// Rows that piece number `piece` has.
__device__ __forceinline__ float piece_rows(const NormArgs& a, const NormTile& t, int piece)
{
    const int left = static_cast<int>(a.pixels) - piece * t.per;
    return static_cast<float>(left < t.per ? (left > 0 ? left : 0) : t.per);
}

// f(vectors..., index in the result) for a thread's rows, B of them loaded
// before the first is worked on.
template <int B, typename T, int V, typename F>
__device__ __forceinline__ void each_row(const NormArgs& a, const Spot& p, F f)
{
    int n = (p.row_end - p.row - p.ty + p.rows - 1) / p.rows;  // rows of this thread; below 1 for none
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + (p.row + p.ty) * a.x_pixel + p.channel;
    const int64_t stride = p.rows * a.x_pixel, advance = static_cast<int64_t>(p.rows) * a.channels;
    int64_t at = (p.image * a.pixels + p.row + p.ty) * a.channels + p.channel;
    for (; n >= B; n -= B) {
        Pack<T, V> q[B];
#pragma unroll
        for (int k = 0; k < B; ++k, x += stride) q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
#pragma unroll
        for (int k = 0; k < B; ++k, at += advance) f(q[k], at);
    }
    Pack<T, V> q[B];
#pragma unroll
    for (int k = 0; k < B - 1; ++k, x += stride)
        if (k < n) q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
#pragma unroll
    for (int k = 0; k < B - 1; ++k, at += advance)
        if (k < n) f(q[k], at);
}

template <int B, typename T, int V, typename F>
__device__ __forceinline__ void each_row_pair(const NormArgs& a, const Spot& p, F f)
{
    int n = (p.row_end - p.row - p.ty + p.rows - 1) / p.rows;
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + (p.row + p.ty) * a.x_pixel + p.channel;
    const T* dy = static_cast<const T*>(a.dy) + p.image * a.dy_image + (p.row + p.ty) * a.dy_pixel + p.channel;
    const int64_t stride = p.rows * a.x_pixel, dstride = p.rows * a.dy_pixel;
    const int64_t advance = static_cast<int64_t>(p.rows) * a.channels;
    int64_t at = (p.image * a.pixels + p.row + p.ty) * a.channels + p.channel;
    for (; n >= B; n -= B) {
        Pack<T, V> q[B], d[B];
#pragma unroll
        for (int k = 0; k < B; ++k, x += stride, dy += dstride) {
            q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
            d[k] = *reinterpret_cast<const Pack<T, V>*>(dy);
        }
#pragma unroll
        for (int k = 0; k < B; ++k, at += advance) f(q[k], d[k], at);
    }
    Pack<T, V> q[B], d[B];
#pragma unroll
    for (int k = 0; k < B - 1; ++k, x += stride, dy += dstride)
        if (k < n) {
            q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
            d[k] = *reinterpret_cast<const Pack<T, V>*>(dy);
        }
#pragma unroll
    for (int k = 0; k < B - 1; ++k, at += advance)
        if (k < n) f(q[k], d[k], at);
}

// f(B vectors, how many of them are rows) for a thread's rows, all loaded
// before f; the count is a constant but for the last.
template <int B, typename T, int V, typename F>
__device__ __forceinline__ void each_batch(const NormArgs& a, const Spot& p, F f)
{
    int n = (p.row_end - p.row - p.ty + p.rows - 1) / p.rows;  // rows of this thread; below 1 for none
    const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + (p.row + p.ty) * a.x_pixel + p.channel;
    const int64_t stride = p.rows * a.x_pixel;
    Pack<T, V> q[B];
    for (; n >= B; n -= B) {
#pragma unroll
        for (int k = 0; k < B; ++k, x += stride) q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
        f(q, B);
    }
#pragma unroll
    for (int k = 0; k < B - 1; ++k, x += stride)
        if (k < n) q[k] = *reinterpret_cast<const Pack<T, V>*>(x);
    if (n > 0) f(q, n);
}

// Running sums of a thread's deviations and their squares, by channel of its
// vector or (ONE) of the whole vector.
template <int V, bool ONE>
struct Moments {
    static constexpr int P = ONE ? 1 : V;
    float origin[P], s[P], q[P];
    int rows, moves_at;  // rows so far; the origin moves when there are so many
    float each;          // 1 / values of moves_at rows

    __device__ __forceinline__ Moments()
    {
#pragma unroll
        for (int i = 0; i < P; ++i) origin[i] = s[i] = q[i] = 0.0f;
        rows = moves_at = 0;
    }

    template <typename T, int B>
    __device__ __forceinline__ void add(const Pack<T, V> (&pack)[B], int n)
    {
        if (rows == 0) {
            float v[V];
            widen(v, pack[0]);
#pragma unroll
            for (int i = 0; i < P; ++i) origin[i] = v[i];
            if (ONE) {  // equal values give exactly that mean
                float d = 0.0f;
#pragma unroll
                for (int i = 1; i < V; ++i) d += v[i] - v[0];
                origin[0] += d * (1.0f / V);
            }
            moves_at = B;
            each = 1.0f / (B * (ONE ? V : 1));
        }
        float row_s[B], row_q[B];  // ONE: of each row, added up in pairs
#pragma unroll
        for (int k = 0; k < B; ++k) {
            row_s[k] = row_q[k] = 0.0f;
            if (k >= n) continue;
            float v[V];
            widen(v, pack[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[i] - origin[ONE ? 0 : i];
                float &to_s = ONE ? row_s[k] : s[ONE ? 0 : i], &to_q = ONE ? row_q[k] : q[ONE ? 0 : i];
                to_s += d;
                to_q = fmaf(d, d, to_q);
            }
        }
        if (ONE) {
            static_assert(B == 4, "pairs of rows");
            s[0] += (row_s[0] + row_s[1]) + (row_s[2] + row_s[3]);
            q[0] += (row_q[0] + row_q[1]) + (row_q[2] + row_q[3]);
        }
        rows += n;
        if (rows != moves_at) return;
        const float values = static_cast<float>(rows * (ONE ? V : 1));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float to = fmaf(s[i], each, origin[i]), d = to - origin[i];  // as far as it moves
            q[i] = fmaf(d, fmaf(values, d, -2.0f * s[i]), q[i]);
            s[i] = fmaf(-values, d, s[i]);
            origin[i] = to;
        }
        moves_at *= 2;
        each *= 0.5f;
    }
};

// (mean, squared deviations) of each row piece by column: a vector (ONE: its
// channels are of one group) or a channel.  Three operations a value; four
// rows' loads in flight a thread, 32 warps an SM (24 where eight channels'
// moments are kept).  16 x 6400 x 256 bf16: 13 us under the profiler, 4.0 TB/s;
// the block's ramps (a first load, the join) are a third of it.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(NT, ONE || V < 8 ? 4 : 3)
norm_partial_kernel(NormArgs a, NormTile t, NormScratch w)
{
    constexpr int P = ONE ? 1 : V;
    __shared__ float s_high[NT * P], s_low[NT * P], s_m2[NT * P];
    __shared__ int s_count[NT];
    pdl_release();
    const Spot p = spot<V>(a, t, blockIdx.x);
    Moments<V, ONE> sums;
    if (p.in)
        each_batch<4, T, V>(a, p, [&](const Pack<T, V>(&pack)[4], int rows) { sums.template add<T, 4>(pack, rows); });
    if (p.ty < p.rows) {
        const int count = sums.rows * (ONE ? V : 1);
        s_count[threadIdx.x] = count;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float m = count ? sums.s[i] / count : 0.0f;
            s_high[threadIdx.x * P + i] = sums.origin[i];
            s_low[threadIdx.x * P + i] = m;
            s_m2[threadIdx.x * P + i] = not_below_0(sums.q[i] - sums.s[i] * m);
        }
    }
    __syncthreads();
    const int width = t.wide * P, columns = a.channels / (ONE ? V : 1);
    const bool by_group = t.values > (ONE ? V : 1);
    for (int c = threadIdx.x; c < width; c += NT) {
        const int column = static_cast<int>(blockIdx.y) * width + c;
        if (column >= columns) continue;
        float n = 0.0f, mean = 0.0f, low = 0.0f, m2 = 0.0f;
        for (int y = 0; y < p.rows; ++y) n += static_cast<float>(s_count[y * t.wide + c / P]);
        if (n == 0.0f) n = 1.0f;
        const float origin = s_high[c], each = 1.0f / n;  // equal values give exactly that mean
        for (int y = 0; y < p.rows; ++y) {
            const int at = y * width + c;
            mean = fmaf(static_cast<float>(s_count[y * t.wide + c / P]) * each, s_high[at] + s_low[at] - origin, mean);
        }
        mean += origin;
        for (int y = 0; y < p.rows; ++y) {
            const int at = y * width + c;
            const float k = static_cast<float>(s_count[y * t.wide + c / P]), d = (s_high[at] - mean) + s_low[at];
            low = fmaf(k, d, low);
            m2 += fmaf(k * d, d, s_m2[at]);
        }
        low *= each;
        m2 = not_below_0(m2 - n * low * low);
        if (by_group) {  // entry c has been read by this thread alone
            s_high[c] = mean;
            s_low[c] = low;
            s_m2[c] = m2;
        } else {
            const int64_t at = (p.image * t.pieces + p.piece) * static_cast<int64_t>(columns) + column;
            w.pa[at] = mean;
            w.pb[at] = m2;
            w.pc[at] = low;
        }
    }
    if (!by_group) return;
    // The tile holds every channel: the columns of a group, alike in count, become one piece.
    __syncthreads();
    const int each = t.values / (ONE ? V : 1);
    const float n = static_cast<float>(p.row_end - p.row) * (ONE ? V : 1), share = 1.0f / each;
    for (int g = threadIdx.x; g < a.groups; g += NT) {
        const float origin = s_high[g * each];
        float mean = 0.0f, low = 0.0f, m2 = 0.0f;
        for (int c = g * each; c < (g + 1) * each; ++c) mean += s_high[c] + s_low[c] - origin;
        mean = fmaf(mean, share, origin);
        for (int c = g * each; c < (g + 1) * each; ++c) {
            const float d = (s_high[c] - mean) + s_low[c];
            low += d;
            m2 += fmaf(n * d, d, s_m2[c]);
        }
        low *= share;
        const int64_t at = (p.image * t.pieces + p.piece) * a.groups + g;
        w.pa[at] = mean;
        w.pb[at] = not_below_0(m2 - n * each * low * low);
        w.pc[at] = low;
    }
}

// Groups that a tile meets, and the threads (a power of two) that join each
// one's pieces.
struct Joint {
    int first, groups, team;
};

template <int V>
__device__ __forceinline__ Joint joint(const NormArgs& a, const NormTile& t)
{
    Joint j;
    const int D = a.channels / a.groups, c0 = static_cast<int>(blockIdx.y) * t.wide * V;
    const int c1 = c0 + t.wide * V < a.channels ? c0 + t.wide * V : a.channels;
    j.first = c0 / D;
    j.groups = (c1 - 1) / D - j.first + 1;
    for (j.team = NT; j.team > 1 && j.team * j.groups > NT; j.team /= 2) {}
    return j;
}

// Sum over each team of a block; every thread calls it.  s: 8 floats.
__device__ __forceinline__ float team_sum(float v, int team, float* s)
{
    for (int o = (team < 32 ? team : 32) / 2; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    if (team > 32) {
        __syncthreads();
        if (lane_id() == 0) s[threadIdx.x / 32] = v;
        __syncthreads();
        const int warps = team / 32, first = static_cast<int>(threadIdx.x) / team * warps;
        v = 0.0f;
        for (int k = 0; k < warps; ++k) v += s[first + k];
    }
    return v;
}

constexpr int MOST_GROUPS = 64 * 8;  // that a tile meets

// mean and rstd of the tile's groups from the pieces (their geometry: from)
// into s_mean, s_rstd; the first piece's block of the tile that holds a
// group's first channel writes them out.
__device__ __forceinline__ void join_moments(const NormArgs& a, const NormTile& from, const Spot& p,
                                             const NormScratch& w, const Joint& j, int first_channel, float* s_mean,
                                             float* s_rstd)
{
    __shared__ float red[NT / 32];
    const int D = a.channels / a.groups, values = from.values, each = D / values, columns = a.channels / values;
    const int items = from.pieces * each, lane = static_cast<int>(threadIdx.x) % j.team;
    const float all = static_cast<float>(a.pixels) * static_cast<float>(D), each_all = 1.0f / all;
    for (int k0 = 0; k0 < j.groups; k0 += NT / j.team) {
        const int k = k0 + static_cast<int>(threadIdx.x) / j.team, g = j.first + (k < j.groups ? k : 0);
        const int64_t base = p.image * from.pieces * columns + static_cast<int64_t>(g) * each;
        // Deviations of the pieces' means from the first piece's: equal means give exactly that mean.
        const float origin = w.pa[base];
        float mean = 0.0f, low = 0.0f, m2 = 0.0f;
#pragma unroll 4
        for (int i = lane; i < items; i += j.team) {
            const int piece = i / each;
            const float n = piece_rows(a, from, piece) * values;
            const float high = w.pa[base + static_cast<int64_t>(piece) * columns + (i - piece * each)];
            if (n > 0.0f) mean = fmaf(high - origin, n * each_all, mean);
        }
        mean = origin + team_sum(mean, j.team, red);
#pragma unroll 4
        for (int i = lane; i < items; i += j.team) {
            const int piece = i / each;
            const int64_t at = base + static_cast<int64_t>(piece) * columns + (i - piece * each);
            const float n = piece_rows(a, from, piece) * values, d = (w.pa[at] - mean) + w.pc[at], m = w.pb[at];
            if (n > 0.0f) {
                low = fmaf(d, n * each_all, low);
                m2 += fmaf(d * n, d, m);
            }
        }
        low = team_sum(low, j.team, red);
        m2 = team_sum(m2, j.team, red);
        if (lane == 0 && k < j.groups) {
            const float m = mean + low, r = 1.0f / sqrtf(not_below_0(m2 / all - low * low) + a.eps);
            s_mean[k] = m;
            s_rstd[k] = r;
            if (p.piece == 0 && g * D >= first_channel) {
                if (a.mean) a.mean[p.image * a.groups + g] = m;
                if (a.rstd) a.rstd[p.image * a.groups + g] = r;
            }
        }
    }
    __syncthreads();
}

// The joined values of the tile's groups, from two planes [batch][groups].
__device__ __forceinline__ void load_joined(const NormArgs& a, const Spot& p, const Joint& j, const float* from_a,
                                            const float* from_b, float* s_a, float* s_b)
{
    for (int k = threadIdx.x; k < j.groups; k += NT) {
        s_a[k] = from_a[p.image * a.groups + j.first + k];
        s_b[k] = from_b[p.image * a.groups + j.first + k];
    }
    __syncthreads();
}

// The results.  16 x 6400 x 256 bf16, silu: 21 us of the two launches' 34, for 52
// MB read again and as much written; the sigmoid's two hardware functions a value take 11 us of their
// pipe, and three blocks an SM (80 registers) hide what latency they can.
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(NT, 3)
norm_apply_kernel(NormArgs a, NormTile t, NormTile from, NormScratch w, bool joined)
{
    constexpr int P = ONE ? 1 : V;
    __shared__ float s_mean[MOST_GROUPS], s_rstd[MOST_GROUPS];
    const Spot p = spot<V>(a, t, gridDim.x - 1 - blockIdx.x);  // the pieces read last come first
    const Joint j = joint<V>(a, t);
    float mean[P], scale[V], shift[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        scale[i] = p.in && a.weight ? load_param<T>(a.weight, a.param_f32, p.channel + i) : 1.0f;
        shift[i] = p.in && a.bias ? load_param<T>(a.bias, a.param_f32, p.channel + i) : 0.0f;
    }
    pdl_wait();
    if (joined) load_joined(a, p, j, a.mean, a.rstd, s_mean, s_rstd);
    else join_moments(a, from, p, w, j, static_cast<int>(blockIdx.y) * t.wide * V, s_mean, s_rstd);
    if (!p.in) return;
    const int D = a.channels / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int g = (p.channel + i) / D - j.first;
        if (i < P) mean[i] = s_mean[g];
        scale[i] *= s_rstd[g];
    }
    T* y = static_cast<T*>(a.out);
    const bool dropping = a.drop.limit < 65536u;
    each_row<4, T, V>(a, p, [&](const Pack<T, V>& q, int64_t at) {
        float v[V];
        widen(v, q);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(v[i] - mean[ONE ? 0 : i], scale[i], shift[i]);
        act_values<T, V>(v, ACT);
        if (dropping) drop<V>(v, static_cast<uint64_t>(at), a.drop);
        store_row<T, V>(y + at, v);
    });
}

// The factors of a thread's channels: z = (x - mean) * scale + bias.
template <typename T, int V, int P>
__device__ __forceinline__ void load_channels(const NormArgs& a, const Spot& p, float (&mean)[P], float (&scale)[V],
                                              float (&bias)[V])
{
    const int D = a.channels / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = p.image * a.groups + (p.channel + i) / D;
        if (i < P) mean[i] = a.mean[g];
        scale[i] = a.rstd[g] * (a.weight ? load_param<T>(a.weight, a.param_f32, p.channel + i) : 1.0f);
        bias[i] = a.bias ? load_param<T>(a.bias, a.param_f32, p.channel + i) : 0.0f;
    }
}

// x - mean, and dz but for the dropout's factor, of one vector.
template <int ACT, typename T, int V, int P>
__device__ __forceinline__ void slope_row(const NormArgs& a, const float (&mean)[P], const float (&scale)[V],
                                          const float (&bias)[V], const Pack<T, V>& x, const Pack<T, V>& dy,
                                          uint64_t at, float (&d)[V], float (&dz)[V])
{
    float z[V];
    widen(d, x);
    widen(dz, dy);
    if (a.drop.limit < 65536u) drop_mask<V>(dz, at, a.drop);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        d[i] -= mean[P == 1 ? 0 : i];
        z[i] = fmaf(d[i], scale[i], bias[i]);
    }
    act_slopes<T, V>(dz, z, ACT);
}

// Sums by channel of dz and dz * (x - mean) of each row piece.  16 x 1600 x 256
// bf16, silu: 14 us under the profiler, latency (seven rows a thread).  8 x 25600
// x 128 fp16, gelu and dropout: 41 us, 35 instructions a value at 16 warps an SM;
// two values an instruction changed nothing.
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(NT, ONE ? 3 : 2)
norm_grad_partial_kernel(NormArgs a, NormTile t, NormScratch w)
{
    constexpr int P = ONE ? 1 : V;
    __shared__ float s_a[NT * V], s_b[NT * V];
    pdl_release();
    const Spot p = spot<V>(a, t, blockIdx.x);
    float sa[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sa[i] = sb[i] = 0.0f;
    if (p.in) {
        float mean[P], scale[V], bias[V];
        load_channels<T, V, P>(a, p, mean, scale, bias);
        each_row_pair<2, T, V>(a, p, [&](const Pack<T, V>& x, const Pack<T, V>& dy, int64_t at) {
            float d[V], dz[V];
            slope_row<ACT>(a, mean, scale, bias, x, dy, static_cast<uint64_t>(at), d, dz);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sa[i] += dz[i];
                sb[i] = fmaf(dz[i], d[i], sb[i]);
            }
        });
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s_a[threadIdx.x * V + i] = sa[i];
        s_b[threadIdx.x * V + i] = sb[i];
    }
    __syncthreads();
    const float factor = a.drop.limit < 65536u ? a.drop.factor : 1.0f;
    for (int c = threadIdx.x; c < t.wide * V; c += NT) {
        const int channel = static_cast<int>(blockIdx.y) * t.wide * V + c;
        if (channel >= a.channels) continue;
        float va = 0.0f, vb = 0.0f;
        for (int y = 0; y < p.rows; ++y) {
            va += s_a[y * t.wide * V + c];
            vb += s_b[y * t.wide * V + c];
        }
        va *= factor;
        vb *= factor;
        const int64_t at = (p.image * t.pieces + p.piece) * static_cast<int64_t>(a.channels) + channel;
        w.pa[at] = va;
        w.pb[at] = vb;
        // For the groups: by column, times the weights.
        const float weight = a.weight ? load_param<T>(a.weight, a.param_f32, channel) : 1.0f;
        s_a[c] = va * weight;  // read by this thread alone so far
        s_b[c] = vb * weight;
    }
    __syncthreads();
    const int width = t.wide * V / t.values, columns = a.channels / t.values;
    for (int c = threadIdx.x; c < width; c += NT) {
        const int column = static_cast<int>(blockIdx.y) * width + c;
        if (column >= columns) continue;
        float va = 0.0f, vb = 0.0f;
        for (int i = 0; i < t.values; ++i) {
            va += s_a[c * t.values + i];
            vb += s_b[c * t.values + i];
        }
        const int64_t at = (p.image * t.pieces + p.piece) * static_cast<int64_t>(columns) + column;
        w.pc[at] = va;
        w.pd[at] = vb;
    }
}

// Sums of du and du * (x - mean) of the tile's groups from the pieces.
__device__ __forceinline__ void join_sums(const NormArgs& a, const NormTile& from, const Spot& p, const NormScratch& w,
                                          const Joint& j, float* s_a, float* s_b)
{
    __shared__ float red[NT / 32];
    const int D = a.channels / a.groups, each = D / from.values, columns = a.channels / from.values;
    const int items = from.pieces * each, lane = static_cast<int>(threadIdx.x) % j.team;
    for (int k0 = 0; k0 < j.groups; k0 += NT / j.team) {
        const int k = k0 + static_cast<int>(threadIdx.x) / j.team, g = j.first + (k < j.groups ? k : 0);
        const int64_t base = p.image * from.pieces * columns + static_cast<int64_t>(g) * each;
        float va = 0.0f, vb = 0.0f;
#pragma unroll 4
        for (int i = lane; i < items; i += j.team) {
            const int piece = i / each;
            const int64_t at = base + static_cast<int64_t>(piece) * columns + (i - piece * each);
            va += w.pc[at];
            vb += w.pd[at];
        }
        va = team_sum(va, j.team, red);
        vb = team_sum(vb, j.team, red);
        if (lane == 0 && k < j.groups) {
            s_a[k] = va;
            s_b[k] = vb;
        }
    }
    __syncthreads();
}

// The join in a launch of its own: a block for each (image, group).
template <bool GRAD>
__global__ void __launch_bounds__(NT)
norm_join_kernel(NormArgs a, NormTile from, NormScratch w)
{
    __shared__ float s_a[1], s_b[1];
    pdl_wait();
    pdl_release();
    const unsigned G = static_cast<unsigned>(a.groups);
    Spot p{};
    p.image = blockIdx.x / G;
    const Joint j{static_cast<int>(blockIdx.x % G), 1, NT};
    if (!GRAD) {
        join_moments(a, from, p, w, j, 0, s_a, s_b);
    } else {
        join_sums(a, from, p, w, j, s_a, s_b);
        if (threadIdx.x == 0) {
            w.ga[blockIdx.x] = s_a[0];
            w.gb[blockIdx.x] = s_b[0];
        }
    }
}

constexpr int PARAMS = 8;  // channels of a block that sums dweight and dbias

// dweight and dbias of PARAMS channels from every image's pieces: 32 threads a
// channel, joined in order.
__device__ __forceinline__ void param_pieces(const NormArgs& a, const NormTile& from, const NormScratch& w, int c0)
{
    __shared__ LongSum s_a[NT], s_b[NT];
    const int x = static_cast<int>(threadIdx.x) % PARAMS, y = static_cast<int>(threadIdx.x) / PARAMS, c = c0 + x;
    LongSum va{}, vb{};
    if (c < a.channels) {
        const unsigned items = static_cast<unsigned>(a.batch) * from.pieces, pieces = from.pieces;
        const int g = c / (a.channels / a.groups);
#pragma unroll 4
        for (unsigned i = y; i < items; i += NT / PARAMS) {
            const int64_t at = static_cast<int64_t>(i) * a.channels + c;
            va.add(w.pa[at]);
            // u = (x - mean) * rstd
            vb.add(__fmul_rn(w.pb[at], a.rstd[static_cast<int64_t>(i / pieces) * a.groups + g]));
        }
    }
    s_a[threadIdx.x] = va;
    s_b[threadIdx.x] = vb;
    __syncthreads();
    if (y == 0 && c < a.channels) {
        for (int k = 1; k < NT / PARAMS; ++k) {
            va.add(s_a[k * PARAMS + x]);
            vb.add(s_b[k * PARAMS + x]);
        }
        if (a.dbias) a.dbias[c] = va.value();
        if (a.dweight) a.dweight[c] = vb.value();
    }
}

// dweight and dbias of channel c: the sums of at most 16 images, added in order.
__device__ __forceinline__ void param_sums(const NormArgs& a, const float* ca, const float* cb, int c)
{
    float va = 0.0f, vb = 0.0f;
    for (int64_t n = 0; n < a.batch; ++n) {
        va += ca[n * a.channels + c];
        vb += cb[n * a.channels + c];
    }
    if (a.dbias) a.dbias[c] = va;
    if (a.dweight) a.dweight[c] = vb;
}

static __global__ void __launch_bounds__(NT)
norm_grad_param_kernel(NormArgs a, NormScratch w)
{
    pdl_wait();
    const int c = static_cast<int>(blockIdx.x) * NT + static_cast<int>(threadIdx.x);
    if (c < a.channels) param_sums(a, w.ca, w.cb, c);
}

// dx; the blocks past the pieces' (the first to run) write dweight and dbias.
// dz is worked out again: keeping it would move 8 bytes a value more.  17 us and
// 50 us under the profiler at the sizes above, 25 and 85 for both launches without.
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(NT, ONE ? 3 : 2)
norm_grad_apply_kernel(NormArgs a, NormTile t, NormTile from, NormScratch w, bool joined)
{
    constexpr int P = ONE ? 1 : V;
    __shared__ float s_a[MOST_GROUPS], s_b[MOST_GROUPS];
    const unsigned block = gridDim.x - 1 - blockIdx.x, main = static_cast<unsigned>(a.batch) * t.pieces;
    if (block >= main) {
        pdl_wait();
        if (blockIdx.y == 0) param_pieces(a, from, w, static_cast<int>(block - main) * PARAMS);
        return;
    }
    const Spot p = spot<V>(a, t, block);
    const Joint j = joint<V>(a, t);
    float mean[P], scale[V], bias[V], m1[P], m2[P];
    if (p.in) load_channels<T, V, P>(a, p, mean, scale, bias);
    pdl_wait();
    if (joined) load_joined(a, p, j, w.ga, w.gb, s_a, s_b);
    else join_sums(a, from, p, w, j, s_a, s_b);
    if (!p.in) return;
    const int D = a.channels / a.groups;
    const float each_all = 1.0f / (static_cast<float>(a.pixels) * static_cast<float>(D));
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int g = (p.channel + i) / D;
        const float r = a.rstd[p.image * a.groups + g];
        m1[i] = -r * s_a[g - j.first] * each_all;
        m2[i] = -(r * s_b[g - j.first] * each_all) * r * r;  // r^3 leaves binary32 where this does not
    }
    each_row_pair<2, T, V>(a, p, [&](const Pack<T, V>& x, const Pack<T, V>& dy, int64_t at) {
        float d[V], dz[V];
        slope_row<ACT>(a, mean, scale, bias, x, dy, static_cast<uint64_t>(at), d, dz);
        if (a.drop.limit < 65536u) {
#pragma unroll
            for (int i = 0; i < V; ++i) dz[i] *= a.drop.factor;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            dz[i] = fmaf(dz[i], scale[i], fmaf(d[i], m2[ONE ? 0 : i], m1[ONE ? 0 : i]));
        store_row<T, V>(static_cast<T*>(a.out) + at, dz);
    });
}

// ------------------------------------------------------------------- clusters
//
// Where one image's slab of whole groups (a few dozen channels of every
// pixel) fits the shared memory of a cluster, it is read once: each block
// keeps its rows, every thread the vectors that it copied itself, the blocks
// exchange their sums through distributed shared memory, and the results are
// written from what they keep.  Small blocks (several to an SM) overlap one's
// loads with another's sums and stores.

// Tile of a cluster: `wide` vectors of V channels (whole groups), the rows
// split over `ctas` blocks of `rows` each.
struct NormCluster {
    int wide, tiles, ctas;
    int rows;
    int groups;     // of a tile, at most NT
    bool shuffles;  // rows and groups are powers of two of lanes
    int held;       // vectors that a thread keeps, at most
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Asynchronous copy of one vector into shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src)
{
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(at), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(at), "l"(src), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// *p of the block `rank` of the cluster = v.
__device__ __forceinline__ void peer_store(float* p, int rank, float v)
{
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at), "f"(v) : "memory");
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

// Sums by group over a block.  Each thread gives N sums for each of its P
// parts (P = 1: its vector lies in one group).  Where rows of the tile and
// groups are powers of two of lanes, lanes of one group join by shuffles and
// the warps' sums by one pass through shared memory; else every thread's
// parts go there and a warp adds up each group.
struct GroupSums {
    float* part;  // [N][NT * P], or [N][8][32]
    float* out;   // [N][groups], groups <= plane
    int wide, each, steps, groups, plane;  // `each` parts of a row of the tile belong to a group
    bool shuffles;

    template <int N, int P>
    __device__ __forceinline__ void operator()(const float (&v)[N][P], const ClusterSpot& p)
    {
        if (P == 1 && shuffles) {
            float u[N];
#pragma unroll
            for (int q = 0; q < N; ++q) {
                u[q] = v[q][0];
                for (int o = 16; o >= wide; o >>= 1) u[q] += __shfl_xor_sync(FULL, u[q], o);
                for (int o = each / 2; o; o >>= 1) u[q] += __shfl_xor_sync(FULL, u[q], o);
            }
            const int lane = static_cast<int>(lane_id());
            if (lane < wide && lane % each == 0)
#pragma unroll
                for (int q = 0; q < N; ++q) part[q * NT + threadIdx.x / 32 * 32 + lane / each] = u[q];
            __syncthreads();
            for (int k = threadIdx.x; k < N * groups; k += NT) {
                const int q = k / groups, g = k % groups;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < NT / 32; ++w) s += part[q * NT + w * 32 + g];
                out[q * plane + g] = s;
            }
            __syncthreads();
            return;
        }
        if (p.ty < steps) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int i = 0; i < P; ++i) part[q * NT * P + (p.ty * wide + p.tx) * P + i] = v[q][i];
        }
        __syncthreads();
        for (int g = static_cast<int>(threadIdx.x) / 32; g < groups; g += NT / 32) {
            float s[N];
#pragma unroll
            for (int q = 0; q < N; ++q) s[q] = 0.0f;
            int y = static_cast<int>(lane_id()) / each, x = static_cast<int>(lane_id()) % each;
            const int dy = 32 / each, dx = 32 % each;
            while (y < steps) {
                const int at = y * wide * P + g * each + x;
#pragma unroll
                for (int q = 0; q < N; ++q) s[q] += part[q * NT * P + at];
                y += dy;
                x += dx;
                if (x >= each) {
                    x -= each;
                    ++y;
                }
            }
#pragma unroll
            for (int q = 0; q < N; ++q) {
                s[q] = warp_sum(s[q]);
                if (lane_id() == 0) out[q * plane + g] = s[q];
            }
        }
        __syncthreads();
    }
};

// ONE: a vector lies in one group (its channels' sums are one).  Two readings
// from shared memory for the moments (the second about the block's mean), one
// for the results; one exchange.  1 x 400 x 256 bf16: 5.8 us with its launch,
// latency.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(NT, 4)
norm_cluster_kernel(NormArgs a, NormCluster t)
{
    constexpr int P = ONE ? 1 : V;  // partial sums of a thread
    extern __shared__ uint4 smem[];
    const int CW = t.wide * V, D = a.channels / a.groups, G = t.groups;
    Pack<T, V>* keep = reinterpret_cast<Pack<T, V>*>(smem) + threadIdx.x;  // [held][NT]
    float* part = reinterpret_cast<float*>(reinterpret_cast<Pack<T, V>*>(smem) + t.held * NT);  // [2][NT * P]
    float* s_weight = part + 2 * NT * P;  // [CW]
    float* s_bias = s_weight + CW;        // [CW]
    float* s_sum = s_bias + CW;           // [2][G]: sums by group
    float* s_piece = s_sum + 2 * G;       // [ctas][3][G]: the blocks' means (high, low) and squares by group
    float* s_mean = s_piece + 3 * t.ctas * G;  // [G]: the image's, by group
    float* s_rstd = s_mean + G;
    const ClusterSpot p = cluster_spot<V>(a, t, D);
    if (t.ctas > 1) cluster_arrive();  // every block has begun: waited for before the first store to a peer
    const int first = p.in ? p.row0 + p.ty : p.row_end;  // a thread outside the map has no rows
    {
        const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + first * a.x_pixel + p.channel;
        const int64_t stride = p.step * a.x_pixel;
        Pack<T, V>* to = keep;
        for (int r = first; r < p.row_end; r += p.step, x += stride, to += NT) copy_async<sizeof(T) * V>(to, x);
    }
    for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
        s_weight[c] = a.weight ? load_param<T>(a.weight, a.param_f32, p.first_channel + c) : 1.0f;
        s_bias[c] = a.bias ? load_param<T>(a.bias, a.param_f32, p.first_channel + c) : 0.0f;
    }
    GroupSums sums{part, s_sum, t.wide, ONE ? D / V : D, p.step, p.groups, G, t.shuffles};
    copies_done();  // a thread reads its own copies alone
    // The block's mean by group, then the deviations from it.
    {
        float s[1][P];
#pragma unroll
        for (int i = 0; i < P; ++i) s[0][i] = 0.0f;
        const Pack<T, V>* from = keep;
#pragma unroll 2
        for (int r = first; r < p.row_end; r += p.step, from += NT) {
            float v[V];
            widen(v, *from);
#pragma unroll
            for (int i = 0; i < V; ++i) s[0][ONE ? 0 : i] += v[i];
        }
        sums.template operator()<1, P>(s, p);
    }
    const float n = static_cast<float>(p.row_end - p.row0) * static_cast<float>(D);
    const float each_n = n > 0.0f ? 1.0f / n : 0.0f;
    float mean_here = 0.0f;  // of the group that this thread publishes
    if (threadIdx.x < p.groups) mean_here = s_sum[threadIdx.x] * each_n;
    {
        float mean[P], s[2][P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            mean[i] = p.in ? s_sum[(p.tx * V + i) / D] * each_n : 0.0f;
            s[0][i] = s[1][i] = 0.0f;
        }
        const Pack<T, V>* from = keep;
#pragma unroll 2
        for (int r = first; r < p.row_end; r += p.step, from += NT) {
            float v[V];
            widen(v, *from);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[i] - mean[ONE ? 0 : i];
                s[0][ONE ? 0 : i] += d;
                s[1][ONE ? 0 : i] = fmaf(d, d, s[1][ONE ? 0 : i]);
            }
        }
        sums.template operator()<2, P>(s, p);
    }
    // Every block's pieces go to every block, which joins them in the same order.
    if (t.ctas > 1) cluster_wait();
    if (threadIdx.x < p.groups) {  // groups <= NT
        const int g = threadIdx.x;
        const float low = s_sum[g] * each_n, m2 = not_below_0(s_sum[G + g] - s_sum[g] * low);
        float* at = s_piece + p.rank * 3 * G + g;
        for (int k = 0; k < t.ctas; ++k) {
            if (t.ctas > 1) {
                peer_store(at, k, mean_here);
                peer_store(at + G, k, low);
                peer_store(at + 2 * G, k, m2);
            } else {
                at[0] = mean_here;
                at[G] = low;
                at[2 * G] = m2;
            }
        }
    }
    if (t.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (threadIdx.x < p.groups) {
        const int g = threadIdx.x;
        const float all = static_cast<float>(a.pixels) * static_cast<float>(D);
        float m = s_piece[g], low = s_piece[G + g], m2 = s_piece[2 * G + g];
        if (t.ctas > 1) {
            const float origin = m, each_all = 1.0f / all;
            float mean = 0.0f;
            auto values = [&](int k) {  // of block k's rows
                const int64_t left = a.pixels - static_cast<int64_t>(k) * t.rows;
                return static_cast<float>(left < t.rows ? (left > 0 ? left : 0) : t.rows) * D;
            };
            for (int k = 1; k < t.ctas; ++k)
                if (values(k) > 0.0f) mean = fmaf(values(k) * each_all, s_piece[k * 3 * G + g] - origin, mean);
            mean += origin;
            low = m2 = 0.0f;
            for (int k = 0; k < t.ctas; ++k) {
                const float w = values(k), d = (s_piece[k * 3 * G + g] - mean) + s_piece[(k * 3 + 1) * G + g];
                if (w == 0.0f) break;
                low = fmaf(d, w * each_all, low);
                m2 += fmaf(d * w, d, s_piece[(k * 3 + 2) * G + g]);
            }
            m2 -= all * low * low;
            m = mean;
        }
        m += low;
        const float r = 1.0f / sqrtf(not_below_0(m2 / all) + a.eps);
        s_mean[g] = m;
        s_rstd[g] = r;
        if (p.rank == 0) {
            const int64_t at = p.image * a.groups + p.first_channel / D + g;
            if (a.mean) a.mean[at] = m;
            if (a.rstd) a.rstd[at] = r;
        }
    }
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
        const int64_t stride = static_cast<int64_t>(p.step) * a.channels;
        int64_t at = (p.image * a.pixels + first) * a.channels + p.channel;
        T* y = static_cast<T*>(a.out) + at;
        const Pack<T, V>* from = keep;
        for (int r = first; r < p.row_end; r += p.step, from += NT, at += stride, y += stride) {
            float v[V];
            widen(v, *from);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = fmaf(v[i] - mean[ONE ? 0 : i], scale[i], shift[i]);
            act_values<T, V>(v, a.act);
            if (a.drop.limit < 65536u) drop<V>(v, static_cast<uint64_t>(at), a.drop);
            store_row<T, V>(y, v);
        }
    }
}

// V numbers of binary32, 16 bytes at a time NT threads apart.
template <int V>
__device__ __forceinline__ void keep_floats(char* at, const float (&v)[V])
{
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        Pack<float, W> q;
#pragma unroll
        for (int j = 0; j < W; ++j) q.v[j] = v[i + j];
        *reinterpret_cast<Pack<float, W>*>(at + (i / W) * NT * W * 4) = q;
    }
}

template <int V>
__device__ __forceinline__ void kept_floats(float (&v)[V], const char* at)
{
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        const Pack<float, W> q = *reinterpret_cast<const Pack<float, W>*>(at + (i / W) * NT * W * 4);
#pragma unroll
        for (int j = 0; j < W; ++j) v[i + j] = q.v[j];
    }
}

// The gradient: x is kept as it came and dz in binary32 (its activation is
// worked out once), in the place that dy was copied to.  The dropout's factor
// is left to the sums and the weights.  Rank 0 writes the image's channel
// sums for dweight and dbias.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(NT, 3)
norm_grad_cluster_kernel(NormArgs a, NormCluster t, NormScratch w)
{
    constexpr int P = ONE ? 1 : V, W = V < 4 ? V : 4;
    constexpr int DZ = NT * V * 4;  // bytes of a pass's dz
    extern __shared__ uint4 smem[];
    const int CW = t.wide * V, D = a.channels / a.groups;
    Pack<T, V>* keep = reinterpret_cast<Pack<T, V>*>(smem) + threadIdx.x;  // [held][NT]
    char* base = reinterpret_cast<char*>(reinterpret_cast<Pack<T, V>*>(smem) + t.held * NT);
    char* keep_dz = base + threadIdx.x * W * 4;                // [held][V / W][NT] of W floats
    float* part = reinterpret_cast<float*>(base + t.held * DZ);  // [2][NT * V]
    float* s_weight = part + 2 * NT * V;  // [CW]
    float* s_bias = s_weight + CW;        // [CW]
    float* s_mine = s_bias + CW;          // [2][CW]: this block's sums by channel
    float* s_image = s_mine + 2 * CW;     // [ctas][2][CW]: the blocks', in rank 0
    float* s_piece = s_image + 2 * t.ctas * CW;  // [ctas][2][G]: the blocks' sums by group, in every block
    const int G = t.groups;
    const ClusterSpot p = cluster_spot<V>(a, t, D);
    if (t.ctas > 1) cluster_arrive();  // every block has begun: waited for before the first store to a peer
    const int first = p.in ? p.row0 + p.ty : p.row_end;  // a thread outside the map has no rows
    {
        const T* x = static_cast<const T*>(a.x) + p.image * a.x_image + first * a.x_pixel + p.channel;
        const T* dy = static_cast<const T*>(a.dy) + p.image * a.dy_image + first * a.dy_pixel + p.channel;
        const int64_t stride = p.step * a.x_pixel, dstride = p.step * a.dy_pixel;
        Pack<T, V>* to = keep;
        char* dto = keep_dz;
        for (int r = first; r < p.row_end; r += p.step) {
            copy_async<sizeof(T) * V>(to, x);
            copy_async<sizeof(T) * V>(dto, dy);
            x += stride;
            dy += dstride;
            to += NT;
            dto += DZ;
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
    const float factor = a.drop.limit < 65536u ? a.drop.factor : 1.0f;
    copies_done();
    __syncthreads();
    float sa[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sa[i] = sb[i] = 0.0f;
    {
        float weight[V], bias[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            weight[i] = s_weight[p.tx * V + i];
            bias[i] = s_bias[p.tx * V + i];
        }
        const int64_t stride = static_cast<int64_t>(p.step) * a.channels;
        int64_t at = (p.image * a.pixels + first) * a.channels + p.channel;
        const Pack<T, V>* from = keep;
        char* dat = keep_dz;
        for (int r = first; r < p.row_end; r += p.step, at += stride, from += NT, dat += DZ) {
            float u[V], z[V], dz[V];
            widen(u, *from);
            widen(dz, *reinterpret_cast<const Pack<T, V>*>(dat));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[i] = (u[i] - mean[ONE ? 0 : i]) * rstd[ONE ? 0 : i];
                z[i] = fmaf(u[i], weight[i], bias[i]);
            }
            if (a.drop.limit < 65536u) drop_mask<V>(dz, static_cast<uint64_t>(at), a.drop);
            act_slopes<T, V>(dz, z, a.act);
            keep_floats<V>(dat, dz);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sa[i] += dz[i];
                sb[i] = fmaf(dz[i], u[i], sb[i]);
            }
        }
    }
    // Sums by channel over the block's rows: lanes of one channel by shuffles
    // where the tile's rows are powers of two of lanes, then `lists` partial
    // sums a channel, then one.
    const bool fast = t.wide <= 32 && (t.wide & (t.wide - 1)) == 0;
    int lists;
    if (fast) {
        lists = NT / 32;
        for (int o = 16; o >= t.wide; o >>= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sa[i] += __shfl_xor_sync(FULL, sa[i], o);
                sb[i] += __shfl_xor_sync(FULL, sb[i], o);
            }
        if (static_cast<int>(lane_id()) < t.wide)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[static_cast<int>(threadIdx.x) / 32 * CW + p.tx * V + i] = sa[i];
                part[NT * V + static_cast<int>(threadIdx.x) / 32 * CW + p.tx * V + i] = sb[i];
            }
    } else {
        lists = CW < NT ? NT / CW : 1;
        if (p.ty < p.step) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[(p.ty * t.wide + p.tx) * V + i] = sa[i];
                part[NT * V + (p.ty * t.wide + p.tx) * V + i] = sb[i];
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < lists * CW; k += NT) {
            float va = 0.0f, vb = 0.0f;
            for (int y = k / CW; y < p.step; y += lists) {
                va += part[y * CW + k % CW];
                vb += part[NT * V + y * CW + k % CW];
            }
            // Entry k is read by this thread alone.
            part[k] = va;
            part[NT * V + k] = vb;
        }
        if (lists > p.step) lists = p.step;
    }
    __syncthreads();
    if (t.ctas > 1) cluster_wait();
    for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
        float va = 0.0f, vb = 0.0f;
        for (int y = 0; y < lists; ++y) {
            va += part[y * CW + c];
            vb += part[NT * V + y * CW + c];
        }
        va *= factor;
        vb *= factor;
        s_mine[c] = va * s_weight[c];
        s_mine[CW + c] = vb * s_weight[c];
        if (t.ctas > 1) {
            peer_store(s_image + p.rank * 2 * CW + c, 0, va);
            peer_store(s_image + (p.rank * 2 + 1) * CW + c, 0, vb);
        } else {
            s_image[c] = va;
            s_image[CW + c] = vb;
        }
    }
    __syncthreads();
    // A thread adds up a small group, a warp a large one.
    const int team = D > 32 ? 32 : 1;
    for (int k = static_cast<int>(threadIdx.x) / team; k < 2 * p.groups; k += NT / team) {
        const int q = k / p.groups, g = k % p.groups, l = static_cast<int>(threadIdx.x) % team;
        float v = 0.0f;
        for (int i = l; i < D; i += team) v += s_mine[q * CW + g * D + i];
        if (team > 1) v = warp_sum(v);
        if (l != 0) continue;
        float* at = s_piece + (p.rank * 2 + q) * G + g;
        if (t.ctas > 1)
            for (int r = 0; r < t.ctas; ++r) peer_store(at, r, v);
        else
            *at = v;
    }
    if (t.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (p.rank == 0)
        for (int c = threadIdx.x; c < CW && p.first_channel + c < a.channels; c += NT) {
            float va = 0.0f, vb = 0.0f;
            for (int r = 0; r < t.ctas; ++r) {
                va += s_image[r * 2 * CW + c];
                vb += s_image[(r * 2 + 1) * CW + c];
            }
            if (a.batch == 1) {  // the image's sums are the gradients
                if (a.dbias) a.dbias[p.first_channel + c] = va;
                if (a.dweight) a.dweight[p.first_channel + c] = vb;
            } else {
                w.ca[p.image * a.channels + p.first_channel + c] = va;
                w.cb[p.image * a.channels + p.first_channel + c] = vb;
            }
        }
    if (p.in) {
        const float each_n = 1.0f / (static_cast<float>(a.pixels) * static_cast<float>(D));
        float m1[P], m2[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int g = (p.tx * V + i) / D;
            float va = 0.0f, vb = 0.0f;
            for (int r = 0; r < t.ctas; ++r) {
                va += s_piece[r * 2 * G + g];
                vb += s_piece[(r * 2 + 1) * G + g];
            }
            m1[i] = va * each_n;
            m2[i] = vb * each_n;
        }
        // dx = dz * (weight * factor * rstd) - (x - mean) * (rstd^2 * m2) - rstd * m1.
        float scale[V];
#pragma unroll
        for (int i = 0; i < V; ++i) scale[i] = s_weight[p.tx * V + i] * factor * rstd[ONE ? 0 : i];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            m1[i] *= -rstd[i];
            m2[i] *= -rstd[i] * rstd[i];
        }
        const int64_t stride = static_cast<int64_t>(p.step) * a.channels;
        T* dx = static_cast<T*>(a.out) + (p.image * a.pixels + first) * a.channels + p.channel;
        const Pack<T, V>* from = keep;
        const char* dat = keep_dz;
#pragma unroll 2
        for (int r = first; r < p.row_end; r += p.step, dx += stride, from += NT, dat += DZ) {
            float x[V], dz[V];
            widen(x, *from);
            kept_floats<V>(dz, dat);
#pragma unroll
            for (int i = 0; i < V; ++i)
                dz[i] = fmaf(dz[i], scale[i], fmaf(x[i] - mean[ONE ? 0 : i], m2[ONE ? 0 : i], m1[ONE ? 0 : i]));
            store_row<T, V>(dx, dz);
        }
    }
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
    t.pieces = static_cast<int>(norm_pieces(a.batch, a.pixels, a.channels));
    t.per = static_cast<int>((a.pixels + t.pieces - 1) / t.pieces);
    // Pieces by group where a block sees every channel and a group has few columns.
    const int D = a.channels / a.groups;
    t.values = D % v == 0 ? v : 1;
    if (t.tiles == 1 && D / t.values <= 16) t.values = D;
    return t;
}

// Launches kernel k over clusters of t.ctas blocks.
template <typename K, typename... Args>
static void launch_clusters(K k, const NormArgs& a, const NormCluster& t, size_t smem, cudaStream_t st, Args... args)
{
    if (smem > 48 * 1024) ensure_dynamic_smem(reinterpret_cast<const void*>(k), smem);
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

// The cluster kernels, where a slab fits (else false).  Small blocks before
// large ones, and row segments of 64 bytes before 32.
template <typename T, int V>
static bool norm_in_clusters(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    const int e = sizeof(T), D = a.channels / a.groups, vecs = a.channels / V;
    // One launch and one reading where latency counts; beyond these sizes streaming is faster.  Us, in clusters and
    // streamed:
    //   forward, 256 channels bf16   1 x 400 pixels 5.7 and 7.0, 1 x 1600 7.4 and 9.5, 1 x 4000 9.4 and 8.1,
    //                                16 x 400 6.9 and 9.1, 16 x 1600 15.6 and 15.0
    //            256 fp32            1 x 400 5.6 and 7.7, 4 x 400 5.8 and 7.8, 1 x 4000 8.1 and 8.8
    //            90, groups of 15    1 x 400 fp32 5.9 and 6.6, 4 x 1600 fp32 7.0 and 8.2, 1 x 1600 bf16 9.1 and 7.6
    //   backward, 256 bf16           1 x 400 5.0 and 8.6, 4 x 400 6.1 and 8.6, 16 x 100 6.4 and 7.9, 16 x 400 13.9 and
    //                                10.7, 64 x 10 29 and 6.8
    //            64 fp16             1 x 400 4.2 and 5.5, 4 x 400 5.1 and 5.6, 16 x 100 7.0 and 5.5
    const double size = static_cast<double>(a.batch) * a.pixels * a.channels * e;
    if (grad ? size > 1.5e6 || a.batch > (a.channels < 256 ? 4 : 16) : size > 4e6 || a.pixels > 2048) return false;
    int whole = 1;  // vectors that hold whole groups: lcm(D, V) / V
    while (whole * V % D != 0) ++whole;
    const int pass = NT * V * (grad ? e + 4 : e);  // bytes that a pass over the block's rows keeps
    for (const int room : {36 * 1024, 72 * 1024, 108 * 1024})
        for (int bytes = 64; bytes >= 32; bytes /= 2) {
            NormCluster t{};
            const int want = bytes / (V * e) > 0 ? bytes / (V * e) : 1;
            t.wide = (want + whole - 1) / whole * whole;
            if (t.wide > vecs) t.wide = vecs;
            if (t.wide > 64) return false;
            t.tiles = (vecs + t.wide - 1) / t.wide;
            const int step = NT / t.wide, most = room / pass;
            const int64_t passes = (a.pixels + step - 1) / step;
            // Blocks enough for the room; while SMs stand idle, until a thread keeps two vectors (1 x 400 x 256 bf16 in 32
            // blocks 5.8 us, in 8 6.7).
            auto more = [&](int64_t ctas) {
                return passes > ctas * most || (passes > ctas * 2 && a.batch * t.tiles * ctas * 2 <= SMS);
            };
            for (t.ctas = 1; t.ctas < 8 && more(t.ctas); t.ctas *= 2) {}
            if (passes > static_cast<int64_t>(t.ctas) * most) continue;
            // Many images of little work each: some 6 ns a block, where streaming takes 17 an image (1000 x 4 pixels bf16:
            // 256 channels, eight blocks an image, 50 us and 17; 90, two, 13 and 17).
            if (a.batch * t.tiles * t.ctas > 4 * SMS && t.tiles * t.ctas > 2) return false;
            t.held = static_cast<int>((passes + t.ctas - 1) / t.ctas);
            t.rows = t.held * step;
            const int CW = t.wide * V;
            t.groups = CW / D;
            if (t.groups > NT) return false;
            const bool one = D % V == 0;
            auto power = [](int n) { return (n & (n - 1)) == 0; };
            t.shuffles = one && t.wide <= 32 && power(t.wide) && power(D / V);
            if (!grad) {
                const size_t smem = static_cast<size_t>(t.held) * pass +
                                    4 * (2 * NT * (one ? 1 : V) + 2 * static_cast<size_t>(CW) + (4 + 3 * t.ctas) * t.groups);
                launch_clusters(one ? norm_cluster_kernel<T, V, true> : norm_cluster_kernel<T, V, false>, a, t, smem, st);
            } else {
                const size_t smem = static_cast<size_t>(t.held) * pass +
                                    4 * (2 * NT * V + (4 + 2 * t.ctas) * static_cast<size_t>(CW) + 2 * t.ctas * t.groups);
                const NormScratch w = scratch(a, ws);
                launch_clusters(one ? norm_grad_cluster_kernel<T, V, true> : norm_grad_cluster_kernel<T, V, false>, a, t,
                                smem, st, w);
                if (a.batch > 1 && (a.dweight || a.dbias))
                    launch_pdl(norm_grad_param_kernel, dim3((a.channels + NT - 1) / NT), dim3(NT), 0, st, a, w);
            }
            return true;
        }
    return false;
}

// The tile with pieces for one wave of `resident` blocks on every SM, at most
// those of the workspace.
inline NormTile one_wave(const NormArgs& a, NormTile t, int resident)
{
    const int64_t wave = static_cast<int64_t>(SMS) * resident / (a.batch * t.tiles);
    const int64_t least = (a.pixels + MOST_ROWS - 1) / MOST_ROWS;
    if (wave < t.pieces) t.pieces = static_cast<int>(wave < least ? least : wave);
    t.per = static_cast<int>((a.pixels + t.pieces - 1) / t.pieces);
    return t;
}

template <typename T, int V, bool ONE, int ACT>
static void norm_streamed(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    const NormTile most = tile(a, V);
    const NormScratch w = scratch(a, ws);
    const dim3 block(NT);
    auto grid = [&](const NormTile& t) { return dim3(static_cast<unsigned>(a.batch * t.pieces), t.tiles); };
    // Whether the join takes a launch of its own.
    auto own = [&](const NormTile& t) { return t.pieces * (a.channels / a.groups / t.values) > OWN_JOIN; };
    if (!grad) {
        static const int sums = resident_blocks(NT, reinterpret_cast<const void*>(norm_partial_kernel<T, V, ONE>));
        static const int rows = resident_blocks(NT, reinterpret_cast<const void*>(norm_apply_kernel<T, V, ONE, ACT>));
        const NormTile t = one_wave(a, most, sums), u = one_wave(a, most, rows);
        NormArgs b = a;
        norm_partial_kernel<T, V, ONE><<<grid(t), block, 0, st>>>(a, t, w);
        const bool joined = own(t);
        if (joined) {
            if (!b.mean) b.mean = w.ga;
            if (!b.rstd) b.rstd = w.gb;
            launch_pdl(norm_join_kernel<false>, dim3(static_cast<unsigned>(a.batch * a.groups)), block, 0, st, b, t, w);
        }
        launch_pdl(norm_apply_kernel<T, V, ONE, ACT>, grid(u), block, 0, st, b, u, t, w, joined);
    } else {
        static const int sums = resident_blocks(NT, reinterpret_cast<const void*>(norm_grad_partial_kernel<T, V, ONE, ACT>));
        static const int rows = resident_blocks(NT, reinterpret_cast<const void*>(norm_grad_apply_kernel<T, V, ONE, ACT>));
        const NormTile t = one_wave(a, most, sums), u = one_wave(a, most, rows);
        norm_grad_partial_kernel<T, V, ONE, ACT><<<grid(t), block, 0, st>>>(a, t, w);
        const unsigned params = a.dweight || a.dbias ? (a.channels + PARAMS - 1) / PARAMS : 0;
        const bool joined = own(t);
        if (joined)
            launch_pdl(norm_join_kernel<true>, dim3(static_cast<unsigned>(a.batch * a.groups)), block, 0, st, a, t, w);
        launch_pdl(norm_grad_apply_kernel<T, V, ONE, ACT>, dim3(grid(u).x + params, u.tiles), block, 0, st, a, u, t, w,
                   joined);
    }
}

template <typename T, int V, bool ONE>
static void norm_streamed(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    switch (a.act) {
    case NMS_ACT_RELU: return norm_streamed<T, V, ONE, NMS_ACT_RELU>(a, ws, st, grad);
    case NMS_ACT_SILU: return norm_streamed<T, V, ONE, NMS_ACT_SILU>(a, ws, st, grad);
    case NMS_ACT_GELU: return norm_streamed<T, V, ONE, NMS_ACT_GELU>(a, ws, st, grad);
    default: return norm_streamed<T, V, ONE, NMS_ACT_NONE>(a, ws, st, grad);
    }
}

template <typename T, int V>
static void norm_width(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    if constexpr (V * sizeof(T) >= 4)
        if (norm_in_clusters<T, V>(a, ws, st, grad)) return;
    if (a.channels / a.groups % V == 0) norm_streamed<T, V, true>(a, ws, st, grad);
    else if constexpr (V > 1) norm_streamed<T, V, false>(a, ws, st, grad);
}

template <typename T>
static void norm_type(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    int v = vector_width(a);
    // Eight-byte vectors that lie in one group before sixteen-byte ones that do not (their sums and moments are kept
    // by channel: 8 x 25600 x 128 in groups of 4, 47 us forward for 40), but where a generator's block serves eight.
    if (a.drop.limit == 65536u && v * sizeof(T) == 16 && a.channels / a.groups % v != 0 && a.channels / a.groups % (v / 2) == 0)
        v /= 2;
    if constexpr (sizeof(T) == 2)
        if (v == 8) return norm_width<T, 8>(a, ws, st, grad);
    if (v == 4) return norm_width<T, 4>(a, ws, st, grad);
    if (v == 2) return norm_width<T, 2>(a, ws, st, grad);
    norm_width<T, 1>(a, ws, st, grad);
}

}  // namespace gbnms
