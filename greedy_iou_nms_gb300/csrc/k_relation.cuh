// Attention weights with a learned bias by buckets of relative position, and
// their gradient.
//
//   probs[b,h,i,:] = softmax over the valid j of scale * scores[b,h,i,j] +
//   table[bucket(i,j)][h]; a pair is masked by a bucket outside the table or
//   by its key's mask, a masked pair has weight 0 whatever its score is, and
//   a row without a valid pair is all zero.
//   da = probs * (dprobs - sum_j probs * dprobs), dscores = scale * da,
//   dtable[u][h] = sum of da over the pairs of bucket u.
//
// Both directions read each operand once and write the result once, so HBM
// bounds them.  A row stays in the registers of its team: L lanes, E elements
// a lane, moved as vectors of EV.  What a row needs besides (its buckets, its
// bias) is the same for many rows, so a team stays with one (query, map) and
// goes through the rows that share it, loading the next row before it works
// on the present one:
//   by image  (one map for all images, no key mask): the rows of one head and
//             query over the images; bias in registers.
//   by head   (a map or mask for each image): the rows of one image and query
//             over the heads; bucket indices in registers, table in shared
//             memory.
// The gradient by head keeps one head instead and goes through images and
// queries, since its sums by bucket are per head.
#pragma once

#include <type_traits>

#include "head.cuh"
#include "internal.h"
#include "relation_plan.h"

namespace gbnms {

constexpr float LOG2E = 1.44269504f;

// 2^x with results below the smallest normal number flushed to zero: such a
// weight is under 2^-126.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Reduction over a team.  L <= 32: neighbouring lanes of a warp; L = 256: the
// block, by way of s (8 floats; alternate between two of them).
template <int L, bool MAX>
__device__ __forceinline__ float team_reduce(float v, float* s)
{
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o; o >>= 1) {
        const float u = __shfl_xor_sync(FULL, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (L > 32) {
        if (lane_id() == 0) s[threadIdx.x / 32] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int k = 1; k < L / 32; ++k) v = MAX ? fmaxf(v, s[k]) : v + s[k];
    }
    return v;
}

template <typename T, int EV, int L, int NV>
__device__ __forceinline__ void load_vectors(Pack<T, EV> (&q)[NV], const T* row, int K, int lane)
{
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int j = (v * L + lane) * EV;
        if (j < K) q[v] = *reinterpret_cast<const Pack<T, EV>*>(row + j);
    }
}

// What a lane knows of its elements' pairs: the bucket index, num_buckets for
// a masked pair or an element past the row, and which are valid, as a mask of
// the packed operand (PACKED: two 16-bit elements to a word) or as bits.
template <typename T, int EV, int NV>
struct Pairs {
    static constexpr bool PACKED = sizeof(T) == 2 && EV % 2 == 0;
    static constexpr int WORDS = PACKED ? NV * EV / 2 : 1;
    Pack<uint16_t, EV> u[NV];
    uint32_t valid[WORDS];

    template <int L>
    __device__ __forceinline__ void set(const Pack<int16_t, EV> (&q)[NV], const uint8_t* mask, int K, int lane, int nb)
    {
        if (!PACKED) valid[0] = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int j = (v * L + lane) * EV;
            const bool in = j < K;
            if (PACKED) {
                Pack<uint8_t, EV> m;
                if (mask && in) m = *reinterpret_cast<const Pack<uint8_t, EV>*>(mask + j);
#pragma unroll
                for (int e = 0; e < EV; e += 2) {
                    uint32_t w = in ? static_cast<uint16_t>(q[v].v[e]) |
                                          static_cast<uint32_t>(static_cast<uint16_t>(q[v].v[e + 1])) << 16
                                    : 0xffffffffu;
                    if (mask && in) w |= (m.v[e] ? 0u : 0xffffu) | (m.v[e + 1] ? 0u : 0xffff0000u);
                    const uint32_t most = static_cast<uint32_t>(nb) * 0x10001u;
                    w = __vminu2(w, most);
                    valid[(v * EV + e) / 2] = ~__vcmpeq2(w, most);
                    u[v].v[e] = static_cast<uint16_t>(w);
                    u[v].v[e + 1] = static_cast<uint16_t>(w >> 16);
                }
            } else {
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    int x = nb;
                    if (in) x = static_cast<uint16_t>(q[v].v[e]);
                    if (x > nb || (mask && in && !mask[j + e])) x = nb;
                    u[v].v[e] = static_cast<uint16_t>(x);
                    valid[0] |= (x < nb ? 1u : 0u) << (v * EV + e);
                }
            }
        }
    }

    // No pair is valid.
    __device__ __forceinline__ void clear(int nb)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < EV; ++e) u[v].v[e] = static_cast<uint16_t>(nb);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) valid[w] = 0;
    }

    // Element e of vector v as binary32, 0 where the pair is masked.
    __device__ __forceinline__ void take(float (&x)[EV], const Pack<T, EV>& q, int v) const
    {
        if (PACKED) {
#pragma unroll
            for (int e = 0; e < EV; e += 2) {
                Pack<T, 2> two{{q.v[e], q.v[e + 1]}};
                uint32_t w = *reinterpret_cast<uint32_t*>(&two) & valid[(v * EV + e) / 2];
                two = *reinterpret_cast<Pack<T, 2>*>(&w);
                x[e] = to_f32(two.v[0]);
                x[e + 1] = to_f32(two.v[1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < EV; ++e) x[e] = (valid[0] >> (v * EV + e)) & 1 ? to_f32(q.v[e]) : 0.0f;
        }
    }
};

// ----------------------------------------------------------------- forward

template <typename T, int EV, int L, int E, bool BY_IMAGE>
__global__ void __launch_bounds__(256, E == 32 ? 2 : E == 16 ? 3 : 4)
relation_softmax_kernel(RelationArgs a, int per)
{
    constexpr int NV = E / EV;
    extern __shared__ float tab[];  // by head: [heads of the chunk][num_buckets + 1]
    __shared__ float red[4][8];
    const int K = static_cast<int>(a.keys), nb = a.num_buckets, H = a.heads;
    const int lane = static_cast<int>(threadIdx.x) % L;
    const int64_t inner = BY_IMAGE ? a.batch : H;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * per, t1 = t0 + per < inner ? t0 + per : inner;
    if (!BY_IMAGE) {
        for (int x = threadIdx.x; x < static_cast<int>(t1 - t0) * (nb + 1); x += 256) {
            const int h = x / (nb + 1), u = x % (nb + 1);
            tab[x] = u < nb ? a.table[static_cast<int64_t>(u) * H + t0 + h] : -INFINITY;
        }
        __syncthreads();
    }
    const int64_t anchors = (BY_IMAGE ? H : a.batch) * a.queries;
    const int64_t want = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L;
    const bool real = want < anchors;  // a team without a row follows another one and stores nothing
    const int64_t anchor = real ? want : anchors - 1, i = anchor % a.queries, outer = anchor / a.queries;
    // Rows of the inner index t: first + t * step.
    const int64_t step = (BY_IMAGE ? H * a.queries : a.queries) * K;
    const int64_t first = (BY_IMAGE ? anchor : outer * H * a.queries + i) * K;
    const T* s = static_cast<const T*>(a.scores) + first + t0 * step;
    T* p = static_cast<T*>(a.out) + first + t0 * step;
    Pack<T, EV> next[NV];
    load_vectors<T, EV, L>(next, s, K, lane);
    Pairs<T, EV, NV> pairs;
    float bias[BY_IMAGE ? E : 1];
    {
        Pack<int16_t, EV> q[NV];
        load_vectors<int16_t, EV, L>(q, a.buckets + ((a.sets == 1 ? 0 : outer) * a.queries + i) * K, K, lane);
        pairs.template set<L>(q, !BY_IMAGE && a.key_mask ? a.key_mask + outer * K : nullptr, K, lane, nb);
    }
    if (BY_IMAGE) {
#pragma unroll
        for (int x = 0; x < E; ++x) {
            const int u = pairs.u[x / EV].v[x % EV];
            bias[x] = u < nb ? a.table[static_cast<int64_t>(u) * H + outer] : -INFINITY;
        }
    }
    const float* row_tab = tab;
    for (int64_t t = t0; t < t1; ++t) {
        Pack<T, EV> cur[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) cur[v] = next[v];
        s += step;
        if (t + 1 < t1) load_vectors<T, EV, L>(next, s, K, lane);
        float x[NV][EV];
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * L * EV >= K) break;
            pairs.take(x[v], cur[v], v);
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                // A masked pair: 0 * scale - inf.
                x[v][e] = fmaf(x[v][e], a.scale, BY_IMAGE ? bias[v * EV + e] : row_tab[pairs.u[v].v[e]]);
                top = fmaxf(top, x[v][e]);
            }
        }
        top = team_reduce<L, true>(top, red[t & 1]);
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * L * EV >= K) break;
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                x[v][e] = exp2_fast((x[v][e] - base) * LOG2E);
                sum += x[v][e];
            }
        }
        sum = team_reduce<L, false>(sum, red[2 + (t & 1)]);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int j = (v * L + lane) * EV;
            if (v * L * EV >= K) break;
            Pack<T, EV> q;
#pragma unroll
            for (int e = 0; e < EV; ++e) q.v[e] = from_f32<T>(x[v][e] * inv);
            if (inv != inv) {  // a row that met an infinity or NaN leaves its masked places 0 all the same
#pragma unroll
                for (int e = 0; e < EV; ++e)
                    if (pairs.u[v].v[e] == nb) q.v[e] = from_f32<T>(0.0f);
            }
            if (j < K && real) *reinterpret_cast<Pack<T, EV>*>(p + j) = q;
        }
        p += step;
        row_tab += nb + 1;
    }
}

// Rows longer than a block holds: one block a row, twice over the keys, the
// first time with a running maximum and sum.
template <typename T>
__global__ void __launch_bounds__(256)
relation_softmax_long_kernel(RelationArgs a, int64_t rows)
{
    __shared__ float red[2][8];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t i = r % a.queries, bh = r / a.queries, b = bh / a.heads;
        const int head = static_cast<int>(bh % a.heads);
        const int16_t* map = a.buckets + ((a.sets == 1 ? 0 : b) * a.queries + i) * a.keys;
        const uint8_t* mask = a.key_mask ? a.key_mask + b * a.keys : nullptr;
        const T* s = static_cast<const T*>(a.scores) + r * a.keys;
        T* p = static_cast<T*>(a.out) + r * a.keys;
        auto logit = [&](int64_t j, float& x) {
            const int u = static_cast<uint16_t>(map[j]);
            if (u >= a.num_buckets || (mask && !mask[j])) return false;
            x = fmaf(to_f32(s[j]), a.scale, a.table[static_cast<int64_t>(u) * a.heads + head]);
            return true;
        };
        float top = -INFINITY, sum = 0.0f, x;
        for (int64_t j = threadIdx.x; j < a.keys; j += 256) {
            if (!logit(j, x)) continue;
            if (x > top) {
                sum *= exp2_fast((top - x) * LOG2E);
                top = x;
            }
            sum += x == -INFINITY ? 0.0f : exp2_fast((x - top) * LOG2E);
        }
        const float all = team_reduce<256, true>(top, red[0]);
        const float base = all == -INFINITY ? 0.0f : all;
        sum = team_reduce<256, false>(top == -INFINITY && sum == 0.0f ? 0.0f : sum * exp2_fast((top - base) * LOG2E),
                                      red[1]);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int64_t j = threadIdx.x; j < a.keys; j += 256)
            p[j] = from_f32<T>(logit(j, x) ? exp2_fast((x - base) * LOG2E) * inv : 0.0f);
        __syncthreads();
    }
}

// ---------------------------------------------------------------- gradient
//
// Sums by bucket: every lane adds to a column of its own in a table
// [num_buckets + 1][columns] of shared memory, so no two lanes collide and the
// order of additions is fixed; the columns are joined in order at the end.
// Masked pairs add 0 to the last row.  With fewer columns than lanes the lanes
// take turns.

// hist[u][lane % columns] += d, lanes of one column in turn.
__device__ __forceinline__ void add_in_turn(float* hist, int u, float d, int columns)
{
    const int lane = static_cast<int>(lane_id());
    for (int turn = 0; turn < 32; turn += columns) {
        if (lane >= turn && lane < turn + columns) hist[u * columns + lane - turn] += d;
        __syncwarp();
    }
}

// column[u * 32] += d for two pairs: both sums are loaded before either is
// stored, and equal buckets add in order.
__device__ __forceinline__ void add_two(float* column, int u0, float d0, int u1, float d1)
{
    float *p0 = column + u0 * 32, *p1 = column + u1 * 32;
    const float v0 = *p0 + d0, old = *p1;
    const float v1 = (u0 == u1 ? v0 : old) + d1;
    *p0 = v0;
    *p1 = v1;
}

// part[u] = sum over the `lists` tables of [num_buckets + 1][columns] at hist.
__device__ __forceinline__ void join_columns(const float* hist, int lists, int columns, int nb, float* part)
{
    __syncthreads();
    const int warps = static_cast<int>(blockDim.x) / 32;
    for (int u = static_cast<int>(threadIdx.x) / 32; u < nb; u += warps) {
        float v = 0.0f;
        for (int c = static_cast<int>(lane_id()); c < lists * columns; c += 32)
            v += hist[(static_cast<size_t>(c / columns) * (nb + 1) + u) * columns + c % columns];
        v = warp_sum(v);
        if (lane_id() == 0) part[u] = v;
    }
}

// One row: da into x (binary32) from the packed operands, dscores stored.
template <typename T, int EV, int L, int NV>
__device__ __forceinline__ void grad_row(float (&x)[NV][EV], const Pack<T, EV> (&pq)[NV], const Pack<T, EV> (&dq)[NV],
                                         const Pairs<T, EV, NV>& pairs, const RelationArgs& a, T* ds, int lane,
                                         bool store, float* red)
{
    const int K = static_cast<int>(a.keys);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (v * L * EV >= K) break;
        float p[EV], d[EV];
        pairs.take(p, pq[v], v);
        pairs.take(d, dq[v], v);
#pragma unroll
        for (int e = 0; e < EV; ++e) dot = fmaf(p[e], d[e], dot);
    }
    dot = team_reduce<L, false>(dot, red);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int j = (v * L + lane) * EV;
        if (v * L * EV >= K) break;
        float p[EV], d[EV];
        pairs.take(p, pq[v], v);
        pairs.take(d, dq[v], v);
        Pack<T, EV> q;
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            x[v][e] = p[e] * (d[e] - dot);
            // A row that met an infinity or NaN leaves its masked places 0 all the same.
            if (!(fabsf(dot) < INFINITY) && pairs.u[v].v[e] == a.num_buckets) x[v][e] = 0.0f;
            q.v[e] = from_f32<T>(a.scale * x[v][e]);
        }
        if (store && j < K) *reinterpret_cast<Pack<T, EV>*>(ds + j) = q;
    }
}

// By image: block (x, y, z) = (query tile, image chunk, head).
template <typename T, int EV, int L, int E>
__global__ void __launch_bounds__(256)
relation_grad_image_kernel(RelationArgs a, int per, int columns, float* part)
{
    constexpr int NV = E / EV;
    extern __shared__ float hist[];  // [num_buckets + 1][columns]
    __shared__ float red[2][8];
    const int K = static_cast<int>(a.keys), nb = a.num_buckets, head = static_cast<int>(blockIdx.z);
    const int lane = static_cast<int>(threadIdx.x) % L;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * per, t1 = t0 + per < a.batch ? t0 + per : a.batch;
    for (int x = threadIdx.x; x < (nb + 1) * columns; x += blockDim.x) hist[x] = 0.0f;
    const int64_t want = static_cast<int64_t>(blockIdx.x) * (blockDim.x / L) + threadIdx.x / L;
    const bool real = want < a.queries;
    const int64_t i = real ? want : a.queries - 1;
    const int64_t step = a.heads * a.queries * K, first = (head * a.queries + i) * K + t0 * step;
    const T* p = static_cast<const T*>(a.probs) + first;
    const T* dp = static_cast<const T*>(a.scores) + first;
    T* ds = static_cast<T*>(a.out) + first;
    Pack<T, EV> pn[NV], dn[NV];
    load_vectors<T, EV, L>(pn, p, K, lane);
    load_vectors<T, EV, L>(dn, dp, K, lane);
    Pairs<T, EV, NV> pairs;
    {
        Pack<int16_t, EV> q[NV];
        load_vectors<int16_t, EV, L>(q, a.buckets + i * K, K, lane);
        pairs.template set<L>(q, nullptr, K, lane, nb);
    }
    float acc[NV][EV];
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k / EV][k % EV] = 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
        Pack<T, EV> pq[NV], dq[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            pq[v] = pn[v];
            dq[v] = dn[v];
        }
        p += step;
        dp += step;
        if (t + 1 < t1) {
            load_vectors<T, EV, L>(pn, p, K, lane);
            load_vectors<T, EV, L>(dn, dp, K, lane);
        }
        float x[NV][EV];
        grad_row<T, EV, L, NV>(x, pq, dq, pairs, a, ds, lane, real, red[t & 1]);
        ds += step;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * L * EV >= K) break;
#pragma unroll
            for (int e = 0; e < EV; ++e) acc[v][e] += x[v][e];
        }
    }
    // The warps add their sums in turn.
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) / 32 == w) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (v * L * EV >= K) break;
#pragma unroll
                for (int e = 0; e < EV; ++e) add_in_turn(hist, real ? pairs.u[v].v[e] : nb, acc[v][e], columns);
            }
        }
    }
    join_columns(hist, 1, columns, nb,
                 part + ((static_cast<int64_t>(head) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * nb);
}

// By head: block (x, y) = (share of the rows, head); each warp has a table of
// its own.
template <typename T, int EV, int L, int E>
__global__ void __launch_bounds__(256)
relation_grad_head_kernel(RelationArgs a, int columns, float* part)
{
    constexpr int NV = E / EV;
    extern __shared__ float hist[];  // [warps][num_buckets + 1][columns]
    __shared__ float red[2][8];
    const int K = static_cast<int>(a.keys), nb = a.num_buckets, head = static_cast<int>(blockIdx.y);
    const int lane = static_cast<int>(threadIdx.x) % L, teams = static_cast<int>(blockDim.x) / L;
    const int warps = static_cast<int>(blockDim.x) / 32;
    for (int x = threadIdx.x; x < warps * (nb + 1) * columns; x += blockDim.x) hist[x] = 0.0f;
    __syncthreads();
    float* mine = hist + static_cast<size_t>(threadIdx.x / 32) * (nb + 1) * columns;
    // Rows are numbered image by image; the block takes `teams` of them at a
    // time.  (image, query) of the team's next row advance without divisions.
    const unsigned Q = static_cast<unsigned>(a.queries), rows = static_cast<unsigned>(a.batch) * Q;
    const unsigned stride = gridDim.x * teams, step_b = stride / Q, step_i = stride % Q;
    unsigned bi = blockIdx.x * teams;
    const unsigned team = threadIdx.x / L;
    unsigned b = (bi + team) / Q, i = (bi + team) % Q;
    Pack<T, EV> pn[NV], dn[NV];
    Pack<int16_t, EV> un[NV];
    int64_t off_next = 0;
    const uint8_t* mask_next = nullptr;
    auto fetch = [&](bool real) {  // a team without a row reads the block's first ones and stores nothing
        const int64_t fb = real ? b : 0, fi = real ? i : 0;
        off_next = ((fb * a.heads + head) * Q + fi) * K;
        mask_next = a.key_mask ? a.key_mask + fb * K : nullptr;
        load_vectors<T, EV, L>(pn, static_cast<const T*>(a.probs) + off_next, K, lane);
        load_vectors<T, EV, L>(dn, static_cast<const T*>(a.scores) + off_next, K, lane);
        load_vectors<int16_t, EV, L>(un, a.buckets + ((a.sets == 1 ? 0 : fb * Q) + fi) * K, K, lane);
    };
    if (bi < rows) fetch(bi + team < rows);
    for (int turn = 0; bi < rows; turn ^= 1) {
        const bool real = bi + team < rows;
        const int64_t off = off_next;
        Pairs<T, EV, NV> pairs;
        pairs.template set<L>(un, mask_next, K, lane, nb);
        if (!real) pairs.clear(nb);
        Pack<T, EV> pq[NV], dq[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            pq[v] = pn[v];
            dq[v] = dn[v];
        }
        bi += stride;
        b += step_b;
        i += step_i;
        if (i >= Q) {
            i -= Q;
            ++b;
        }
        if (bi < rows) fetch(bi + team < rows);
        float x[NV][EV];
        grad_row<T, EV, L, NV>(x, pq, dq, pairs, a, static_cast<T*>(a.out) + off, lane, real, red[turn]);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * L * EV >= K) break;
            if (columns == 32) {
                float* column = mine + lane_id();
                if (EV == 1) {
                    if (v & 1) continue;
                    if (v + 1 < NV && (v + 1) * L < K)
                        add_two(column, pairs.u[v].v[0], x[v][0], pairs.u[v + 1 < NV ? v + 1 : v].v[0],
                                x[v + 1 < NV ? v + 1 : v][0]);
                    else
                        column[pairs.u[v].v[0] * 32] += x[v][0];
                } else {
#pragma unroll
                    for (int e = 0; e + 1 < EV; e += 2)
                        add_two(column, pairs.u[v].v[e], x[v][e], pairs.u[v].v[e + 1], x[v][e + 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < EV; ++e) add_in_turn(mine, pairs.u[v].v[e], x[v][e], columns);
            }
        }
    }
    join_columns(hist, warps, columns, nb, part + (static_cast<int64_t>(head) * gridDim.x + blockIdx.x) * nb);
}

// Rows longer than a block holds: one warp a row, twice over the keys.
template <typename T>
__global__ void __launch_bounds__(256)
relation_grad_long_kernel(RelationArgs a, int columns, float* part)
{
    extern __shared__ float hist[];
    const int warps = static_cast<int>(blockDim.x) / 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int head = static_cast<int>(blockIdx.y), nb = a.num_buckets;
    for (int x = threadIdx.x; x < warps * (nb + 1) * columns; x += blockDim.x) hist[x] = 0.0f;
    __syncthreads();
    float* mine = hist + static_cast<size_t>(warp) * (nb + 1) * columns;
    for (int64_t bi = static_cast<int64_t>(blockIdx.x) * warps + warp; bi < a.batch * a.queries;
         bi += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t b = bi / a.queries, i = bi % a.queries, off = ((b * a.heads + head) * a.queries + i) * a.keys;
        const T* dp = static_cast<const T*>(a.scores) + off;
        const T* p = static_cast<const T*>(a.probs) + off;
        T* ds = static_cast<T*>(a.out) + off;
        const int16_t* map = a.buckets + (a.sets == 1 ? i : bi) * a.keys;
        const uint8_t* mask = a.key_mask ? a.key_mask + b * a.keys : nullptr;
        auto bucket = [&](int64_t j) {
            const int u = static_cast<uint16_t>(map[j]);
            return u < nb && (!mask || mask[j]) ? u : nb;
        };
        float dot = 0.0f;
        for (int64_t j = lane_id(); j < a.keys; j += 32)
            if (bucket(j) < nb) dot = fmaf(to_f32(p[j]), to_f32(dp[j]), dot);
        dot = warp_sum(dot);
        for (int64_t j0 = 0; j0 < a.keys; j0 += 32) {
            const int64_t j = j0 + lane_id();
            const int u = j < a.keys ? bucket(j) : nb;
            const float da = u < nb ? to_f32(p[j]) * (to_f32(dp[j]) - dot) : 0.0f;
            if (j < a.keys) ds[j] = from_f32<T>(a.scale * da);
            add_in_turn(mine, u, da, columns);
        }
    }
    join_columns(hist, warps, columns, nb, part + (static_cast<int64_t>(head) * gridDim.x + blockIdx.x) * nb);
}

// ------------------------------------------------------------------- launches

// Elements that every row of the operands can be moved by.
inline int relation_vector(const RelationArgs& a, int most)
{
    auto fits = [&](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const int e = a.type == NMS_TYPE_F32 ? 4 : 2;
    for (int v = most; v > 1; v = v == 8 ? 2 : 1)
        if (a.keys % v == 0 && fits(a.scores, v * e) && fits(a.probs, v * e) && fits(a.out, v * e) &&
            fits(a.buckets, v * 2) && (!a.key_mask || fits(a.key_mask, v)))
            return v;
    return 1;
}

// f(EV, L, E as integral constants) for the row's shape.
template <typename T, typename F>
inline void relation_shape(const RelationArgs& a, F f)
{
    constexpr int MOST = sizeof(T) == 2 ? 8 : 4;
    auto shape = [&](auto ev) {
        using std::integral_constant;
        if (a.keys <= 64) f(ev, integral_constant<int, 8>{}, integral_constant<int, 8>{});
        else if (a.keys <= 128) f(ev, integral_constant<int, 16>{}, integral_constant<int, 8>{});
        else if (a.keys <= 256) f(ev, integral_constant<int, 32>{}, integral_constant<int, 8>{});
        else if (a.keys <= 512) f(ev, integral_constant<int, 32>{}, integral_constant<int, 16>{});
        else if (a.keys <= 1024) f(ev, integral_constant<int, 32>{}, integral_constant<int, 32>{});
        else f(ev, integral_constant<int, 256>{}, integral_constant<int, 32>{});
    };
    const int v = relation_vector(a, MOST);
    if (v == MOST) shape(std::integral_constant<int, MOST>{});
    else if (v == 2) shape(std::integral_constant<int, 2>{});
    else shape(std::integral_constant<int, 1>{});
}

template <typename T>
inline void softmax_type(const RelationArgs& a, cudaStream_t st)
{
    if (a.keys > RELATION_MOST) {
        const int64_t rows = a.batch * a.heads * a.queries;
        relation_softmax_long_kernel<T><<<static_cast<unsigned>(rows < 152 * 8 ? rows : 152 * 8), 256, 0, st>>>(a, rows);
        return;
    }
    relation_shape<T>(a, [&](auto ev, auto l, auto e) {
        constexpr int EV = decltype(ev)::value, L = decltype(l)::value, E = decltype(e)::value;
        const bool image = relation_by_image(a);
        const int64_t anchors = (image ? a.heads : a.batch) * a.queries, inner = image ? a.batch : a.heads;
        const int64_t blocks = (anchors + 256 / L - 1) / (256 / L);
        // Chunks of the inner index: enough blocks for every SM eight times over.
        int64_t chunks = (152 * 8 + blocks - 1) / blocks;
        if (chunks > inner) chunks = inner;
        if (!image) {  // the chunk's tables have to fit
            const int64_t most = 96 * 1024 / (4 * (a.num_buckets + 1));
            if (chunks < (inner + most - 1) / most) chunks = (inner + most - 1) / most;
        }
        if (chunks > 65535) chunks = 65535;
        const int per = static_cast<int>((inner + chunks - 1) / chunks);
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((inner + per - 1) / per));
        if (image) {
            relation_softmax_kernel<T, EV, L, E, true><<<grid, 256, 0, st>>>(a, per);
        } else {
            const size_t smem = 4 * static_cast<size_t>(per) * (a.num_buckets + 1);
            ensure_dynamic_smem(reinterpret_cast<const void*>(relation_softmax_kernel<T, EV, L, E, false>), smem);
            relation_softmax_kernel<T, EV, L, E, false><<<grid, 256, smem, st>>>(a, per);
        }
    });
}

template <typename T>
inline void grad_type(const RelationArgs& a, float* part, cudaStream_t st)
{
    const bool image = relation_by_image(a) && a.keys <= RELATION_MOST;
    const RelationGradPlan p = relation_grad_plan(a.batch, a.heads, a.queries, a.keys, a.num_buckets, image);
    const size_t table = 4 * static_cast<size_t>(a.num_buckets + 1) * p.columns;
    if (a.keys > RELATION_MOST) {
        ensure_dynamic_smem(reinterpret_cast<const void*>(relation_grad_long_kernel<T>), table * p.warps);
        relation_grad_long_kernel<T><<<dim3(static_cast<unsigned>(p.blocks), a.heads), p.warps * 32, table * p.warps,
                                       st>>>(a, p.columns, part);
        return;
    }
    relation_shape<T>(a, [&](auto ev, auto l, auto e) {
        constexpr int EV = decltype(ev)::value, L = decltype(l)::value, E = decltype(e)::value;
        if (image) {
            auto* k = relation_grad_image_kernel<T, EV, L, E>;
            ensure_dynamic_smem(reinterpret_cast<const void*>(k), table);
            k<<<dim3(static_cast<unsigned>(p.blocks), static_cast<unsigned>(p.chunks), a.heads), p.warps * 32, table,
                st>>>(a, static_cast<int>(p.per), p.columns, part);
        } else {
            auto* k = relation_grad_head_kernel<T, EV, L, E>;
            ensure_dynamic_smem(reinterpret_cast<const void*>(k), table * p.warps);
            k<<<dim3(static_cast<unsigned>(p.blocks), a.heads), p.warps * 32, table * p.warps, st>>>(a, p.columns,
                                                                                                    part);
        }
    });
}

}  // namespace gbnms
