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
// bounds them.  A row stays in the registers of its team: L lanes, NV vectors
// of EV elements a lane.  What a row needs besides (its buckets, its
// bias) is the same for many rows, so a team stays with one (query, map) and
// goes through the rows that share it, several short ones at a time, or
// loading the next long one before it works on the present one:
//   by image  (one map for all images, no key mask): the rows of one head and
//             query over the images; bias in registers.
//   by head   (a map or mask for each image): the rows of one image and query
//             over the heads; bucket indices in registers, table in shared
//             memory.
// The gradient by head keeps one head instead and goes through images and
// queries, since its sums by bucket are per head.
//
// Measured (us; TB/s of what has to move): weights 2304 x 8 x 49 x 49 fp16, one
// map, 47 (3.8), issue: 27 instructions a place; 16 x 8 x 1000 x 1000 bf16, a map
// by image, 104 (5.2); 4 x 8 x 2000 x 2000 fp32 187 (5.6).  Gradient 1600 x 8 x
// 64 x 64 fp16, one map, 69 (4.6); 16 x 8 x 1000 x 1000 bf16, 225 buckets, a map
// by image, 218 (3.7), latency: 12 warps an SM beside their tables of sums.
// Odd lengths above 128 keys go element by element and take twice as long.
#pragma once

#include <type_traits>

#include "head.cuh"
#include "internal.h"
#include "relation_plan.h"

namespace gbnms {

// A weight below 2^-126 is flushed to zero (exp2_fast).

// Reductions over a team, of R rows at once.  L <= 32: neighbouring lanes of
// a warp; L = 256: the block, by way of s (8 floats; alternate between two of
// them), R = 1.
template <int L, bool MAX, int R>
__device__ __forceinline__ void team_reduce(float (&v)[R], float* s)
{
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float u = __shfl_xor_sync(FULL, v[r], o);
            v[r] = MAX ? fmaxf(v[r], u) : v[r] + u;
        }
    if (L > 32) {
        if (lane_id() == 0) s[threadIdx.x / 32] = v[0];
        __syncthreads();
        v[0] = s[0];
#pragma unroll
        for (int k = 1; k < L / 32; ++k) v[0] = MAX ? fmaxf(v[0], s[k]) : v[0] + s[k];
    }
}

// 0xffff in each half (byte pair) of x whose top bit is set.
__device__ __forceinline__ uint32_t spread_top_bits(uint32_t x)
{
    uint32_t y;
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(y) : "r"(x));
    return y;
}

// The same from the top bits of the low (HIGH: high) two bytes.
template <bool HIGH>
__device__ __forceinline__ uint32_t spread_byte_bits(uint32_t x)
{
    uint32_t y;
    if (HIGH) asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(y) : "r"(x));
    else asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void unpack_two(uint32_t w, float& lo, float& hi, __nv_bfloat16)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_two(uint32_t w, float& lo, float& hi, __half)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
}
__device__ __forceinline__ void unpack_two(uint32_t, float&, float&, float) {}  // never called

__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(__half x) { return __half_as_ushort(x); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
__device__ __forceinline__ float of_bits(uint32_t w, float) { return __uint_as_float(w); }
__device__ __forceinline__ float of_bits(uint32_t w, __half) { return to_f32(__ushort_as_half(static_cast<unsigned short>(w))); }
__device__ __forceinline__ float of_bits(uint32_t w, __nv_bfloat16) { return __uint_as_float(w << 16); }

// How a team holds a row: L lanes by NV vectors of EV elements, of which all
// but the last SLACK vectors lie inside every row that the shape serves.
template <typename T_, int EV_, int L_, int NV_, int SLACK_>
struct Shape {
    using T = T_;
    static constexpr int EV = EV_, L = L_, NV = NV_, SLACK = SLACK_, E = EV * NV;
    // Two 16-bit elements to a word.
    static constexpr bool PACKED = sizeof(T) == 2 && EV % 2 == 0;
    // Blocks that an SM holds at least (the launches count on it).
    static constexpr int BLOCKS = E > 16 ? (PACKED ? 2 : 1) : E > 8 ? 2 : 3;
    static constexpr int GRAD_BLOCKS = E > 16 ? 1 : E > 8 ? 2 : 3;
    // Rows that a team works on at a time: short ones side by side, to have enough loads and shuffles under way.
    static constexpr int ROWS = L > 32 || E > 16 ? 1 : E > 8 ? 2 : 4;

    static __device__ __forceinline__ int first(int v, int lane) { return (v * L + lane) * EV; }
    static __device__ __forceinline__ bool inside(int v, int lane, int K)
    {
        return v < NV - SLACK || first(v, lane) < K;
    }
    // A row's vectors; one past the row reads the row's start instead.
    template <typename U>
    static __device__ __forceinline__ void load(Pack<U, EV> (&q)[NV], const U* row, int K, int lane)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            q[v] = *reinterpret_cast<const Pack<U, EV>*>(row + (inside(v, lane, K) ? first(v, lane) : 0));
    }
    // Vector v as binary32.
    static __device__ __forceinline__ void widen(float (&x)[EV], const Pack<T, EV>& q)
    {
        if constexpr (PACKED) {
#pragma unroll
            for (int e = 0; e < EV; e += 2)
                unpack_two(reinterpret_cast<const uint32_t*>(&q)[e / 2], x[e], x[e + 1], T{});
        } else {
#pragma unroll
            for (int e = 0; e < EV; ++e) x[e] = to_f32(q.v[e]);
        }
    }
};

// Bucket indices of a lane's elements, num_buckets for a masked pair or an
// element past the row: two to a word when PACKED.
template <typename S>
struct Buckets {
    uint32_t u[S::PACKED ? S::E / 2 : S::E];

    // From the map's vectors and (or NULL) the key mask's.
    __device__ __forceinline__ void set(const Pack<int16_t, S::EV> (&q)[S::NV], const Pack<uint8_t, S::EV> (&key)[S::NV],
                                        bool keyed, int K, int lane, int nb)
    {
        constexpr int EV = S::EV;
#pragma unroll
        for (int v = 0; v < S::NV; ++v) {
            const bool in = S::inside(v, lane, K);
            if constexpr (S::PACKED) {
                uint32_t on[(EV + 3) / 4];  // top bit of a byte: the key takes part
#pragma unroll
                for (int k = 0; k < (EV + 3) / 4; ++k) {
                    uint32_t m = 0xffffffffu;
                    if (keyed)
                        m = EV >= 4 ? reinterpret_cast<const uint32_t*>(&key[v])[k]
                                    : *reinterpret_cast<const uint16_t*>(&key[v]);
                    on[k] = ((m & 0x7f7f7f7fu) + 0x7f7f7f7fu) | m;
                }
#pragma unroll
                for (int e = 0; e < EV; e += 2) {
                    uint32_t w = reinterpret_cast<const uint32_t*>(&q[v])[e / 2];
                    if (keyed)
                        w |= ~(e % 4 ? spread_byte_bits<true>(on[e / 4]) : spread_byte_bits<false>(on[e / 4]));
                    if (!in) w = 0xffffffffu;
                    u[(v * EV + e) / 2] = __vminu2(w, static_cast<uint32_t>(nb) * 0x10001u);
                }
            } else {
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    const uint32_t x = static_cast<uint16_t>(q[v].v[e]), most = static_cast<uint32_t>(nb);
                    u[v * EV + e] = !in || x > most || (keyed && !key[v].v[e]) ? most : x;
                }
            }
        }
    }

    __device__ __forceinline__ void clear(int nb)
    {
#pragma unroll
        for (int k = 0; k < (S::PACKED ? S::E / 2 : S::E); ++k)
            u[k] = static_cast<uint32_t>(nb) * (S::PACKED ? 0x10001u : 1u);
    }

    __device__ __forceinline__ int operator()(int v, int e) const
    {
        const int k = v * S::EV + e;
        if (!S::PACKED) return static_cast<int>(u[k]);
        return static_cast<int>(k & 1 ? u[k / 2] >> 16 : u[k / 2] & 0xffffu);
    }
};

// Ones over the operands of valid pairs: packed like Buckets, or a word for
// each element, or beyond eight unpacked elements a bit each.
template <typename S>
struct Valid {
    static constexpr bool BITS = !S::PACKED && S::E > 8;
    uint32_t m[S::PACKED ? S::E / 2 : BITS ? 1 : S::E];

    __device__ __forceinline__ void set(const Buckets<S>& b, int nb)
    {
        if constexpr (S::PACKED) {
            // nb - u is 0 in a masked half and 1 .. 1024 else: the sum carries into its top bit.
#pragma unroll
            for (int k = 0; k < S::E / 2; ++k)
                m[k] = spread_top_bits(static_cast<uint32_t>(nb) * 0x10001u - b.u[k] + 0x7fff7fffu);
        } else {
            if (BITS) m[0] = 0;
#pragma unroll
            for (int k = 0; k < S::E; ++k) {
                const bool ok = b.u[k] != static_cast<uint32_t>(nb);
                if (BITS) m[0] |= (ok ? 1u : 0u) << k;
                else m[k] = ok ? 0xffffffffu : 0u;
            }
        }
    }

    // Vector v as binary32, 0 where the pair is masked.
    __device__ __forceinline__ void take(float (&x)[S::EV], const Pack<typename S::T, S::EV>& q, int v) const
    {
        constexpr int EV = S::EV;
        if constexpr (S::PACKED) {
#pragma unroll
            for (int e = 0; e < EV; e += 2)
                unpack_two(reinterpret_cast<const uint32_t*>(&q)[e / 2] & m[(v * EV + e) / 2], x[e], x[e + 1],
                           typename S::T{});
        } else {
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                const int k = v * EV + e;
                if (BITS) x[e] = (m[0] >> k) & 1u ? to_f32(q.v[e]) : 0.0f;
                else x[e] = of_bits(bits_of(q.v[e]) & m[k], typename S::T{});
            }
        }
    }
};

// ----------------------------------------------------------------- staging
//
// Short rows of odd lengths: read and written element by element they cost a
// memory request for every few bytes (57% of the SM's request slots at 2304 x
// 8 x 49 x 49 fp16).  Neighbouring teams' rows of one image are one stretch of
// memory, a multiple of 16 bytes long but for the last block's; so, where an
// image's rows are a multiple of that too, the block moves it as 16-byte
// vectors through shared memory, the next rows' while it works on the present
// ones'.
template <typename S>
struct Stretch {
    using T = typename S::T;
    static constexpr bool USED = S::EV == 1 && S::L <= 16;
    static constexpr int VE = 16 / sizeof(T), TEAMS = 256 / S::L;
    static constexpr int MOST = (TEAMS * S::NV * S::L / VE + 255) / 256;  // vectors of a thread
    int whole, all;  // elements of the block's stretch: in whole vectors, and in all

    __device__ __forceinline__ explicit Stretch(int n) : whole(n / VE * VE), all(n) {}

    // buf[0 .. all) = from[0 .. all), asynchronously.
    __device__ __forceinline__ void fetch(T* buf, const T* from) const
    {
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int at = (k * 256 + static_cast<int>(threadIdx.x)) * VE;
            if (at < whole) {
                const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(buf + at));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from + at) : "memory");
            }
        }
        const int last = whole + static_cast<int>(threadIdx.x);
        if (last < all) buf[last] = from[last];
    }
    static __device__ __forceinline__ void fetched()
    {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    // to[0 .. all) = buf[0 .. all).
    __device__ __forceinline__ void put(const T* buf, T* to) const
    {
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int at = (k * 256 + static_cast<int>(threadIdx.x)) * VE;
            if (at < whole) *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(buf + at);
        }
        const int last = whole + static_cast<int>(threadIdx.x);
        if (last < all) to[last] = buf[last];
    }
};

// Whether an image's rows and the operands lie on 16-byte boundaries.
template <typename S>
inline bool stretches(const RelationArgs& a)
{
    auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    return Stretch<S>::USED && static_cast<int64_t>(a.heads) * a.queries * a.keys % Stretch<S>::VE == 0 &&
           aligned(a.scores) && aligned(a.probs) && aligned(a.out);
}

// ----------------------------------------------------------------- forward

template <typename S, bool BY_IMAGE, bool STAGED>
__global__ void __launch_bounds__(256, S::BLOCKS)
relation_softmax_kernel(RelationArgs a, unsigned per)
{
    using T = typename S::T;
    constexpr int EV = S::EV, NV = S::NV, L = S::L;
    // By head: [heads of the chunk][num_buckets + 1], -inf last.  Staged: two times R rows' stretches.
    extern __shared__ __align__(16) float tab[];
    __shared__ float red[4][8];
    using Rows = Stretch<S>;
    const int K = static_cast<int>(a.keys), nb = a.num_buckets, H = a.heads;
    const int lane = static_cast<int>(threadIdx.x) % L;
    // Unsigned: up to 2^31 - 1 images, and the loop counts past them.
    const unsigned inner = static_cast<unsigned>(BY_IMAGE ? a.batch : H);
    const unsigned t0 = blockIdx.y * per, t1 = t0 + per < inner ? t0 + per : inner;
    if (!BY_IMAGE) {
        for (int x = threadIdx.x; x < static_cast<int>(t1 - t0) * (nb + 1); x += 256) {
            const int h = x / (nb + 1), u = x % (nb + 1);
            tab[x] = u < nb ? a.table[static_cast<int64_t>(u) * H + t0 + h] : -INFINITY;
        }
        __syncthreads();
    }
    const unsigned Q = static_cast<unsigned>(a.queries);
    const unsigned anchors = static_cast<unsigned>(BY_IMAGE ? H : a.batch) * Q;
    const unsigned want = blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool real = want < anchors;  // a team without a row follows another one and stores nothing
    const unsigned anchor = real ? want : anchors - 1, outer = anchor / Q, i = anchor % Q;
    // Rows of the inner index t: first + t * step.
    const int64_t step = (BY_IMAGE ? static_cast<int64_t>(H) * Q : static_cast<int64_t>(Q)) * K;
    const int64_t first = (BY_IMAGE ? static_cast<int64_t>(anchor) : static_cast<int64_t>(outer) * H * Q + i) * K;
    const T* s = static_cast<const T*>(a.scores) + first + t0 * step;
    T* p = static_cast<T*>(a.out) + first + t0 * step;
    constexpr int R = S::ROWS;
    Pack<T, EV> next[R][NV];
    if (R == 1 && !STAGED) S::load(next[0], s, K, lane);
    T* const stage = reinterpret_cast<T*>(tab);
    const int pitch = Rows::TEAMS * K, team = static_cast<int>(threadIdx.x) / L;
    const unsigned rows_left = anchors - blockIdx.x * Rows::TEAMS;
    const Rows rows(static_cast<int>(rows_left < Rows::TEAMS ? rows_left : Rows::TEAMS) * K);
    const int64_t start = t0 * step + static_cast<int64_t>(blockIdx.x) * pitch;
    const T* from = static_cast<const T*>(a.scores) + start;
    T* to_all = static_cast<T*>(a.out) + start;
    auto fetch = [&](unsigned t, int half) {
#pragma unroll
        for (int r = 0; r < R; ++r, from += step)
            if (t + r < t1) rows.fetch(stage + (half * R + r) * pitch, from);
    };
    int half = 0;
    if (STAGED) fetch(t0, 0);
    Buckets<S> bucket;
    float bias[BY_IMAGE ? S::E : 1];
    {
        Pack<int16_t, EV> q[NV];
        Pack<uint8_t, EV> key[NV];
        S::load(q, a.buckets + (static_cast<int64_t>(a.sets == 1 ? 0 : outer) * Q + i) * K, K, lane);
        const bool keyed = !BY_IMAGE && a.key_mask;
        if (keyed) S::load(key, a.key_mask + static_cast<int64_t>(outer) * K, K, lane);
        bucket.set(q, key, keyed, K, lane, nb);
    }
    if (BY_IMAGE) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                const int u = bucket(v, e);
                bias[v * EV + e] = u < nb ? a.table[static_cast<int64_t>(u) * H + outer] : -INFINITY;
            }
    }
    const float* row_tab = tab;
    for (unsigned t = t0; t < t1; t += R) {
        float x[R][NV][EV], top[R], sum[R], inv[R];
        T* mine[R];  // staged: the team's row
        if constexpr (STAGED) {
            Rows::fetched();
            if (t + R < t1) fetch(t + R, half ^ 1);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mine[r] = stage + (half * R + r) * pitch + team * K;
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    x[r][v][0] = real && t + r < t1 ? to_f32(mine[r][S::inside(v, lane, K) ? S::first(v, lane) : 0]) : 0.0f;
            }
        } else {
            if (R > 1) {  // past the last row: that row again, not stored
#pragma unroll
                for (int r = 0; r < R; ++r) S::load(next[r], s + (t + r < t1 ? r : t1 - 1 - t) * step, K, lane);
            }
            s += R * step;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < NV; ++v) S::widen(x[r][v], next[r][v]);
            if (R == 1 && t + 1 < t1) S::load(next[0], s, K, lane);
        }
        auto bias_of = [&](int r, int v, int e) {
            return BY_IMAGE ? bias[v * EV + e] : row_tab[(t + r < t1 ? r : 0) * (nb + 1) + bucket(v, e)];
        };
        // A masked pair's logit is -inf, or NaN if its score is NaN or infinite; the maximum passes over both.
#pragma unroll
        for (int r = 0; r < R; ++r) {
            top[r] = -INFINITY;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    x[r][v][e] = fmaf(x[r][v][e], a.scale, bias_of(r, v, e));
                    top[r] = fmaxf(top[r], x[r][v][e]);
                }
        }
        team_reduce<L, true>(top, red[t & 1]);
        bool odd = false;  // a row met a NaN or +inf
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float base = top[r] == -INFINITY ? 0.0f : top[r];
            sum[r] = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    x[r][v][e] = exp2_fast((x[r][v][e] - base) * LOG2E);
                    sum[r] += x[r][v][e];
                }
        }
        team_reduce<L, false>(sum, red[2 + (t & 1)]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            inv[r] = sum[r] == 0.0f ? 0.0f : reciprocal(sum[r]);
            odd |= inv[r] != inv[r];
        }
        if (__any_sync(FULL, odd)) {  // perhaps of masked pairs alone: once more without those
            if (L > 32) __syncthreads();  // red is still being read
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sum[r] = 0.0f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < EV; ++e) {
                        if (bias_of(r, v, e) == -INFINITY) x[r][v][e] = 0.0f;
                        sum[r] += x[r][v][e];
                    }
            }
            team_reduce<L, false>(sum, red[2 + (t & 1)]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                inv[r] = sum[r] == 0.0f ? 0.0f : reciprocal(sum[r]);
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < EV; ++e)
                        x[r][v][e] = bias_of(r, v, e) == -INFINITY ? 0.0f : x[r][v][e] * inv[r];
                inv[r] = 1.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (t + r >= t1) break;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int e = 0; e < EV; ++e) x[r][v][e] *= inv[r];
                T* to = STAGED ? mine[r] : p;
                if (real && S::inside(v, lane, K))
                    *reinterpret_cast<Pack<T, EV>*>(to + S::first(v, lane)) = pack_results<T, EV>(x[r][v]);
            }
            p += step;
        }
        row_tab += R * (nb + 1);
        if constexpr (STAGED) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r, to_all += step)
                if (t + r < t1) rows.put(stage + (half * R + r) * pitch, to_all);
            half ^= 1;
        }
    }
}

// Rows longer than a block holds: one block a row, twice over the keys, the
// first time with a running maximum and sum.  4 x 8 x 100 x 9000 bf16: 126 us,
// 1.0 TB/s, element by element; a row is not split, so few of them leave SMs idle
// (eight of a million keys: 3 ms).
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
            const float bias = a.table[static_cast<int64_t>(u) * a.heads + head];
            x = fmaf(to_f32(s[j]), a.scale, bias);
            return bias != -INFINITY;
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
        float all[1] = {top}, total[1];
        team_reduce<256, true>(all, red[0]);
        const float base = all[0] == -INFINITY ? 0.0f : all[0];
        total[0] = top == -INFINITY && sum == 0.0f ? 0.0f : sum * exp2_fast((top - base) * LOG2E);
        team_reduce<256, false>(total, red[1]);
        const float inv = total[0] == 0.0f ? 0.0f : reciprocal(total[0]);
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

// R rows: da into p from probs p and gradients d (0 where masked), dscores
// stored for the first `stored` of them, `step` elements apart.
template <typename S, int R>
__device__ __forceinline__ void grad_rows(float (&p)[R][S::NV][S::EV], float (&d)[R][S::NV][S::EV],
                                          const Buckets<S>& bucket, const RelationArgs& a, typename S::T* ds,
                                          int64_t step, int lane, int stored, float* red)
{
    constexpr int EV = S::EV, NV = S::NV;
    const int K = static_cast<int>(a.keys);
    float dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        dot[r] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < EV; ++e) dot[r] = fmaf(p[r][v][e], d[r][v][e], dot[r]);
    }
    team_reduce<S::L, false>(dot, red);
    bool odd = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        odd |= !(fabsf(dot[r]) < INFINITY);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < EV; ++e) p[r][v][e] *= d[r][v][e] - dot[r];
    }
    if (__any_sync(FULL, odd)) {
        // A row that met an infinity or NaN leaves its masked places 0 all the same.
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e)
                    if (bucket(v, e) == a.num_buckets) p[r][v][e] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= stored) break;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[EV];
#pragma unroll
            for (int e = 0; e < EV; ++e) y[e] = a.scale * p[r][v][e];
            if (S::inside(v, lane, K))
                *reinterpret_cast<Pack<typename S::T, EV>*>(ds + r * step + S::first(v, lane)) =
                    pack_results<typename S::T, EV>(y);
        }
    }
}

// By image: block (x, y, z) = (query tile, image chunk, head).
template <typename S>
__global__ void __launch_bounds__(256, S::GRAD_BLOCKS)
relation_grad_image_kernel(RelationArgs a, unsigned per, int columns, float* part)
{
    using T = typename S::T;
    constexpr int EV = S::EV, NV = S::NV, L = S::L;
    extern __shared__ float hist[];  // [num_buckets + 1][columns]
    __shared__ float red[2][8];
    const int K = static_cast<int>(a.keys), nb = a.num_buckets, head = static_cast<int>(blockIdx.z);
    const int lane = static_cast<int>(threadIdx.x) % L;
    const unsigned batch = static_cast<unsigned>(a.batch);  // the loop counts past it
    const unsigned t0 = blockIdx.y * per, t1 = t0 + per < batch ? t0 + per : batch;
    for (int x = threadIdx.x; x < (nb + 1) * columns; x += 256) hist[x] = 0.0f;
    const unsigned Q = static_cast<unsigned>(a.queries), want = blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool real = want < Q;
    const int64_t i = real ? want : Q - 1;
    const int64_t step = static_cast<int64_t>(a.heads) * Q * K;
    const int64_t first = (static_cast<int64_t>(head) * Q + i) * K + t0 * step;
    const T* p = static_cast<const T*>(a.probs) + first;
    const T* dp = static_cast<const T*>(a.scores) + first;
    T* ds = static_cast<T*>(a.out) + first;
    constexpr int R = S::ROWS;
    Pack<T, EV> pn[R][NV], dn[R][NV];
    if (R == 1) {
        S::load(pn[0], p, K, lane);
        S::load(dn[0], dp, K, lane);
    }
    Buckets<S> bucket;
    Valid<S> valid;
    auto map = [&]() {
        Pack<int16_t, EV> q[NV];
        Pack<uint8_t, EV> key[NV];
        S::load(q, a.buckets + i * K, K, lane);
        bucket.set(q, key, false, K, lane, nb);
    };
    map();
    valid.set(bucket, nb);
    float acc[NV][EV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < EV; ++e) acc[v][e] = 0.0f;
    for (unsigned t = t0; t < t1; t += R) {
        const int rows = t + R < t1 ? R : static_cast<int>(t1 - t);
        if (R > 1) {  // past the last row: that row again, neither stored nor added
#pragma unroll
            for (int r = 0; r < R; ++r) {
                S::load(pn[r], p + (r < rows ? r : rows - 1) * step, K, lane);
                S::load(dn[r], dp + (r < rows ? r : rows - 1) * step, K, lane);
            }
        }
        p += R * step;
        dp += R * step;
        float x[R][NV][EV], d[R][NV][EV];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                valid.take(x[r][v], pn[r][v], v);
                valid.take(d[r][v], dn[r][v], v);
            }
        if (R == 1 && t + 1 < t1) {
            S::load(pn[0], p, K, lane);
            S::load(dn[0], dp, K, lane);
        }
        grad_rows<S, R>(x, d, bucket, a, ds, step, lane, real ? rows : 0, red[t & 1]);
        ds += R * step;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) break;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) acc[v][e] += x[r][v][e];
        }
    }
    // The warps add their sums in turn (the map is read again: its indices need not live through the loop).
    map();
    if (!real) bucket.clear(nb);
    for (int w = 0; w < 8; ++w) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) / 32 == w) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) add_in_turn(hist, bucket(v, e), acc[v][e], columns);
        }
    }
    join_columns(hist, 1, columns, nb,
                 part + ((static_cast<int64_t>(head) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * nb);
}

// By head: block (x, y) = (share of the rows, head); each warp has a table of
// its own, of COLUMNS columns: 32 (one a lane), 16 (lanes l and l + 16 share
// one), or fewer, taken in turns (0: `columns` says how many).
template <typename S, int COLUMNS>
__global__ void __launch_bounds__(COLUMNS == 16 ? 32 * RELATION_PAIR_WARPS : 256, COLUMNS == 16 ? 2 : 1)
relation_grad_head_kernel(RelationArgs a, int columns, float* part)
{
    using T = typename S::T;
    constexpr int EV = S::EV, NV = S::NV, L = S::L;
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
    Pack<uint8_t, EV> kn[NV];
    int64_t off_next = 0;
    const bool keyed = a.key_mask != nullptr;
    auto fetch = [&](bool real) {  // a team without a row reads the first one and stores nothing
        const int64_t fb = real ? b : 0, fi = real ? i : 0;
        off_next = ((fb * a.heads + head) * Q + fi) * K;
        S::load(pn, static_cast<const T*>(a.probs) + off_next, K, lane);
        S::load(dn, static_cast<const T*>(a.scores) + off_next, K, lane);
        S::load(un, a.buckets + ((a.sets == 1 ? 0 : fb * Q) + fi) * K, K, lane);
        if (keyed) S::load(kn, a.key_mask + fb * K, K, lane);
    };
    // The next row is loaded ahead, but for long rows element by element, whose loads would not fit the registers.
    constexpr bool AHEAD = EV > 1 || NV <= 16;
    if (AHEAD && bi < rows) fetch(bi + team < rows);
    for (int turn = 0; bi < rows; turn ^= 1) {
        const bool real = bi + team < rows;
        if (!AHEAD) fetch(real);
        T* ds = static_cast<T*>(a.out) + off_next;
        Buckets<S> bucket;
        Valid<S> valid;
        bucket.set(un, kn, keyed, K, lane, nb);
        if (!real) bucket.clear(nb);
        valid.set(bucket, nb);
        float x[1][NV][EV], d[1][NV][EV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            valid.take(x[0][v], pn[v], v);
            valid.take(d[0][v], dn[v], v);
        }
        bi += stride;
        b += step_b;
        i += step_i;
        if (i >= Q) {
            i -= Q;
            ++b;
        }
        if (AHEAD && bi < rows) fetch(bi + team < rows);
        grad_rows<S, 1>(x, d, bucket, a, ds, 0, lane, real ? 1 : 0, red[turn]);
        if (COLUMNS == 32) {
            float* column = mine + lane_id();
#pragma unroll
            for (int k = 0; k + 1 < S::E; k += 2)
                add_two(column, bucket(k / EV, k % EV), x[0][k / EV][k % EV], bucket((k + 1) / EV, (k + 1) % EV),
                        x[0][(k + 1) / EV][(k + 1) % EV]);
            if (S::E % 2) column[bucket(NV - 1, EV - 1) * 32] += x[0][NV - 1][EV - 1];
        } else if (COLUMNS == 16) {
            // Where both lanes of a column hold pairs of one bucket the lower adds for the two, and the upper adds what it
            // has to the last row (nothing to row 0 if that bucket is the last row, the masked pairs'): their rows always
            // differ.  The barrier orders an element's additions before the next one's, which may meet the other lane's
            // rows.  A branch in place of the upper's other row takes 306 us for 220 (16 x 8 x 1000 x 1000 bf16).
            float* column = mine + lane_id() % 16;
            const bool lower = lane_id() < 16;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    const int u = bucket(v, e), other = __shfl_xor_sync(FULL, u, 16);
                    const float d = x[0][v][e], more = __shfl_xor_sync(FULL, d, 16);
                    const bool same = u == other;
                    column[(same && !lower ? (u == nb ? 0 : nb) : u) * 16] += same ? d + more : d;
                    __syncwarp();
                }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < EV; ++e) add_in_turn(mine, bucket(v, e), x[0][v][e], columns);
        }
    }
    join_columns(hist, warps, columns, nb, part + (static_cast<int64_t>(head) * gridDim.x + blockIdx.x) * nb);
}

// Rows longer than a block holds: one warp a row, twice over the keys.  4 x 8 x
// 100 x 9000 bf16: 285 us; eight rows of a million keys 20 ms.
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
    for (int v = most; v > 1; v /= 2)
        if (a.keys % v == 0 && fits(a.scores, v * e) && fits(a.probs, v * e) && fits(a.out, v * e) &&
            fits(a.buckets, v * 2) && (!a.key_mask || fits(a.key_mask, v)))
            return v;
    return 1;
}

// f(Shape) with the first of the vector counts NV that holds the row; each
// count serves the rows that the one before does not.
template <typename T, int EV, int L, int PREV, typename F>
inline void pick_count(const RelationArgs&, F) {}

template <typename T, int EV, int L, int PREV, int NV, int... MORE, typename F>
inline void pick_count(const RelationArgs& a, F f)
{
    if (a.keys <= NV * L * EV || sizeof...(MORE) == 0) f(Shape<T, EV, L, NV, NV - PREV>{});
    else pick_count<T, EV, L, NV, MORE...>(a, f);
}

// f(Shape) for the row's length and vector width.  Eight lanes a row up to 64
// keys, 16 up to 128, a warp up to 1024, a block up to 8192.
template <typename T, bool GRAD, typename F>
inline void relation_shape(const RelationArgs& a, F f)
{
    constexpr int MOST = sizeof(T) == 2 ? 8 : 4;
    const int v = relation_vector(a, MOST);
    const int64_t K = a.keys;
    if (v == 8) {
        if constexpr (MOST == 8) {
            if (K <= 64) pick_count<T, 8, 8, 0, 1>(a, f);
            else if (K <= 128) pick_count<T, 8, 16, 0, 1>(a, f);
            else if (K <= 1024) pick_count<T, 8, 32, 0, 1, 2, 3, 4>(a, f);
            else pick_count<T, 8, 256, 0, 1, 2, 4>(a, f);
        }
    } else if (v == 4) {
        if (K <= 64) pick_count<T, 4, 8, 0, 1, 2>(a, f);
        else if (K <= 128) pick_count<T, 4, 16, 1, 2>(a, f);
        else if (K <= 1024) pick_count<T, 4, 32, 1, 2, 3, 4, 6, 8>(a, f);
        else pick_count<T, 4, 256, 1, 2, 4, 8>(a, f);
    } else if (v == 2) {
        if (K <= 64) pick_count<T, 2, 8, 0, 1, 2, 3, 4>(a, f);
        else if (K <= 128) pick_count<T, 2, 16, 2, 4>(a, f);
        else if (K <= 1024) pick_count<T, 2, 32, 2, 4, 8, 12, 16>(a, f);
        else pick_count<T, 2, 256, 2, 8, 16>(a, f);
    } else {
        if (K <= 64) pick_count<T, 1, 8, 0, 1, 2, 4, 6, 7, 8>(a, f);
        else if (K <= 128) pick_count<T, 1, 16, 4, 6, 8>(a, f);
        else if (GRAD && K <= 1024) pick_count<T, 1, 32, 4, 6, 8, 12, 16, 24, 32>(a, f);
        else if (!GRAD && K <= 512) pick_count<T, 1, 32, 4, 6, 8, 12, 16>(a, f);
        else if (!GRAD) pick_count<T, 1, 256, 2, 3, 4, 8, 16, 32>(a, f);
        else pick_count<T, 1, 256, 4, 8, 16, 32>(a, f);
    }
}

constexpr int64_t blocks_over(int64_t n, int64_t each) { return (n + each - 1) / each; }

template <typename T>
inline void softmax_type(const RelationArgs& a, cudaStream_t st)
{
    if (a.keys > RELATION_MOST) {
        const int64_t rows = a.batch * a.heads * a.queries;
        relation_softmax_long_kernel<T><<<static_cast<unsigned>(rows < SMS * 8 ? rows : SMS * 8), 256, 0, st>>>(a, rows);
        return;
    }
    relation_shape<T, false>(a, [&](auto shape) {
        using S = decltype(shape);
        const bool image = relation_by_image(a);
        const int64_t anchors = (image ? a.heads : a.batch) * a.queries, inner = image ? a.batch : a.heads;
        const int64_t blocks = blocks_over(anchors, 256 / S::L);
        const bool staged = image && stretches<S>(a);
        size_t smem = staged ? 2 * S::ROWS * sizeof(T) * Stretch<S>::TEAMS * a.keys : 0;
        // Chunks of the inner index: one wave of resident blocks.
        static const int held = resident_blocks(256, reinterpret_cast<const void*>(relation_softmax_kernel<S, true, false>));
        const int fit = staged ? static_cast<int>(220 * 1024 / (smem + 1024)) : held;
        int64_t chunks = SMS * (!image ? S::BLOCKS : fit < held ? fit : held) / blocks;
        if (chunks < 1) chunks = 1;
        if (chunks > inner) chunks = inner;
        if (!image) {  // the chunk's tables have to fit
            const int64_t most = 40 * 1024 / (4 * (a.num_buckets + 1));
            if (chunks < blocks_over(inner, most)) chunks = blocks_over(inner, most);
        }
        const unsigned per = static_cast<unsigned>(blocks_over(inner, chunks));
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(blocks_over(inner, per)));
        auto run = [&](auto* kernel) {
            if (smem > 40 * 1024) ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
            kernel<<<grid, 256, smem, st>>>(a, per);
        };
        if (image) {
            if constexpr (Stretch<S>::USED) {
                if (staged) return run(relation_softmax_kernel<S, true, true>);
            }
            run(relation_softmax_kernel<S, true, false>);
        } else {
            smem = 4 * static_cast<size_t>(per) * (a.num_buckets + 1);
            run(relation_softmax_kernel<S, false, false>);
        }
    });
}

template <typename T>
inline void grad_type(const RelationArgs& a, float* part, cudaStream_t st)
{
    const bool image = relation_grad_by_image(a);
    const RelationGradPlan p = relation_grad_plan(a.batch, a.heads, a.queries, a.keys, a.num_buckets, image);
    const size_t table = 4 * static_cast<size_t>(a.num_buckets + 1) * p.columns;
    if (a.keys > RELATION_MOST) {
        ensure_dynamic_smem(reinterpret_cast<const void*>(relation_grad_long_kernel<T>), table * p.warps);
        relation_grad_long_kernel<T><<<dim3(static_cast<unsigned>(p.blocks), a.heads), p.warps * 32, table * p.warps,
                                       st>>>(a, p.columns, part);
        return;
    }
    relation_shape<T, true>(a, [&](auto shape) {
        using S = decltype(shape);
        if (image) {
            relation_grad_image_kernel<S><<<dim3(static_cast<unsigned>(p.blocks), static_cast<unsigned>(p.chunks),
                                                 a.heads), 256, table, st>>>(a, static_cast<unsigned>(p.per), p.columns,
                                                                             part);
        } else {
            auto* k = p.columns == 32 ? relation_grad_head_kernel<S, 32> : relation_grad_head_kernel<S, 0>;
            if constexpr (S::L <= 32)
                if (p.columns == 16) k = relation_grad_head_kernel<S, 16>;
            ensure_dynamic_smem(reinterpret_cast<const void*>(k), table * p.warps);
            k<<<dim3(static_cast<unsigned>(p.blocks), a.heads), p.warps * 32, table * p.warps, st>>>(a, p.columns,
                                                                                                    part);
        }
    });
}

}  // namespace gbnms
