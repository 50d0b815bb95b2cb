// Device helpers shared by the operators of a trainable detection head
// (k_norm.cu, k_dropout.cu, k_relation.cu): element types, activations and
// the counter-based generator.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "head.h"

namespace gbnms {

// V consecutive elements moved by one access of sizeof(T) * V bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// One rounding, to nearest even, of a result held in binary32.
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T> __device__ __forceinline__ uint32_t pack_two(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack_two<__half>(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack_two<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack_two<float>(float, float) { return 0; }  // never called

// Rounds EV results to their type.
template <typename T, int EV>
__device__ __forceinline__ Pack<T, EV> pack_results(const float (&x)[EV])
{
    Pack<T, EV> q;
    if constexpr (sizeof(T) == 2 && EV % 2 == 0) {
#pragma unroll
        for (int e = 0; e < EV; e += 2) reinterpret_cast<uint32_t*>(&q)[e / 2] = pack_two<T>(x[e], x[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < EV; ++e) q.v[e] = from_f32<T>(x[e]);
    }
    return q;
}

// A norm parameter: binary32, or the type of the features.
template <typename T>
__device__ __forceinline__ float load_param(const void* p, int is_f32, int64_t i)
{
    return is_f32 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const T*>(p)[i]);
}

// ------------------------------------------------------------------- dropout
//
// Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): counter (block, offset), key the seed.  A block's
// four words are eight 16-bit fields, low half first, one for each of the
// elements 8 * block .. 8 * block + 7; an element is kept iff its field is
// below DropArgs::limit.
__device__ __forceinline__ uint4 philox(uint64_t block, const DropArgs& d)
{
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = d.offset_lo, c3 = d.offset_hi, k0 = d.key_lo, k1 = d.key_hi;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0, n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c1 = static_cast<uint32_t>(b);
        c3 = static_cast<uint32_t>(a);
        c0 = n0;
        c2 = n2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// v[i] = 0 for the dropped of the elements first .. first + V - 1 (first a
// multiple of V, so they lie in one block), whatever their value was; the
// caller applies the factor.  A field is compared in the top half of a word.
template <int V>
__device__ __forceinline__ void drop_mask(float (&v)[V], uint64_t first, const DropArgs& d)
{
    const uint4 w = philox(first >> 3, d);
    const uint32_t limit = d.limit << 16;
    if (V == 8) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (i & 1 ? x[i / 2] : x[i / 2] << 16) < limit ? v[i] : 0.0f;
    } else {
        // The parts of a block one after another: from word at / 2 on, and within it from field at % 2 on.
        const int at = static_cast<int>(first & 7);
        uint32_t x0 = at < 4 ? w.x : w.z, x1 = at < 4 ? w.y : w.w;
        if (V < 4 && (at & 2)) x0 = x1;
        if (V < 2 && (at & 1)) x0 = x0 & 0xffff0000u;
        else if (V < 2) x0 <<= 16;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t word = i < 2 ? x0 : x1;
            v[i] = (V < 2 ? word : i & 1 ? word : word << 16) < limit ? v[i] : 0.0f;
        }
    }
}

template <int V>
__device__ __forceinline__ void drop(float (&v)[V], uint64_t first, const DropArgs& d)
{
    drop_mask<V>(v, first, d);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= d.factor;
}

// ---------------------------------------------------------------- activation
//
// The hardware's 2^x and 1/x (each right to about 2^-22 of its result) carry
// the sigmoid, which is right to 2^-22 (1 + |z|) of itself (2^-126 and below is
// 0), and the normal distribution.

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float LOG2E = 1.44269504f;

__device__ __forceinline__ float sigmoid(float z) { return reciprocal(1.0f + exp2_fast(-LOG2E * z)); }

// The normal distribution function and density at z, for features of type T.
// The tail beyond x = |z| is the density times Mills' ratio, which is t = 1 / (1
// + c x) times a polynomial, fitted with weights until its largest errors were
// equal.
//   binary32: degree 8 in 1 - t, whose roundings are small where the tail is
//     large; for z < 0 within 2^-24 (20 + 2 z^2) of itself.
//   16 bits: degree 6 in t: within 2^-21, and for -10 < z < 0 within 3e-5 of
//     itself, a sixteenth of half a step of binary16.
// A polynomial of degree 4 of small absolute error alone, off by 5e-4 of the
// tail at -4, takes 85 us for 87 (gradient of 8 x 25600 x 128 fp16 with dropout) and
// 96 for 98 (of 16 x 6400 x 256 fp32).
template <typename T>
__device__ __forceinline__ float normal_cdf(float z, float& density)
{
    const float x = fabsf(z);
    float q, t;
    if constexpr (sizeof(T) == 4) {
        density = 0.398942280f * exp2_fast(-0.5f * LOG2E * z * z);
        t = reciprocal(fmaf(0.26f, x, 1.0f));
        const float s = 0.26f * fminf(x, 0x1.fffffep127f) * t;  // of an infinity, where t is 0, a number too
        q = fmaf(0.0790923014f, s, -0.237447441f);
        q = fmaf(q, s, 0.101926945f);
        q = fmaf(q, s, 0.350009143f);
        q = fmaf(q, s, -0.0844072327f);
        q = fmaf(q, s, -1.44065559f);
        q = fmaf(q, s, 2.83110499f);
        q = fmaf(q, s, -2.59284019f);
        q = fmaf(q, s, 1.25331414f);
    } else {
        density = exp2_fast(fmaf(-0.5f * LOG2E * z, z, -1.32574806f));  // log2 of 1 / sqrt(2 pi)
        t = reciprocal(fmaf(0.34f, x, 1.0f));
        q = fmaf(0.110553453f, t, -0.494552710f);
        q = fmaf(q, t, 0.647315039f);
        q = fmaf(q, t, -0.0634329129f);
        q = fmaf(q, t, 0.385721482f);
        q = fmaf(q, t, 0.326906588f);
        q = fmaf(q, t, 0.340803222f);
    }
    const float tail = q * t * density;
    return z < 0.0f ? tail : 1.0f - tail;
}

// v = act(v), one uniform branch for V elements; T: the features' type.
template <typename T, int V>
__device__ __forceinline__ void act_values(float (&v)[V], int act)
{
    if (act == NMS_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i]);
    } else if (act == NMS_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    } else if (act == NMS_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float density;
            v[i] *= normal_cdf<T>(v[i], density);
        }
    }
}

// d *= act'(z).
template <typename T, int V>
__device__ __forceinline__ void act_slopes(float (&d)[V], const float (&z)[V], int act)
{
    if (act == NMS_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float r = sigmoid(z[i]);
            d[i] *= r * fmaf(z[i], 1.0f - r, 1.0f);
        }
    } else if (act == NMS_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = z[i] > 0.0f ? d[i] : 0.0f;
    } else if (act == NMS_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float density;
            const float cdf = normal_cdf<T>(z[i], density);
            d[i] *= fmaf(z[i], density, cdf);
        }
    }
}

// ----------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// A sum of any number of terms: what each addition rounds off is added up
// beside it (Neumaier, 1974), so that roundings that go one way do not mount.
struct LongSum {
    float sum, off;
    __device__ __forceinline__ void add(float v)
    {
        const float t = __fadd_rn(sum, v);
        off += fabsf(sum) >= fabsf(v) ? (sum - t) + v : (v - t) + sum;
        sum = t;
    }
    __device__ __forceinline__ void add(const LongSum& o)
    {
        add(o.sum);
        off += o.off;
    }
    // An infinite sum has left no number in `off`.
    __device__ __forceinline__ float value() const { return fabsf(off) < INFINITY ? sum + off : sum; }
};

// --------------------------------------------------------------------- host

// Blocks of so many threads of a kernel that an SM holds.
inline int resident_blocks(int threads, const void* kernel)
{
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) == cudaSuccess && n > 0 ? n : 1;
}

}  // namespace gbnms
