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

__device__ __forceinline__ uint32_t philox_field(const uint4& w, int i)
{
    const uint32_t x = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
    return (i & 1) ? x >> 16 : x & 0xffffu;
}

// v[0..V) *= mask / keep for the elements first .. first + V - 1 (first a
// multiple of V, so they lie in one block).  A dropped element is 0 whatever
// its value was.
template <int V>
__device__ __forceinline__ void drop(float (&v)[V], uint64_t first, const DropArgs& d)
{
    const uint4 w = philox(first >> 3, d);
    if (V == 8) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = philox_field(w, i) < d.limit ? v[i] * d.factor : 0.0f;
    } else {
        const int at = static_cast<int>(first & 7);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = philox_field(w, at + i) < d.limit ? v[i] * d.factor : 0.0f;
    }
}

// ---------------------------------------------------------------- activation

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if (ACT == NMS_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == NMS_ACT_SILU) return z / (1.0f + expf(-z));
    if (ACT == NMS_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if (ACT == NMS_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (ACT == NMS_ACT_SILU) {
        const float r = 1.0f / (1.0f + expf(-z));
        return r * fmaf(z, 1.0f - r, 1.0f);
    }
    if (ACT == NMS_ACT_GELU)
        return fmaf(0.39894228f * z, expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.70710678f)));
    return 1.0f;
}

// ----------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

}  // namespace gbnms
