// The 16-bit parts of a binary32 number that stand for it on the tensor cores:
// three of bfloat16 (see k_product_split.cu), or two where 16 bits are what the
// other operand has.
#pragma once

#include "head.cuh"

namespace gbnms {

// x = h + m + l.  Where x rounds to an infinity (and is none) its first part is
// cut instead; of a NaN the first part is all there is.  An infinity is the last
// part, with 1 of its sign as the first: the last part is multiplied by first parts
// only (and first by last), which are 0 for 0 alone, so that products with infinities
// are what they are in binary32 (infinity times 0 a NaN); a first part of infinity met
// the zeros in other numbers' lower parts.
template <int V>
__device__ __forceinline__ void split_parts(const float (&x)[V], Pack<__nv_bfloat16, V>& h, Pack<__nv_bfloat16, V>& m,
                                            Pack<__nv_bfloat16, V>& l)
{
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const bool finite = fabsf(x[k]) < INFINITY;
        h.v[k] = __float2bfloat16_rn(x[k]);
        if (finite && fabsf(to_f32(h.v[k])) == INFINITY) h.v[k] = __float2bfloat16_rz(x[k]);
        const float rest = finite ? x[k] - to_f32(h.v[k]) : 0.0f;
        m.v[k] = __float2bfloat16_rn(rest);
        l.v[k] = __float2bfloat16_rn(rest - to_f32(m.v[k]));
        if (fabsf(x[k]) == INFINITY) {
            l.v[k] = h.v[k];
            h.v[k] = __float2bfloat16_rn(copysignf(1.0f, x[k]));
        }
    }
}

__device__ __forceinline__ __half cut(float x, __half) { return __float2half_rz(x); }
__device__ __forceinline__ __nv_bfloat16 cut(float x, __nv_bfloat16) { return __float2bfloat16_rz(x); }

// x = h + l, to 2^-18 of itself (bfloat16), or to 2^-22 and 2^-25 (binary16).  The
// same of what rounds to an infinity, and of infinities and NaN.
template <typename T, int V>
__device__ __forceinline__ void split_two(const float (&x)[V], Pack<T, V>& h, Pack<T, V>& l)
{
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const bool finite = fabsf(x[k]) < INFINITY;
        h.v[k] = from_f32<T>(x[k]);
        if (finite && fabsf(to_f32(h.v[k])) == INFINITY) h.v[k] = cut(x[k], T());
        l.v[k] = from_f32<T>(finite ? x[k] - to_f32(h.v[k]) : 0.0f);
    }
}

}  // namespace gbnms
