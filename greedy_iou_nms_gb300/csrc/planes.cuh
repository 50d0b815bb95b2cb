// The three bfloat16 parts of a binary32 number that stand for it on the tensor
// cores (see k_product_split.cu).
#pragma once

#include "head.cuh"

namespace gbnms {

// x = h + m + l.  Where x rounds to an infinity (and is none) its first part is
// cut instead; of a NaN or an infinity the first part is all there is.
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
    }
}

}  // namespace gbnms
