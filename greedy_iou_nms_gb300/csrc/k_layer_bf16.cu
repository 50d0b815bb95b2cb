// Layer normalisation of bfloat16 rows.
#include "k_layer.cuh"

namespace gbnms {

int64_t launch_layer_bf16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    return launch_layer_type<__nv_bfloat16>(a, parts, grad, st);
}

}  // namespace gbnms
