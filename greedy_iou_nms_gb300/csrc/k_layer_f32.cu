// Layer normalisation of binary32 rows.
#include "k_layer.cuh"

namespace gbnms {

int64_t launch_layer_f32(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    return launch_layer_type<float>(a, parts, grad, st);
}

}  // namespace gbnms
