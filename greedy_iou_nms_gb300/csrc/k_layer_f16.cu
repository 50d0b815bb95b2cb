// Layer normalisation of binary16 rows.
#include "k_layer.cuh"

namespace gbnms {

int64_t launch_layer_f16(const LayerArgs& a, float* parts, bool grad, cudaStream_t st)
{
    return launch_layer_type<__half>(a, parts, grad, st);
}

}  // namespace gbnms
