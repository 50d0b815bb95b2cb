// The relation kernels for one element type (a translation unit of its own:
// they compile in parallel).
#include "k_relation.cuh"

namespace gbnms {

void relation_softmax_f32(const RelationArgs& a, cudaStream_t st) { softmax_type<float>(a, st); }
void relation_grad_f32(const RelationArgs& a, float* part, cudaStream_t st) { grad_type<float>(a, part, st); }

}  // namespace gbnms
