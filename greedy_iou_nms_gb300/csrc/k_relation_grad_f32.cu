// The gradient of the relation weights for one element type (translation
// units of their own compile in parallel).
#include "k_relation.cuh"

namespace gbnms {

void relation_grad_f32(const RelationArgs& a, float* part, cudaStream_t st) { grad_type<float>(a, part, st); }

}  // namespace gbnms
