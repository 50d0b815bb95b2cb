// The relation kernels for one element type (a translation unit of its own:
// they compile in parallel).
#include "k_relation.cuh"

namespace gbnms {

void relation_softmax_bf16(const RelationArgs& a, cudaStream_t st) { softmax_type<__nv_bfloat16>(a, st); }
void relation_grad_bf16(const RelationArgs& a, float* part, cudaStream_t st) { grad_type<__nv_bfloat16>(a, part, st); }

}  // namespace gbnms
