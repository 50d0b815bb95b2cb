// The relation weights for one element type (translation units of their own
// compile in parallel).
#include "k_relation.cuh"

namespace gbnms {

void relation_softmax_f16(const RelationArgs& a, cudaStream_t st) { softmax_type<__half>(a, st); }

}  // namespace gbnms
