// Group normalisation for one element type (translation units of their own
// compile in parallel).
#include "k_norm.cuh"

namespace gbnms {

void norm_f32(const NormArgs& a, void* ws, cudaStream_t st, bool grad) { norm_type<float>(a, ws, st, grad); }

}  // namespace gbnms
