// Group normalisation for one element type (translation units of their own
// compile in parallel).
#include "k_norm.cuh"

namespace gbnms {

void norm_f16(const NormArgs& a, void* ws, cudaStream_t st, bool grad) { norm_type<__half>(a, ws, st, grad); }

}  // namespace gbnms
