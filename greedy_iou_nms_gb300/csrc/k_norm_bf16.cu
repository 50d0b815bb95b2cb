// Group normalisation for one element type (translation units of their own
// compile in parallel).
#include "k_norm.cuh"

namespace gbnms {

void norm_bf16(const NormArgs& a, void* ws, cudaStream_t st, bool grad) { norm_type<__nv_bfloat16>(a, ws, st, grad); }

}  // namespace gbnms
