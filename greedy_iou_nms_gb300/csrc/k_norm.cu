// Group normalisation: the scratch's size and the dispatch by type
// (k_norm.cuh has the kernels).
#include "k_norm.cuh"

namespace gbnms {

size_t norm_workspace_bytes(int64_t batch, int64_t pixels, int channels, int groups)
{
    const size_t image = static_cast<size_t>(batch) * channels;
    return 16 * image * norm_pieces(batch, pixels, channels) + 8 * image + 8 * static_cast<size_t>(batch) * groups + 256;
}

void norm_f32(const NormArgs& a, void* ws, cudaStream_t st, bool grad);
void norm_f16(const NormArgs& a, void* ws, cudaStream_t st, bool grad);
void norm_bf16(const NormArgs& a, void* ws, cudaStream_t st, bool grad);

static void norm_any(const NormArgs& a, void* ws, cudaStream_t st, bool grad)
{
    if (a.type == NMS_TYPE_F32) norm_f32(a, ws, st, grad);
    else if (a.type == NMS_TYPE_F16) norm_f16(a, ws, st, grad);
    else norm_bf16(a, ws, st, grad);
}

void launch_norm(const NormArgs& a, void* workspace, cudaStream_t st) { norm_any(a, workspace, st, false); }
void launch_norm_grad(const NormArgs& a, void* workspace, cudaStream_t st) { norm_any(a, workspace, st, true); }

}  // namespace gbnms
