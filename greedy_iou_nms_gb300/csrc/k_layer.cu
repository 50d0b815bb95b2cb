// Layer normalisation: launches by type, and the join of the parameters'
// gradients.
#include "k_layer.cuh"

namespace gbnms {

namespace {

// A column's parts go to SLOTS threads in turn; their sums are joined in order by
// one thread, or in a tree by a warp where there are many.
template <int COLUMNS, int SLOTS>
__global__ void __launch_bounds__(COLUMNS * SLOTS)
column_join_kernel(const float* parts, int64_t blocks, int64_t columns, int64_t split, float* first, float* second)
{
    __shared__ LongSum sums[SLOTS][COLUMNS + 1];
    pdl_wait();  // the parts are there
    const int64_t e = static_cast<int64_t>(blockIdx.x) * COLUMNS + threadIdx.x;
    LongSum s{0.0f, 0.0f};
    if (e < columns) {
        constexpr int AHEAD = 4;
        for (int64_t b = threadIdx.y; b < blocks; b += AHEAD * SLOTS) {
            float v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[k] = b + k * SLOTS < blocks ? parts[(b + k * SLOTS) * columns + e] : 0.0f;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (b + k * SLOTS < blocks) s.add(v[k]);
        }
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    const int thread = threadIdx.y * COLUMNS + threadIdx.x;
    int64_t c = static_cast<int64_t>(blockIdx.x) * COLUMNS;
    if constexpr (SLOTS > 32) {
        const int warp = thread / 32, lane = thread % 32;
        if (warp >= COLUMNS) return;
        c += warp;
        s = sums[lane][warp];
#pragma unroll
        for (int k = 32; k < SLOTS; k += 32) s.add(sums[k + lane][warp]);
#pragma unroll
        for (int o = 16; o; o >>= 1) s.add(LongSum{__shfl_down_sync(FULL, s.sum, o), __shfl_down_sync(FULL, s.off, o)});
        if (lane) return;
    } else {
        if (thread >= COLUMNS) return;
        c += thread;
        s = sums[0][thread];
#pragma unroll
        for (int k = 1; k < SLOTS; ++k) s.add(sums[k][thread]);
    }
    if (c < columns) {
        float* out = c < split ? first : second;
        if (out) out[c < split ? c : c - split] = s.value();
    }
}

template <int COLUMNS, int SLOTS>
void launch_join(const float* parts, int64_t blocks, int64_t columns, int64_t split, float* first, float* second, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((columns + COLUMNS - 1) / COLUMNS));
    cfg.blockDim = dim3(COLUMNS, SLOTS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, column_join_kernel<COLUMNS, SLOTS>, parts, blocks, columns, split, first, second);
}

int64_t launch_rows(const LayerArgs& args, float* parts, bool grad, cudaStream_t st)
{
    LayerArgs a = args;
    a.once = beyond_l2((grad ? 3 : 2) * (a.type == NMS_TYPE_F32 ? 4 : 2) * a.rows * a.width);
    if (a.type == NMS_TYPE_F32) return launch_layer_f32(a, parts, grad, st);
    if (a.type == NMS_TYPE_F16) return launch_layer_f16(a, parts, grad, st);
    return launch_layer_bf16(a, parts, grad, st);
}

}  // namespace

void launch_layer_norm(const LayerArgs& a, cudaStream_t st) { launch_rows(a, nullptr, false, st); }

size_t layer_grad_workspace_bytes(int64_t rows, int width)
{
    int64_t most = 0;
    for (const bool single : {false, true}) {
        const LayerShape s = layer_shape(width, single);
        const int64_t blocks = layer_grad_blocks(rows, s.team, layer_grad_resident(s.team, s.values));
        if (blocks > most) most = blocks;
    }
    return static_cast<size_t>(most) * 2 * width * sizeof(float);
}

void launch_layer_grad(const LayerArgs& a, void* workspace, cudaStream_t st)
{
    float* parts = a.dweight || a.dbias ? static_cast<float*>(workspace) : nullptr;
    const int64_t blocks = launch_rows(a, parts, true, st);
    if (!parts) return;
    launch_column_join(parts, blocks, 2 * static_cast<int64_t>(a.width), a.width, a.dweight,
                       a.dbias, st);
}

void launch_column_join(const float* parts, int64_t blocks, int64_t columns, int64_t split, float* first, float* second,
                        cudaStream_t st)
{
    if (blocks <= 32) launch_join<64, 4>(parts, blocks, columns, split, first, second, st);
    else if (blocks <= 256) launch_join<32, 16>(parts, blocks, columns, split, first, second, st);
    else launch_join<8, 128>(parts, blocks, columns, split, first, second, st);
}

}  // namespace gbnms
