// The bucket map of relative positions, the dispatch of the relation kernels
// (k_relation.cuh) by type and the last step of their gradient.
#include "head.cuh"
#include "internal.h"
#include "relation_plan.h"

namespace gbnms {

// --------------------------------------------------------------------- map

constexpr int BK_THREADS = 256;

// buckets[set][i][j] = sum over the axes of lut[axis][clamp(k - q)], -1 when
// a part is negative or the sum does not fit.
__global__ void __launch_bounds__(BK_THREADS)
relation_buckets_kernel(BucketArgs a)
{
    const int64_t all = a.sets * a.queries * a.keys, step = static_cast<int64_t>(gridDim.x) * BK_THREADS;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * BK_THREADS + threadIdx.x; e < all; e += step) {
        const int64_t j = e % a.keys, row = e / a.keys, i = row % a.queries, set = row / a.queries;
        const int32_t* q = a.q_pos + ((a.q_sets == 1 ? 0 : set) * a.queries + i) * a.axes;
        const int32_t* k = a.k_pos + ((a.k_sets == 1 ? 0 : set) * a.keys + j) * a.axes;
        int64_t sum = 0;
        bool masked = false;
        for (int x = 0; x < a.axes; ++x) {
            int64_t d = static_cast<int64_t>(k[x]) - q[x];
            d = d < -a.reach ? -a.reach : (d > a.reach ? a.reach : d);
            const int part = a.lut[x * (2 * a.reach + 1) + a.reach + d];
            masked |= part < 0;
            sum += part;
        }
        a.buckets[e] = static_cast<int16_t>(masked || sum > 32767 ? -1 : sum);
    }
}

void launch_relation_buckets(const BucketArgs& a, cudaStream_t st)
{
    const int64_t want = (a.sets * a.queries * a.keys + BK_THREADS - 1) / BK_THREADS;
    relation_buckets_kernel<<<static_cast<unsigned>(want < SMS * 64 ? want : SMS * 64), BK_THREADS, 0, st>>>(a);
}

// ---------------------------------------------------------------- dispatch

void relation_softmax_f32(const RelationArgs& a, cudaStream_t st);
void relation_softmax_f16(const RelationArgs& a, cudaStream_t st);
void relation_softmax_bf16(const RelationArgs& a, cudaStream_t st);
void relation_grad_f32(const RelationArgs& a, float* part, cudaStream_t st);
void relation_grad_f16(const RelationArgs& a, float* part, cudaStream_t st);
void relation_grad_bf16(const RelationArgs& a, float* part, cudaStream_t st);

void launch_relation_softmax(const RelationArgs& a, cudaStream_t st)
{
    if (a.type == NMS_TYPE_F32) relation_softmax_f32(a, st);
    else if (a.type == NMS_TYPE_F16) relation_softmax_f16(a, st);
    else relation_softmax_bf16(a, st);
}

// Lanes of a row's team (k_relation.cuh).
static int team_lanes(int64_t keys) { return keys <= 64 ? 8 : keys <= 128 ? 16 : keys <= 1024 ? 32 : 256; }

RelationGradPlan relation_grad_plan(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets,
                                    bool image)
{
    RelationGradPlan p{};
    const int lanes = keys > RELATION_MOST ? 32 : team_lanes(keys);
    if (image) {
        // One table a block, small enough for several blocks on an SM.
        p.columns = (num_buckets + 1) * 128 <= 46 * 1024 ? 32 : 8;
        p.warps = 8;
        const int64_t teams = 256 / lanes;
        p.blocks = (queries + teams - 1) / teams;
        const int64_t held = (keys + lanes - 1) / lanes;  // elements a lane
        const int resident = held <= 8 ? 3 : held <= 16 ? 2 : 1;
        const int64_t want = SMS * resident / (p.blocks * heads);  // one wave
        p.chunks = want < 1 ? 1 : want > batch ? batch : want;
        p.per = (batch + p.chunks - 1) / p.chunks;
        p.chunks = (batch + p.per - 1) / p.per;
        return p;
    }
    // A table a warp: 32 columns if six warps' fit, else fewer.
    constexpr int ROOM = 208 * 1024;
    const int need = lanes == 256 ? 8 : 6;
    for (p.columns = 32; p.columns > 4 && need * (num_buckets + 1) * 4 * p.columns > ROOM; p.columns /= 2) {}
    const int fit = ROOM / ((num_buckets + 1) * 4 * p.columns);
    p.warps = fit > 8 ? 8 : fit;
    const int64_t teams = p.warps * 32 / lanes, rows = batch * queries, want = (rows + teams - 1) / teams;
    const int resident = ROOM / (p.warps * (num_buckets + 1) * 4 * p.columns);
    const int64_t most = (SMS * static_cast<int64_t>(resident < 4 ? resident : 4) + heads - 1) / heads;
    p.blocks = want < most ? want : most;
    p.chunks = 1;
    return p;
}

size_t relation_grad_workspace_bytes(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets)
{
    if (batch == 0 || queries == 0 || keys == 0) return 256;
    const int64_t a = relation_grad_plan(batch, heads, queries, keys, num_buckets, false).parts();
    const int64_t b = relation_grad_plan(batch, heads, queries, keys, num_buckets, true).parts();
    return 4 * static_cast<size_t>(heads) * (a > b ? a : b) * num_buckets + 256;
}

// dtable[u][h] = sum over the parts [heads][parts][num_buckets], eight warps
// a block over 32 buckets, each warp every eighth part.
__global__ void __launch_bounds__(256)
relation_table_kernel(const float* part, int64_t parts, int num_buckets, int heads, float* dtable)
{
    __shared__ float s[8][32];
    const int u = static_cast<int>(blockIdx.x) * 32 + static_cast<int>(lane_id()), w = static_cast<int>(threadIdx.x) / 32;
    const int h = static_cast<int>(blockIdx.y);
    float v = 0.0f;
    if (u < num_buckets)
        for (int64_t k = w; k < parts; k += 8) v += part[(h * parts + k) * num_buckets + u];
    s[w][lane_id()] = v;
    __syncthreads();
    if (w == 0 && u < num_buckets) {
        for (int k = 1; k < 8; ++k) v += s[k][lane_id()];
        dtable[static_cast<int64_t>(u) * heads + h] = v;
    }
}

void launch_relation_grad(const RelationArgs& a, void* workspace, cudaStream_t st)
{
    float* part = static_cast<float*>(workspace);
    if (a.type == NMS_TYPE_F32) relation_grad_f32(a, part, st);
    else if (a.type == NMS_TYPE_F16) relation_grad_f16(a, part, st);
    else relation_grad_bf16(a, part, st);
    const int64_t parts = relation_grad_plan(a.batch, a.heads, a.queries, a.keys, a.num_buckets,
                                             relation_by_image(a) && a.keys <= RELATION_MOST).parts();
    relation_table_kernel<<<dim3((a.num_buckets + 31) / 32, a.heads), 256, 0, st>>>(part, parts, a.num_buckets,
                                                                                     a.heads, a.dtable);
}

}  // namespace gbnms
