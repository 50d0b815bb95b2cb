// Attention weights with a learned bias by buckets of relative position, and
// their gradient.
//
//   probs[b,h,i,:] = softmax over the valid j of scale * scores[b,h,i,j] +
//   table[bucket(i,j)][h]; a pair is masked by a bucket outside the table or
//   by its key's mask, a masked pair has weight 0 whatever its score is, and
//   a row without a valid pair is all zero.
//   da = probs * (dprobs - sum_j probs * dprobs), dscores = scale * da,
//   dtable[u][h] = sum of da over the pairs of bucket u.
#include "head.cuh"
#include "internal.h"

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
    relation_buckets_kernel<<<static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64), BK_THREADS, 0, st>>>(a);
}

// ----------------------------------------------------------------- softmax

// Row r of [batch][heads][queries]: its head, map row and key mask row.
struct RowAt {
    int head;
    const int16_t* map;
    const uint8_t* mask;
};

__device__ __forceinline__ RowAt row_at(const RelationArgs& a, int64_t r)
{
    RowAt w;
    const int64_t i = r % a.queries, bh = r / a.queries, b = bh / a.heads;
    w.head = static_cast<int>(bh % a.heads);
    w.map = a.buckets + ((a.sets == 1 ? 0 : b) * a.queries + i) * a.keys;
    w.mask = a.key_mask ? a.key_mask + b * a.keys : nullptr;
    return w;
}

// The bucket of a valid pair, else -1.
__device__ __forceinline__ int valid_bucket(const RelationArgs& a, const RowAt& w, int64_t j)
{
    const int u = w.map[j];
    return u >= 0 && u < a.num_buckets && (!w.mask || w.mask[j]) ? u : -1;
}

constexpr int RW = 8;  // warps of a block, one row each

template <typename T>
__global__ void __launch_bounds__(RW * 32)
relation_softmax_kernel(RelationArgs a, int64_t rows)
{
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * RW + threadIdx.x / 32; r < rows;
         r += static_cast<int64_t>(gridDim.x) * RW) {
        const RowAt w = row_at(a, r);
        const T* s = static_cast<const T*>(a.scores) + r * a.keys;
        T* p = static_cast<T*>(a.out) + r * a.keys;
        auto value = [&](int64_t j, int u) {
            return fmaf(to_f32(s[j]), a.scale, a.table[static_cast<int64_t>(u) * a.heads + w.head]);
        };
        float top = -INFINITY;
        for (int64_t j = lane_id(); j < a.keys; j += 32) {
            const int u = valid_bucket(a, w, j);
            if (u >= 0) top = fmaxf(top, value(j, u));
        }
        top = warp_max(top);
        if (top == -INFINITY) top = 0.0f;
        float sum = 0.0f;
        for (int64_t j = lane_id(); j < a.keys; j += 32) {
            const int u = valid_bucket(a, w, j);
            if (u >= 0) sum += expf(value(j, u) - top);
        }
        sum = warp_sum(sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int64_t j = lane_id(); j < a.keys; j += 32) {
            const int u = valid_bucket(a, w, j);
            p[j] = from_f32<T>(u >= 0 ? expf(value(j, u) - top) * inv : 0.0f);
        }
    }
}

template <typename T>
static void softmax_type(const RelationArgs& a, cudaStream_t st)
{
    const int64_t rows = a.batch * a.heads * a.queries, want = (rows + RW - 1) / RW;
    relation_softmax_kernel<T><<<static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64), RW * 32, 0, st>>>(a, rows);
}

void launch_relation_softmax(const RelationArgs& a, cudaStream_t st)
{
    if (a.type == NMS_TYPE_F32) softmax_type<float>(a, st);
    else if (a.type == NMS_TYPE_F16) softmax_type<__half>(a, st);
    else softmax_type<__nv_bfloat16>(a, st);
}

// ---------------------------------------------------------------- gradient
//
// A block's warps share nothing: every lane adds its pairs to a column of its
// own in its warp's [num_buckets][32] table of sums in shared memory (lane =
// bank, so no two lanes collide and the order of additions is fixed), and the
// columns are joined in order at the end.

// Blocks per head and warps per block (functions of the shape alone).
struct GradPlan {
    int warps, blocks;
};

static GradPlan grad_plan(int64_t batch, int heads, int64_t queries, int num_buckets)
{
    GradPlan p;
    const int fit = 200 * 1024 / (num_buckets * 128);
    p.warps = fit > 8 ? 8 : fit;
    const int64_t rows = batch * queries, want = (rows + p.warps - 1) / p.warps;
    const int64_t most = (152 * 2 + heads - 1) / heads;
    p.blocks = static_cast<int>(want < most ? want : most);
    if (p.blocks < 1) p.blocks = 1;
    return p;
}

size_t relation_grad_workspace_bytes(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets)
{
    (void)keys;
    return 4 * static_cast<size_t>(heads) * grad_plan(batch, heads, queries, num_buckets).blocks * num_buckets + 256;
}

template <typename T>
__global__ void relation_grad_kernel(RelationArgs a, float* part)
{
    extern __shared__ float sums[];
    const int warps = static_cast<int>(blockDim.x) / 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int head = static_cast<int>(blockIdx.y);
    float* mine = sums + static_cast<size_t>(warp) * a.num_buckets * 32 + lane_id();
    for (int u = 0; u < a.num_buckets; ++u) mine[u * 32] = 0.0f;
    for (int64_t bi = static_cast<int64_t>(blockIdx.x) * warps + warp; bi < a.batch * a.queries;
         bi += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t r = (bi / a.queries * a.heads + head) * a.queries + bi % a.queries;
        const RowAt w = row_at(a, r);
        const T* dp = static_cast<const T*>(a.scores) + r * a.keys;
        const T* p = static_cast<const T*>(a.probs) + r * a.keys;
        T* ds = static_cast<T*>(a.out) + r * a.keys;
        float dot = 0.0f;
        for (int64_t j = lane_id(); j < a.keys; j += 32)
            if (valid_bucket(a, w, j) >= 0) dot = fmaf(to_f32(p[j]), to_f32(dp[j]), dot);
        dot = warp_sum(dot);
        for (int64_t j = lane_id(); j < a.keys; j += 32) {
            const int u = valid_bucket(a, w, j);
            float da = 0.0f;
            if (u >= 0) {
                da = to_f32(p[j]) * (to_f32(dp[j]) - dot);
                mine[u * 32] += da;
            }
            ds[j] = from_f32<T>(a.scale * da);
        }
    }
    __syncthreads();
    float* out = part + (static_cast<size_t>(head) * gridDim.x + blockIdx.x) * a.num_buckets;
    for (int u = warp; u < a.num_buckets; u += warps) {
        float v = 0.0f;
        for (int k = 0; k < warps; ++k) v += sums[(static_cast<size_t>(k) * a.num_buckets + u) * 32 + lane_id()];
        v = warp_sum(v);
        if (lane_id() == 0) out[u] = v;
    }
}

// dtable[u][h] = sum over the blocks, one thread each.
__global__ void relation_table_kernel(const float* part, int blocks, int num_buckets, int heads, float* dtable)
{
    const int at = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
    if (at >= num_buckets * heads) return;
    const int u = at % num_buckets, h = at / num_buckets;
    float v = 0.0f;
    for (int b = 0; b < blocks; ++b) v += part[(static_cast<size_t>(h) * blocks + b) * num_buckets + u];
    dtable[static_cast<size_t>(u) * heads + h] = v;
}

template <typename T>
static void grad_type(const RelationArgs& a, float* part, cudaStream_t st)
{
    const GradPlan p = grad_plan(a.batch, a.heads, a.queries, a.num_buckets);
    const size_t smem = static_cast<size_t>(p.warps) * a.num_buckets * 128;
    ensure_dynamic_smem(reinterpret_cast<const void*>(relation_grad_kernel<T>), smem);
    relation_grad_kernel<T><<<dim3(p.blocks, a.heads), p.warps * 32, smem, st>>>(a, part);
    relation_table_kernel<<<(a.num_buckets * a.heads + 127) / 128, 128, 0, st>>>(part, p.blocks, a.num_buckets,
                                                                                  a.heads, a.dtable);
}

void launch_relation_grad(const RelationArgs& a, void* workspace, cudaStream_t st)
{
    float* part = static_cast<float*>(workspace);
    if (a.type == NMS_TYPE_F32) grad_type<float>(a, part, st);
    else if (a.type == NMS_TYPE_F16) grad_type<__half>(a, part, st);
    else grad_type<__nv_bfloat16>(a, part, st);
}

}  // namespace gbnms
