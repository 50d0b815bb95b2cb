// The bucket map of relative positions, the dispatch of the relation kernels
// (k_relation.cuh) by type and the last step of their gradient.
#include "head.cuh"
#include "internal.h"
#include "relation_plan.h"

namespace gbnms {

// --------------------------------------------------------------------- map

constexpr int BK_THREADS = 128, BK_EACH = 4, BK_ROWS = 4, BK_TABLE = 4096;

// buckets[set][i][j] = sum over the axes of lut[axis][clamp(k - q)], -1 when
// a part is negative or the sum does not fit.  A block takes BK_THREADS *
// BK_EACH keys (four neighbours a thread) of BK_ROWS queries of one set; the
// tables lie in shared memory where they fit and serve several rows
// (SHARED), else they come from L1.  16 x 300 x 300, two axes: 4.8 us, latency.
template <int AXES, bool SHARED>
__global__ void __launch_bounds__(BK_THREADS)
relation_buckets_kernel(BucketArgs a, unsigned tiles)
{
    __shared__ int s_lut[SHARED ? BK_TABLE : 1];
    const int width = 2 * a.reach + 1, axes = AXES < NMS_RELATION_MAX_AXES ? AXES : a.axes;
    if (SHARED) {
        for (int x = threadIdx.x; x < axes * width; x += BK_THREADS) s_lut[x] = a.lut[x];
        __syncthreads();
    }
    const int* lut = (SHARED ? s_lut : a.lut) + a.reach;
    const unsigned Q = static_cast<unsigned>(a.queries), set = blockIdx.x / tiles, first = blockIdx.x % tiles * BK_ROWS;
    const int32_t* q = a.q_pos + static_cast<int64_t>(a.q_sets == 1 ? 0 : set) * Q * axes;
    const int32_t* k = a.k_pos + (a.k_sets == 1 ? 0 : set) * a.keys * axes;
    const bool wide = a.keys % 4 == 0 && reinterpret_cast<uintptr_t>(a.buckets) % 8 == 0;
    for (int64_t j0 = (static_cast<int64_t>(blockIdx.y) * BK_THREADS + threadIdx.x) * BK_EACH; j0 < a.keys;
         j0 += static_cast<int64_t>(gridDim.y) * BK_THREADS * BK_EACH) {
        const int here = a.keys - j0 < BK_EACH ? static_cast<int>(a.keys - j0) : BK_EACH;
        int at[BK_EACH][AXES];
#pragma unroll
        for (int e = 0; e < BK_EACH; ++e)
#pragma unroll
            for (int x = 0; x < AXES; ++x) at[e][x] = x < axes ? k[(j0 + (e < here ? e : 0)) * axes + x] : 0;
#pragma unroll
        for (int r = 0; r < BK_ROWS; ++r) {
            const unsigned i = first + r;
            if (i >= Q) break;
            int sum[BK_EACH] = {}, signs[BK_EACH] = {};
#pragma unroll
            for (int x = 0; x < AXES; ++x) {
                if (x >= axes) break;
                // Keys are clamped to the reach about the query: no difference leaves 32 bits.
                const int from = q[static_cast<int64_t>(i) * axes + x];
                const int64_t least = static_cast<int64_t>(from) - a.reach, most = static_cast<int64_t>(from) + a.reach;
                const int lo = least < INT32_MIN ? INT32_MIN : static_cast<int>(least);
                const int hi = most > INT32_MAX ? INT32_MAX : static_cast<int>(most);
#pragma unroll
                for (int e = 0; e < BK_EACH; ++e) {
                    const int part = lut[x * width + (min(max(at[e][x], lo), hi) - from)];
                    signs[e] |= part;
                    sum[e] += min(part, 32768);
                }
            }
            Pack<int16_t, BK_EACH> out;
#pragma unroll
            for (int e = 0; e < BK_EACH; ++e)
                out.v[e] = static_cast<int16_t>(signs[e] < 0 || sum[e] > 32767 ? -1 : sum[e]);
            int16_t* to = a.buckets + (static_cast<int64_t>(set) * Q + i) * a.keys + j0;
            if (wide) {
                *reinterpret_cast<Pack<int16_t, BK_EACH>*>(to) = out;
            } else {
#pragma unroll
                for (int e = 0; e < BK_EACH; ++e)
                    if (e < here) to[e] = out.v[e];
            }
        }
    }
}

void launch_relation_buckets(const BucketArgs& a, cudaStream_t st)
{
    const int64_t chunks = (a.keys + BK_THREADS * BK_EACH - 1) / (BK_THREADS * BK_EACH);
    const unsigned tiles = static_cast<unsigned>((a.queries + BK_ROWS - 1) / BK_ROWS);
    const dim3 grid(static_cast<unsigned>(a.sets) * tiles, static_cast<unsigned>(chunks < 4096 ? chunks : 4096));
    const bool shared = a.queries >= BK_ROWS && a.axes * (2 * a.reach + 1) <= BK_TABLE;
    auto run = [&](auto kernel) { kernel<<<grid, BK_THREADS, 0, st>>>(a, tiles); };
    if (a.axes == 1) shared ? run(relation_buckets_kernel<1, true>) : run(relation_buckets_kernel<1, false>);
    else if (a.axes == 2) shared ? run(relation_buckets_kernel<2, true>) : run(relation_buckets_kernel<2, false>);
    else shared ? run(relation_buckets_kernel<4, true>) : run(relation_buckets_kernel<4, false>);
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
        const int64_t least = (batch + 1023) / 1024;  // chains of at most 1024 additions
        p.chunks = want < least ? least : want > batch ? batch : want;
        if (p.chunks > 65535) p.chunks = 65535;  // of a grid's second axis
        p.per = (batch + p.chunks - 1) / p.chunks;
        p.chunks = (batch + p.per - 1) / p.per;
        return p;
    }
    // A table a warp, in all of an SM's shared memory: 32 columns if twelve
    // warps' fit, else 16 and two blocks of up to six warps if four each fit,
    // else 32 or fewer for one block of six warps.
    constexpr int ROOM = 208 * 1024;
    const int row = 4 * (num_buckets + 1), need = lanes == 256 ? 8 : 6;
    const bool pairs = lanes <= 32 && keys <= RELATION_MOST;  // 16 columns: the kernel whose lanes share them
    if (pairs && 12 * 32 * row > ROOM && 4 * 16 * row <= ROOM / 2) {
        p.columns = 16;
        const int fit = ROOM / 2 / (16 * row);
        p.warps = fit > RELATION_PAIR_WARPS ? RELATION_PAIR_WARPS : fit;
    } else {
        for (p.columns = 32; p.columns > 4 && need * p.columns * row > ROOM; p.columns /= 2) {}
        const int fit = ROOM / (p.columns * row), most = pairs && p.columns == 16 ? RELATION_PAIR_WARPS : 8;
        p.warps = fit > most ? most : fit;
    }
    const int64_t teams = p.warps * 32 / lanes, rows = batch * queries, want = (rows + teams - 1) / teams;
    const int resident = ROOM / (p.warps * p.columns * row);
    const int64_t most = (SMS * static_cast<int64_t>(resident < 4 ? resident : 4) + heads - 1) / heads;
    p.blocks = want < most ? want : most;
    p.chunks = 1;
    return p;
}

// Images from which the gradient of one map for all goes by image.  A block by image ends with a table of sums for
// its few queries, which costs the more the more elements a lane holds; by head the tables are few, but each image's
// rows cost more, most where lanes take turns at the columns.  Us by image and by head, 8 heads:
//   rows up to 320 keys            2 x 300 x 300 bf16     25 and 29    64 x 300 x 300           73 and 109
//   lanes in turns                 4 x 200 x 1100 bf16    82 and 91    2 x 200 x 1100           76 and 56
//   up to 16 elements, 16 bits     16 x 512 x 512 bf16    75 and 68    64 x 512 x 512          166 and 194
//   more                           16 x 1000 x 1000 bf16 326 and 202   2 x 1000 x 1000         205 and 50
//   binary32, odd rows             8 x 1000 x 1000 fp32  302 and 294   2 x 1000 x 1000         218 and 97
static int64_t images_to_go_by(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets, bool packed)
{
    if (keys <= 320) return 2;
    const RelationGradPlan head = relation_grad_plan(batch, heads, queries, keys, num_buckets, false);
    const int lanes = team_lanes(keys);
    if (head.columns < (lanes <= 32 ? 16 : 32)) return 4;  // turns
    return !packed ? 8 : (keys + lanes - 1) / lanes <= 16 ? 16 : 64;
}

bool relation_grad_by_image(const RelationArgs& a)
{
    return relation_by_image(a) && a.keys <= RELATION_MOST &&
           a.batch >= images_to_go_by(a.batch, a.heads, a.queries, a.keys, a.num_buckets,
                                      a.type != NMS_TYPE_F32 && a.keys % 2 == 0);
}

size_t relation_grad_workspace_bytes(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets)
{
    if (batch == 0 || queries == 0 || keys == 0) return 256;
    const int64_t a = relation_grad_plan(batch, heads, queries, keys, num_buckets, false).parts();
    // By image as well where the type, the map and the mask may have it so.
    const int64_t least = images_to_go_by(batch, heads, queries, keys, num_buckets, false);
    const bool image = keys <= RELATION_MOST && batch >= least;
    const int64_t b = image ? relation_grad_plan(batch, heads, queries, keys, num_buckets, true).parts() : 0;
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
                                             relation_grad_by_image(a)).parts();
    relation_table_kernel<<<dim3((a.num_buckets + 31) / 32, a.heads), 256, 0, st>>>(part, parts, a.num_buckets,
                                                                                     a.heads, a.dtable);
}

}  // namespace gbnms
