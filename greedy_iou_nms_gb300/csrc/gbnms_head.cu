// The C entry points of the operators of a trainable detection head: group
// normalisation with activation and dropout, dropout, and attention weights
// with a bias by relative position.  Argument checks and launches; no host
// synchronisation, no allocation.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "head.h"
#include "internal.h"

using namespace gbnms;

namespace {

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

nms_status cuda_status() { return cudaGetLastError() == cudaSuccess ? NMS_OK : NMS_ERR_CUDA; }

bool known_type(int32_t t) { return t == NMS_TYPE_F32 || t == NMS_TYPE_F16 || t == NMS_TYPE_BF16; }

uintptr_t type_bytes(int32_t t) { return t == NMS_TYPE_F32 ? 4 : 2; }

bool bad_probability(double p) { return !(p >= 0.0 && p <= 1.0); }

DropArgs drop_args(double p, uint64_t seed, uint64_t offset)
{
    DropArgs d;
    d.key_lo = static_cast<uint32_t>(seed);
    d.key_hi = static_cast<uint32_t>(seed >> 32);
    d.offset_lo = static_cast<uint32_t>(offset);
    d.offset_hi = static_cast<uint32_t>(offset >> 32);
    d.limit = static_cast<uint32_t>(std::floor((1.0 - p) * 65536.0 + 0.5));
    d.factor = d.limit ? static_cast<float>(65536.0 / d.limit) : 0.0f;
    return d;
}

// a * b for non-negative a, b, or -1 when it passes `most`.
int64_t product(int64_t a, int64_t b, int64_t most)
{
    if (a == 0 || b == 0) return 0;
    return a > most / b ? -1 : a * b;
}

constexpr int64_t kMostElements = int64_t(1) << 40;
constexpr int64_t kMostRows = INT32_MAX;

// Shape of a feature map: 0, or the status to return.
nms_status check_map(int64_t batch, int64_t pixels, int32_t channels, int32_t groups)
{
    if (batch < 0 || pixels < 0 || channels < 1 || groups < 1 || channels % groups != 0) return NMS_ERR_INVALID_ARG;
    if (channels > NMS_NORM_MAX_CHANNELS || batch > NMS_NORM_MAX_BATCH || pixels > NMS_NORM_MAX_PIXELS ||
        batch * groups > INT32_MAX || product(batch * channels, pixels, kMostElements) < 0)
        return NMS_ERR_CAPACITY;
    return NMS_OK;
}

// Strides of a feature map: rows that do not overlap, images in order.
bool bad_strides(int64_t image, int64_t pixel, int64_t batch, int64_t pixels, int32_t channels)
{
    if (pixels > 1 && pixel < channels) return true;
    if (batch > 1 && image < 0) return true;
    return pixel < 0 || image < 0 || product(pixel, pixels, kMostElements) < 0 || product(image, batch, kMostElements) < 0;
}

}  // namespace

extern "C" nms_status nms_group_norm_workspace_size(int64_t batch, int64_t pixels, int32_t channels, int32_t groups,
                                                    size_t* bytes)
{
    if (!bytes) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_map(batch, pixels, channels, groups);
    if (s != NMS_OK) return s;
    *bytes = batch == 0 ? 256 : norm_workspace_bytes(batch, pixels, channels, groups);
    return NMS_OK;
}

extern "C" nms_status nms_group_norm_run(const void* x, int64_t x_image, int64_t x_pixel, int32_t type, int64_t batch,
                                         int64_t pixels, int32_t channels, int32_t groups, const void* weight,
                                         const void* bias, int32_t param_type, float eps, int32_t act, double drop_p,
                                         uint64_t seed, uint64_t offset, void* y, float* mean, float* rstd,
                                         void* workspace, size_t workspace_bytes, void* stream)
{
    if (!known_type(type) || (param_type != NMS_TYPE_F32 && param_type != type)) return NMS_ERR_INVALID_ARG;
    if (act < NMS_ACT_NONE || act > NMS_ACT_GELU || !(eps >= 0.0f) || std::isinf(eps) || bad_probability(drop_p))
        return NMS_ERR_INVALID_ARG;
    const nms_status s = check_map(batch, pixels, channels, groups);
    if (s != NMS_OK) return s;
    if (bad_strides(x_image, x_pixel, batch, pixels, channels)) return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type), pe = type_bytes(param_type);
    if (batch > 0 && pixels > 0 && (!x || !y || misaligned(x, e) || misaligned(y, e))) return NMS_ERR_INVALID_ARG;
    if (misaligned(weight, pe) || misaligned(bias, pe) || misaligned(mean, 4) || misaligned(rstd, 4))
        return NMS_ERR_INVALID_ARG;
    if (batch == 0) return NMS_OK;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < norm_workspace_bytes(batch, pixels, channels, groups))
        return NMS_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (pixels == 0) {
        const size_t stats = static_cast<size_t>(batch) * groups * sizeof(float);
        if (mean) cudaMemsetAsync(mean, 0, stats, st);
        if (rstd) cudaMemsetAsync(rstd, 0, stats, st);
        return cuda_status();
    }
    NormArgs a{};
    a.x = x;
    a.x_image = x_image;
    a.x_pixel = x_pixel;
    a.type = type;
    a.batch = batch;
    a.pixels = pixels;
    a.channels = channels;
    a.groups = groups;
    a.weight = weight;
    a.bias = bias;
    a.param_f32 = param_type == NMS_TYPE_F32;
    a.eps = eps;
    a.act = act;
    a.drop = drop_args(drop_p, seed, offset);
    a.out = y;
    a.mean = mean;
    a.rstd = rstd;
    launch_norm(a, workspace, st);
    return cuda_status();
}

extern "C" nms_status nms_group_norm_grad_run(const void* dy, int64_t dy_image, int64_t dy_pixel, const void* x,
                                              int64_t x_image, int64_t x_pixel, int32_t type, int64_t batch,
                                              int64_t pixels, int32_t channels, int32_t groups, const float* mean,
                                              const float* rstd, const void* weight, const void* bias,
                                              int32_t param_type, int32_t act, double drop_p, uint64_t seed,
                                              uint64_t offset, void* dx, float* dweight, float* dbias,
                                              void* workspace, size_t workspace_bytes, void* stream)
{
    if (!known_type(type) || (param_type != NMS_TYPE_F32 && param_type != type)) return NMS_ERR_INVALID_ARG;
    if (act < NMS_ACT_NONE || act > NMS_ACT_GELU || bad_probability(drop_p)) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_map(batch, pixels, channels, groups);
    if (s != NMS_OK) return s;
    if (bad_strides(x_image, x_pixel, batch, pixels, channels) ||
        bad_strides(dy_image, dy_pixel, batch, pixels, channels))
        return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type), pe = type_bytes(param_type);
    const bool empty = batch == 0 || pixels == 0;
    if (!empty && (!x || !dy || !dx || !mean || !rstd || misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e)))
        return NMS_ERR_INVALID_ARG;
    if (misaligned(weight, pe) || misaligned(bias, pe) || misaligned(mean, 4) || misaligned(rstd, 4) ||
        misaligned(dweight, 4) || misaligned(dbias, 4))
        return NMS_ERR_INVALID_ARG;
    if (!empty && (!workspace || misaligned(workspace, 256) ||
                   workspace_bytes < norm_workspace_bytes(batch, pixels, channels, groups)))
        return NMS_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (empty) {
        if (dweight) cudaMemsetAsync(dweight, 0, channels * sizeof(float), st);
        if (dbias) cudaMemsetAsync(dbias, 0, channels * sizeof(float), st);
        return cuda_status();
    }
    NormArgs a{};
    a.x = x;
    a.x_image = x_image;
    a.x_pixel = x_pixel;
    a.dy = dy;
    a.dy_image = dy_image;
    a.dy_pixel = dy_pixel;
    a.type = type;
    a.batch = batch;
    a.pixels = pixels;
    a.channels = channels;
    a.groups = groups;
    a.weight = weight;
    a.bias = bias;
    a.param_f32 = param_type == NMS_TYPE_F32;
    a.act = act;
    a.drop = drop_args(drop_p, seed, offset);
    a.out = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dweight = dweight;
    a.dbias = dbias;
    launch_norm_grad(a, workspace, st);
    return cuda_status();
}

extern "C" nms_status nms_dropout_run(const void* x, const void* residual, int32_t type, int64_t n, double drop_p,
                                      uint64_t seed, uint64_t offset, void* y, void* stream)
{
    if (!known_type(type) || n < 0 || bad_probability(drop_p)) return NMS_ERR_INVALID_ARG;
    if (n > kMostElements) return NMS_ERR_CAPACITY;
    if (n == 0) return NMS_OK;
    const uintptr_t e = type_bytes(type);
    if (!x || !y || misaligned(x, e) || misaligned(y, e) || misaligned(residual, e)) return NMS_ERR_INVALID_ARG;
    cudaGetLastError();
    launch_dropout(x, residual, y, type, n, drop_args(drop_p, seed, offset), static_cast<cudaStream_t>(stream));
    return cuda_status();
}

extern "C" nms_status nms_relation_buckets_run(const int32_t* q_pos, int64_t q_sets, const int32_t* k_pos,
                                               int64_t k_sets, int64_t queries, int64_t keys, int32_t axes,
                                               const int32_t* lut, int32_t reach, int16_t* buckets, void* stream)
{
    if (q_sets < 0 || k_sets < 0 || queries < 0 || keys < 0 || axes < 1 || reach < 0) return NMS_ERR_INVALID_ARG;
    if (q_sets != k_sets && q_sets != 1 && k_sets != 1) return NMS_ERR_INVALID_ARG;
    if (axes > NMS_RELATION_MAX_AXES || reach > NMS_RELATION_MAX_REACH) return NMS_ERR_CAPACITY;
    const int64_t sets = q_sets == 1 ? k_sets : q_sets;
    const int64_t rows = product(sets, queries, kMostRows);
    if (rows < 0 || product(rows, keys, kMostElements) < 0) return NMS_ERR_CAPACITY;
    if (rows == 0 || keys == 0) return NMS_OK;
    if (!q_pos || !k_pos || !lut || !buckets || misaligned(q_pos, 4) || misaligned(k_pos, 4) || misaligned(lut, 4) ||
        misaligned(buckets, 2))
        return NMS_ERR_INVALID_ARG;
    cudaGetLastError();
    BucketArgs a{q_pos, k_pos, q_sets, k_sets, sets, queries, keys, axes, lut, reach, buckets};
    launch_relation_buckets(a, static_cast<cudaStream_t>(stream));
    return cuda_status();
}

// What both directions of the relation check; fills the shared arguments.
static nms_status check_relation(int32_t type, int64_t batch, int32_t heads, int64_t queries, int64_t keys,
                                 int64_t sets, int32_t num_buckets, float scale)
{
    if (!known_type(type) || batch < 0 || heads < 1 || queries < 0 || keys < 0 || num_buckets < 1 ||
        (sets != 1 && sets != batch) || !std::isfinite(scale))
        return NMS_ERR_INVALID_ARG;
    if (heads > NMS_RELATION_MAX_HEADS || num_buckets > NMS_RELATION_MAX_BUCKETS) return NMS_ERR_CAPACITY;
    const int64_t bh = product(batch, heads, kMostRows), rows = bh < 0 ? -1 : product(bh, queries, kMostRows);
    if (rows < 0 || product(rows, keys, kMostElements) < 0) return NMS_ERR_CAPACITY;
    return NMS_OK;
}

extern "C" nms_status nms_relation_softmax_run(const void* scores, int32_t type, int64_t batch, int32_t heads,
                                               int64_t queries, int64_t keys, const int16_t* buckets, int64_t sets,
                                               const float* table, int32_t num_buckets, const uint8_t* key_mask,
                                               float scale, void* probs, void* stream)
{
    const nms_status s = check_relation(type, batch, heads, queries, keys, sets, num_buckets, scale);
    if (s != NMS_OK) return s;
    if (batch == 0 || queries == 0 || keys == 0) return NMS_OK;
    const uintptr_t e = type_bytes(type);
    if (!scores || !buckets || !table || !probs || misaligned(scores, e) || misaligned(probs, e) ||
        misaligned(buckets, 2) || misaligned(table, 4))
        return NMS_ERR_INVALID_ARG;
    cudaGetLastError();
    RelationArgs a{};
    a.scores = scores;
    a.out = probs;
    a.type = type;
    a.batch = batch;
    a.queries = queries;
    a.keys = keys;
    a.heads = heads;
    a.buckets = buckets;
    a.sets = sets;
    a.table = table;
    a.num_buckets = num_buckets;
    a.key_mask = key_mask;
    a.scale = scale;
    launch_relation_softmax(a, static_cast<cudaStream_t>(stream));
    return cuda_status();
}

extern "C" nms_status nms_relation_grad_workspace_size(int64_t batch, int32_t heads, int64_t queries, int64_t keys,
                                                       int32_t num_buckets, size_t* bytes)
{
    if (!bytes) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_relation(NMS_TYPE_F32, batch, heads, queries, keys, 1, num_buckets, 1.0f);
    if (s != NMS_OK) return s;
    *bytes = relation_grad_workspace_bytes(batch, heads, queries, keys, num_buckets);
    return NMS_OK;
}

extern "C" nms_status nms_relation_softmax_grad_run(const void* dprobs, const void* probs, int32_t type,
                                                    int64_t batch, int32_t heads, int64_t queries, int64_t keys,
                                                    const int16_t* buckets, int64_t sets, int32_t num_buckets,
                                                    const uint8_t* key_mask, float scale, void* dscores,
                                                    float* dtable, void* workspace, size_t workspace_bytes,
                                                    void* stream)
{
    const nms_status s = check_relation(type, batch, heads, queries, keys, sets, num_buckets, scale);
    if (s != NMS_OK) return s;
    if (!dtable || misaligned(dtable, 4)) return NMS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (batch == 0 || queries == 0 || keys == 0) {
        cudaMemsetAsync(dtable, 0, sizeof(float) * num_buckets * heads, st);
        return cuda_status();
    }
    const uintptr_t e = type_bytes(type);
    if (!dprobs || !probs || !buckets || !dscores || misaligned(dprobs, e) || misaligned(probs, e) ||
        misaligned(dscores, e) || misaligned(buckets, 2))
        return NMS_ERR_INVALID_ARG;
    if (!workspace || misaligned(workspace, 256) ||
        workspace_bytes < relation_grad_workspace_bytes(batch, heads, queries, keys, num_buckets))
        return NMS_ERR_WORKSPACE;
    RelationArgs a{};
    a.scores = dprobs;
    a.probs = probs;
    a.out = dscores;
    a.type = type;
    a.batch = batch;
    a.queries = queries;
    a.keys = keys;
    a.heads = heads;
    a.buckets = buckets;
    a.sets = sets;
    a.num_buckets = num_buckets;
    a.key_mask = key_mask;
    a.scale = scale;
    a.dtable = dtable;
    launch_relation_grad(a, workspace, st);
    return cuda_status();
}
