// Host-side launchers of the detection-head operators (gbnms_head.cu calls
// them after its checks).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gbnms {

constexpr int SMS = 152;  // of a GB300; launches are sized by it

// Dropout of one call: an element is kept when its 16-bit field is below
// limit (65536: every element), and a kept one is multiplied by factor.
struct DropArgs {
    uint32_t key_lo, key_hi, offset_lo, offset_hi;
    uint32_t limit;
    float factor;
};

// One feature map [batch][pixels][channels]; strides count elements, the
// channels of a pixel are consecutive.
struct NormArgs {
    const void* x;
    int64_t x_image, x_pixel;
    const void* dy;  // gradient only
    int64_t dy_image, dy_pixel;
    int type;
    int64_t batch, pixels;
    int channels, groups;
    const void* weight;  // NULL: 1
    const void* bias;    // NULL: 0
    int param_f32;       // weight and bias are binary32 (else of `type`)
    float eps;
    int act;
    DropArgs drop;
    void* out;    // y, or dx; contiguous
    float* mean;  // [batch][groups]; the gradient reads them
    float* rstd;
    float* dweight;  // gradient only; may be NULL
    float* dbias;
};

// Scratch of either direction (they share the layout).
size_t norm_workspace_bytes(int64_t batch, int64_t pixels, int channels, int groups);
void launch_norm(const NormArgs& a, void* workspace, cudaStream_t st);
void launch_norm_grad(const NormArgs& a, void* workspace, cudaStream_t st);

// y = drop(x) (+ residual) over n contiguous elements.
void launch_dropout(const void* x, const void* residual, void* y, int type, int64_t n, const DropArgs& d,
                    cudaStream_t st);

// Bucket map of relative positions.
struct BucketArgs {
    const int32_t* q_pos;
    const int32_t* k_pos;
    int64_t q_sets, k_sets, sets, queries, keys;
    int axes;
    const int32_t* lut;
    int reach;
    int16_t* buckets;
};
void launch_relation_buckets(const BucketArgs& a, cudaStream_t st);

struct RelationArgs {
    const void* scores;  // forward: scores; gradient: the incoming gradient
    const void* probs;   // gradient only
    void* out;           // forward: probs; gradient: dscores
    int type;
    int64_t batch, queries, keys;
    int heads;
    const int16_t* buckets;
    int64_t sets;  // 1, or batch
    const float* table;
    int num_buckets;
    const uint8_t* key_mask;  // [batch][keys] or NULL
    float scale;
    float* dtable;  // gradient only, [num_buckets][heads]
};
void launch_relation_softmax(const RelationArgs& a, cudaStream_t st);
size_t relation_grad_workspace_bytes(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets);
void launch_relation_grad(const RelationArgs& a, void* workspace, cudaStream_t st);

}  // namespace gbnms
