// Which way the relation kernels take, and the geometry of their gradient.
#pragma once

#include "head.h"

namespace gbnms {

constexpr int64_t RELATION_MOST = 8192;  // keys of a row that a block holds

constexpr int RELATION_PAIR_WARPS = 6;  // of a block whose lanes share 16 columns, at most

// One map for all images: the weights' kernel goes by image.  Us by image and by head, 8 heads: 512 x 49 x 49 bf16 15
// and 21, 64 x 300 x 300 50 and 67, 16 x 1000 x 1000 99 and 104, 8 x 1496 x 1496 159 and 198; two images of long rows
// are within a sixth either way (1000 x 1000 23 and 19).
inline bool relation_by_image(const RelationArgs& a) { return a.sets == 1 && !a.key_mask && a.batch > 1; }

// Whether the gradient does too.
bool relation_grad_by_image(const RelationArgs& a);

// Geometry of the gradient, a function of the shapes alone but for `image`
// (the workspace is sized for either).
struct RelationGradPlan {
    int columns, warps;
    int64_t blocks, chunks, per;  // blocks of rows (or query tiles); image chunks
    int64_t parts() const { return blocks * chunks; }
};

RelationGradPlan relation_grad_plan(int64_t batch, int heads, int64_t queries, int64_t keys, int num_buckets,
                                    bool image);

}  // namespace gbnms
