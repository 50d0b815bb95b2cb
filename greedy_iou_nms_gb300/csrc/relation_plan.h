// Which way the relation kernels take, and the geometry of their gradient.
#pragma once

#include "head.h"

namespace gbnms {

constexpr int64_t RELATION_MOST = 8192;  // keys of a row that a block holds

constexpr int RELATION_PAIR_WARPS = 6;  // of a block whose lanes share 16 columns, at most

inline bool relation_by_image(const RelationArgs& a) { return a.sets == 1 && !a.key_mask && a.batch > 1; }

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
