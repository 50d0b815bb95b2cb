// Host-side launchers of a transformer block's operators (gbnms_block.cu calls
// them after its checks).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "head.h"

namespace gbnms {

// Rows of `width` consecutive elements; strides count elements.
struct LayerArgs {
    const void* x;
    int64_t x_row;
    const void* second;  // forward: the residual added to x, gradient: the gradient added to dx; or NULL
    int64_t second_row;
    const void* dy;  // gradient only
    int64_t dy_row;
    int type;
    int64_t rows;
    int width;
    const void* weight;  // NULL: 1
    const void* bias;    // NULL: 0
    int param_f32;       // weight and bias are binary32 (else of `type`)
    float eps;
    void* out;    // y, or dx; contiguous
    void* sum;    // forward: x + residual; contiguous
    float* mean;  // [rows]; the gradient reads them
    float* rstd;
    float* dweight;  // gradient only; may be NULL
    float* dbias;
    bool once;  // the operands are more than L2 keeps (set by the launcher)
};
void launch_layer_norm(const LayerArgs& a, cudaStream_t st);
size_t layer_grad_workspace_bytes(int64_t rows, int width);
void launch_layer_grad(const LayerArgs& a, void* workspace, cudaStream_t st);

// Vectors [batch][tokens][heads][dim]; strides count elements.
struct RotaryArgs {
    const void* x;
    int64_t x_batch, x_token, x_head;
    int type;
    int64_t batch, tokens;
    int heads, dim;
    const void* positions;  // [sets][tokens][axes], int32 or binary32
    int64_t sets;           // 1, or batch
    int fractions;          // positions are binary32
    int axes;
    const int64_t* lut;  // [2][pairs]: turns by position in units of 2^-64, axis
    int pairs;
    int halves, inverse;
    void* y;
    int64_t y_batch, y_token, y_head;
    bool once;  // the vectors are more than L2 keeps (set by the launcher)
};
void launch_rotary(const RotaryArgs& a, cudaStream_t st);

// sums[c] = the parts' sum in column c, parts [blocks][columns]; the first
// `split` columns go to one array, the others to a second (either may be NULL).
void launch_column_join(const float* parts, int64_t blocks, int64_t columns, int64_t split, float* first, float* second,
                        cudaStream_t st);

// How long, in ns, a wait of the tensor-core products that this host thread
// launches lasts before it gives up; a tile's whole sum has five times as long
// (2^31 of k take a second).  gbnms_product_patience() sets it, for tests.
inline uint64_t& product_patience()
{
    static thread_local uint64_t ns = 2000000000;
    return ns;
}

// out = act(A B^T + bias) + residual, A m x k, B n x k.
struct ProductArgs {
    const void* a;  // [m][k], or [k][m] with a_across; rows a_row apart
    const void* b;  // [n][k], or [k][n] with b_across
    const void* a_low;  // 16 bits: what a's elements left out when they were rounded, laid out like a; or NULL
    int64_t a_row, b_row;
    int a_across, b_across;
    int type;
    int64_t m, n, k;
    const void* bias;  // [n] or NULL
    int bias_f32;
    int act;
    const void* residual;  // [m][n], rows residual_row apart, or NULL
    int64_t residual_row;
    void* out;        // [m][n] contiguous
    void* pre;        // A B^T + bias [m][n] contiguous, or NULL
    int32_t* status;  // or NULL
    int segments;     // 1; more: stretches of k whose sums go to parts [segments][m][n] in place of out
    float* parts;
    float* scratch;  // 16 bits: product_scratch_bytes()
};
// What 16-bit products keep there for sums over k (the larger one of two products').
size_t product_scratch_bytes(int type, int64_t k);
// Binary32, by the plain arithmetic units.  False: the driver refused a launch.
bool launch_product_f32(const ProductArgs& p, cudaStream_t st);
// Binary32, by the tensor cores: operands of three planes of 16 bits, as
// launch_split_rows leaves them.
bool launch_product_split(const ProductArgs& p, cudaStream_t st);
// Rows of binary32 and their planes [3][rows][to_row], to_row a multiple of 8.
struct SplitRows {
    const float* from;
    int64_t from_row, rows, width;
    void* to;
    int64_t to_row;
};
void launch_split_rows(const SplitRows* of, int count, cudaStream_t st);  // one or two operands
// out = sums over the parts [segments][n], of any type, in order.
void launch_join_parts(const float* parts, int segments, int64_t n, void* out, int type, cudaStream_t st);
// 16 bits, by the tensor cores: operands and their rows start at multiples of
// 16 bytes and do not overlap.
bool launch_product_tc(const ProductArgs& p, cudaStream_t st);
// Rows of 16-bit elements to rows `to_row` apart, a multiple of 8.
struct CopyRows {
    const void* from;
    int64_t from_row, rows, width;
    void* to;
    int64_t to_row;
};
void launch_copy_rows(const CopyRows* of, int count, cudaStream_t st);  // one or two operands

// dz = dy * act'(pre) [rows][width], rows dz_row apart (none: dz NULL), and
// the sums of its columns before they are rounded (none: dbias NULL).
struct SlopeArgs {
    const void* dy;
    int64_t dy_row;
    const void* pre;  // contiguous; NULL: act is none
    int type;
    int64_t rows, width;
    int act;
    void* dz;
    int64_t dz_row;
    void* low;     // 16 bits: what rounding dz left out, like dz; or NULL
    void* planes;  // binary32: dz as planes [3][rows][dz_row] in place of dz
    float* dbias;
};
size_t slope_workspace_bytes(int64_t rows, int64_t width);
void launch_slope(const SlopeArgs& s, void* workspace, cudaStream_t st);

}  // namespace gbnms
