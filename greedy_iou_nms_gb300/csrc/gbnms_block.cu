// The C entry points of a transformer block's operators: linear layer, layer
// normalisation and rotary positions.  Argument checks and launches; no host
// synchronisation, no allocation.
#include <cmath>
#include <cstdint>

#include "block.h"
#include "common.cuh"

using namespace gbnms;

namespace {

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

nms_status cuda_status() { return cudaGetLastError() == cudaSuccess ? NMS_OK : NMS_ERR_CUDA; }

bool known_type(int32_t t) { return t == NMS_TYPE_F32 || t == NMS_TYPE_F16 || t == NMS_TYPE_BF16; }

uintptr_t type_bytes(int32_t t) { return t == NMS_TYPE_F32 ? 4 : 2; }

constexpr int64_t kMostElements = int64_t(1) << 38;
constexpr int64_t kMostRows = INT32_MAX;

// Whether n rows at a stride reach beyond kMostElements.
bool too_far(int64_t n, int64_t stride) { return n > 0 && stride > kMostElements / n; }

size_t round_up(size_t bytes) { return (bytes + 255) / 256 * 256; }

int64_t padded(int64_t width) { return (width + 7) / 8 * 8; }

nms_status check_linear(int32_t type, int64_t rows, int32_t inner, int32_t outer)
{
    if (!known_type(type) || rows < 0 || inner < 1 || outer < 1) return NMS_ERR_INVALID_ARG;
    static_assert(int64_t(NMS_LINEAR_MAX_WIDTH) * NMS_LINEAR_MAX_WIDTH <= kMostElements, "a weight has no more");
    if (inner > NMS_LINEAR_MAX_WIDTH || outer > NMS_LINEAR_MAX_WIDTH || rows > kMostRows || too_far(rows, inner) ||
        too_far(rows, outer))
        return NMS_ERR_CAPACITY;
    return NMS_OK;
}

bool bad_row(int64_t row, int64_t rows) { return row < 0 || too_far(rows, row); }

// Whether the tensor cores' loads cannot take an operand of 16 bits as it lies.
bool uneven(int32_t type, const void* p, int64_t row, int64_t rows, int64_t width)
{
    return type != NMS_TYPE_F32 && (misaligned(p, 16) || row % 8 != 0 || row < width);
}

size_t copy_bytes(int64_t rows, int64_t width) { return round_up(2 * rows * padded(width)); }

// Multiplications from which a binary32 product is worth making planes for, where k
// is short: 300 x 256 x 1024, 2^26.2, took 14.6 us by them and 16.4 on the plain
// units; 300 x 256 x 512, 2^25.2, 14.4 and 12.5.
constexpr int64_t SPLIT_LEAST = int64_t(1) << 26;

size_t plane_bytes(int64_t rows, int64_t width) { return round_up(3 * 2 * rows * padded(width)); }

// Whether a binary32 product of m x n results goes by planes to the tensor cores:
// from SPLIT_LEAST multiplications on; from a thirty-second of them where k is long,
// so that there are few results (70 x 64 of k = 2816: 16.8 us by planes, 24.5 on the
// plain units; 43 x 192 of 3776: 18.7 and 30.8).  A weight's gradient also where it
// is few results of many rows (64 x 64 of 100000: 54 us and 592), but of up to 32
// rows not: a tile has 128, and x need be read once only (10 x 3624 of 14309: 57 us
// by few_across_kernel, 178 by planes; 32 x 3500 of 18000: 161 and 214).
bool by_planes(int32_t type, int64_t m, int64_t n, int64_t k, bool gradient)
{
    if (type != NMS_TYPE_F32) return false;
    if (m <= (gradient ? 32 : 16)) return false;
    if (gradient && k >= 8192) return true;
    return m * n >= (k >= 1024 ? SPLIT_LEAST / 32 : SPLIT_LEAST) / k;
}

// Stretches of k of a weight's gradient on the tensor cores: where clusters of
// eight leave half of the SMs idle, one for each SM; and no sum over more than 2^18
// of k, as none of a width is, so that a chain in binary32 has 2^12 additions at most.
// `low`: dz comes in two parts, each of which goes through k.
int gradient_segments(int32_t type, int64_t m, int64_t n, int64_t k, bool low)
{
    if (type == NMS_TYPE_F32 && m <= 32) {  // blocks of few_across_kernel: two an SM
        const int64_t columns = m <= 16 ? 128 : 64, fill = 2 * SMS / ((n + columns - 1) / columns), most = k / 1024, want = fill < most ? fill : most;
        const int64_t least = (k + (1 << 16) - 1) >> 16;  // a thread's chain: 2^13 products
        return static_cast<int>(want > least ? want : least);
    }
    if (type == NMS_TYPE_F32 && !by_planes(type, m, n, k, true)) return 1;
    const int64_t width = type == NMS_TYPE_F32 ? 128 : 64, tiles = ((m + 127) / 128) * ((n + width - 1) / width);
    int64_t segments = (k + (1 << 18) - 1) >> 18;
    if (low && segments > 1) segments *= 2;
    if (tiles * 8 <= SMS / 2 && k >= 8192) {
        const int64_t fill = SMS / tiles, most = k / 512;
        const int64_t want = fill < most ? fill : most;
        if (want > segments) segments = want;
    }
    return static_cast<int>(segments);
}

size_t parts_bytes(int segments, int64_t m, int64_t n) { return segments > 1 ? round_up(4 * segments * m * n) : 0; }

// An operand of a product: itself, or what the tensor cores take in its place.
struct Operand {
    const void* p;
    int64_t row, rows, width;
    const void* planes = nullptr;
};

// An operand's place among the planes, which the workspace moves on behind.
SplitRows as_split(Operand& o, char*& workspace)
{
    o.planes = workspace;
    workspace += plane_bytes(o.rows, o.width);
    return {static_cast<const float*>(o.p), o.row, o.rows, o.width, const_cast<void*>(o.planes), padded(o.width)};
}

// The product, its operands made ready in the workspace, which moves on.
bool launch_product(ProductArgs& q, Operand& a, Operand& b, bool as_planes, char*& workspace, cudaStream_t st)
{
    SplitRows split[2];
    CopyRows copy[2];
    int splits = 0, copies = 0;
    for (Operand* o : {&a, &b}) {
        if (as_planes && !o->planes) {
            split[splits++] = as_split(*o, workspace);
        } else if (uneven(q.type, o->p, o->row, o->rows, o->width)) {
            copy[copies++] = {o->p, o->row, o->rows, o->width, workspace, padded(o->width)};
            o->p = workspace;
            o->row = padded(o->width);
            workspace += copy_bytes(o->rows, o->width);
        }
    }
    if (splits) launch_split_rows(split, splits, st);
    if (copies) launch_copy_rows(copy, copies, st);
    q.a = as_planes ? a.planes : a.p;
    q.b = as_planes ? b.planes : b.p;
    q.a_row = as_planes ? padded(a.width) : a.row;
    q.b_row = as_planes ? padded(b.width) : b.row;
    if (as_planes) return launch_product_split(q, st);
    return q.type == NMS_TYPE_F32 ? launch_product_f32(q, st) : launch_product_tc(q, st);
}

}  // namespace

// Not among the public entries: see product_patience().
extern "C" void gbnms_product_patience(uint64_t ns) { product_patience() = ns; }

extern "C" nms_status nms_linear_workspace_size(int32_t type, int64_t rows, int32_t inner, int32_t outer,
                                                int32_t aligned, size_t* bytes)
{
    if (!bytes) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_linear(type, rows, inner, outer);
    if (s != NMS_OK) return s;
    *bytes = 0;
    if (rows == 0) return NMS_OK;
    if (by_planes(type, rows, outer, inner, false)) *bytes = plane_bytes(rows, inner) + plane_bytes(outer, inner);
    else if (type != NMS_TYPE_F32 && !aligned) *bytes = copy_bytes(rows, inner) + copy_bytes(outer, inner);
    *bytes += product_scratch_bytes(type, inner);
    return NMS_OK;
}

extern "C" nms_status nms_linear_run(const void* x, int64_t x_row, int32_t type, int64_t rows, int32_t inner,
                                     const void* weight, int64_t weight_row, int32_t outer, const void* bias,
                                     int32_t bias_type, int32_t act, const void* residual, int64_t residual_row,
                                     void* y, void* pre, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                                     void* stream)
{
    const nms_status s = check_linear(type, rows, inner, outer);
    if (s != NMS_OK) return s;
    if ((bias_type != NMS_TYPE_F32 && bias_type != type) || act < NMS_ACT_NONE || act > NMS_ACT_GELU)
        return NMS_ERR_INVALID_ARG;
    if (bad_row(x_row, rows) || bad_row(weight_row, outer) || bad_row(residual_row, rows)) return NMS_ERR_INVALID_ARG;
    if (misaligned(bias, type_bytes(bias_type)) || misaligned(dev_status, 4)) return NMS_ERR_INVALID_ARG;
    if (rows == 0) return NMS_OK;
    const uintptr_t e = type_bytes(type);
    if (!x || !weight || !y || misaligned(x, e) || misaligned(weight, e) || misaligned(y, e) || misaligned(pre, e) ||
        misaligned(residual, e))
        return NMS_ERR_INVALID_ARG;
    const bool aligned = !uneven(type, x, x_row, rows, inner) && !uneven(type, weight, weight_row, outer, inner);
    size_t need;
    nms_linear_workspace_size(type, rows, inner, outer, aligned, &need);
    if (need && (!workspace || misaligned(workspace, 256) || workspace_bytes < need)) return NMS_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    char* rest = static_cast<char*>(workspace);
    float* const scratch = reinterpret_cast<float*>(rest);
    rest += product_scratch_bytes(type, inner);
    Operand a{x, x_row, rows, inner}, b{weight, weight_row, outer, inner};
    ProductArgs p{};
    p.type = type;
    p.m = rows;
    p.n = outer;
    p.k = inner;
    p.bias = bias;
    p.bias_f32 = bias_type == NMS_TYPE_F32;
    p.act = act;
    p.residual = residual;
    p.residual_row = residual ? residual_row : 0;
    p.out = y;
    p.pre = pre;
    p.status = dev_status;
    p.scratch = scratch;
    p.segments = 1;
    if (!launch_product(p, a, b, by_planes(type, rows, outer, inner, false), rest, st)) return NMS_ERR_CUDA;
    return cuda_status();
}

extern "C" nms_status nms_linear_grad_workspace_size(int32_t type, int64_t rows, int32_t inner, int32_t outer,
                                                     int32_t aligned, size_t* bytes)
{
    if (!bytes) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_linear(type, rows, inner, outer);
    if (s != NMS_OK) return s;
    *bytes = 0;
    if (rows == 0) return NMS_OK;
    // dz, of 16 bits in two parts, and its columns' sums; the weight's gradient's parts.
    const bool two = type != NMS_TYPE_F32;
    *bytes = (two ? 2 : 1) * round_up(type_bytes(type) * rows * padded(outer)) + round_up(slope_workspace_bytes(rows, outer));
    *bytes += parts_bytes(gradient_segments(type, outer, inner, rows, two), outer, inner);
    *bytes += product_scratch_bytes(type, outer > rows ? outer : rows);
    if (by_planes(type, rows, inner, outer, false) || by_planes(type, outer, inner, rows, true))
        *bytes += plane_bytes(rows, outer) + plane_bytes(outer, inner) + plane_bytes(rows, inner);
    else if (type != NMS_TYPE_F32 && !aligned)
        *bytes += copy_bytes(rows, inner) + copy_bytes(outer, inner);
    return NMS_OK;
}

extern "C" nms_status nms_linear_grad_run(const void* dy, int64_t dy_row, const void* x, int64_t x_row, int32_t type,
                                          int64_t rows, int32_t inner, const void* weight, int64_t weight_row,
                                          int32_t outer, const void* pre, int32_t act, void* dx, void* dweight,
                                          float* dbias, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                                          void* stream)
{
    const nms_status s = check_linear(type, rows, inner, outer);
    if (s != NMS_OK) return s;
    const bool rounded = act >= 0 && (act & NMS_ACT_ROUND_SLOPES);
    if (rounded) act &= ~NMS_ACT_ROUND_SLOPES;
    if (act < NMS_ACT_NONE || act > NMS_ACT_GELU) return NMS_ERR_INVALID_ARG;
    if (bad_row(dy_row, rows) || bad_row(x_row, rows) || bad_row(weight_row, outer)) return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type);
    if (misaligned(dx, e) || misaligned(dweight, e) || misaligned(dbias, 4) || misaligned(dev_status, 4))
        return NMS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (rows == 0) {
        if (dweight) cudaMemsetAsync(dweight, 0, e * outer * inner, st);
        if (dbias) cudaMemsetAsync(dbias, 0, sizeof(float) * outer, st);
        return cuda_status();
    }
    if (!dy || misaligned(dy, e) || misaligned(x, e) || misaligned(weight, e) || misaligned(pre, e) ||
        (dx && !weight) || (dweight && !x) || (act != NMS_ACT_NONE && !pre))
        return NMS_ERR_INVALID_ARG;
    const bool dy_uneven = uneven(type, dy, dy_row, rows, outer);
    const bool aligned = !dy_uneven && !(x && uneven(type, x, x_row, rows, inner)) &&
                         !(weight && uneven(type, weight, weight_row, outer, inner));
    size_t need;
    nms_linear_grad_workspace_size(type, rows, inner, outer, aligned, &need);
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < need) return NMS_ERR_WORKSPACE;
    // With SiLU and GELU dz has more bits than dy: of 16 bits it goes to the products in two parts, dz rounded and what
    // that left out (ReLU passes dy on).  4800 x 1024 -> 4096 bf16 with SiLU: 132 us, dx and dweight off by 1.7e-3 of
    // their size, which is their own rounding; by dz rounded 80 us and 2.3e-3.
    const bool low = type != NMS_TYPE_F32 && (act == NMS_ACT_SILU || act == NMS_ACT_GELU) && !rounded && (dx || dweight);
    char* rest = static_cast<char*>(workspace) + round_up(e * rows * padded(outer));
    void* const lower = low ? rest : nullptr;
    if (type != NMS_TYPE_F32) rest += round_up(e * rows * padded(outer));
    void* sums = rest;
    rest += round_up(slope_workspace_bytes(rows, outer));
    const bool dx_planes = by_planes(type, rows, inner, outer, false), dw_planes = by_planes(type, outer, inner, rows, true);
    const bool products = dx || dweight, changed = products && (act != NMS_ACT_NONE || dy_uneven);
    // What reads dz for its sums or slopes makes its planes on the way, where nothing else takes it; without slopes only
    // where it moves 16 bytes at a time (557 wide, 18205 rows, none: 270 us that way and 250 with a pass of their own).
    const bool whole = outer % 4 == 0 && dy_row % 4 == 0 && !misaligned(dy, 16);
    const bool planes = products && (!dx || dx_planes) && (!dweight || dw_planes) && (changed || (dbias && whole));
    const bool copied = changed && !planes;
    Operand z{copied ? workspace : dy, copied ? padded(outer) : dy_row, rows, outer};
    if (planes) {
        z.planes = rest;
        rest += plane_bytes(rows, outer);
    }
    if (copied || planes || dbias) {
        SlopeArgs a{};
        a.dy = dy;
        a.dy_row = dy_row;
        a.pre = act != NMS_ACT_NONE ? pre : nullptr;
        a.type = type;
        a.rows = rows;
        a.width = outer;
        a.act = act;
        a.dz = copied ? workspace : nullptr;
        a.dz_row = padded(outer);
        a.low = lower;
        a.planes = const_cast<void*>(z.planes);
        a.dbias = dbias;
        launch_slope(a, sums, st);
    }
    float* const scratch = reinterpret_cast<float*>(rest);
    rest += product_scratch_bytes(type, outer > rows ? outer : rows);
    Operand xs{x, x_row, rows, inner}, ws{weight, weight_row, outer, inner};
    if (planes && dx && dweight) {  // both products' other operands at once
        const SplitRows split[2] = {as_split(ws, rest), as_split(xs, rest)};
        launch_split_rows(split, 2, st);
    }
    ProductArgs p{};
    p.type = type;
    p.act = NMS_ACT_NONE;
    p.status = dev_status;
    p.a_low = lower;
    p.scratch = scratch;
    p.b_across = 1;
    p.n = inner;
    p.segments = 1;
    if (dx) {
        p.m = rows;
        p.k = outer;
        p.out = dx;
        if (!launch_product(p, z, ws, dx_planes, rest, st)) return NMS_ERR_CUDA;
    }
    if (dweight) {
        p.a_across = 1;
        p.m = outer;
        p.k = rows;
        p.out = dweight;
        p.segments = gradient_segments(type, outer, inner, rows, low);
        if (p.segments > 1) {
            p.parts = reinterpret_cast<float*>(rest);
            rest += parts_bytes(p.segments, outer, inner);
        }
        if (!launch_product(p, z, xs, dw_planes, rest, st)) return NMS_ERR_CUDA;
        // The join of columns is made for many parts of few results.
        if (p.segments > 32 && type == NMS_TYPE_F32)
            launch_column_join(p.parts, p.segments, static_cast<int64_t>(outer) * inner, static_cast<int64_t>(outer) * inner,
                               static_cast<float*>(dweight), nullptr, st);
        else if (p.segments > 1)
            launch_join_parts(p.parts, p.segments, static_cast<int64_t>(outer) * inner, dweight, type, st);
    }
    return cuda_status();
}

static nms_status check_layer(int32_t type, int32_t param_type, int64_t rows, int32_t width)
{
    if (!known_type(type) || (param_type != NMS_TYPE_F32 && param_type != type) || rows < 0 || width < 1)
        return NMS_ERR_INVALID_ARG;
    if (width > NMS_LAYER_MAX_WIDTH || rows > kMostRows) return NMS_ERR_CAPACITY;
    return NMS_OK;
}

extern "C" nms_status nms_layer_norm_run(const void* x, int64_t x_row, const void* residual, int64_t residual_row,
                                         int32_t type, int64_t rows, int32_t width, const void* weight,
                                         const void* bias, int32_t param_type, float eps, void* y, void* sum,
                                         float* mean, float* rstd, void* stream)
{
    const nms_status s = check_layer(type, param_type, rows, width);
    if (s != NMS_OK) return s;
    if (!(eps >= 0.0f) || std::isinf(eps) || bad_row(x_row, rows) || bad_row(residual_row, rows) ||
        (rows > 0 && (residual != nullptr) != (sum != nullptr)))
        return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type), pe = type_bytes(param_type);
    if (misaligned(weight, pe) || misaligned(bias, pe) || misaligned(mean, 4) || misaligned(rstd, 4))
        return NMS_ERR_INVALID_ARG;
    if (rows == 0) return NMS_OK;
    if (!x || !y || misaligned(x, e) || misaligned(y, e) || misaligned(residual, e) || misaligned(sum, e))
        return NMS_ERR_INVALID_ARG;
    cudaGetLastError();
    LayerArgs a{};
    a.x = x;
    a.x_row = x_row;
    a.second = residual;
    a.second_row = residual ? residual_row : 0;
    a.type = type;
    a.rows = rows;
    a.width = width;
    a.weight = weight;
    a.bias = bias;
    a.param_f32 = param_type == NMS_TYPE_F32;
    a.eps = eps;
    a.out = y;
    a.sum = sum;
    a.mean = mean;
    a.rstd = rstd;
    launch_layer_norm(a, static_cast<cudaStream_t>(stream));
    return cuda_status();
}

extern "C" nms_status nms_layer_norm_workspace_size(int64_t rows, int32_t width, size_t* bytes)
{
    if (!bytes) return NMS_ERR_INVALID_ARG;
    const nms_status s = check_layer(NMS_TYPE_F32, NMS_TYPE_F32, rows, width);
    if (s != NMS_OK) return s;
    *bytes = rows == 0 ? 0 : round_up(layer_grad_workspace_bytes(rows, width));
    return NMS_OK;
}

extern "C" nms_status nms_layer_norm_grad_run(const void* dy, int64_t dy_row, const void* x, int64_t x_row,
                                              const void* dsum, int64_t dsum_row, int32_t type, int64_t rows,
                                              int32_t width, const float* mean, const float* rstd, const void* weight,
                                              int32_t param_type, void* dx, float* dweight, float* dbias,
                                              void* workspace, size_t workspace_bytes, void* stream)
{
    const nms_status s = check_layer(type, param_type, rows, width);
    if (s != NMS_OK) return s;
    if (bad_row(dy_row, rows) || bad_row(x_row, rows) || bad_row(dsum_row, rows)) return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type);
    if (misaligned(weight, type_bytes(param_type)) || misaligned(mean, 4) || misaligned(rstd, 4) ||
        misaligned(dweight, 4) || misaligned(dbias, 4))
        return NMS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (rows == 0) {
        if (dweight) cudaMemsetAsync(dweight, 0, sizeof(float) * width, st);
        if (dbias) cudaMemsetAsync(dbias, 0, sizeof(float) * width, st);
        return cuda_status();
    }
    if (!dy || !x || !dx || !mean || !rstd || misaligned(dy, e) || misaligned(x, e) || misaligned(dx, e) ||
        misaligned(dsum, e))
        return NMS_ERR_INVALID_ARG;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < layer_grad_workspace_bytes(rows, width))
        return NMS_ERR_WORKSPACE;
    LayerArgs a{};
    a.x = x;
    a.x_row = x_row;
    a.second = dsum;
    a.second_row = dsum ? dsum_row : 0;
    a.dy = dy;
    a.dy_row = dy_row;
    a.type = type;
    a.rows = rows;
    a.width = width;
    a.weight = weight;
    a.param_f32 = param_type == NMS_TYPE_F32;
    a.out = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dweight = dweight;
    a.dbias = dbias;
    launch_layer_grad(a, workspace, st);
    return cuda_status();
}

extern "C" nms_status nms_rotary_run(const void* x, int64_t x_batch, int64_t x_token, int64_t x_head, int32_t type,
                                     int64_t batch, int64_t tokens, int32_t heads, int32_t dim, const void* positions,
                                     int32_t position_type, int64_t sets, int32_t axes, const int64_t* lut,
                                     int32_t pairs, int32_t halves, int32_t inverse, void* y, int64_t y_batch,
                                     int64_t y_token, int64_t y_head, void* stream)
{
    if (!known_type(type) || (position_type != NMS_TYPE_F32 && position_type != NMS_POSITION_I32) || batch < 0 ||
        tokens < 0 || heads < 0 || dim < 1 || axes < 1 || pairs < 0 || pairs > dim / 2 || (sets != 1 && sets != batch))
        return NMS_ERR_INVALID_ARG;
    if (axes > NMS_ROTARY_MAX_AXES || dim > NMS_ROTARY_MAX_DIM || heads > (1 << 20) || batch > kMostRows ||
        tokens > kMostRows || batch * tokens > kMostRows || static_cast<int64_t>(heads) * dim > kMostRows ||
        too_far(batch * tokens, static_cast<int64_t>(heads) * dim))
        return NMS_ERR_CAPACITY;
    const bool empty = batch == 0 || tokens == 0 || heads == 0;
    if (empty) return NMS_OK;
    for (const int64_t* st : {&x_batch, &y_batch})
        if (bad_row(*st, batch)) return NMS_ERR_INVALID_ARG;
    if (bad_row(x_token, tokens) || bad_row(y_token, tokens) || bad_row(x_head, heads) || bad_row(y_head, heads))
        return NMS_ERR_INVALID_ARG;
    const uintptr_t e = type_bytes(type);
    if (!x || !y || misaligned(x, e) || misaligned(y, e) || (pairs > 0 && (!positions || !lut)) ||
        misaligned(positions, 4) || misaligned(lut, 8))
        return NMS_ERR_INVALID_ARG;
    cudaGetLastError();
    RotaryArgs a{x,     x_batch, x_token, x_head, type,  batch,  tokens,  heads, dim,     positions, sets,
                 position_type == NMS_TYPE_F32,   axes,  lut,    pairs,   halves != 0,    inverse != 0, y,
                 y_batch, y_token, y_head};
    launch_rotary(a, static_cast<cudaStream_t>(stream));
    return cuda_status();
}
