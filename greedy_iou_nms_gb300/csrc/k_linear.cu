// Matrix products of binary32 operands with bias, activation and residual in
// their epilogue, on the plain arithmetic units, and the copy of 16-bit rows
// whose places the tensor cores' loads cannot take.
//
// product_kernel, for what by_planes() (gbnms_block.cu) does not send to the tensor
// cores (k_product_split.cu): products of less than 2^26 multiplications, 2^21 where
// k is 1024 and more.  A block has a tile of 64 x 64 results, its 256 threads 4 x 4
// of them each.  Few tiles: the blocks of a cluster share one, each a stretch of k,
// and add up their parts through distributed shared memory, in order.
//
// Up to 16 rows are a stream of the weight, whose elements are used once a row:
// few_along_kernel reads it straight to registers, all of an SM's warps at once,
// few_across_kernel has it copied ahead.  The gradient of a weight of up to 32 rows
// is such a stream of x.
#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

namespace {

constexpr int PR_DEPTH = 16;   // of a step along k
constexpr int PR_STAGES = 3;   // steps in shared memory
constexpr int PR_TILE = 64, PR_STRIDE = PR_TILE + 4;

// One operand's way to shared memory, [k][m or n], element by element
// (cp.async), so that any stride and start will do and either order of the
// operand.  Element i of a thread lies i * delta behind its first.
template <bool ACROSS>
struct Feed {
    static constexpr int TILE = PR_TILE, STRIDE = PR_STRIDE, N = TILE * PR_DEPTH / 256;
    const float* from;
    int64_t delta, step;
    uint32_t to;
    int64_t left_mn, left_k;  // elements from this thread's first on
    __device__ __forceinline__ Feed(const float* p, int64_t row, int64_t mn0, int64_t mns, int64_t k0, int64_t ks,
                                    const void* shared)
    {
        const int t = threadIdx.x, mn = ACROSS ? t % TILE : t / PR_DEPTH, k = ACROSS ? t / TILE : t % PR_DEPTH;
        from = p + (ACROSS ? (k0 + k) * row + mn0 + mn : (mn0 + mn) * row + k0 + k);
        delta = ACROSS ? (256 / TILE) * row : (256 / PR_DEPTH) * row;
        step = ACROSS ? PR_DEPTH * row : PR_DEPTH;
        to = static_cast<uint32_t>(__cvta_generic_to_shared(shared)) + 4 * (k * STRIDE + mn);
        left_mn = mns - mn0 - mn;
        left_k = ks - k;
    }
    // The next step; what lies outside becomes 0.
    __device__ __forceinline__ void next(int stage)
    {
        const float* p = from;
        const uint32_t at = to + stage * (PR_DEPTH * STRIDE * 4);
#pragma unroll
        for (int i = 0; i < N; ++i, p += delta) {
            const bool in = ACROSS ? left_mn > 0 && left_k > i * (256 / TILE) : left_k > 0 && left_mn > i * (256 / PR_DEPTH);
            const uint32_t dst = at + 4 * i * (ACROSS ? (256 / TILE) * STRIDE : 256 / PR_DEPTH);
            if (in) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(p) : "memory");
            else asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(0.0f) : "memory");
        }
        from += step;
        left_k -= PR_DEPTH;
    }
};

// The sum over the cluster's blocks of what each has at its own `at`.
__device__ __forceinline__ float cluster_sum(const float* at, int split)
{
    const uint32_t own = static_cast<uint32_t>(__cvta_generic_to_shared(at));
    float v[8], sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < split) {
            uint32_t peer;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(own), "r"(q));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[q]) : "r"(peer));
        }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < split) sum += v[q];
    return sum;
}

// What a result gets added.
struct Addends {
    float bias, residual;
    __device__ __forceinline__ Addends(const ProductArgs& p, int64_t m, int64_t n)
        : bias(p.bias ? __ldg(static_cast<const float*>(p.bias) + n) : 0.0f),
          residual(p.residual ? static_cast<const float*>(p.residual)[m * p.residual_row + n] : 0.0f)
    {
    }
    __device__ __forceinline__ Addends() {}
};

__device__ __forceinline__ void finish(const ProductArgs& p, int64_t m, int64_t n, float sum, const Addends& add)
{
    float z[1] = {sum + add.bias};
    if (p.pre) static_cast<float*>(p.pre)[m * p.n + n] = z[0];
    act_values<float>(z, p.act);
    static_cast<float*>(p.out)[m * p.n + n] = z[0] + add.residual;
}

template <bool A_ACROSS, bool B_ACROSS>
__global__ void __launch_bounds__(256, 3)
product_kernel(const ProductArgs p, int64_t tiles_n, int split)
{
    static_assert(PR_TILE <= 2 * PR_STAGES * PR_DEPTH, "a block's part fits in the stages");
    extern __shared__ __align__(16) float stages[];  // [2][PR_STAGES][PR_DEPTH][PR_STRIDE]; then the block's part
    float* const as = stages;
    float* const bs = stages + PR_STAGES * PR_DEPTH * PR_STRIDE;
    const int64_t tile = blockIdx.x / split, rank = blockIdx.x - tile * split;
    const int64_t tm = tile / tiles_n, tn = tile - tm * tiles_n;
    const int64_t m0 = tm * PR_TILE, n0 = tn * PR_TILE;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {}, total[4][4] = {};
    const int64_t all = (p.k + PR_DEPTH - 1) / PR_DEPTH, each = (all + split - 1) / split;
    const int64_t from = min(p.k, rank * each * PR_DEPTH), count = min(p.k - from, each * PR_DEPTH);  // of k, this block's
    Feed<A_ACROSS> a(static_cast<const float*>(p.a), p.a_row, m0, p.m, from, count, as);
    Feed<B_ACROSS> b(static_cast<const float*>(p.b), p.b_row, n0, p.n, from, count, bs);
    const int64_t steps = (count + PR_DEPTH - 1) / PR_DEPTH;
#pragma unroll
    for (int s = 0; s < PR_STAGES - 1; ++s) {
        if (s < steps) {
            a.next(s);
            b.next(s);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int at = 0, ahead = PR_STAGES - 1;
    for (int64_t s = 0; s < steps; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(PR_STAGES - 2) : "memory");
        __syncthreads();  // step s is there, and step s - 1 is no longer read
        if (s + PR_STAGES - 1 < steps) {
            a.next(ahead);
            b.next(ahead);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const float* const ak = as + at * PR_DEPTH * PR_STRIDE;
        const float* const bk = bs + at * PR_DEPTH * PR_STRIDE;
#pragma unroll
        for (int k = 0; k < PR_DEPTH; ++k) {
            alignas(16) float x[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; i += 4)
                *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(ak + k * PR_STRIDE + i * 16 + ty * 4);
#pragma unroll
            for (int j = 0; j < 4; j += 4)
                *reinterpret_cast<float4*>(w + j) = *reinterpret_cast<const float4*>(bk + k * PR_STRIDE + j * 16 + tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
        }
        // Sums of 256 products, added up: a chain over all of k would round off with k.
        if (s % 16 == 15 || s + 1 == steps) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    total[i][j] += acc[i][j];
                    acc[i][j] = 0.0f;
                }
        }
        at = at + 1 == PR_STAGES ? 0 : at + 1;
        ahead = ahead + 1 == PR_STAGES ? 0 : ahead + 1;
    }
    __syncthreads();  // the stages are no longer read
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 4)
            *reinterpret_cast<float4*>(stages + ((i / 4) * 64 + ty * 4 + i % 4) * PR_STRIDE + j * 16 + tx * 4) =
                make_float4(total[i][j], total[i][j + 1], total[i][j + 2], total[i][j + 3]);
    // From shared memory a warp's results are neighbours in a row.
    if (split == 1) {
        __syncthreads();
        for (int e0 = threadIdx.x; e0 < PR_TILE * PR_TILE; e0 += 8 * 256) {
            Addends add[8];  // the residual may be what is written: read before the first of these results
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (e0 + i * 256) / PR_TILE, c = (e0 + i * 256) % PR_TILE;
                if (m0 + r < p.m && n0 + c < p.n) add[i] = Addends(p, m0 + r, n0 + c);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (e0 + i * 256) / PR_TILE, c = (e0 + i * 256) % PR_TILE;
                if (m0 + r < p.m && n0 + c < p.n) finish(p, m0 + r, n0 + c, stages[r * PR_STRIDE + c], add[i]);
            }
        }
        return;
    }
    cluster_barrier();
    const int rows = PR_TILE / split;
    for (int e = threadIdx.x; e < rows * PR_TILE; e += 256) {
        const int r = static_cast<int>(rank) * rows + e / PR_TILE, c = e % PR_TILE;
        if (m0 + r < p.m && n0 + c < p.n) 
            finish(p, m0 + r, n0 + c, cluster_sum(stages + r * PR_STRIDE + c, split), Addends(p, m0 + r, n0 + c));
    }
    __syncwarp();
    cluster_barrier();  // no block leaves while another reads its part
}

// Results of up to R rows and eight columns a block; B's rows are columns of the
// result.  Four of a block's warps share four columns, each a quarter of k.
template <int R, int V>
__global__ void __launch_bounds__(256)
few_along_kernel(const ProductArgs p)
{
    __shared__ float parts[8][4 * R];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, quarter = warp % 4;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 8 + warp / 4 * 4;
    const float* const x = static_cast<const float*>(p.a);
    const float* const w = static_cast<const float*>(p.b);
    float acc[4][R] = {};
    for (int64_t k = (quarter * 32 + lane) * V; k < p.k; k += 128 * V) {  // V divides k
        Pack<float, V> wv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n0 + c < p.n) wv[c] = *reinterpret_cast<const Pack<float, V>*>(w + (n0 + c) * p.b_row + k);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= p.m) break;
            const Pack<float, V> xv = *reinterpret_cast<const Pack<float, V>*>(x + r * p.a_row + k);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[c][r] = fmaf(xv.v[i], wv[c].v[i], acc[c][r]);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = warp_sum(acc[c][r]);
            if (lane == 0) parts[warp][c * R + r] = sum;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 8 * R; e += 256) {
        const int r = e / 8, c = e % 8, first = c / 4 * 4, at = c % 4 * R + r;
        const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + c;
        if (r < p.m && n < p.n)
            finish(p, r, n, ((parts[first][at] + parts[first + 1][at]) + parts[first + 2][at]) + parts[first + 3][at],
                   Addends(p, r, n));
    }
}

constexpr int FEW_CHUNK = 32, FEW_STAGES = 4;
template <int R> constexpr int FEW_PITCH = R == 1 ? 1 : R + 4;  // of A's chunk: 32 lanes fill it over its columns
template <int R, int V> constexpr int FEW_STAGE = FEW_CHUNK * 32 * V + FEW_CHUNK * FEW_PITCH<R>;  // floats
template <int R, int V>
constexpr int FEW_SMEM = 4 * (FEW_STAGES * FEW_STAGE<R, V> > 9 * R * 32 * V ? FEW_STAGES * FEW_STAGE<R, V> : 9 * R * 32 * V);

// BYTES to shared memory, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void copy_or_zero(float* to, const float* from, bool in)
{
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(in ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(from), "n"(BYTES), "r"(in ? BYTES : 0) : "memory");
}

// Results of up to R rows and 32 V columns a cluster, B lying across: a block
// has a stretch of k, in chunks of 32 on their way to shared memory three ahead, a
// warp four rows of B of each chunk, a lane V columns.  The gradient of a weight
// of up to 32 rows (A across too) has segments of k along the grid's second axis.
// HBM bounds it, and from 16 rows on its arithmetic as much: gradient of 8 x 8192 by a
// weight of 8192 x 8192 52 us (5.2 TB/s; a chunk at a time through registers 100), 16 x
// 4096 by 11008 x 4096 51; two blocks an SM, without that bound 84.
template <int R, int V>
__global__ void __launch_bounds__(256, 2)
few_across_kernel(const ProductArgs p, int split)
{
    extern __shared__ __align__(16) float dynamic[];
    constexpr int COLUMNS = 32 * V, EACH = FEW_CHUNK / 8, PITCH = FEW_PITCH<R>;
    float* const stages = dynamic;                            // [FEW_STAGES], a chunk's rows of B [EACH][256][V], of A [FEW_CHUNK][PITCH]
    float* const parts = dynamic;                             // after them [8][R][COLUMNS]
    float* const sums = parts + 8 * R * COLUMNS;              // [R][COLUMNS]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t group = blockIdx.x / split, rank = blockIdx.x - group * split;
    const int64_t n = group * COLUMNS + lane * V;
    const float* const x = static_cast<const float*>(p.a);
    const float* const w = static_cast<const float*>(p.b) + n;
    const int64_t sharers = static_cast<int64_t>(p.segments) * split;
    const int64_t each = ((p.k + sharers - 1) / sharers + FEW_CHUNK - 1) / FEW_CHUNK * FEW_CHUNK;
    const int64_t first = min(p.k, (static_cast<int64_t>(blockIdx.y) * split + rank) * each), last = min(p.k, first + each);
    // A chunk on its way; what is not there becomes 0.
    auto fetch = [&](int64_t k0, int stage) {
        float* const to = stages + stage * FEW_STAGE<R, V>;
        if (k0 < last) {
#pragma unroll
            for (int q = 0; q < EACH; ++q) {
                const int64_t k = k0 + warp * EACH + q;
                const bool in = n < p.n && k < last;  // V divides n
                copy_or_zero<4 * V>(to + (q * 256 + threadIdx.x) * V, in ? w + k * p.b_row : static_cast<const float*>(p.b), in);
            }
#pragma unroll
            for (int e = threadIdx.x; e < FEW_CHUNK * R; e += 256) {
                const int r = p.a_across ? e % R : e / FEW_CHUNK, c = p.a_across ? e / R : e % FEW_CHUNK;
                const bool in = r < p.m && k0 + c < last;
                const int64_t at = p.a_across ? (k0 + c) * p.a_row + r : r * p.a_row + k0 + c;
                copy_or_zero<4>(to + EACH * 256 * V + c * PITCH + r, in ? x + at : x, in);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float acc[R][V] = {};
#pragma unroll
    for (int s = 0; s < FEW_STAGES - 1; ++s) fetch(first + s * FEW_CHUNK, s);
    int at = 0, ahead = FEW_STAGES - 1;
    for (int64_t k0 = first; k0 < last; k0 += FEW_CHUNK) {
        asm volatile("cp.async.wait_group %0;" ::"n"(FEW_STAGES - 2) : "memory");
        __syncthreads();  // this chunk is there, and the last one no longer read
        fetch(k0 + (FEW_STAGES - 1) * FEW_CHUNK, ahead);
        const float* const now = stages + at * FEW_STAGE<R, V>;
        const float* const xs = now + EACH * 256 * V + warp * EACH * PITCH;
#pragma unroll
        for (int q = 0; q < EACH; ++q) {
            const Pack<float, V> wv = *reinterpret_cast<const Pack<float, V>*>(now + (q * 256 + threadIdx.x) * V);
            constexpr int TOGETHER = R == 1 ? 1 : 4;
#pragma unroll
            for (int r = 0; r < R; r += TOGETHER) {
                const Pack<float, TOGETHER> xv = *reinterpret_cast<const Pack<float, TOGETHER>*>(xs + q * PITCH + r);
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[r + j][i] = fmaf(xv.v[j], wv.v[i], acc[r + j][i]);
            }
        }
        at = at + 1 == FEW_STAGES ? 0 : at + 1;
        ahead = ahead + 1 == FEW_STAGES ? 0 : ahead + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stages are no longer read
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) parts[(warp * R + r) * COLUMNS + lane * V + i] = acc[r][i];
    __syncthreads();
    for (int e = threadIdx.x; e < R * COLUMNS; e += 256) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) sum += parts[q * R * COLUMNS + e];
        sums[e] = sum;
    }
    cluster_barrier();
    for (int e = static_cast<int>(rank) * 256 + threadIdx.x; e < R * COLUMNS; e += 256 * split) {
        const int r = e / COLUMNS, c = e % COLUMNS;
        const int64_t at = group * COLUMNS + c;
        if (r >= p.m || at >= p.n) continue;
        const float sum = cluster_sum(sums + e, split);
        if (p.segments > 1) p.parts[(blockIdx.y * p.m + r) * p.n + at] = sum;
        else finish(p, r, at, sum, Addends(p, r, at));
    }
    __syncwarp();
    cluster_barrier();  // no block leaves while another reads its sums
}

template <typename T>
__global__ void __launch_bounds__(256)
join_parts_kernel(const float* parts, int segments, int64_t n, T* out)
{
    pdl_wait();  // the parts are there
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        constexpr int AHEAD = 8;
        float sum = 0.0f;
        for (int s = 0; s < segments; s += AHEAD) {
            float v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[k] = s + k < segments ? parts[(s + k) * n + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) sum += v[k];
        }
        out[i] = from_f32<T>(sum);
    }
}

// Eight elements of a row a thread.
__global__ void __launch_bounds__(256)
copy_rows_kernel(const CopyRows first, const CopyRows second)
{
    const int64_t n0 = first.rows * (first.to_row / 8), n = n0 + second.rows * (second.to_row / 8);
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < n; at += static_cast<int64_t>(gridDim.x) * 256) {
        const CopyRows& c = at < n0 ? first : second;
        const int64_t i = at < n0 ? at : at - n0, parts = c.to_row / 8, row = i / parts, e = (i - row * parts) * 8;
        const uint16_t* p = static_cast<const uint16_t*>(c.from) + row * c.from_row + e;
        Pack<uint16_t, 8> q;
#pragma unroll
        for (int k = 0; k < 8; ++k) q.v[k] = e + k < c.width ? p[k] : 0;
        *reinterpret_cast<Pack<uint16_t, 8>*>(static_cast<uint16_t*>(c.to) + row * c.to_row + e) = q;
    }
}

}  // namespace

// A kernel over clusters of `split` blocks of 256 threads.
template <typename Kernel, typename... Args>
static bool launch_clusters(Kernel kernel, int64_t clusters, int split, int segments, int smem, cudaStream_t st, Args... args)
{
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return false;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * split), segments);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

static bool even(const void* p, int64_t row, int v) { return reinterpret_cast<uintptr_t>(p) % (4 * v) == 0 && row % v == 0; }

template <int R, int V>
static bool launch_few_across(const ProductArgs& p, cudaStream_t st)
{
    constexpr int COLUMNS = 32 * V;
    const int64_t groups = (p.n + COLUMNS - 1) / COLUMNS;
    // A gradient's blocks run all at once; the others' stretches are short.
    const int64_t most = p.a_across ? SMS * 2 : SMS * 4;
    int split = 1;
    while (split < 8 && groups * p.segments * split * 2 <= most && p.k / p.segments >= split * 128) split *= 2;
    return launch_clusters(few_across_kernel<R, V>, groups, split, p.segments, FEW_SMEM<R, V>, st, p, split);
}

template <int R>
static bool launch_few(const ProductArgs& p, cudaStream_t st)
{
    if (p.b_across)
        return p.n % 4 == 0 && even(p.b, p.b_row, 4) ? launch_few_across<R, 4>(p, st) : launch_few_across<R, 1>(p, st);
    const unsigned grid = static_cast<unsigned>((p.n + 7) / 8);
    if (p.k % 4 == 0 && even(p.a, p.a_row, 4) && even(p.b, p.b_row, 4)) few_along_kernel<R, 4><<<grid, 256, 0, st>>>(p);
    else few_along_kernel<R, 1><<<grid, 256, 0, st>>>(p);
    return true;
}

static bool launch_tiles(const ProductArgs& p, cudaStream_t st)
{
    constexpr int SMEM = 2 * PR_STAGES * PR_DEPTH * PR_STRIDE * 4;
    const int64_t tiles_n = (p.n + PR_TILE - 1) / PR_TILE, tiles = ((p.m + PR_TILE - 1) / PR_TILE) * tiles_n;
    const int64_t steps = (p.k + PR_DEPTH - 1) / PR_DEPTH;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= SMS * 4 && steps >= split * 8) split *= 2;
    if (p.a_across) return launch_clusters(product_kernel<true, true>, tiles, split, 1, SMEM, st, p, tiles_n, split);
    if (p.b_across) return launch_clusters(product_kernel<false, true>, tiles, split, 1, SMEM, st, p, tiles_n, split);
    return launch_clusters(product_kernel<false, false>, tiles, split, 1, SMEM, st, p, tiles_n, split);
}

bool launch_product_f32(const ProductArgs& p, cudaStream_t st)
{
    if (p.m <= 16) {
        if (p.m == 1) return launch_few<1>(p, st);
        return p.m <= 4 ? launch_few<4>(p, st) : p.m <= 8 ? launch_few<8>(p, st) : launch_few<16>(p, st);
    }
    // 32 sums of two columns each are as many registers as 16 of four.
    if (p.m <= 32 && p.a_across)
        return p.n % 2 == 0 && even(p.b, p.b_row, 2) ? launch_few_across<32, 2>(p, st) : launch_few_across<32, 1>(p, st);
    return launch_tiles(p, st);
}

void launch_join_parts(const float* parts, int segments, int64_t n, void* out, int type, cudaStream_t st)
{
    const int64_t want = (n + 255) / 256, most = SMS * 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (type == NMS_TYPE_F32) cudaLaunchKernelEx(&cfg, join_parts_kernel<float>, parts, segments, n, static_cast<float*>(out));
    else if (type == NMS_TYPE_F16)
        cudaLaunchKernelEx(&cfg, join_parts_kernel<__half>, parts, segments, n, static_cast<__half*>(out));
    else cudaLaunchKernelEx(&cfg, join_parts_kernel<__nv_bfloat16>, parts, segments, n, static_cast<__nv_bfloat16*>(out));
}

void launch_copy_rows(const CopyRows* of, int count, cudaStream_t st)
{
    CopyRows second{};
    if (count > 1) second = of[1];
    const int64_t n = of[0].rows * (of[0].to_row / 8) + second.rows * (second.to_row / 8);
    const int64_t want = (n + 255) / 256, most = SMS * 8;
    copy_rows_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, st>>>(of[0], second);
}

}  // namespace gbnms
