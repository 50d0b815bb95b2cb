// Matrix products of binary32 operands with bias, activation and residual in
// their epilogue, on the plain arithmetic units: a block has a tile of TILE x
// TILE results, its 256 threads S x S of them each.  And the copy of 16-bit
// rows whose places the tensor cores' loads cannot take.
#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

namespace {

constexpr int PR_DEPTH = 16;   // of a step along k
constexpr int PR_STAGES = 4;   // steps in shared memory

// One operand's way to shared memory, [k][m or n], element by element
// (cp.async), so that any stride and start will do and either order of the
// operand.  Element i of a thread lies i * delta behind its first.
template <int TILE, bool ACROSS>
struct Feed {
    static constexpr int N = TILE * PR_DEPTH / 256, STRIDE = TILE + 4;
    const float* from;
    int64_t delta, step;
    uint32_t to;
    int64_t left_mn, left_k;  // elements from this thread's first on
    __device__ __forceinline__ Feed(const float* p, int64_t row, int64_t mn0, int64_t mns, int64_t ks, const void* shared)
    {
        const int t = threadIdx.x, mn = ACROSS ? t % TILE : t / PR_DEPTH, k = ACROSS ? t / TILE : t % PR_DEPTH;
        from = p + (ACROSS ? k * row + mn0 + mn : (mn0 + mn) * row + k);
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

template <int S, bool A_ACROSS, bool B_ACROSS>
__global__ void __launch_bounds__(256)
product_kernel(const ProductArgs p, int64_t tiles_n)
{
    using T = float;
    constexpr int TILE = 16 * S, STRIDE = TILE + 4;
    extern __shared__ __align__(16) float stages[];  // [2][PR_STAGES][PR_DEPTH][STRIDE]
    float* const as = stages;
    float* const bs = stages + PR_STAGES * PR_DEPTH * STRIDE;
    const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
    const int64_t m0 = tm * TILE, n0 = tn * TILE;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[S][S] = {}, total[S][S] = {};
    Feed<TILE, A_ACROSS> a(static_cast<const float*>(p.a), p.a_row, m0, p.m, p.k, as);
    Feed<TILE, B_ACROSS> b(static_cast<const float*>(p.b), p.b_row, n0, p.n, p.k, bs);
    const int64_t steps = (p.k + PR_DEPTH - 1) / PR_DEPTH;
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
        const float* const ak = as + at * PR_DEPTH * STRIDE;
        const float* const bk = bs + at * PR_DEPTH * STRIDE;
#pragma unroll
        for (int k = 0; k < PR_DEPTH; ++k) {
            alignas(16) float x[S], w[S];
#pragma unroll
            for (int i = 0; i < S; i += 4) {
                *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(ak + k * STRIDE + i * 16 + ty * 4);
                *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(bk + k * STRIDE + i * 16 + tx * 4);
            }
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < S; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
        }
        // Sums of 256 products, added up: a chain over all of k would round off with k.
        if (s % 16 == 15 || s + 1 == steps) {
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    total[i][j] += acc[i][j];
                    acc[i][j] = 0.0f;
                }
        }
        at = at + 1 == PR_STAGES ? 0 : at + 1;
        ahead = ahead + 1 == PR_STAGES ? 0 : ahead + 1;
    }
    T* out = static_cast<T*>(p.out);
    T* pre = static_cast<T*>(p.pre);
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int64_t m = m0 + (i / 4) * 64 + ty * 4 + i % 4;
        if (m >= p.m) continue;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int64_t n = n0 + (j / 4) * 64 + tx * 4 + j % 4;
            if (n >= p.n) continue;
            float z[1] = {total[i][j] + (p.bias ? load_param<T>(p.bias, p.bias_f32, n) : 0.0f)};
            if (pre) pre[m * p.n + n] = from_f32<T>(z[0]);
            act_values<T>(z, p.act);
            if (p.residual) z[0] += to_f32(static_cast<const T*>(p.residual)[m * p.residual_row + n]);
            out[m * p.n + n] = from_f32<T>(z[0]);
        }
    }
}

// Eight elements of a row a thread.
__global__ void __launch_bounds__(256)
copy_rows_kernel(const uint16_t* from, int64_t from_row, int64_t rows, int64_t width, uint16_t* to, int64_t to_row)
{
    const int64_t parts = (width + 7) / 8, n = rows * parts;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / parts, e = (i - row * parts) * 8;
        const uint16_t* p = from + row * from_row + e;
        Pack<uint16_t, 8> q;
#pragma unroll
        for (int k = 0; k < 8; ++k) q.v[k] = e + k < width ? p[k] : 0;
        *reinterpret_cast<Pack<uint16_t, 8>*>(to + row * to_row + e) = q;
    }
}

}  // namespace

template <int S>
static void launch_tiles(const ProductArgs& p, cudaStream_t st)
{
    constexpr int TILE = 16 * S, SMEM = 2 * PR_STAGES * PR_DEPTH * (TILE + 4) * 4;
    const int64_t tiles_n = (p.n + TILE - 1) / TILE, tiles = ((p.m + TILE - 1) / TILE) * tiles_n;
    auto run = [&](auto kernel) {
        if (SMEM > 48 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        kernel<<<static_cast<unsigned>(tiles), 256, SMEM, st>>>(p, tiles_n);
    };
    if (p.a_across) run(product_kernel<S, true, true>);
    else p.b_across ? run(product_kernel<S, false, true>) : run(product_kernel<S, false, false>);
}

void launch_product_f32(const ProductArgs& p, cudaStream_t st)
{
    if (((p.m + 127) / 128) * ((p.n + 127) / 128) >= SMS) launch_tiles<8>(p, st);
    else launch_tiles<4>(p, st);
}

void launch_copy_rows(const void* from, int64_t from_row, int64_t rows, int64_t width, void* to, int64_t to_row,
                      cudaStream_t st)
{
    const int64_t want = (rows * ((width + 7) / 8) + 255) / 256, most = SMS * 8;
    copy_rows_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, st>>>(
        static_cast<const uint16_t*>(from), from_row, rows, width, static_cast<uint16_t*>(to), to_row);
}

}  // namespace gbnms
