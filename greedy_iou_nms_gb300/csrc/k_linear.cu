// Matrix products of binary32 operands with bias, activation and residual in
// their epilogue, on the plain arithmetic units: a block has a tile of TILE x
// TILE results, its 256 threads S x S of them each.  And the copy of 16-bit
// rows whose places the tensor cores' loads cannot take.
#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

namespace {

constexpr int PR_DEPTH = 16;  // of a step along k

// A step of one operand in registers: element i of a thread is at (mn, k).
template <typename T, int TILE>
struct Step {
    static constexpr int N = TILE * PR_DEPTH / 256;
    float v[N];
    __device__ __forceinline__ static void place(int i, int across, int& mn, int& k)
    {
        const int at = i * 256 + threadIdx.x;
        if (across) {
            mn = at % TILE;
            k = at / TILE;
        } else {
            k = at % PR_DEPTH;
            mn = at / PR_DEPTH;
        }
    }
    __device__ __forceinline__ void load(const T* p, int64_t row, int across, int64_t mn0, int64_t mns, int64_t k0,
                                         int64_t ks)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int mn, k;
            place(i, across, mn, k);
            const int64_t a = mn0 + mn, b = k0 + k;
            v[i] = a < mns && b < ks ? to_f32(p[across ? b * row + a : a * row + b]) : 0.0f;
        }
    }
    __device__ __forceinline__ void store(float (*s)[TILE + 4], int across) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int mn, k;
            place(i, across, mn, k);
            s[k][mn] = v[i];
        }
    }
};

template <typename T, int S>
__global__ void __launch_bounds__(256)
product_kernel(const ProductArgs p, int64_t tiles_n)
{
    constexpr int TILE = 16 * S;
    __shared__ float as[2][PR_DEPTH][TILE + 4], bs[2][PR_DEPTH][TILE + 4];
    const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
    const int64_t m0 = tm * TILE, n0 = tn * TILE;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[S][S] = {}, total[S][S] = {};
    Step<T, TILE> a, b;
    const int64_t steps = (p.k + PR_DEPTH - 1) / PR_DEPTH;
    auto load = [&](int64_t s) {
        a.load(static_cast<const T*>(p.a), p.a_row, p.a_across, m0, p.m, s * PR_DEPTH, p.k);
        b.load(static_cast<const T*>(p.b), p.b_row, p.b_across, n0, p.n, s * PR_DEPTH, p.k);
    };
    load(0);
    a.store(as[0], p.a_across);
    b.store(bs[0], p.b_across);
    __syncthreads();
    for (int64_t s = 0; s < steps; ++s) {
        const int at = static_cast<int>(s & 1);
        if (s + 1 < steps) load(s + 1);
#pragma unroll
        for (int k = 0; k < PR_DEPTH; ++k) {
            alignas(16) float x[S], w[S];
#pragma unroll
            for (int i = 0; i < S; i += 4) {
                *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(&as[at][k][i * 16 + ty * 4]);
                *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(&bs[at][k][i * 16 + tx * 4]);
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
        if (s + 1 < steps) {
            a.store(as[at ^ 1], p.a_across);
            b.store(bs[at ^ 1], p.b_across);
            __syncthreads();
        }
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

void launch_product_f32(const ProductArgs& p, cudaStream_t st)
{
    auto tiles = [&](int64_t t) { return ((p.m + t - 1) / t) * ((p.n + t - 1) / t); };
    if (tiles(128) >= SMS)
        product_kernel<float, 8><<<static_cast<unsigned>(tiles(128)), 256, 0, st>>>(p, (p.n + 127) / 128);
    else
        product_kernel<float, 4><<<static_cast<unsigned>(tiles(64)), 256, 0, st>>>(p, (p.n + 63) / 64);
}

void launch_copy_rows(const void* from, int64_t from_row, int64_t rows, int64_t width, void* to, int64_t to_row,
                      cudaStream_t st)
{
    const int64_t want = (rows * ((width + 7) / 8) + 255) / 256, most = SMS * 8;
    copy_rows_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, st>>>(
        static_cast<const uint16_t*>(from), from_row, rows, width, static_cast<uint16_t*>(to), to_row);
}

}  // namespace gbnms
