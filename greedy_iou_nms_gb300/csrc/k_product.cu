// Matrix products of 16-bit operands on the tensor cores (tcgen05), with bias,
// activation and residual in the epilogue:
//   out[m][n] = act(sum_k A[m][k] B[n][k] + bias[n]) + residual[m][n].
//
// A block has tiles of 128 x BN results.  One thread feeds a ring of shared-
// memory stages by TMA (64 columns of k a stage, 128-byte swizzle), one thread
// issues the matrix instructions, whose accumulators lie in tensor memory, and
// eight warps carry accumulators to the outputs: those of one tile while the
// next one is multiplied (two sets of accumulators).  An operand that lies
// across ([k][m], as both do for a weight's gradient) is taken as it lies: the
// instruction reads either order, only boxes and descriptors differ.
//
// Two blocks on neighbouring SMs share a tile of 256 x BN where there are tiles
// enough (PAIR): one thread's instructions work on both SMs' tensor cores, each
// of which has its own 128 rows of A and half of B's in shared memory.  A block
// alone moves 96 KB there for 512 cycles of multiplying (a stage of 48 KB in, and
// out), 192 bytes a cycle of the 128 that shared memory has; a block of a pair 64
// KB.  16384 x 4096 x 4096: bf16 without activation 286 us, 1.92 PFLOP/s, within
// 6% of torch's own product on the same card; fp16 with gelu and residual 328, and
// 380 back to back, where the power limit sets the clock (338 without either).
//
// Few rows of A (a step of serving): A and B change places, so that the long
// side fills the 128 lanes and BN is 16 to 64.  Few tiles: the blocks of a
// cluster share one, each a stretch of k, and add up their parts through
// distributed shared memory, in order.
//
// Long sums: see product_stretch().  An operand of two parts (low_of): k twice.
#include <atomic>

#include "tensor_core.cuh"

namespace gbnms {

namespace {

// BB: rows of B in a block's stage.
template <int BB> constexpr int TC_STAGES = BB == 256 ? 4 : BB == 128 ? 6 : 8;
template <int BB> constexpr int TC_RING = TC_STAGES<BB> * (A_BYTES + BB * TC_K * 2);  // from a multiple of 1024 on

struct TcArgs {
    int a_across, b_across;
    int64_t m, n, k;
    int64_t tiles_m, tiles_n;
    int split;     // blocks of a cluster, which share a tile along k
    int segments;  // stretches of k whose sums go to parts [segments][m][n], 1: none
    float* parts;
    const void* bias;
    int bias_f32, act;
    const void* residual;
    int64_t residual_m, residual_n;  // strides
    void* out;
    void* pre;
    int64_t out_m, out_n;  // strides of out and pre
    int vector;            // rows of out, pre and residual start at multiples of 16 bytes
    int stretch;           // steps along k whose products an accumulator adds up
    float* scratch;        // sums of longer ones so far: of each block TC_M x BN
    Patience patience;
    int low_of;            // operand that comes in two parts (1: A, 2: B, 0: none)
    int32_t* status;
};

// One result.
template <typename T>
__device__ __forceinline__ void finish_one(const TcArgs& p, int64_t m, int64_t n, float sum, float bias, T residual)
{
    float z[1] = {sum + bias};
    const int64_t at = m * p.out_m + n * p.out_n;
    if (p.pre) static_cast<T*>(p.pre)[at] = from_f32<T>(z[0]);
    act_values<T>(z, p.act);
    if (p.residual) z[0] += to_f32(residual);
    static_cast<T*>(p.out)[at] = from_f32<T>(z[0]);
}

// N results of one m; the residual, which may be what is written, is read before
// the first of them.
template <typename T, int N>
__device__ __forceinline__ void finish_some(const TcArgs& p, int64_t m, int64_t n, const float (&sum)[N], const float* bias, int bias_step)
{
    T r[N];
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (n + i < p.n) r[i] = static_cast<const T*>(p.residual)[m * p.residual_m + (n + i) * p.residual_n];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (n + i < p.n) finish_one<T>(p, m, n + i, sum[i], bias[i * bias_step], r[i]);
}

// A warp's 32 rows of 32 results, on their way between one row a lane, as
// tensor memory gives them, and 64 consecutive bytes of a row for four lanes, as
// memory likes them: through shared memory, rows TC_PITCH bytes apart.  (Rows of
// 16 bytes a lane straight to memory: 349 us for 16384 x 4096 x 4096 with gelu
// and residual, 34 for 4864 x 1024 x 4096 without.)
constexpr int TC_PITCH = 80, TC_PATCH = 32 * TC_PITCH;

template <typename T>
struct Patch {
    using Vec = Pack<T, 8>;
    char* own;   // this lane's row
    char* part;  // this lane's 16 bytes of row lane / 4; eight rows further, the next
    __device__ __forceinline__ Patch(char* patch, int lane)
        : own(patch + lane * TC_PITCH), part(patch + lane / 4 * TC_PITCH + lane % 4 * 16)
    {
    }
    // Rows row .. row + 31 (lane's part at `at`, rows `stride` apart) of which there are m.
    __device__ __forceinline__ static void fetch(Vec (&v)[4], const T* at, int64_t stride, int64_t row, int64_t m, int lane)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = row + i * 8 + lane / 4;
            if (r < m) v[i] = *reinterpret_cast<const Vec*>(at + r * stride + lane % 4 * 8);
        }
    }
    __device__ __forceinline__ void spread(const Vec (&v)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<Vec*>(part + i * 8 * TC_PITCH) = v[i];
        __syncwarp();
    }
    __device__ __forceinline__ void take(Vec (&v)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const Vec*>(own + i * 16);
        __syncwarp();
    }
    // The same of rows that start anywhere: a lane has a column, the 32 rows one after another.
    __device__ __forceinline__ void spread_columns(const T* at, int64_t stride, int64_t row, int64_t m, int64_t columns,
                                                   int lane) const
    {
        T* const patch = reinterpret_cast<T*>(own - lane * TC_PITCH) + lane;
        T v[32];  // all on their way before the first is put down
#pragma unroll
        for (int r = 0; r < 32; ++r)
            if (lane < columns && row + r < m) v[r] = at[(row + r) * stride + lane];
#pragma unroll
        for (int r = 0; r < 32; ++r) patch[r * (TC_PITCH / 2)] = v[r];
        __syncwarp();
    }
    __device__ __forceinline__ void put_columns(const float (&z)[32], T* at, int64_t stride, int64_t row, int64_t m,
                                                int64_t columns, int lane) const
    {
        const T* const patch = reinterpret_cast<const T*>(own - lane * TC_PITCH) + lane;
        leave(z);
        if (lane < columns)
            for (int r = 0; r < 32 && row + r < m; ++r) at[(row + r) * stride + lane] = patch[r * (TC_PITCH / 2)];
        __syncwarp();
    }
    // One row a lane.
    __device__ __forceinline__ void leave(const float (&z)[32]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = z[8 * i + k];
            *reinterpret_cast<Vec*>(own + i * 16) = pack_results<T, 8>(e);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void put(const float (&z)[32], T* at, int64_t stride, int64_t row, int64_t m, int lane) const
    {
        leave(z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = row + i * 8 + lane / 4;
            if (r < m) *reinterpret_cast<Vec*>(at + r * stride + lane % 4 * 8) = *reinterpret_cast<const Vec*>(part + i * 8 * TC_PITCH);
        }
        __syncwarp();
    }
};

// A thread's sums of a stretch of k, TC_WRITERS apart: added to, and left.
template <int N>
__device__ __forceinline__ void take_sums(float (&v)[N], const float* at)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += at[i * TC_WRITERS];
}
template <int N>
__device__ __forceinline__ void leave_sums(const float (&v)[N], float* at)
{
#pragma unroll
    for (int i = 0; i < N; ++i) at[i * TC_WRITERS] = v[i];
}

// SWAP: A's rows are results' columns (the operands changed places); bias by m.
template <typename T, int BN, bool SWAP, bool PAIR>
__global__ void __launch_bounds__(TC_THREADS, 1)
product_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_low, const TcArgs p)
{
    constexpr int BB = PAIR ? BN / 2 : BN, ROWS = PAIR ? 2 * TC_M : TC_M;  // of B in this block, of A in a tile
    constexpr int STAGES = TC_STAGES<BB>, B_BYTES = BB * TC_K * 2, STAGE = A_BYTES + B_BYTES;
    constexpr int COLUMNS = 2 * BN < 32 ? 32 : 2 * BN;  // of tensor memory
    constexpr int CHUNK = BN >= 64 ? 32 : 8;            // columns that a thread carries at a time
    extern __shared__ char dynamic[];
    __shared__ alignas(8) uint64_t bars[2 * STAGES + 4];
    __shared__ uint32_t tensor_at;
    __shared__ float lost_s;  // 0; a NaN when a part of this block is none
    __shared__ alignas(16) float bias_s[2][SWAP ? TC_M : BN];
    const uint32_t ring = (shared_address(dynamic) + 1023) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = shared_address(bars), empty = full + 8 * STAGES, done = empty + 8 * STAGES, free_ = done + 16;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            barrier_init(full + 8 * s, 1);
            barrier_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            barrier_init(done + 8 * b, 1);
            barrier_init(free_ + 8 * b, (PAIR ? 2 : 1) * TC_WRITERS / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        lost_s = 0.0f;
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(&tensor_at)),
                         "n"(COLUMNS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(&tensor_at)),
                         "n"(COLUMNS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (PAIR) cluster_barrier();  // the other block's barriers are there
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tensor = tensor_at;
    pdl_wait();
    const int share = PAIR ? 2 : p.split, rank = static_cast<int>(blockIdx.x) % share;  // of the cluster
    // An operand of two parts goes through k twice, its lower part first: what sums so small lose counts for nothing.
    const int once = static_cast<int>((p.k + TC_K - 1) / TC_K), low = p.low_of ? once : 0, steps = low + once;
    const int64_t tiles = p.tiles_m * p.tiles_n, items = tiles * p.segments;
    const int sharers = p.segments > 1 ? p.segments : p.split, each = (steps + sharers - 1) / sharers;
    // Item t: a tile and this block's stretch of k.
    auto item = [&](int64_t t, int& first, int& last) {
        const int segment = p.segments > 1 ? static_cast<int>(t / tiles) : PAIR ? 0 : rank;
        first = min(steps, segment * each);
        last = min(steps, first + each);
        return tile_place(p.segments > 1 ? t - segment * tiles : t, p.tiles_m, p.tiles_n, ROWS, BN);
    };
    // The stretch of steps from `from` on (lower parts count for nothing).
    auto stretch_end = [&](int from, int last) { return min(last, max(from, low) + p.stretch); };
    const int64_t tile0 = blockIdx.x / share, tile_step = gridDim.x / share;
    bool waited = true;  // false: a wait gave up

    if (warp == 0 && lane == 0) {  // ---- operands to the ring
        int s = 0, turn = 0;
        for (int64_t t = tile0; t < items && waited; t += tile_step) {
            int first, last;
            const Place at = item(t, first, last);
            const int m = static_cast<int>(at.m) + (PAIR ? rank * TC_M : 0), n = static_cast<int>(at.n) + (PAIR ? rank * BB : 0);
            for (int k = first; k < last; ++k) {
                waited = barrier_wait(empty + 8 * s, turn ^ 1, p.patience);
                if (!waited) break;
                const uint32_t bar = full + 8 * s, a = ring + s * STAGE, b = a + A_BYTES;
                if (!PAIR) barrier_expect(bar, STAGE);
                else if (rank == 0) barrier_expect(bar, 2 * STAGE);
                const int lower = k < low ? p.low_of : 0, x = (k < low ? k : k - low) * TC_K;
                const CUtensorMap* const from_a = lower == 1 ? &map_low : &map_a;
                const CUtensorMap* const from_b = lower == 2 ? &map_low : &map_b;
                if (p.a_across) {
#pragma unroll
                    for (int h = 0; h < TC_M / 64; ++h) tma_load<PAIR>(a + h * HALF_BYTES, from_a, m + 64 * h, x, bar);
                } else {
                    tma_load<PAIR>(a, from_a, x, m, bar);
                }
                if (BB >= 64 && p.b_across) {
#pragma unroll
                    for (int h = 0; h < BB / 64; ++h) tma_load<PAIR>(b + h * HALF_BYTES, from_b, n + 64 * h, x, bar);
                } else {
                    tma_load<PAIR>(b, from_b, x, n, bar);
                }
                if (++s == STAGES) {
                    s = 0;
                    turn ^= 1;
                }
            }
        }
    } else if (warp == 1 && lane == 0 && (!PAIR || rank == 0)) {  // ---- matrix instructions
        const uint32_t form = instruction_form<T>(p.a_across, p.b_across, ROWS, BN);
        const uint64_t form_a = operand_form(p.a_across), form_b = operand_form(p.b_across);
        const uint32_t step_a = p.a_across ? 128 : 2, step_b = p.b_across ? 128 : 2;  // 16 of k, in 16 bytes
        int s = 0, turn = 0, set = 0, set_turn = 0;
        for (int64_t t = tile0; t < items && waited; t += tile_step) {
            int first, last;
            item(t, first, last);
            do {
                const int end = stretch_end(first, last);
                waited = barrier_wait(free_ + 8 * set, set_turn ^ 1, p.patience);
                if (!waited) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int k = first; k < end; ++k) {
                    waited = barrier_wait(full + 8 * s, turn, p.patience);
                    if (!waited) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    // Descriptors have 14 bits of an address; a cluster's blocks have their rank above bit 23 of it.
                    const uint32_t a = ((ring + s * STAGE) & 0x3ffff) >> 4, b = a + A_BYTES / 16;
#pragma unroll
                    for (int i = 0; i < TC_K / 16; ++i)
                        mma<PAIR>(tensor + set * BN, form_a | (a + i * step_a), form_b | (b + i * step_b), form,
                                  k > first || i > 0);
                    mma_commit<PAIR>(empty + 8 * s);
                    if (++s == STAGES) {
                        s = 0;
                        turn ^= 1;
                    }
                }
                if (!waited) break;
                mma_commit<PAIR>(done + 8 * set);
                set_turn ^= set;
                set ^= 1;
                first = end;
            } while (first < last);
        }
    } else if (warp >= 2) {  // ---- results
        const int writer = threadIdx.x - 64, quarter = warp % 4, row = quarter * 32 + lane, side = (warp - 2) / 4;
        char* const ring_at = dynamic + (ring - shared_address(dynamic));
        const Patch<T> patch(ring_at + STAGES * STAGE + (warp - 2) * TC_PATCH, lane);
        float* const mine = p.scratch + (static_cast<int64_t>(blockIdx.x) * (BN / 2) - side * (BN / 2)) * TC_WRITERS + writer;
        int set = 0, turn = 0, tile_set = 0;
        for (int64_t t = tile0; t < items; t += tile_step, tile_set ^= 1) {
            int first, last;
            Place at = item(t, first, last);
            if (PAIR) at.m += rank * TC_M;
            const int64_t bias0 = SWAP ? at.m : at.n, biases = SWAP ? p.m : p.n;
            for (int e = writer; e < (SWAP ? TC_M : BN); e += TC_WRITERS)
                bias_s[tile_set][e] = p.bias && bias0 + e < biases ? load_param<T>(p.bias, p.bias_f32, bias0 + e) : 0.0f;
            asm volatile("bar.sync 1, %0;" ::"n"(TC_WRITERS) : "memory");
            const int64_t row0 = at.m + quarter * 32;  // this warp's first
            const int c0 = side * (BN / 2);            // and its columns: BN / 2 from here on
            Pack<T, 8> ahead[4];                       // of the residual
            const bool more = !SWAP && p.vector && p.residual;
            auto fetch = [&](int c) {
                if (at.n + c + 32 <= p.n)
                    Patch<T>::fetch(ahead, static_cast<const T*>(p.residual) + at.n + c, p.residual_m, row0, p.m, lane);
            };
            const int64_t m = at.m + row;
            // Stretch by stretch: sums that are not the tile's last wait in the scratch memory, each thread's own.
            for (int from = first;;) {
                const int end = stretch_end(from, last);
                const bool begun = from > first, ends = end == last;
                if (more && ends && (PAIR || p.split == 1)) fetch(c0);
                if (waited) waited = barrier_wait(done + 8 * set, turn, p.patience, 5);
                // Given up: no number comes out of what should have been summed.
                const float lost = waited ? 0.0f : NAN;
                __syncwarp();
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t acc = tensor + set * BN + (static_cast<uint32_t>(quarter * 32) << 16);
                if (!PAIR && p.split > 1) {
                    // The block's part to its own shared memory: the ring is empty by now (or the part is none, and a copy may
                    // still land on it).
                    if (!waited) lost_s = NAN;
                    float* part = reinterpret_cast<float*>(ring_at) + row * (BN + 4);
#pragma unroll
                    for (int c = c0; c < c0 + BN / 2; c += 8) {
                        float v[8];
                        tensor_load(v, acc + c);
                        if (begun) take_sums(v, mine + c * TC_WRITERS);
                        if (!ends) {
                            leave_sums(v, mine + c * TC_WRITERS);
                            continue;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) part[c + i] = first < last ? v[i] : 0.0f;
                    }
                } else {
#pragma unroll 1
                    for (int c = c0; c < c0 + BN / 2; c += CHUNK) {
                        float v[CHUNK];
                        __syncwarp();
                        tensor_load(v, acc + c);
                        if (lost != 0.0f) {
#pragma unroll
                            for (int i = 0; i < CHUNK; ++i) v[i] = lost;
                        }
                        if (begun) take_sums(v, mine + c * TC_WRITERS);
                        if (!ends) {
                            leave_sums(v, mine + c * TC_WRITERS);
                            continue;
                        }
                        if (!SWAP && p.segments > 1) {
                            // Of a stretch without steps nothing was summed.
                            float* part = p.parts + (t / tiles * p.m + m) * p.n + at.n + c;
                            if (m < p.m) {
#pragma unroll
                                for (int i = 0; i < CHUNK; i += 4) {
                                    if (first == last) v[i] = v[i + 1] = v[i + 2] = v[i + 3] = lost;
                                    if (p.n % 4 == 0 && at.n + c + i < p.n) {
                                        *reinterpret_cast<float4*>(part + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                                    } else {
#pragma unroll
                                        for (int j = i; j < i + 4; ++j)
                                            if (at.n + c + j < p.n) part[j] = v[j];
                                    }
                                }
                            }
                        } else if constexpr (SWAP) {
                            if (m < p.m) finish_some<T>(p, m, at.n + c, v, &bias_s[tile_set][row], 0);
                        } else {
                            const bool whole = p.vector && at.n + c + CHUNK <= p.n;
                            const int64_t columns = p.n - (at.n + c);
                            Pack<T, 8> add[4];
                            if (whole && more) {
                                patch.spread(ahead);
                                if (c + CHUNK < c0 + BN / 2) fetch(c + CHUNK);
                                patch.take(add);
                            } else if (p.residual) {
                                patch.spread_columns(static_cast<const T*>(p.residual) + at.n + c, p.residual_m, row0, p.m, columns,
                                                 lane);
                                patch.take(add);
                            }
#pragma unroll
                            for (int i = 0; i < CHUNK; i += 4) {
                                const float4 b = *reinterpret_cast<const float4*>(&bias_s[tile_set][c + i]);
                                v[i] += b.x;
                                v[i + 1] += b.y;
                                v[i + 2] += b.z;
                                v[i + 3] += b.w;
                            }
                            auto put = [&](void* to) {
                                T* const t = static_cast<T*>(to) + at.n + c;
                                if (whole) patch.put(v, t, p.out_m, row0, p.m, lane);
                                else patch.put_columns(v, t, p.out_m, row0, p.m, columns, lane);
                            };
                            if (p.pre) put(p.pre);
                            act_values<T, CHUNK>(v, p.act);
                            if (p.residual) {
#pragma unroll
                                for (int i = 0; i < CHUNK; ++i) v[i] += to_f32(add[i / 8].v[i % 8]);
                            }
                            put(p.out);
                        }
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                // A warp that does not wait any more does not speak for those that still read.
                if (lane == 0 && waited) {
                    if constexpr (PAIR) barrier_arrive_at(peer_address(free_ + 8 * set, 0));
                    else barrier_arrive(free_ + 8 * set);
                }
                turn ^= set;
                set ^= 1;
                if (ends) break;
                from = end;
            }
            if (!PAIR && p.split > 1) break;  // one tile a cluster
        }
    }
    __syncwarp();
    if (!PAIR && p.split > 1) {
        cluster_barrier();
        if (!waited) settle(p.status);
        if (warp >= 2) {
            // This block's rows of the tile, the parts added in the blocks' order.
            const Place at = tile_place(tile0, p.tiles_m, p.tiles_n, ROWS, BN);
            const int rows = TC_M / p.split, writer = threadIdx.x - 64;
            for (int e = writer; e < rows * BN / 4; e += TC_WRITERS) {
                const int r = rank * rows + (SWAP ? e % rows : e / (BN / 4)), c = 4 * (SWAP ? e / rows : e % (BN / 4));
                if (at.m + r >= p.m || at.n + c >= p.n) continue;
                const uint32_t from = ring + 4 * (r * (BN + 4) + c);
                float v[8][4], lost[8];
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b < p.split)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v[b][0]), "=f"(v[b][1]), "=f"(v[b][2]), "=f"(v[b][3])
                                     : "r"(peer_address(from, b)));
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b < p.split)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(lost[b]) : "r"(peer_address(shared_address(&lost_s), b)));
                float sum[4] = {};
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b < p.split) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] += v[b][i] + lost[b];
                    }
                finish_some<T>(p, at.m + r, at.n + c, sum, &bias_s[0][SWAP ? r : c], SWAP ? 0 : 1);
            }
        }
        __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    // No block leaves while another reads its shared memory or arrives at its barriers, or something of its own is in
    // flight.
    if ((PAIR || p.split == 1) && __syncthreads_or(!waited)) settle(p.status);
    __syncwarp();
    if (PAIR || p.split > 1) cluster_barrier();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) {
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(COLUMNS));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(COLUMNS));
    }
}

// --------------------------------------------------------------------- host

// Rows of an operand, 64 columns a box (128 bytes: one swizzle span).
bool encode(CUtensorMap* map, int type, const void* p, int64_t width, int64_t rows, int64_t row, int box_rows)
{
    const cuuint64_t size[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(row) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    const EncodeTiled fn = encoder();
    return fn && fn(map, type == NMS_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void*>(p), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int BN, bool SWAP, bool PAIR>
bool launch_tile(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& low, const TcArgs& p, cudaStream_t st)
{
    auto kernel = product_tc_kernel<T, BN, SWAP, PAIR>;
    constexpr int SMEM = 1024 + TC_RING<PAIR ? BN / 2 : BN> + (SWAP ? 0 : TC_WRITERS / 32 * TC_PATCH);
    // Once for each device: the attribute belongs to the kernel on the current one.
    static std::atomic<uint64_t> ready{0};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return false;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return false;
        if (device < 64) ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t items = p.tiles_m * p.tiles_n * p.segments;
    const int share = PAIR ? 2 : p.split;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(items * share < SMS ? items * share : SMS / share * share));
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = share;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, b, low, p) == cudaSuccess;
}

template <typename T>
bool launch_type(int bn, bool swap, bool pair, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& low,
                 const TcArgs& p, cudaStream_t st)
{
    if (swap) {
        if (bn == 16) return launch_tile<T, 16, true, false>(a, b, low, p, st);
        if (bn == 32) return launch_tile<T, 32, true, false>(a, b, low, p, st);
        return launch_tile<T, 64, true, false>(a, b, low, p, st);
    }
    if (pair) return bn == 128 ? launch_tile<T, 128, false, true>(a, b, low, p, st) : launch_tile<T, 256, false, true>(a, b, low, p, st);
    if (bn == 64) return launch_tile<T, 64, false, false>(a, b, low, p, st);
    if (bn == 128) return launch_tile<T, 128, false, false>(a, b, low, p, st);
    return launch_tile<T, 256, false, false>(a, b, low, p, st);
}

}  // namespace

// Products of k that the tensor cores add up by themselves of 16-bit operands.  They
// cut each product below 2^-25 of the sum so far (counted in the sum's power of two)
// and the sum below 2^-23 after every 16 of them, so k are off by up to k (2^-25 +
// 2^-27): with these 0.31 of the half step that a result is rounded by anyway.
// Longer sums are added up in binary32, to nearest.
static int64_t product_stretch(int type) { return type == NMS_TYPE_F16 ? 1 << 12 : 1 << 15; }

// A block an SM at most, each with the largest tile's sums.
size_t product_scratch_bytes(int type, int64_t k)
{
    return type != NMS_TYPE_F32 && k > product_stretch(type) ? sizeof(float) * SMS * TC_M * 256 : 0;
}

bool launch_product_tc(const ProductArgs& q, cudaStream_t st)
{
    TcArgs p{};
    const bool swap = q.m <= 64 && !q.a_across;
    bool pair = false;
    p.k = q.k;
    p.bias = q.bias;
    p.bias_f32 = q.bias_f32;
    p.act = q.act;
    p.residual = q.residual;
    p.out = q.out;
    p.pre = q.pre;
    p.status = q.status;
    p.patience = patience();
    p.stretch = static_cast<int>(product_stretch(q.type) / TC_K);
    p.scratch = q.scratch;
    p.low_of = !q.a_low ? 0 : swap ? 2 : 1;
    p.segments = q.segments;
    p.parts = q.parts;
    const void *a = q.a, *b = q.b;
    int64_t a_row = q.a_row, b_row = q.b_row;
    int bn;
    if (swap) {
        a = q.b;
        b = q.a;
        a_row = q.b_row;
        b_row = q.a_row;
        p.a_across = q.b_across;
        p.b_across = q.a_across;
        p.m = q.n;
        p.n = q.m;
        p.residual_m = p.out_m = 1;
        p.residual_n = q.residual_row;
        p.out_n = q.n;
        bn = q.m <= 16 ? 16 : q.m <= 32 ? 32 : 64;
    } else {
        p.a_across = q.a_across;
        p.b_across = q.b_across;
        p.m = q.m;
        p.n = q.n;
        p.residual_m = q.residual_row;
        p.out_m = q.n;
        p.residual_n = p.out_n = 1;
        auto aligned = [](const void* v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; };
        p.vector = q.n % 8 == 0 && aligned(q.out) && aligned(q.pre) && aligned(q.residual) && q.residual_row % 8 == 0;
        // The tile whose waves cost least: a tile takes its width (a third more where one block has it alone, see above)
        // and a fixed part.
        bn = 0;
        int64_t best = 0;
        for (int two = 1; two >= 0; --two)
            for (int w : {256, 128, 64}) {
                if (two && w == 64) continue;
                const int64_t rows = two ? 2 * TC_M : TC_M, slots = two ? SMS / 2 : SMS;
                const int64_t tiles = ((p.m + rows - 1) / rows) * ((p.n + w - 1) / w) * p.segments;
                const int64_t cost = ((tiles + slots - 1) / slots) * ((two ? 3 * w : 4 * w) + 192);
                if (bn == 0 || cost < best) {
                    bn = w;
                    pair = two;
                    best = cost;
                }
            }
    }
    const int64_t rows = pair ? 2 * TC_M : TC_M;
    p.tiles_m = (p.m + rows - 1) / rows;
    p.tiles_n = (p.n + bn - 1) / bn;
    const int64_t tiles = p.tiles_m * p.tiles_n, steps = (p.k + TC_K - 1) / TC_K * (q.a_low ? 2 : 1);
    p.split = 1;
    // Joining the parts costs a few microseconds: 300 x 256 x 1024, four stages a tile, took 7.7 us by two blocks a tile
    // and 5.5 by one; 16 x 1024 x 4096, sixteen stages, 6.2 by four and 6.6 by two.
    while (!pair && p.segments == 1 && p.split < 8 && tiles * p.split * 2 <= SMS && steps >= p.split * 8) p.split *= 2;
    auto encode_a = [&](CUtensorMap* map, const void* at) {
        return p.a_across ? encode(map, q.type, at, p.m, p.k, a_row, 64) : encode(map, q.type, at, p.k, p.m, a_row, TC_M);
    };
    auto encode_b = [&](CUtensorMap* map, const void* at) {
        return p.b_across ? encode(map, q.type, at, p.n, p.k, b_row, 64)
                          : encode(map, q.type, at, p.k, p.n, b_row, pair ? bn / 2 : bn);
    };
    CUtensorMap map_a, map_b, map_low;
    if (!encode_a(&map_a, a) || !encode_b(&map_b, b)) return false;
    if (!p.low_of) map_low = map_a;  // not used
    else if (!(swap ? encode_b(&map_low, q.a_low) : encode_a(&map_low, q.a_low))) return false;
    return q.type == NMS_TYPE_F16 ? launch_type<__half>(bn, swap, pair, map_a, map_b, map_low, p, st)
                                  : launch_type<__nv_bfloat16>(bn, swap, pair, map_a, map_b, map_low, p, st);
}

}  // namespace gbnms
