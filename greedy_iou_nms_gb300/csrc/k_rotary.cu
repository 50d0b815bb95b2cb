// Rotary positions on several axes: the pair i of a vector's elements turns by
// position[axis(i)] * frequency(i).
//
// The angle is kept as a fraction of a turn in units of 2^-64: position times
// the table's turns per position, a 64-bit product whose overflow is whole
// turns.  So a position far into a history loses nothing (a binary32 angle of
// 10^6 radians is off by 0.03), at the price of a few integer instructions; the
// fraction's top 32 bits go on to the sine.
//
// HBM bounds it, so an angle's sine and cosine are worked out once for all heads
// of a token: a block has a run of tokens, makes their table in shared memory
// and then goes through the tokens' vectors in the order in which they lie.  48
// warps an SM with one access pair each in flight hide more than 32 with two (79
// us for 91 at 4 x 25600 x 16 x 64 bf16) or 24 with four; with the table no larger
// than its run and streaming accesses 72, 5.8 TB/s.
#include "block.h"
#include "head.cuh"
#include "internal.h"
#include "once.cuh"

namespace gbnms {

namespace {

constexpr int RO_THREADS = 256;
constexpr int RO_TABLE = 4096;  // sines and cosines of a block at most, 32 KB
// Tokens of a block at most.  Blocks that start at different times overlap one's table with another's stream: 16 took
// 79 us for 4 x 25600 x 16 x 64 bf16, 64 took 90, 4 took 104.
constexpr int RO_TOKENS = 16;

struct RotaryPlan {
    int units;       // accesses of a vector: turned pairs of them, then copied ones
    int turned;      // of these the turned pairs
    int64_t each;    // accesses of a token: of all its heads
    int slots;       // threads of a block that share a token
    int run;         // tokens of a block
    int64_t tokens;  // of all
};

// Fraction of a turn, in units of 2^-64, of position p; `known` is false where
// there is none (a NaN, an infinity or beyond 2^31).
__device__ __forceinline__ uint64_t turns(float p, uint64_t f, bool& known)
{
    known = fabsf(p) < 0x1p31f;
    const float whole = floorf(known ? p : 0.0f);
    const float part = (known ? p : 0.0f) - whole;  // exact but for positions in (-2^-24, 0): at most 1
    const uint64_t bits = static_cast<uint64_t>(part * 0x1p32f);
    // part * f = bits * f / 2^32: the table's top half gives it to 2^-32 of a turn over the position's 2^-32.
    return static_cast<uint64_t>(static_cast<int64_t>(whole)) * f + bits * (f >> 32);
}

// Sine and cosine of pair i at one token; a pair whose axis the positions do
// not have is not turned.
__device__ __forceinline__ void sine(const RotaryArgs& a, const void* at, int i, float& s, float& c)
{
    const uint64_t f = static_cast<uint64_t>(__ldg(a.lut + i));
    const int64_t axis = __ldg(a.lut + a.pairs + i);
    if (axis < 0 || axis >= a.axes) {
        s = 0.0f;
        c = 1.0f;
        return;
    }
    bool known = true;
    uint64_t t;
    if (a.fractions) t = turns(__ldg(static_cast<const float*>(at) + axis), f, known);
    else t = static_cast<uint64_t>(static_cast<int64_t>(__ldg(static_cast<const int32_t*>(at) + axis))) * f;
    // The nearest quarter turn and what is left of it, an eighth at most, so that rounding it to binary32 is off by
    // 2^-27 of a half turn and not by 2^-25.
    const int32_t half = static_cast<int32_t>(t >> 32);
    const uint32_t quarter = (static_cast<uint32_t>(half) + 0x20000000u) >> 30;
    const float r = static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(half) - (quarter << 30))) * 0x1p-31f;
    // Sine and cosine of pi r, |r| <= 1/4: polynomials in r^2 whose largest error is least, 2^-28 of the sine (whose
    // first factor is pi in two parts) and 2^-34.
    const float r2 = r * r;
    const float sr = fmaf(r, 3.14159274f, r * fmaf(r2, fmaf(r2, fmaf(r2, -0.589012210f, 2.54976105f), -5.16770768f), -9.76113e-08f));
    const float cr = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, 0.231429548f, -1.33505846f), 4.05870790f), -4.93480217f), 1.0f);
    s = quarter & 1 ? cr : sr;
    c = quarter & 1 ? sr : cr;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
    if (!known) s = c = NAN;
    if (a.inverse) s = -s;
}

// VP: pairs of an item, two accesses of VP elements.  An item behind the turned
// ones is one access of copied elements.
template <typename T, int VP, bool HALVES>
__global__ void __launch_bounds__(RO_THREADS, 6)
rotary_kernel(const RotaryArgs a, const RotaryPlan plan)
{
    using Vec = Pack<T, VP>;
    constexpr int BATCH = sizeof(Vec) == 16 ? 1 : 4;  // tokens of a thread on their way
    extern __shared__ __align__(16) float2 table[];   // cosine, sine [run][pairs]
    __shared__ int64_t places[RO_TOKENS][3];          // of a token's vectors in x and y, of its positions
    const int64_t token0 = static_cast<int64_t>(blockIdx.x) * plan.run;
    const int run = static_cast<int>(min(static_cast<int64_t>(plan.run), plan.tokens - token0));
    for (int i = threadIdx.x; i < run; i += RO_THREADS) {
        const int64_t batch = (token0 + i) / a.tokens, token = token0 + i - batch * a.tokens;
        places[i][0] = batch * a.x_batch + token * a.x_token;
        places[i][1] = batch * a.y_batch + token * a.y_token;
        places[i][2] = (a.sets == 1 ? token : token0 + i) * a.axes;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < run * a.pairs; i += RO_THREADS) {
        const int at = static_cast<unsigned>(i) / static_cast<unsigned>(a.pairs);
        float s, c;
        sine(a, static_cast<const int32_t*>(a.positions) + places[at][2], i - at * a.pairs, s, c);
        table[i] = make_float2(c, s);
    }
    __syncthreads();
    // A thread has one item, or every so many items, of each of its tokens, so that its place in a vector is worked
    // out once: `slots` threads a token.
    const uint64_t policy = once_policy(a.once);
    const int slot = threadIdx.x % plan.slots, first = threadIdx.x / plan.slots, step = RO_THREADS / plan.slots;
    if (first >= step) return;
    for (int64_t item = slot; item < plan.each; item += plan.slots) {
        const int64_t head = item / plan.units;
        const int unit = static_cast<int>(item - head * plan.units);
        const bool turned = unit < plan.turned;
        const int e = !turned ? 2 * a.pairs + (unit - plan.turned) * VP : HALVES ? unit * VP : 2 * unit * VP;
        const int apart = HALVES ? a.pairs : VP;
        const T* x = static_cast<const T*>(a.x) + head * a.x_head + e;
        T* y = static_cast<T*>(a.y) + head * a.y_head + e;
        const float2* turn = table + unit * VP;
        for (int at = first; at < run; at += BATCH * step) {
            Vec p[BATCH], q[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
                if (at + b * step < run) {
                    const T* from = x + places[at + b * step][0];
                    p[b] = load_once(reinterpret_cast<const Vec*>(from), policy);
                    if (turned) q[b] = load_once(reinterpret_cast<const Vec*>(from + apart), policy);
                }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int token = at + b * step;
                if (token >= run) break;
                T* to = y + places[token][1];
                if (!turned) {
                    *reinterpret_cast<Vec*>(to) = p[b];
                    continue;
                }
                const float2* t2 = turn + token * a.pairs;
                float2 t[VP];
                if constexpr (VP == 1) {
                    t[0] = t2[0];
                } else {
#pragma unroll
                    for (int i = 0; i < VP; i += 2) {
                        const float4 two = *reinterpret_cast<const float4*>(t2 + i);
                        t[i] = make_float2(two.x, two.y);
                        t[i + 1] = make_float2(two.z, two.w);
                    }
                }
                float u[VP], v[VP];
                if constexpr (HALVES || VP == 1) {
#pragma unroll
                    for (int i = 0; i < VP; ++i) {
                        const float c = to_f32(p[b].v[i]), d = to_f32(q[b].v[i]);
                        u[i] = fmaf(c, t[i].x, -d * t[i].y);
                        v[i] = fmaf(d, t[i].x, c * t[i].y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VP; i += 2) {
                        const float2 f = t[i / 2], g = t[VP / 2 + i / 2];
                        const float c0 = to_f32(p[b].v[i]), c1 = to_f32(p[b].v[i + 1]);
                        const float d0 = to_f32(q[b].v[i]), d1 = to_f32(q[b].v[i + 1]);
                        u[i] = fmaf(c0, f.x, -c1 * f.y);
                        u[i + 1] = fmaf(c1, f.x, c0 * f.y);
                        v[i] = fmaf(d0, g.x, -d1 * g.y);
                        v[i + 1] = fmaf(d1, g.x, d0 * g.y);
                    }
                }
                store_once(reinterpret_cast<Vec*>(to), pack_results<T, VP>(u), policy);
                store_once(reinterpret_cast<Vec*>(to + apart), pack_results<T, VP>(v), policy);
            }
        }
    }
}

template <typename T>
void launch(const RotaryArgs& a, cudaStream_t st)
{
    constexpr int MOST = 16 / sizeof(T);
    auto even = [](const void* p, int64_t s0, int64_t s1, int64_t s2) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % MOST == 0 && s1 % MOST == 0 && s2 % MOST == 0;
    };
    const bool wide = a.pairs % MOST == 0 && a.dim % MOST == 0 && even(a.x, a.x_batch, a.x_token, a.x_head) &&
                      even(a.y, a.y_batch, a.y_token, a.y_head);
    const int vp = wide ? MOST : 1;
    RotaryPlan p;
    p.turned = a.pairs / vp;
    p.units = p.turned + (a.dim - 2 * a.pairs) / vp;
    p.each = static_cast<int64_t>(a.heads) * p.units;
    p.slots = static_cast<int>(p.each < RO_THREADS ? p.each : RO_THREADS);
    p.tokens = a.batch * a.tokens;
    // Runs as long as leave every SM a few blocks.
    const int64_t most = a.pairs ? RO_TABLE / a.pairs : RO_TOKENS, share = p.tokens / (SMS * 8);
    p.run = static_cast<int>(share < 1 ? 1 : share < most ? share : most);
    if (p.run > RO_TOKENS) p.run = RO_TOKENS;
    const unsigned grid = static_cast<unsigned>((p.tokens + p.run - 1) / p.run);
    const size_t table = sizeof(float2) * p.run * a.pairs;
    auto run = [&](auto kernel) { kernel<<<grid, RO_THREADS, table, st>>>(a, p); };
    if (wide) a.halves ? run(rotary_kernel<T, MOST, true>) : run(rotary_kernel<T, MOST, false>);
    else a.halves ? run(rotary_kernel<T, 1, true>) : run(rotary_kernel<T, 1, false>);
}

}  // namespace

void launch_rotary(const RotaryArgs& args, cudaStream_t st)
{
    RotaryArgs a = args;
    a.once = beyond_l2(2 * (a.type == NMS_TYPE_F32 ? 4 : 2) * a.batch * a.tokens * a.heads * a.dim);
    if (a.type == NMS_TYPE_F32) launch<float>(a, st);
    else if (a.type == NMS_TYPE_F16) launch<__half>(a, st);
    else launch<__nv_bfloat16>(a, st);
}

}  // namespace gbnms
