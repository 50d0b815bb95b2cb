// Rotary positions on several axes: the pair i of a vector's elements turns by
// position[axis(i)] * frequency(i).
//
// The angle is kept as a fraction of a turn in units of 2^-64: position times
// the table's turns per position, a 64-bit product whose overflow is whole
// turns.  So a position far into a history loses nothing (a binary32 angle of
// 10^6 radians is off by 0.03), at the price of a few integer instructions; the
// fraction's top 32 bits go to sincospif.
//
// A thread has VP pairs of one token and goes through its heads, so an angle's
// sine and cosine are worked out once for all of them.
#include "block.h"
#include "head.cuh"
#include "internal.h"

namespace gbnms {

namespace {

constexpr int RO_THREADS = 256;
#ifndef RO_ENOUGH
#define RO_ENOUGH 2048
#endif

struct RotaryPlan {
    int units;       // threads' shares of a token: turned ones, then copied ones
    int turned;      // of these the turned ones
    int head_parts;  // threads that share a token's heads
    int head_step;   // heads of each
    int64_t items;   // threads in all
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
    float sr, cr;
    sincospif(static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(half) - (quarter << 30))) * 0x1p-31f, &sr,
              &cr);
    s = quarter & 1 ? cr : sr;
    c = quarter & 1 ? sr : cr;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
    if (!known) s = c = NAN;
    if (a.inverse) s = -s;
}

// n / d of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d)
{
    if (((n | d) >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}

// VP: pairs of a thread; with VP > 1 they are two accesses of VP elements a head.
template <typename T, int VP, int HB, bool HALVES>
__global__ void __launch_bounds__(RO_THREADS, 3)
rotary_kernel(const RotaryArgs a, const RotaryPlan plan)
{
    const int64_t item = static_cast<int64_t>(blockIdx.x) * RO_THREADS + threadIdx.x;
    if (item >= plan.items) return;
    const int64_t rest = quotient(item, plan.units);
    const int unit = static_cast<int>(item - rest * plan.units);
    const int64_t at = quotient(rest, plan.head_parts);  // token of all
    const int part = static_cast<int>(rest - at * plan.head_parts);
    const int64_t batch = quotient(at, a.tokens), token = at - batch * a.tokens;
    const int first = part * plan.head_step, last = min(a.heads, first + plan.head_step);
    const T* x = static_cast<const T*>(a.x) + batch * a.x_batch + token * a.x_token + first * a.x_head;
    T* y = static_cast<T*>(a.y) + batch * a.y_batch + token * a.y_token + first * a.y_head;
    using Vec = Pack<T, VP>;
    if (unit >= plan.turned) {  // elements behind the pairs
        const int64_t e = 2 * static_cast<int64_t>(a.pairs) + static_cast<int64_t>(unit - plan.turned) * VP;
        for (int h = first; h < last; ++h, x += a.x_head, y += a.y_head)
            *reinterpret_cast<Vec*>(y + e) = *reinterpret_cast<const Vec*>(x + e);
        return;
    }
    const int pair = unit * VP;
    // Elements of the two accesses: first and second of each pair, or pairs one after another.
    const int e0 = HALVES ? pair : 2 * pair, e1 = HALVES ? pair + a.pairs : 2 * pair + VP;
    const int64_t where = ((a.sets == 1 ? 0 : batch) * a.tokens + token) * a.axes;
    float s[VP], c[VP];
    Vec lo[HB], hi[HB];
#pragma unroll
    for (int b = 0; b < HB; ++b)
        if (first + b < last) {
            lo[b] = *reinterpret_cast<const Vec*>(x + b * a.x_head + e0);
            hi[b] = *reinterpret_cast<const Vec*>(x + b * a.x_head + e1);
        }
#pragma unroll
    for (int i = 0; i < VP; ++i) sine(a, static_cast<const int32_t*>(a.positions) + where, pair + i, s[i], c[i]);
    for (int h = first; h < last; h += HB) {
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            if (h + b >= last) break;
            const Vec p = lo[b], q = hi[b];
            if (h + HB + b < last) {  // the next heads' while these are worked on
                lo[b] = *reinterpret_cast<const Vec*>(x + (HB + b) * a.x_head + e0);
                hi[b] = *reinterpret_cast<const Vec*>(x + (HB + b) * a.x_head + e1);
            }
            float u[VP], v[VP];
            if constexpr (HALVES || VP == 1) {
#pragma unroll
                for (int i = 0; i < VP; ++i) {
                    const float pi = to_f32(p.v[i]), qi = to_f32(q.v[i]);
                    u[i] = fmaf(pi, c[i], -qi * s[i]);
                    v[i] = fmaf(qi, c[i], pi * s[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VP; i += 2) {
                    const int k = i / 2, m = VP / 2 + k;
                    const float p0 = to_f32(p.v[i]), p1 = to_f32(p.v[i + 1]), q0 = to_f32(q.v[i]), q1 = to_f32(q.v[i + 1]);
                    u[i] = fmaf(p0, c[k], -p1 * s[k]);
                    u[i + 1] = fmaf(p1, c[k], p0 * s[k]);
                    v[i] = fmaf(q0, c[m], -q1 * s[m]);
                    v[i + 1] = fmaf(q1, c[m], q0 * s[m]);
                }
            }
            *reinterpret_cast<Vec*>(y + b * a.y_head + e0) = pack_results<T, VP>(u);
            *reinterpret_cast<Vec*>(y + b * a.y_head + e1) = pack_results<T, VP>(v);
        }
        x += HB * a.x_head;
        y += HB * a.y_head;
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
    // A thread takes all heads of its token once there are threads enough for every SM without splitting them.
    const int64_t tokens = a.batch * a.tokens, whole = tokens * p.units, enough = static_cast<int64_t>(SMS) * RO_ENOUGH;
    p.head_step = a.heads;
    while (p.head_step > 1 && whole * ((a.heads + p.head_step - 1) / p.head_step) < enough)
        p.head_step = (p.head_step + 1) / 2;
    p.head_parts = (a.heads + p.head_step - 1) / p.head_step;
    p.items = whole * p.head_parts;
    const unsigned grid = static_cast<unsigned>((p.items + RO_THREADS - 1) / RO_THREADS);
    auto run = [&](auto kernel) { kernel<<<grid, RO_THREADS, 0, st>>>(a, p); };
    if (wide) a.halves ? run(rotary_kernel<T, MOST, 2, true>) : run(rotary_kernel<T, MOST, 2, false>);
    else a.halves ? run(rotary_kernel<T, 1, 4, true>) : run(rotary_kernel<T, 1, 4, false>);
}

}  // namespace

void launch_rotary(const RotaryArgs& a, cudaStream_t st)
{
    if (a.type == NMS_TYPE_F32) launch<float>(a, st);
    else if (a.type == NMS_TYPE_F16) launch<__half>(a, st);
    else launch<__nv_bfloat16>(a, st);
}

}  // namespace gbnms
