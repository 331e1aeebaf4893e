// Rotary positions: pairs of channels of every head turned by position times
// frequency.
//
// y1 = amp (x1 cos - x2 sin), y2 = amp (x2 cos + x1 sin), the angle reduced exactly (turn_of):
// cosine and sine are right to a few 2^-24 at any position. One angle serves all
// heads of a step: a thread takes some pairs of a step and goes through its heads
// with their cosines in registers. Bound by memory: x is read and written once.
#include "layers.h"

namespace symnmf {

namespace {

// Sine and cosine of pos times freq (radians). The turns' whole part is taken off exactly: pos as
// two numbers that float64 holds (52 and 11 bits), freq / 2 pi as two, the large product by an fma
// that takes its own whole turns off before it rounds. What is left is right to 2^-42 turns at any
// position (freq up to 1) and goes to float32 with its remainder, whose first order is added to the
// functions' values.
__device__ __forceinline__ void turn_of(int64_t pos, double freq, float* sine, float* cosine) {
    constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;  // 1 / 2 pi
    const double f = freq * kTurn, f_rest = fma(freq, kTurn, -f) + freq * kTurnRest;
    const double far = (double)(pos & ~int64_t(2047)), near = (double)(pos & 2047);
    double turns = fma(far, f, -rint(far * f)) + fma(near, f, far * f_rest);
    turns -= rint(turns);
    const float u = (float)turns, du = (float)((turns - u) * 6.283185307179586);
    float s, c;
    sincospif(2.f * u, &s, &c);
    *sine = fmaf(c, du, s);
    *cosine = fmaf(-s, du, c);
}

// P pairs of each of U heads, all asked for before the first is turned: (CLOSE) 2 P elements
// at x, or P at x and P at x + gap. copy: they stay as they are (0 times an infinity would
// not).
template <class T, int P, bool CLOSE, int U>
__device__ __forceinline__ void turn(const T* x, int64_t xs, T* y, int64_t ys, int gap, bool copy,
                                     const float (&c)[P], const float (&s)[P]) {
    constexpr int V = CLOSE ? 2 * P : P;
    Vec<T, V> v[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = load_vec<T, V>(x + u * xs);
        if (!CLOSE) w[u] = load_vec<T, V>(x + u * xs + gap);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            T& p = CLOSE ? v[u].e[2 * i] : v[u].e[i];
            T& q = CLOSE ? v[u].e[(2 * i + 1) % V] : w[u].e[i];
            const float a = to_f32(p), b = to_f32(q);
            const T pt = from_f32<T>(a * c[i] - b * s[i]), qt = from_f32<T>(b * c[i] + a * s[i]);
            p = copy ? p : pt;
            q = copy ? q : qt;
        }
        store_vec<T, V>(y + u * ys, v[u]);
        if (!CLOSE) store_vec<T, V>(y + u * ys + gap, w[u]);
    }
}

// A thread: one step, `per` of its heads, and one group of P pairs or, past those, 2 P
// channels that stay (one or two for P = 1). Threads of a step lie next to one another, and
// all take the same path. Four heads in flight: 108.5 us for 32768 steps of 32 heads of 128
// bf16 (5.0 TB/s, the copy's rate) against 118 with two. The angles show where a step has one
// head (100000 steps of 128: 20.6 us at a floor of 10).
template <class T, int P, bool CLOSE>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int64_t first, int groups,
                                                     int splits, int per) {
    const int64_t id = (first + blockIdx.x) * 256 + threadIdx.x;
    const int grp = (int)(id % groups);
    const int64_t rest = id / groups;
    const int split = (int)(rest % splits);
    const int64_t n = rest / splits;
    if (n >= a.batch * a.steps) return;
    const int64_t b = n / a.steps, t = n % a.steps;
    const int half = a.dims / 2, turned = half / P, p0 = grp * P;
    const bool copy = grp >= turned;
    int at = a.interleaved ? 2 * p0 : p0, gap = a.interleaved ? P : half;
    float c[P], s[P];
    if (copy) {
        at = 2 * p0;  // dims = 2 P turned
        gap = at + P < a.width ? P : 0;
#pragma unroll
        for (int i = 0; i < P; ++i) c[i] = s[i] = 0.f;
    } else {
        const int64_t pa = b * a.pos_b + t * a.pos_t;
        const int64_t pos = a.pos_type == kI32 ? static_cast<const int32_t*>(a.pos)[pa]
                                               : static_cast<const int64_t*>(a.pos)[pa];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            turn_of(pos, a.freqs[p0 + i], &s[i], &c[i]);
            c[i] *= a.amplitude;
            s[i] *= a.inverse ? -a.amplitude : a.amplitude;
        }
    }
    const int h0 = split * per;
    int left = a.heads - h0;
    if (left > per) left = per;
    const T* x = static_cast<const T*>(a.x) + b * a.x_b + t * a.x_t + h0 * a.x_h + at;
    T* y = static_cast<T*>(a.out) + b * a.o_b + t * a.o_t + h0 * a.o_h + at;
    constexpr int U = 4;
    for (; left >= U; left -= U, x += U * a.x_h, y += U * a.o_h)
        turn<T, P, CLOSE, U>(x, a.x_h, y, a.o_h, gap, copy, c, s);
    for (; left > 0; --left, x += a.x_h, y += a.o_h)
        turn<T, P, CLOSE, 1>(x, a.x_h, y, a.o_h, gap, copy, c, s);
}

template <class T, int P>
hipError_t rotary_as(const RotaryArgs& a, hipStream_t st) {
    const int groups = a.dims / 2 / P + (a.width - a.dims + 2 * P - 1) / (2 * P);
    // heads are split over threads until a few hundred thousand of them are there
    const int64_t n = a.batch * a.steps * groups;
    int64_t splits = (1 << 18) / (n ? n : 1);
    if (splits > a.heads) splits = a.heads;
    if (splits < 1) splits = 1;
    const int per = (int)((a.heads + splits - 1) / splits);
    splits = (a.heads + per - 1) / per;
    const int64_t blocks = (n * splits + 255) / 256;
    return in_launches(blocks, [&](int64_t first, unsigned k) {
        if (P > 1 && a.interleaved)
            rotary_kernel<T, P, (P > 1)><<<k, 256, 0, st>>>(a, first, groups, (int)splits, per);
        else
            rotary_kernel<T, P, false><<<k, 256, 0, st>>>(a, first, groups, (int)splits, per);
    });
}

// 16 bytes of neighbouring pairs, or twice 8 of pairs apart, where dims and the rest of the
// width allow it; otherwise single elements (65536 steps of 32 heads of 24 bf16, 12 turned: 97 us,
// 16 turned 55 interleaved and 76 in halves).
template <class T>
hipError_t rotary_type(const RotaryArgs& a, hipStream_t st) {
    constexpr int P = 8 / sizeof(T);
    return a.dims / 2 % P == 0 && (a.width - a.dims) % (2 * P) == 0 ? rotary_as<T, P>(a, st)
                                                                    : rotary_as<T, 1>(a, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st) {
    switch (a.type) {
        case kBF16: return rotary_type<bf16_t>(a, st);
        case kF16: return rotary_type<f16_t>(a, st);
        default: return rotary_type<float>(a, st);
    }
}

}  // namespace symnmf
