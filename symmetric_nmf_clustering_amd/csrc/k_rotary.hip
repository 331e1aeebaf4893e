// Rotary positions: pairs of channels of every head turned by position times
// frequency.
//
// y1 = amp (x1 cos - x2 sin), y2 = amp (x2 cos + x1 sin), the angle in 64 bits: as
// turns (position times frequency over 2 pi) less their whole part, whose cosine
// and sine float32 then has to a few 2^-24 at any position. One angle serves all
// heads of a step: a thread takes some pairs of a step and goes through its heads
// with their cosines in registers. Bound by memory: x is read and written once.
#include "layers.h"

namespace symnmf {

namespace {

// P pairs next to one another, of U heads: all asked for before the first is turned.
template <class T, int P, bool INTER, int U>
__device__ __forceinline__ void turn(const T* x, int64_t xs, T* y, int64_t ys, int half,
                                     const float (&c)[P], const float (&s)[P]) {
    if constexpr (INTER) {
        Vec<T, 2 * P> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_vec<T, 2 * P>(x + u * xs);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float a = to_f32(v[u].e[2 * i]), b = to_f32(v[u].e[2 * i + 1]);
                v[u].e[2 * i] = from_f32<T>(a * c[i] - b * s[i]);
                v[u].e[2 * i + 1] = from_f32<T>(b * c[i] + a * s[i]);
            }
            store_vec<T, 2 * P>(y + u * ys, v[u]);
        }
    } else {
        Vec<T, P> v[U], w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = load_vec<T, P>(x + u * xs);
            w[u] = load_vec<T, P>(x + u * xs + half);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float a = to_f32(v[u].e[i]), b = to_f32(w[u].e[i]);
                v[u].e[i] = from_f32<T>(a * c[i] - b * s[i]);
                w[u].e[i] = from_f32<T>(b * c[i] + a * s[i]);
            }
            store_vec<T, P>(y + u * ys, v[u]);
            store_vec<T, P>(y + u * ys + half, w[u]);
        }
    }
}

// A thread: one step, `per` of its heads, and one group of P pairs (or, past the pairs,
// 2 P channels that stay as they are). Threads of a step lie next to one another.
template <class T, int P, bool INTER>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int64_t first, int groups,
                                                     int splits, int per) {
    const int64_t id = (first + blockIdx.x) * 256 + threadIdx.x;
    const int grp = (int)(id % groups);
    const int64_t rest = id / groups;
    const int split = (int)(rest % splits);
    const int64_t n = rest / splits;
    if (n >= a.batch * a.steps) return;
    const int64_t b = n / a.steps, t = n % a.steps;
    const int half = a.dims / 2, turned = half / P;
    const T* x = static_cast<const T*>(a.x) + b * a.x_b + t * a.x_t;
    T* y = static_cast<T*>(a.out) + b * a.o_b + t * a.o_t;
    const int h0 = split * per;
    int h1 = h0 + per;
    if (h1 > a.heads) h1 = a.heads;
    if (grp >= turned) {
        const int c = a.dims + (grp - turned) * 2 * P;
        for (int h = h0; h < h1; ++h) {
            if (c + 2 * P <= a.width) {
                store_vec<T, 2 * P>(y + h * a.o_h + c, load_vec<T, 2 * P>(x + h * a.x_h + c));
            } else {
                for (int i = c; i < a.width; ++i) y[h * a.o_h + i] = x[h * a.x_h + i];
            }
        }
        return;
    }
    const int64_t at = b * a.pos_b + t * a.pos_t;
    const double pos = a.pos_type == kI32 ? (double)static_cast<const int32_t*>(a.pos)[at]
                                          : (double)static_cast<const int64_t*>(a.pos)[at];
    const int p0 = grp * P;
    float c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        constexpr double kTurn = 0.15915494309189533577;  // 1 / 2 pi
        const double turns = pos * a.freqs[p0 + i] * kTurn;
        const float f = (float)(turns - rint(turns));
        sincospif(2.f * f, &s[i], &c[i]);
        c[i] *= a.amplitude;
        s[i] *= a.inverse ? -a.amplitude : a.amplitude;
    }
    const int at_x = INTER ? 2 * p0 : p0;
    x += h0 * a.x_h + at_x;
    y += h0 * a.o_h + at_x;
    int left = h1 - h0;
    constexpr int U = 4;
    for (; left >= U; left -= U, x += U * a.x_h, y += U * a.o_h)
        turn<T, P, INTER, U>(x, a.x_h, y, a.o_h, half, c, s);
    for (; left > 0; --left, x += a.x_h, y += a.o_h)
        turn<T, P, INTER, 1>(x, a.x_h, y, a.o_h, half, c, s);
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
        if (a.interleaved)
            rotary_kernel<T, P, true><<<k, 256, 0, st>>>(a, first, groups, (int)splits, per);
        else
            rotary_kernel<T, P, false><<<k, 256, 0, st>>>(a, first, groups, (int)splits, per);
    });
}

template <class T>
hipError_t rotary_type(const RotaryArgs& a, hipStream_t st) {
    constexpr int P = 8 / sizeof(T);  // 16 bytes of interleaved pairs, twice 8 of halves
    return a.dims / 2 % P == 0 ? rotary_as<T, P>(a, st) : rotary_as<T, 1>(a, st);
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
