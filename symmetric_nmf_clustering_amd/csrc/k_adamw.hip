// AdamW over many tensors in one launch, states in 32 or 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
//
// In 8 bits a state is float8 e4m3 (finite, 4 bits of exponent, 3 of mantissa) times
// one float32 scale for each 256 elements, the largest of them over 448. v is held as
// its root, which spans half as many powers of two. A root above zero never becomes
// zero (it is held as the least code): sqrt(v) = 0 beside m != 0 would send the
// parameter off by m / eps. The update itself uses the new m and v before they are
// rounded. Every block's largest element is held to float32, so that all of a block
// decays with it; a code that is off by half a step puts a root at most 2^-4 off.
//
// The betas and 1 - lr wd are not rounded to float32, whose error every step would repeat: the
// memory of beta2 = 0.99999 would be 0.14% off, a weight decay of 1e-6 a step 1.3%. (A beta goes
// in as two numbers, the decay as p - lr wd p.)
//
// Arithmetic is float32: six codes of m in 10^7 lie on the other side of a rounding's border than
// in float64 (of v's root less than one; m rounded once to float32 alone makes four). Through
// float64 the 8-bit step takes 284 us instead of 228, and 278 where only waves with a value near a
// border go there.
//
// Bound by memory: a workgroup takes 2048 elements of one tensor, a thread 8 that lie
// next to one another; 32 lanes share an 8-bit block. Which tensor is found from the
// tensors' first workgroups, in the kernel's arguments. 108 million parameters: bf16 with
// float32 masters and states (28 bytes each) 622 us, 4.8 TB/s; bf16 with 8-bit states (10
// bytes) 226 us, 4.8 TB/s.
#include <cfloat>

#include "layers.h"

namespace symnmf {

namespace {

constexpr int kTensors = 48;  // of one launch: arguments stay below 4 KiB
constexpr int kEach = 8, kChunk = 256 * kEach;

struct AdamLaunch {
    AdamTensor t[kTensors];
    uint32_t first[kTensors];  // workgroup
    int32_t count;
    float b1, c1, b2, c2;     // betas and 1 - betas
    float b1_rest, b2_rest;   // what float32 leaves of the betas
    float decay, rate, root;  // lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float eps, grad_scale;
    double beta1, beta2, lr, weight_decay, step;
    const int64_t* step_dev;
    const float* lr_dev;
    const float* grad_scale_dev;
};
static_assert(sizeof(AdamLaunch) <= 4000, "kernel arguments");

// The three factors of the update that depend on the step and the rate.
__host__ __device__ inline void factors(double step, double lr, double beta1, double beta2,
                                        double wd, float* decay, float* rate, float* root) {
    *decay = (float)(lr * wd);
    *rate = (float)(lr / (1.0 - pow(beta1, step)));
    *root = (float)(1.0 / sqrt(1.0 - pow(beta2, step)));
}

template <class T>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    if (n == 8) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < 8 / V; ++q) {
            const Vec<T, V> u = load_vec<T, V>(p + q * V);
#pragma unroll
            for (int j = 0; j < V; ++j) v[q * V + j] = to_f32(u.e[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f32(p[j]) : 0.f;
    }
}
template <class T>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
    if (n == 8) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < 8 / V; ++q) {
            Vec<T, V> u;
#pragma unroll
            for (int j = 0; j < V; ++j) u.e[j] = from_f32<T>(v[q * V + j]);
            store_vec<T, V>(p + q * V, u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = from_f32<T>(v[j]);
    }
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int n, float (&v)[8]) {
    uint32_t w[2] = {0, 0};
    if (n == 8) {
        const Vec<uint8_t, 8> u = load_vec<uint8_t, 8>(p);
        __builtin_memcpy(w, &u, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
    typedef float f32p __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const f32p a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
        const f32p b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
        v[4 * q + 0] = a[0];
        v[4 * q + 1] = a[1];
        v[4 * q + 2] = b[0];
        v[4 * q + 3] = b[1];
    }
}

// A block's elements (32 lanes, 8 each) as codes and their scale. What is not finite
// becomes NaN and leaves the others' scale alone.
template <bool ROOT>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int n, const float (&v)[8]) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = fabsf(v[j]);
        top = x < INFINITY ? fmaxf(top, x) : top;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 32));
    top = fmaxf(top, 0x1p-100f);
    const float up = 448.f / top;
    if ((threadIdx.x & 31) == 0 && n > 0) *scale = top / 448.f;
    uint32_t w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float y = v[4 * q + j];
            x[j] = fabsf(y) < INFINITY ? y * up : NAN;
            // below the least code, but not zero
            if (ROOT && y > 0.f) x[j] = fmaxf(x[j], 0x1p-9f);
            if (ROOT && !(y < INFINITY)) x[j] = NAN;
        }
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
        w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], c, true);
    }
    if (n == 8) {
        Vec<uint8_t, 8> u;
        __builtin_memcpy(&u, w, 8);
        store_vec<uint8_t, 8>(p, u);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
}

template <class P, class G, bool LOW>
__global__ __launch_bounds__(256) void adamw_kernel(AdamLaunch a, uint32_t first) {
    const uint32_t id = first + blockIdx.x;
    int lo = 0, hi = a.count - 1;  // the last tensor whose first workgroup is at most id
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= id)
            lo = mid;
        else
            hi = mid - 1;
    }
    const AdamTensor& t = a.t[lo];
    float decay = a.decay, rate = a.rate, root = a.root;
    if (a.step_dev || a.lr_dev) {
        __shared__ float f[3];
        if (threadIdx.x == 0)
            factors(a.step_dev ? (double)*a.step_dev : a.step, a.lr_dev ? (double)*a.lr_dev : a.lr,
                    a.beta1, a.beta2, a.weight_decay, &f[0], &f[1], &f[2]);
        __syncthreads();
        decay = f[0];
        rate = f[1];
        root = f[2];
    }
    const float gs = a.grad_scale_dev ? a.grad_scale * *a.grad_scale_dev : a.grad_scale;
    const int64_t at = (int64_t)(id - a.first[lo]) * kChunk + threadIdx.x * kEach;
    const int64_t left = t.n - at;
    const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    const int64_t block = at / kAdamBlock;
    if (!LOW && n == 0) return;  // (in 8 bits all lanes take part in the blocks' maxima)

    float g[8], m[8], v[8], p[8];
    P* pp = static_cast<P*>(t.param) + at;
    load8<G>(static_cast<const G*>(t.grad) + at, n, g);
    // what m is kept with, as two numbers; of codes, by their scale
    float k1 = a.b1, k1_rest = a.b1_rest;
    if (LOW) {
        const float ms = n ? t.m_scale[block] : 0.f, vs = n ? t.v_scale[block] : 0.f;
        load_codes(static_cast<const uint8_t*>(t.m) + at, n, m);
        load_codes(static_cast<const uint8_t*>(t.v) + at, n, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] *= vs;  // (not vs * vs, which is 0 where the roots' squares are not yet)
            v[j] *= v[j];
        }
        k1 = a.b1 * ms;
        k1_rest = fmaf(a.b1, ms, -k1) + a.b1_rest * ms;
    } else {
        load8<float>(static_cast<const float*>(t.m) + at, n, m);
        load8<float>(static_cast<const float*>(t.v) + at, n, v);
    }
    if (t.master)
        load8<float>(t.master + at, n, p);
    else
        load8<P>(pp, n, p);
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = g[j] * gs;
        m[j] = fmaf(k1, m[j], fmaf(k1_rest, m[j], a.c1 * x));
        // (a second moment past float32's range stays infinite; no code is)
        const float rest = LOW ? v[j] : fminf(v[j], FLT_MAX);
        v[j] = fmaf(a.b2, v[j], fmaf(a.b2_rest, rest, a.c2 * (x * x)));
        r[j] = sqrtf(v[j]);
        // (an infinite parameter, a mask's, stays)
        const float kept = fmaf(-decay, __builtin_amdgcn_fmed3f(p[j], -FLT_MAX, FLT_MAX), p[j]);
        p[j] = fmaf(-rate, m[j] / (r[j] * root + a.eps), kept);
    }
    if (n) store8<P>(pp, n, p);
    if (t.master && n) store8<float>(t.master + at, n, p);
    if (LOW) {
        store_codes<false>(static_cast<uint8_t*>(t.m) + at, t.m_scale + block, n, m);
        store_codes<true>(static_cast<uint8_t*>(t.v) + at, t.v_scale + block, n, r);
    } else {
        store8<float>(static_cast<float*>(t.m) + at, n, m);
        store8<float>(static_cast<float*>(t.v) + at, n, v);
    }
}

template <class P, class G>
hipError_t launch_as(const AdamLaunch& l, bool low, uint32_t blocks, hipStream_t st) {
    return in_launches(blocks, [&](int64_t first, unsigned n) {
        if (low)
            adamw_kernel<P, G, true><<<n, 256, 0, st>>>(l, (uint32_t)first);
        else
            adamw_kernel<P, G, false><<<n, 256, 0, st>>>(l, (uint32_t)first);
    });
}

template <class P>
hipError_t launch_param(const AdamLaunch& l, int grad_type, bool low, uint32_t blocks,
                        hipStream_t st) {
    switch (grad_type) {
        case kBF16: return launch_as<P, bf16_t>(l, low, blocks, st);
        case kF16: return launch_as<P, f16_t>(l, low, blocks, st);
        default: return launch_as<P, float>(l, low, blocks, st);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, hipStream_t st) {
    AdamLaunch l{};
    l.beta1 = a.beta1, l.beta2 = a.beta2, l.lr = a.lr, l.weight_decay = a.weight_decay;
    l.step = a.step;
    l.b1 = (float)a.beta1, l.c1 = (float)(1.0 - a.beta1), l.b1_rest = (float)(a.beta1 - l.b1);
    l.b2 = (float)a.beta2, l.c2 = (float)(1.0 - a.beta2), l.b2_rest = (float)(a.beta2 - l.b2);
    l.eps = (float)a.eps;
    l.grad_scale = a.grad_scale;
    l.step_dev = a.step_dev, l.lr_dev = a.lr_dev, l.grad_scale_dev = a.grad_scale_dev;
    factors(a.step, a.lr, a.beta1, a.beta2, a.weight_decay, &l.decay, &l.rate, &l.root);
    for (int32_t i = 0; i < a.count;) {
        int64_t blocks = 0;
        l.count = 0;
        for (; i < a.count && l.count < kTensors; ++i) {
            const int64_t n = (a.tensors[i].n + kChunk - 1) / kChunk;
            if (n == 0) continue;
            if (blocks + n > 0xffffffffLL) break;  // (the sizes' limits keep n itself below)
            l.t[l.count] = a.tensors[i];
            l.first[l.count++] = (uint32_t)blocks;
            blocks += n;
        }
        if (l.count == 0) continue;
        hipError_t e;
        switch (a.param_type) {
            case kBF16:
                e = launch_param<bf16_t>(l, a.grad_type, a.bits == 8, (uint32_t)blocks, st);
                break;
            case kF16:
                e = launch_param<f16_t>(l, a.grad_type, a.bits == 8, (uint32_t)blocks, st);
                break;
            default:
                e = launch_param<float>(l, a.grad_type, a.bits == 8, (uint32_t)blocks, st);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace symnmf
