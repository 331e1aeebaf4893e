// Log probabilities of given tokens under softmax(scale * logits), with the
// entropy and the top alternatives of every row, and their gradient.
//
// Per row, with z the logits, M = max z, k = scale log2(e), t_j = k (z_j - M):
//   s = sum 2^t_j, u = sum t_j 2^t_j,
//   lse = scale M + ln s,  logp = scale z_tok - lse,  H = ln s - ln(2) u / s.
// The row is read once with running M, s and u (rescaled when M grows). Long
// rows are cut into slices whose (M, s, u) a second kernel joins.
//
// Alternatives: the logits are seen in groups of 8 columns whose maxima are
// kept in LDS. Order groups by their best element (larger value, then lower
// column): the m best elements lie in the m first groups, because an element
// outside them is beaten by the best element of each. So after the one pass
// only m groups are read again.
//
// A column whose logit is -inf is excluded: probability 0, never an
// alternative. A row with no column left has lse = -inf, logp = -inf and
// entropy 0. NaN or +inf in a row makes its results NaN.
#include <float.h>

#include "common.h"
#include "seq.h"

namespace symnmf {
namespace {

constexpr int kGroup = 8;          // columns per group
constexpr int kMaxGroups = 8192;   // groups of one slice (32 per thread)
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// Order of (value, column) as one number: larger is better. -0 equals 0; a NaN
// counts as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
    if (!(v > -INFINITY)) v = -INFINITY;
    v += 0.f;  // -0 -> 0
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
constexpr uint32_t kOrdNegInf = 0x007fffffu;  // ordered(-inf)

struct Stat {
    float m, s, u;
};
__device__ __forceinline__ Stat stat_none() { return {-FLT_MAX, 0.f, 0.f}; }
// u += t e with the t of an excluded column (-inf) held finite: its e is 0.
__device__ __forceinline__ void stat_rescale(Stat& a, float m, float k) {
    const float t = k * (a.m - m);  // <= 0
    const float f = __builtin_amdgcn_exp2f(t);
    a.u = f * fmaf(fmaxf(t, -1000.f), a.s, a.u);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ Stat stat_join(Stat a, Stat b, float k) {
    const float m = fmaxf(a.m, b.m);
    stat_rescale(a, m, k);
    stat_rescale(b, m, k);
    return {m, a.s + b.s, a.u + b.u};
}
__device__ __forceinline__ Stat stat_shfl_xor(Stat a, int o) {
    return {__shfl_xor(a.m, o, 64), __shfl_xor(a.s, o, 64), __shfl_xor(a.u, o, 64)};
}

struct RowOut {
    const void* tokens;
    int token_type;
    float* logp;
    float* entropy;
    float* lse;
    float* top_logp;
    int32_t* top_ids;
};

// lse and entropy of a row from its joined statistics.
__device__ __forceinline__ void row_stats(const Stat& a, float scale, float& lse, float& h) {
    const float ls = __logf(a.s);
    lse = a.s == 0.f ? -INFINITY : fmaf(scale, a.m, ls);
    h = a.s == 0.f ? 0.f : fmaxf(ls - kLn2 * (a.u / a.s), 0.f);
    if (a.s != a.s || a.m == INFINITY) lse = h = __builtin_nanf("");
}
// The log probability of a logit z in a row whose joined statistics are `a`.
__device__ __forceinline__ float row_logp(const Stat& a, float scale, float z) {
    if (a.s != a.s || z != z || a.m == INFINITY) return __builtin_nanf("");
    if (z == -INFINITY) return -INFINITY;
    return scale * (z - a.m) - __logf(a.s);
}
__device__ __forceinline__ int64_t token_at(const RowOut& o, int64_t row) {
    return o.token_type == kI32 ? (int64_t)((const int32_t*)o.tokens)[row]
                                : ((const int64_t*)o.tokens)[row];
}
template <class T>
__device__ void put_token(const RowOut& o, const Stat& a, float scale, const T* z, int64_t row,
                          int64_t vocab) {
    float lse, h;
    row_stats(a, scale, lse, h);
    const int64_t tok = token_at(o, row);
    o.logp[row] = tok < 0 ? 0.f
                  : tok < vocab ? row_logp(a, scale, to_f32(z[tok]))
                                : __builtin_nanf("");
    if (o.entropy) o.entropy[row] = h;
    if (o.lse) o.lse[row] = lse;
}
__device__ __forceinline__ void put_top(const RowOut& o, const Stat& a, float scale, int64_t row,
                                        int top, int r, uint64_t key) {
    const uint32_t ord = (uint32_t)(key >> 32);
    const bool none = ord <= kOrdNegInf;
    float lp = none ? -INFINITY : row_logp(a, scale, unordered(ord));
    if (a.s != a.s || a.m == INFINITY) lp = __builtin_nanf("");
    o.top_logp[row * top + r] = lp;
    o.top_ids[row * top + r] = none ? -1 : (int32_t)~(uint32_t)key;
}

// ---- long rows -------------------------------------------------------------------

// A slice of a row per workgroup: elements [lo, hi) of it, lo on a group
// boundary. Groups start at addresses that a vector load can take: group q
// holds the columns [8 q - sh, 8 q - sh + 8), sh the row start's distance (in
// elements) from the last such address.
template <class T>
__device__ __forceinline__ void load_group(const T* row, int64_t c, int64_t vocab,
                                           float (&z)[kGroup]) {
    constexpr int V = 16 / sizeof(T);
    if (c >= 0 && c + kGroup <= vocab) {
#pragma unroll
        for (int q = 0; q < kGroup / V; ++q) {
            const Vec<T, V> v = load_vec<T, V>(row + c + q * V);
#pragma unroll
            for (int u = 0; u < V; ++u) z[q * V + u] = to_f32(v.e[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            z[u] = c + u >= 0 && c + u < vocab ? to_f32(row[c + u]) : -INFINITY;
    }
}

// part: per (row, slice) the statistics; cand: per (row, slice) `top` keys. With
// one slice the row's outputs are written here.
template <class T>
__global__ __launch_bounds__(256) void logprob_slice_kernel(
    const T* __restrict__ logits, int64_t vocab, int64_t ld, float scale, int groups_per_slice,
    int nslice, int top, Stat* __restrict__ part, uint64_t* __restrict__ cand, RowOut out) {
    extern __shared__ __align__(16) char smem[];
    __shared__ Stat wst[4];
    __shared__ uint64_t best[256];
    __shared__ uint64_t won[kMaxTop * 32];
    __shared__ int nwon;
    float* gmax = reinterpret_cast<float*>(smem);
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const int64_t row = blockIdx.x / nslice;
    const int slice = blockIdx.x % nslice;
    const T* z = logits + row * ld;
    const int sh = (int)((reinterpret_cast<uintptr_t>(z) % 16) / sizeof(T));
    const int64_t all = (vocab + sh + kGroup - 1) / kGroup;
    const int64_t g_lo = (int64_t)slice * groups_per_slice;
    const int ng = (int)(all - g_lo < groups_per_slice ? all - g_lo : groups_per_slice);
    const float k = scale * kLog2e;
    Stat a = stat_none();
    uint64_t mine = 0;
    for (int g = t; g < ng; g += 256) {
        float v[kGroup];
        load_group<T>(z, (g_lo + g) * kGroup - sh, vocab, v);
        float mx = v[0];
#pragma unroll
        for (int u = 1; u < kGroup; ++u) mx = fmaxf(mx, v[u]);
        if (mx > a.m) stat_rescale(a, mx, k);
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const float d = k * (v[u] - a.m);
            const float e = __builtin_amdgcn_exp2f(d);
            a.s += e;
            a.u = fmaf(e, fmaxf(d, -1000.f), a.u);
        }
        if (top) {
            gmax[g] = mx;
            const uint64_t key = ((uint64_t)ordered(mx) << 32) | (uint32_t)~g;
            mine = key > mine ? key : mine;
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a = stat_join(a, stat_shfl_xor(a, o), k);
    if (lane == 0) wst[w] = a;
    if (t == 0) nwon = 0;
    best[t] = mine;
    __syncthreads();
    a = stat_join(stat_join(wst[0], wst[1], k), stat_join(wst[2], wst[3], k), k);
    if (t == 0) {
        if (nslice > 1)
            part[row * nslice + slice] = a;
        else
            put_token<T>(out, a, scale, z, row, vocab);
    }
    if (!top) return;
    // The groups that can be among the first `top` belong to the `top` threads
    // whose best group is best: each thread ranks its own.
    int rank = 0;
    for (int q = 0; q < 256; ++q) rank += best[q] > mine;
    if (mine && rank < top) {
        for (int g = t; g < ng; g += 256) {
            const int at = atomicAdd(&nwon, 1);
            won[at] = ((uint64_t)ordered(gmax[g]) << 32) | (uint32_t)~g;
        }
    }
    __syncthreads();
    const int n = nwon;
    // of those, the `top` first, in order, into best[]
    if (t < kMaxTop) best[t] = 0;
    __syncthreads();
    for (int q = t; q < n; q += 256) {
        const uint64_t key = won[q];
        int r = 0;
        for (int p = 0; p < n && r < top; ++p) r += won[p] > key;
        if (r < top) best[r] = key;
    }
    __syncthreads();
    // one element per thread of the chosen groups
    uint64_t key = 0;
    if (t < top * kGroup) {
        const uint64_t gk = best[t / kGroup];
        if (gk) {
            const int64_t c = (g_lo + (int64_t)(~(uint32_t)gk)) * kGroup - sh + t % kGroup;
            if (c >= 0 && c < vocab)
                key = ((uint64_t)ordered(to_f32(z[c])) << 32) | (uint32_t)~(uint32_t)c;
        }
    }
    __syncthreads();
    best[t] = key;
    __syncthreads();
    if (t < top * kGroup) {
        int r = 0;
        for (int q = 0; q < top * kGroup; ++q) r += best[q] > key || (best[q] == key && q < t);
        if (r < top) {
            if (nslice > 1)
                cand[(row * nslice + slice) * top + r] = key;
            else
                put_top(out, a, scale, row, top, r, key);
        }
    }
}

// Joins a row's slices: statistics, then the `top` best of their candidates.
template <class T>
__global__ __launch_bounds__(256) void logprob_join_kernel(const T* __restrict__ logits,
                                                           int64_t vocab, int64_t ld, float scale,
                                                           int nslice, int top,
                                                           const Stat* __restrict__ part,
                                                           const uint64_t* __restrict__ cand,
                                                           RowOut out) {
    __shared__ uint64_t red[4];
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x;
    const float k = scale * kLog2e;
    Stat a = stat_none();
    for (int s = t & 63; s < nslice; s += 64) a = stat_join(a, part[row * nslice + s], k);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a = stat_join(a, stat_shfl_xor(a, o), k);
    if (t == 0) put_token<T>(out, a, scale, logits + row * ld, row, vocab);
    const int n = nslice * top;
    uint64_t below = ~0ull;
    for (int r = 0; r < top; ++r) {
        uint64_t m = 0;
        for (int q = t; q < n; q += 256) {
            const uint64_t key = cand[row * n + q];
            if (key < below && key > m) m = key;
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const uint64_t v = __shfl_xor((unsigned long long)m, o, 64);
            m = v > m ? v : m;
        }
        if ((t & 63) == 0) red[t >> 6] = m;
        __syncthreads();
        for (int q = 0; q < 4; ++q) m = red[q] > m ? red[q] : m;
        __syncthreads();
        if (t == 0) put_top(out, a, scale, row, top, r, m);
        below = m;
    }
}

// ---- short rows ------------------------------------------------------------------

constexpr int kShortCols = 512;  // 8 columns for each of a wave's lanes
constexpr int kShortPer = 8;

// A row per group of `gl` lanes (a power of two <= 64); lane l holds the
// columns l, l + gl, ...
template <class T>
__global__ __launch_bounds__(256) void logprob_short_kernel(const T* __restrict__ logits,
                                                            int64_t count, int vocab, int64_t ld,
                                                            float scale, int gl_log2, int top,
                                                            RowOut out) {
    const int gl = 1 << gl_log2;
    const int l = threadIdx.x & (gl - 1);
    const int64_t row0 = (int64_t)blockIdx.x * (256 >> gl_log2) + (threadIdx.x >> gl_log2);
    const bool on = row0 < count;
    const int64_t row = on ? row0 : count - 1;
    const T* z = logits + row * ld;
    const float k = scale * kLog2e;
    float v[kShortPer];
    float m = -FLT_MAX;
#pragma unroll
    for (int u = 0; u < kShortPer; ++u) {
        const int c = l + (u << gl_log2);
        v[u] = c < vocab ? to_f32(z[c]) : -INFINITY;
        m = fmaxf(m, v[u]);
    }
    for (int o = gl >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    Stat a = {m, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kShortPer; ++u) {
        const float d = k * (v[u] - m);
        const float e = __builtin_amdgcn_exp2f(d);
        a.s += e;
        a.u = fmaf(e, fmaxf(d, -1000.f), a.u);
    }
    for (int o = gl >> 1; o >= 1; o >>= 1) {
        a.s += __shfl_xor(a.s, o, 64);
        a.u += __shfl_xor(a.u, o, 64);
    }
    if (on && l == 0) put_token<T>(out, a, scale, z, row, vocab);
    uint64_t below = ~0ull;
    for (int r = 0; r < top; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int u = 0; u < kShortPer; ++u) {
            const int c = l + (u << gl_log2);
            const uint64_t key = ((uint64_t)ordered(v[u]) << 32) | (uint32_t)~c;
            if (c < vocab && key < below && key > best) best = key;
        }
        for (int o = gl >> 1; o >= 1; o >>= 1) {
            const uint64_t q = __shfl_xor((unsigned long long)best, o, 64);
            best = q > best ? q : best;
        }
        if (on && l == 0) put_top(out, a, scale, row, top, r, best);
        below = best;
    }
}

// ---- gradient ----------------------------------------------------------------------

// dlogits_j = scale (w ([j = tok] - p_j) - q p_j (logp_j + H)), w = dlogp (0
// without a token), q = dentropy. grid: (column tiles, rows).
template <class T>
__global__ __launch_bounds__(256) void logprob_grad_kernel(LogprobArgs p, int aligned) {
    constexpr int V = 16 / sizeof(T);
    const int64_t row = (int64_t)blockIdx.y + (int64_t)blockIdx.z * 65535;
    if (row >= p.count) return;
    const T* z = (const T*)p.logits + row * p.ld;
    T* d = (T*)p.dlogits + row * p.ldd;
    const float scale = p.scale, lse = p.lse[row], h = p.entropy ? p.entropy[row] : 0.f;
    const float q = p.dentropy ? p.dentropy[row] : 0.f;
    const int64_t tok = p.token_type == kI32 ? (int64_t)((const int32_t*)p.tokens)[row]
                                             : ((const int64_t*)p.tokens)[row];
    const float w = tok < 0 ? 0.f : tok < p.vocab ? p.dlogp[row] : __builtin_nanf("");
    const bool empty = lse == -INFINITY;
    const int sh = aligned ? (int)((reinterpret_cast<uintptr_t>(z) % 16) / sizeof(T)) : 0;
    auto one = [&](float v, int64_t c) {
        const float lp = fmaf(scale, v, -lse);
        const float pr = __builtin_amdgcn_exp2f(lp * kLog2e);
        float g = -pr * (w + q * (fmaxf(lp, -1e30f) + h));
        if (c == tok) g += w;
        return empty ? 0.f : scale * g;
    };
    const int64_t step = (int64_t)gridDim.x * 256 * V;
    for (int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V - sh; c < p.vocab; c += step) {
        if (aligned && c >= 0 && c + V <= p.vocab) {
            const Vec<T, V> v = load_vec<T, V>(z + c);
            Vec<T, V> o;
#pragma unroll
            for (int u = 0; u < V; ++u) o.e[u] = from_f32<T>(one(to_f32(v.e[u]), c + u));
            store_vec<T, V>(d + c, o);
        } else {
            for (int u = 0; u < V; ++u)
                if (c + u >= 0 && c + u < p.vocab)
                    d[c + u] = from_f32<T>(one(to_f32(z[c + u]), c + u));
        }
    }
}

// ---- plans -------------------------------------------------------------------------

struct SlicePlan {
    int groups, nslice;
};
// As few slices as the LDS allows, more where there are few rows: about 1024
// workgroups, each with at least one group per thread.
SlicePlan slice_plan(int64_t vocab, int64_t count) {
    const int64_t all = (vocab + 7 + kGroup - 1) / kGroup;  // whatever the row's alignment
    int64_t n = (all + kMaxGroups - 1) / kMaxGroups;
    const int64_t want = (1024 + count - 1) / count;
    const int64_t most = (all + 255) / 256;
    if (n < want) n = want < most ? want : most;
    SlicePlan p;
    p.groups = (int)((all + n - 1) / n);
    p.nslice = (int)((all + p.groups - 1) / p.groups);
    return p;
}

template <class T>
hipError_t logprobs_run(const LogprobArgs& a, hipStream_t st) {
    const RowOut o{a.tokens, a.token_type, a.logp, a.entropy, a.lse, a.top_logp, a.top_ids};
    if (a.vocab <= kShortCols) {
        int lg = 0;
        while (lg < 6 && (int64_t)(kShortPer / 2) << lg < a.vocab) ++lg;
        const int64_t per = 256 >> lg;
        hipLaunchKernelGGL((logprob_short_kernel<T>), dim3((unsigned)((a.count + per - 1) / per)),
                           dim3(256), 0, st, (const T*)a.logits, a.count, (int)a.vocab, a.ld,
                           a.scale, lg, a.top, o);
        return hipGetLastError();
    }
    const SlicePlan p = slice_plan(a.vocab, a.count);
    Stat* part = (Stat*)a.ws;
    uint64_t* cand =
        (uint64_t*)((char*)a.ws + ((size_t)a.count * p.nslice * sizeof(Stat) + 255) / 256 * 256);
    hipLaunchKernelGGL((logprob_slice_kernel<T>), dim3((unsigned)(a.count * p.nslice)), dim3(256),
                       a.top ? (size_t)p.groups * 4 : 0, st, (const T*)a.logits, a.vocab, a.ld,
                       a.scale, p.groups, p.nslice, a.top, part, cand, o);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.nslice == 1) return e;
    hipLaunchKernelGGL((logprob_join_kernel<T>), dim3((unsigned)a.count), dim3(256), 0, st,
                       (const T*)a.logits, a.vocab, a.ld, a.scale, p.nslice, a.top, part, cand, o);
    return hipGetLastError();
}

template <class T>
hipError_t grad_run(const LogprobArgs& a, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int aligned =
        reinterpret_cast<uintptr_t>(a.logits) % 16 == reinterpret_cast<uintptr_t>(a.dlogits) % 16 &&
        (a.ld - a.ldd) % V == 0;
    int64_t tiles = (a.vocab + V + 256 * V * 4 - 1) / (256 * V * 4);
    if (tiles < 1) tiles = 1;
    const unsigned gy = (unsigned)(a.count < 65535 ? a.count : 65535);
    const unsigned gz = (unsigned)((a.count + 65534) / 65535);
    hipLaunchKernelGGL((logprob_grad_kernel<T>), dim3((unsigned)tiles, gy, gz), dim3(256), 0, st, a,
                       aligned);
    return hipGetLastError();
}

}  // namespace

size_t logprob_ws_bytes(int64_t vocab, int top, int64_t count) {
    if (vocab <= kShortCols || count == 0) return 256;
    const SlicePlan p = slice_plan(vocab, count);
    return ((size_t)count * p.nslice * sizeof(Stat) + 255) / 256 * 256 +
           (size_t)count * p.nslice * (size_t)top * 8 + 256;
}

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t st) {
    return a.type == kF32    ? logprobs_run<float>(a, st)
           : a.type == kBF16 ? logprobs_run<bf16_t>(a, st)
                             : logprobs_run<f16_t>(a, st);
}
hipError_t launch_logprobs_grad(const LogprobArgs& a, hipStream_t st) {
    return a.type == kF32    ? grad_run<float>(a, st)
           : a.type == kBF16 ? grad_run<bf16_t>(a, st)
                             : grad_run<f16_t>(a, st);
}

}  // namespace symnmf
