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

#include <algorithm>

#include "common.h"
#include "seq.h"

namespace symnmf {
namespace {

constexpr int kGroup = 8;          // columns per group
constexpr int kMaxSlice = 256 << 10;  // bytes of one slice (maxima: an eighth of it in LDS)
constexpr int kMaxSlices = 64;        // slices of one row: a lane each when they are joined
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// Order of (value, column) as one number: larger is better. -0 equals 0; a NaN
// counts as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
    const int b = __float_as_int(fmaxf(v, -INFINITY) + 0.f);  // -0 + 0 is 0
    return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
constexpr uint32_t kOrdNegInf = 0x007fffffu;  // ordered(-inf)

// ---- best of a wave ----------------------------------------------------------------

// The largest of the wave's values, in every lane (a scalar): row shifts
// inside each 16 lanes, then broadcasts across rows; lane 63 ends with it.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto step = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xf, 0xf, false));
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xf, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// (ordered value, index): better is a larger value, then a lower index. An
// ordered value of 0 is nothing.
struct Cand {
    uint32_t ord, idx;
};
__device__ __forceinline__ bool better(Cand a, Cand b) {
    return a.ord > b.ord || (a.ord == b.ord && a.idx < b.idx);
}
__device__ __forceinline__ Cand best_of(Cand a, Cand b) { return better(a, b) ? a : b; }
// The best of the wave's candidates, in every lane.
__device__ __forceinline__ Cand wave_best(Cand c, int& lane) {
    const uint32_t m = wave_max(c.ord);
    uint64_t at = __ballot(c.ord == m);
    lane = __ffsll((unsigned long long)at) - 1;
    Cand r{m, (uint32_t)__builtin_amdgcn_readlane((int)c.idx, lane)};
    for (at &= at - 1; at; at &= at - 1) {  // equal values: the lowest index
        const int l = __ffsll((unsigned long long)at) - 1;
        const uint32_t i = (uint32_t)__builtin_amdgcn_readlane((int)c.idx, l);
        if (i < r.idx) {
            r.idx = i;
            lane = l;
        }
    }
    return r;
}

// How many of the candidates of lanes 0, step, 2 step, ... (n of them) are better
// than this lane's.
__device__ __forceinline__ int rank_among(Cand c, int n, int step = 1) {
    const uint64_t key = (uint64_t)c.ord << 32 | (uint32_t)~c.idx;
    int r = 0;
    for (int j = 0; j < n * step; j += step) {
        const uint32_t ord = (uint32_t)__builtin_amdgcn_readlane((int)c.ord, j);
        const uint32_t idx = (uint32_t)__builtin_amdgcn_readlane((int)c.idx, j);
        r += ((uint64_t)ord << 32 | (uint32_t)~idx) > key;
    }
    return r;
}
// The candidate of the lane whose rank is r (nothing if there is none).
__device__ __forceinline__ Cand of_rank(Cand c, int rank, int r) {
    const uint64_t at = __ballot(rank == r);
    if (!at) return Cand{0, 0};
    const int l = __ffsll((unsigned long long)at) - 1;
    return Cand{(uint32_t)__builtin_amdgcn_readlane((int)c.ord, l),
                (uint32_t)__builtin_amdgcn_readlane((int)c.idx, l)};
}
// Appends the candidates of the lanes whose `on` is set to a list of kFew in LDS;
// returns the list's new length (past kFew: it did not fit).
constexpr int kFew = 64;
__device__ __forceinline__ int append(Cand* list, int n, bool on, Cand c) {
    const uint64_t m = __ballot(on);
    const int at = n + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1ull));
    if (on && at < kFew) list[at] = c;
    return n + __popcll(m);
}

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
// v[op]... over the wave, in every lane (a scalar): row shifts inside each 16
// lanes, then broadcasts across rows; lane 63 ends with it. `none` is what op
// leaves unchanged.
template <class F>
__device__ __forceinline__ float wave_fold(float v, float none, F&& op) {
    auto from = [&](auto x) { return __int_as_float(x(__float_as_int(none), __float_as_int(v))); };
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x111, 0xf, 0xf, false); }));
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x112, 0xf, 0xf, false); }));
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x114, 0xf, 0xf, false); }));
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x118, 0xf, 0xf, false); }));
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x142, 0xf, 0xf, false); }));
    v = op(v, from([](int o, int x) { return __builtin_amdgcn_update_dpp(o, x, 0x143, 0xf, 0xf, false); }));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// The wave's statistics joined, in every lane: one rescaling to the common
// maximum, then plain sums.
__device__ __forceinline__ Stat stat_wave(Stat a, float k) {
    stat_rescale(a, wave_fold(a.m, -FLT_MAX, [](float x, float y) { return fmaxf(x, y); }), k);
    a.s = wave_fold(a.s, 0.f, [](float x, float y) { return x + y; });
    a.u = wave_fold(a.u, 0.f, [](float x, float y) { return x + y; });
    return a;
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
// A row's token and its logit: two loads one after the other. Rows in registers ask
// for them before the row (50000 x 800, top 5: 46.2 us, after it 48.4); waves that
// stream a row would wait for the first before they begin (20000 x 2000: 31.8, after
// it 29.6).
struct Token {
    int64_t id;
    float z;
};
template <class T>
__device__ __forceinline__ Token token_of(const RowOut& o, const T* z, int64_t row,
                                          int64_t vocab) {
    const int64_t id = token_at(o, row);
    return {id, to_f32(z[id >= 0 && id < vocab ? id : 0])};
}
__device__ __forceinline__ void put_token(const RowOut& o, const Stat& a, float scale,
                                          int64_t row, int64_t vocab, const Token& tok) {
    float lse, h;
    row_stats(a, scale, lse, h);
    o.logp[row] = tok.id < 0 ? 0.f
                  : tok.id < vocab ? row_logp(a, scale, tok.z)
                                   : __builtin_nanf("");
    if (o.entropy) o.entropy[row] = h;
    if (o.lse) o.lse[row] = lse;
}
__device__ __forceinline__ void put_top(const RowOut& o, const Stat& a, float scale, int64_t row,
                                        int top, int r, Cand c) {
    const bool none = c.ord <= kOrdNegInf;
    float lp = none ? -INFINITY : row_logp(a, scale, unordered(c.ord));
    if (a.s != a.s || a.m == INFINITY) lp = __builtin_nanf("");
    o.top_logp[row * top + r] = lp;
    o.top_ids[row * top + r] = none ? -1 : (int32_t)c.idx;
}

// ---- long rows -------------------------------------------------------------------

// WAVES waves per (row, slice); a workgroup of at least 256 threads. Each thread
// takes four groups (of a tile of 256 WAVES) at a time, the next four already
// on their way; a row's last group may be partial and is read element by
// element. Group maxima are kept in the logits' own type (exact).
template <class T, int WAVES>
__global__ __launch_bounds__(WAVES < 4 ? 256 : 64 * WAVES) void logprob_slice_kernel(
    const T* __restrict__ logits, int64_t items, int64_t vocab, int64_t ld, float scale,
    int groups_per_slice, int nslice, int top, Stat* __restrict__ part, Cand* __restrict__ cand,
    RowOut out, int64_t first) {
    extern __shared__ __align__(16) char smem[];
    constexpr int V = 16 / sizeof(T), NV = kGroup / V, Q = 4, N = 64 * WAVES;
    constexpr int SLOTS = WAVES < 4 ? 4 / WAVES : 1;
    __shared__ Stat wst[WAVES];
    __shared__ Cand leads[SLOTS][N > 2 * kFew ? N : 2 * kFew];
    const int slot = threadIdx.x / N, t = threadIdx.x % N, lane = t & 63, w = t >> 6;
    const int64_t item = (first + blockIdx.x) * SLOTS + slot;
    if (item >= items) return;  // whole waves, and with several to an item whole workgroups
    T* gmax = reinterpret_cast<T*>(smem) + (int64_t)slot * groups_per_slice;
    Cand* lead = leads[slot];
    const int64_t row = item / nslice;
    const int slice = (int)(item % nslice);
    const T* z = logits + row * ld;
    const int64_t all = (vocab + kGroup - 1) / kGroup;
    const int64_t g_lo = (int64_t)slice * groups_per_slice;
    const int ng = (int)max((int64_t)0, min(all - g_lo, (int64_t)groups_per_slice));
    const T* zs = z + g_lo * kGroup;  // group g of the slice begins at zs + 8 g
    const int g_end = ng > 0 && g_lo + ng == all && vocab % kGroup ? ng - 1 : ng;
    const float k = scale * kLog2e;
    Stat a = stat_none();
    float best = -INFINITY;  // the thread's best group, compared as a float: its
    int best_g = t;          // ordered key is made once, after the loop

    Vec<T, V> cur[Q][NV], nxt[Q][NV];
    auto fetch = [&](Vec<T, V>(&to)[Q][NV], int g0) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int g = g0 + q * N;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (g < g_end) {
                    to[q][i] = load_vec<T, V>(zs + (int64_t)g * kGroup + i * V);
                } else {
#pragma unroll
                    for (int u = 0; u < V; ++u) to[q][i].e[u] = from_f32<T>(-INFINITY);
                }
            }
        }
    };
    auto take = [&](const float (&v)[kGroup]) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const float d = k * (v[u] - a.m);
            const float e = __builtin_amdgcn_exp2f(d);
            a.s += e;
            a.u = fmaf(e, fmaxf(d, -1000.f), a.u);
        }
    };
    auto keep = [&](int g, float mx) {
        gmax[g] = from_f32<T>(mx);
        if (mx > best) {  // groups come in order: the first of equals stays
            best = mx;
            best_g = g;
        }
    };
    fetch(cur, t);
    for (int g0 = t; g0 - t < g_end; g0 += N * Q) {
        fetch(nxt, g0 + N * Q);
        float mx[Q], all_mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            mx[q] = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int u = 0; u < V; ++u) mx[q] = fmaxf(mx[q], to_f32(cur[q][i].e[u]));
            all_mx = fmaxf(all_mx, mx[q]);
        }
        if (all_mx > a.m) stat_rescale(a, all_mx, k);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int g = g0 + q * N;
            if (g - t >= g_end) break;  // nothing for the whole wave
            float v[kGroup];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int u = 0; u < V; ++u) v[i * V + u] = to_f32(cur[q][i].e[u]);
            take(v);
            if (top && g < g_end) keep(g, mx[q]);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < NV; ++i) cur[q][i] = nxt[q][i];
    }
    if (g_end < ng && g_end % N == t) {  // the partial group
        float v[kGroup], mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const int64_t c = (g_lo + g_end) * kGroup + u;
            v[u] = c < vocab ? to_f32(z[c]) : -INFINITY;
            mx = fmaxf(mx, v[u]);
        }
        if (mx > a.m) stat_rescale(a, mx, k);
        take(v);
        if (top) keep(g_end, mx);
    }
    // Groups of -inf alone are led by the first of them, so the leaders differ.
    Cand mine{t < ng ? ordered(best) : 0u, (uint32_t)best_g};
    a = stat_wave(a, k);
    if (WAVES > 1) {
        if (lane == 0) wst[w] = a;
        lead[t] = mine;
        __syncthreads();
        if (w != 0) return;
        a = stat_wave(lane < WAVES ? wst[lane] : stat_none(), k);
        mine = lead[t];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) mine = best_of(mine, lead[t + 64 * i]);
    }
    wave_lds_sync();  // gmax is read below, and lead written
    if (lane == 0) {
        if (nslice > 1)
            part[item] = a;
        else
            put_token(out, a, scale, row, vocab, token_of(out, z, row, vocab));
    }
    if (!top) return;
    // One wave picks the groups: lane l leads the groups g = l (mod 64). The
    // `top`-th best leader bounds the `top`-th best group and element from
    // below, so groups from it on, and their elements that reach its value, hold
    // all that is wanted. Mostly those are few enough for a lane each, and then
    // counting who is better ranks them at once (20000 x 2000, top 20:
    // 46.7 us; picking one by one 88.9. 16 x 100000: 20.9 and 27.7).
    {
        Cand* list = lead;        // kFew groups
        Cand* elems = lead + kFew;  // kFew elements
        Cand low;
        int ngr = 0, nel = 0;
        // Sixteen leaders of four lanes serve for up to 8, 32 of two for up to 16.
        const Cand own = mine;
        if (top <= 16) {
            Cand m = best_of(own, Cand{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)own.ord, 0xB1, 0xf, 0xf, false),
                                       (uint32_t)__builtin_amdgcn_update_dpp(0, (int)own.idx, 0xB1, 0xf, 0xf, false)});
            if (top <= 8) {
                m = best_of(m, Cand{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)m.ord, 0x4E, 0xf, 0xf, false),
                                    (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m.idx, 0x4E, 0xf, 0xf, false)});
                low = of_rank(m, (lane & 3) ? 64 : rank_among(m, 16, 4), top - 1);
            } else {
                low = of_rank(m, (lane & 1) ? 64 : rank_among(m, 32, 2), top - 1);
            }
        } else {
            low = of_rank(own, rank_among(own, 64), top - 1);
        }
        if (ng <= 64 * top) {  // look all groups over
            for (int g = lane; g - lane < ng; g += 64) {
                const Cand c{g < ng ? ordered(to_f32(gmax[g])) : 0u, (uint32_t)g};
                ngr = append(list, ngr, c.ord && !better(low, c), c);
            }
        } else {  // look over the groups of the lanes whose best reaches the bound
            for (uint64_t at = __ballot(!better(low, own)); at && ngr <= kFew; at &= at - 1) {
                const int owner = __ffsll((unsigned long long)at) - 1;
                for (int g = owner + 64 * lane; g - 64 * lane < ng; g += 4096) {
                    const Cand c{g < ng ? ordered(to_f32(gmax[g])) : 0u, (uint32_t)g};
                    ngr = append(list, ngr, c.ord && !better(low, c), c);
                }
            }
        }
        if (ngr <= kFew) {
            wave_lds_sync();
            for (int e = lane; e - lane < ngr * kGroup; e += 64) {
                Cand c{0, 0};
                if (e < ngr * kGroup) {
                    const int64_t col = (g_lo + list[e / kGroup].idx) * kGroup + e % kGroup;
                    if (col < vocab) c = Cand{ordered(to_f32(z[col])), (uint32_t)col};
                }
                nel = append(elems, nel, c.ord && c.ord >= low.ord, c);
            }
            if (nel <= kFew) {
                wave_lds_sync();
                const Cand c = lane < nel ? elems[lane] : Cand{0, 0};
                int at = rank_among(c, nel);
                if (lane >= nel) at = lane;  // fewer than `top` there are
                if (at >= top) return;
                if (nslice > 1)
                    cand[item * top + at] = c;
                else
                    put_top(out, a, scale, row, top, at, c);
                return;
            }
        }
        wave_lds_sync();
    }
    // Many equal or ordered logits: one by one. After a lane's best is taken the
    // wave looks its groups over for the next.
    Cand chosen[4] = {};  // of the groups chosen, those of ranks lane / 8 + 8 q
    for (int r = 0; r < top; ++r) {
        int owner;
        const Cand b = wave_best(mine, owner);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if ((lane >> 3) + 8 * q == r) chosen[q] = b;
        if (b.ord == 0) break;
        Cand next{0, 0};
        for (int g = owner + 64 * lane; g < ng; g += 4096) {
            const Cand c{ordered(to_f32(gmax[g])), (uint32_t)g};
            if (better(b, c)) next = best_of(c, next);
        }
        int unused;
        next = wave_best(next, unused);
        if (lane == owner) mine = next;
    }
    // their elements, four to a lane, and the best of those
    Cand el[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        el[q] = Cand{0, 0};
        const int64_t c = (g_lo + chosen[q].idx) * kGroup + (lane & 7);
        if (chosen[q].ord && c < vocab) el[q] = Cand{ordered(to_f32(z[c])), (uint32_t)c};
    }
    Cand got{0, 0};  // lane r keeps the r-th
    for (int r = 0; r < top; ++r) {
        const Cand m01 = best_of(el[0], el[1]), m23 = best_of(el[2], el[3]);
        int unused;
        const Cand b = wave_best(best_of(m01, m23), unused);
        if (lane == r) got = b;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (el[q].idx == b.idx) el[q].ord = 0;
    }
    if (lane >= top) return;
    if (nslice > 1)
        cand[item * top + lane] = got;
    else
        put_top(out, a, scale, row, top, lane, got);
}

// Joins a row's slices (at most 64), a wave per row: statistics, then the `top`
// best of the slices' lists. Each list is in order: lane l holds the head of
// list l.
template <class T>
__global__ __launch_bounds__(64) void logprob_join_kernel(const T* __restrict__ logits,
                                                          int64_t vocab, int64_t ld, float scale,
                                                          int nslice, int top,
                                                          const Stat* __restrict__ part,
                                                          const Cand* __restrict__ cand,
                                                          RowOut out, int64_t first) {
    __shared__ Cand list[kMaxTop][kMaxSlices];
    const int64_t row = first + blockIdx.x;
    const int lane = threadIdx.x;
    const float k = scale * kLog2e;
    const bool on = lane < nslice;
    const Cand* c = cand + (row * nslice + lane) * top;
    Stat a = on ? part[row * nslice + lane] : stat_none();
    for (int r = 0; r < top; ++r) list[r][lane] = on ? c[r] : Cand{0, 0};  // the lane's own
    a = stat_wave(a, k);
    if (lane == 0)
        put_token(out, a, scale, row, vocab, token_of(out, logits + row * ld, row, vocab));
    if (!top) return;
    Cand mine = list[0][lane], got{0, 0};
    if (nslice >= top) {  // as for a slice's groups: the `top`-th best head bounds what is wanted
        __shared__ Cand few[64];
        const Cand low = of_rank(mine, rank_among(mine, nslice), top - 1);
        int n = 0;
        for (int r = 0; r < top; ++r) {
            const Cand c = list[r][lane];
            const int m = append(few, n, c.ord && !better(low, c), c);
            if (m == n) break;
            n = m;
        }
        if (n <= 64) {
            wave_lds_sync();
            const Cand c = lane < n ? few[lane] : Cand{0, 0};
            const int rank = lane < n ? rank_among(c, n) : lane;
            if (rank < top) put_top(out, a, scale, row, top, rank, c);
            return;
        }
    }
    int at = 0;
    for (int r = 0; r < top; ++r) {
        int owner;
        const Cand b = wave_best(mine, owner);
        if (lane == r) got = b;
        if (lane == owner) mine = ++at < top ? list[at][lane] : Cand{0, 0};
    }
    if (lane < top) put_top(out, a, scale, row, top, lane, got);
}

// ---- short rows ------------------------------------------------------------------

// Up to these columns, a row lies in the registers of a few lanes: 1024 (50000 x
// 1000 bf16: 26.5 us, by the kernel for long rows 35.2; top 5: 47.4 and 54.0; 20000 x
// 2000, top 5: 41.3 and 28.9). Alternatives of fp32 rows have no short key (below)
// and stop at 512 (50000 x 1000, top 5: 74.0 us and 62.4).
constexpr int kShortBits = 10, kShortCols = 1 << kShortBits;
bool short_row(int64_t vocab, int top, int bytes) {
    return vocab <= (bytes == 2 || top == 0 ? kShortCols : kShortCols / 2);
}

// Exchanges across a group of 2^lg lanes, one step per bit, for reductions that
// leave every lane of the group with the result: within 16 lanes by lane
// permutes of the register file (the mirrors serve as xor 4 and 8 once 4 and 8
// lanes agree), past that through LDS permutes.
template <class F>
__device__ __forceinline__ void group_steps(int lg, F&& step) {
    if (lg > 0) step([](int v) { return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, false); });
    if (lg > 1) step([](int v) { return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, false); });
    if (lg > 2) step([](int v) { return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false); });
    if (lg > 3) step([](int v) { return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false); });
    if (lg > 4) step([](int v) { return __shfl_xor(v, 16, 64); });
    if (lg > 5) step([](int v) { return __shfl_xor(v, 32, 64); });
}

// A row per group of 2^lg lanes; lane l holds the column groups l, l + 2^lg, ...
// (NG of them), all in registers.
template <class T, int NG>
__global__ __launch_bounds__(256) void logprob_short_kernel(const T* __restrict__ logits,
                                                            int64_t count, int vocab, int64_t ld,
                                                            float scale, int lg, int top,
                                                            RowOut out, int64_t first) {
    constexpr int NS = NG * kGroup, V = 16 / sizeof(T);
    const int l = threadIdx.x & ((1 << lg) - 1);
    const int64_t row0 = (first + blockIdx.x) * (256 >> lg) + (threadIdx.x >> lg);
    const bool on = row0 < count;
    const int64_t row = on ? row0 : count - 1;
    const T* z = logits + row * ld;
    const float k = scale * kLog2e;
    const Token tok = token_of(out, z, row, vocab);
    float v[NS];
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const int c = (l + (i << lg)) * kGroup;
        if (c + kGroup <= vocab) {
#pragma unroll
            for (int q = 0; q < kGroup; q += V) {
                const Vec<T, V> x = load_vec<T, V>(z + c + q);
#pragma unroll
                for (int u = 0; u < V; ++u) v[i * kGroup + q + u] = to_f32(x.e[u]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                v[i * kGroup + u] = c + u < vocab ? to_f32(z[c + u]) : -INFINITY;
        }
    }
#pragma unroll
    for (int u = 0; u < NS; ++u) m = fmaxf(m, v[u]);
    group_steps(lg, [&](auto x) { m = fmaxf(m, __int_as_float(x(__float_as_int(m)))); });
    Stat a = {m, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NS; ++u) {
        const float d = k * (v[u] - m);
        const float e = __builtin_amdgcn_exp2f(d);
        a.s += e;
        a.u = fmaf(e, fmaxf(d, -1000.f), a.u);
    }
    group_steps(lg, [&](auto x) {
        a.s += __int_as_float(x(__float_as_int(a.s)));
        a.u += __int_as_float(x(__float_as_int(a.u)));
    });
    if (on && l == 0) put_token(out, a, scale, row, vocab, tok);
    if (!top) return;
    // The lanes of the group hold one alternative each and write them together.
    const int mask = (1 << lg) - 1;
    Cand got{0, 0};
    auto put = [&](int r, Cand b) {
        if (l == (r & mask)) got = b;
        const int first = r & ~mask;
        if (((r & mask) == mask || r == top - 1) && on && first + l <= r)
            put_top(out, a, scale, row, top, first + l, got);
    };
    if constexpr (sizeof(T) == 2) {
        // Sixteen-bit logits: the order's upper 19 bits tell them apart (8 of exponent,
        // 10 of mantissa at most), so value and column make one key, and the best key
        // under the last one is last - 1 - min(last - 1 - key), where the keys from
        // the last on wrap round to large numbers. Places past the row count as -inf.
        uint32_t key[NS], last = ~0u;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int c = (l + ((u / kGroup) << lg)) * kGroup + u % kGroup;
            const uint32_t o = ordered(v[u]) >> (13 - kShortBits);
            key[u] = (o & -(1u << kShortBits)) | (uint32_t)(kShortCols - 1 - c);
        }
        for (int r = 0; r < top; ++r) {
            const uint32_t below = max(last, 1u) - 1;
            uint32_t d = below;  // that of key 0: nothing
#pragma unroll
            for (int u = 0; u < NS; ++u) d = min(d, below - key[u]);
            group_steps(lg, [&](auto x) { d = min(d, (uint32_t)x((int)d)); });
            last = below - d;
            uint32_t o = last >> kShortBits << 13;
            if (last && !(o >> 31)) o |= 0x1fffu;  // negative numbers' lower bits
            put(r, Cand{o, kShortCols - 1 - (last & (kShortCols - 1))});
        }
        return;
    }
    uint32_t ord[NS];
#pragma unroll
    for (int u = 0; u < NS; ++u) {
        const int c = (l + ((u / kGroup) << lg)) * kGroup + u % kGroup;
        ord[u] = c < vocab ? ordered(v[u]) : 0u;
    }
    for (int r = 0; r < top; ++r) {
        uint32_t bo = ord[0];
        int bu = 0;
#pragma unroll
        for (int u = 1; u < NS; ++u)
            if (ord[u] > bo) {
                bo = ord[u];
                bu = u;
            }
        Cand b{bo, (uint32_t)((l + ((bu / kGroup) << lg)) * kGroup + bu % kGroup)};
        const uint32_t own = b.idx;
        group_steps(lg, [&](auto x) {
            b = best_of(b, Cand{(uint32_t)x((int)b.ord), (uint32_t)x((int)b.idx)});
        });
        put(r, b);
        const int gone = own == b.idx ? bu : -1;  // the lane that held it
#pragma unroll
        for (int u = 0; u < NS; ++u) ord[u] = u == gone ? 0u : ord[u];
    }
}

// ---- gradient ----------------------------------------------------------------------

// dlogits_j = scale (w ([j = tok] - p_j) - q p_j (logp_j + H)), w = dlogp (0
// without a token), q = dentropy. grid: (column tiles, groups of rows).
// Rows of few columns share a workgroup, 2^lx lanes to each. Accesses start at
// 16-byte boundaries where the rows of both arrays allow it (`aligned`; 2048 x
// 100003 bf16: 153 us, from the rows' own starts 171).
//
// ln p = scale z - lse takes lse's rounding into p: |lse| 2^-24 of it. Up to
// kLseFar that is 4e-6 at most; past it the row is read again for its M and ln s,
// which keep those bits as in the forward, in ln p = scale (z - M) - ln s. They
// are taken where they round to the lse given (or, where scale M overflows, to
// its infinity), so an lse of more columns than these stays what it was given
// for. Such a row is one wave's or one workgroup's (the first of those that share
// it), which has read it when it begins to write, since it may write in place
// (bf16, near and far: 50000 x 500 25 and 45 us, 2048 x 100003 155 and 320, 16 x
// 100000 11 and 43).
constexpr float kLseFar = 64.f;

// M and s of a row (u is not needed), by the n lanes of t = 0 ... n - 1 that share
// it: up to 64 of one wave, or a workgroup's 256. All have read when it returns.
template <class T>
__device__ Stat row_again(const T* z, int64_t vocab, float k, int t, int n) {
    __shared__ Stat wst[4];
    constexpr int V = 16 / sizeof(T);
    Stat a = stat_none();
    for (int64_t c = (int64_t)t * V; c < vocab; c += (int64_t)n * V) {
        float v[V], m = a.m;
#pragma unroll
        for (int u = 0; u < V; ++u) v[u] = -INFINITY;
        if (c + V <= vocab) {
            const Vec<T, V> x = load_vec<T, V>(z + c);
#pragma unroll
            for (int u = 0; u < V; ++u) v[u] = to_f32(x.e[u]);
        } else {
            for (int u = 0; u < V; ++u)
                if (c + u < vocab) v[u] = to_f32(z[c + u]);
        }
#pragma unroll
        for (int u = 0; u < V; ++u) m = fmaxf(m, v[u]);
        if (m > a.m) stat_rescale(a, m, k);
#pragma unroll
        for (int u = 0; u < V; ++u) a.s += __builtin_amdgcn_exp2f(k * (v[u] - a.m));
    }
    auto join = [&](float m, float s) {
        const float both = fmaxf(a.m, m);
        stat_rescale(a, both, k);
        a.s += s * __builtin_amdgcn_exp2f(k * (m - both));
    };
    for (int o = 1; o < min(n, 64); o <<= 1) {
        const float m = __shfl_xor(a.m, o, 64), s = __shfl_xor(a.s, o, 64);
        join(m, s);
    }
    if (n > 64) {
        if ((t & 63) == 0) wst[t >> 6] = a;
        __syncthreads();
        a = wst[0];
        for (int w = 1; w < 4; ++w) join(wst[w].m, wst[w].s);
    }
    return a;
}

template <class T>
__global__ __launch_bounds__(256) void logprob_grad_kernel(LogprobArgs p, int aligned, int lx) {
    constexpr int V = 16 / sizeof(T);
    const int64_t row = ((int64_t)blockIdx.y << (8 - lx)) + (threadIdx.x >> lx);
    if (row >= p.count) return;
    const T* z = (const T*)p.logits + row * p.ld;
    T* d = (T*)p.dlogits + row * p.ldd;
    const float scale = p.scale, lse = p.lse[row], h = p.entropy ? p.entropy[row] : 0.f;
    const float q = p.dentropy ? p.dentropy[row] : 0.f;
    const int64_t tok = p.token_type == kI32 ? (int64_t)((const int32_t*)p.tokens)[row]
                                             : ((const int64_t*)p.tokens)[row];
    const float w = tok < 0 ? 0.f : tok < p.vocab ? p.dlogp[row] : __builtin_nanf("");
    bool empty = lse == -INFINITY;
    float ref = 0.f, off = lse;  // ln p = scale (z - ref) - off
    // this lane among those that share the row, and how many they are
    int t = (int)(threadIdx.x & ((1 << lx) - 1)) + ((int)blockIdx.x << lx);
    int n = (int)gridDim.x << lx;
    if (fabsf(lse) > kLseFar) {  // a row's lanes agree
        n = lx == 7 ? 64 : 1 << lx;
        if (t >= n) return;  // whole waves or whole workgroups
        const Stat a = row_again<T>(z, p.vocab, scale * kLog2e, t, n);
        const float ls = __logf(a.s), full = fmaf(scale, a.m, ls);
        if (a.s > 0.f && (full == lse || fabsf(full - lse) <= fabsf(lse) * 4.7683716e-7f)) {  // 2^-21
            ref = a.m;
            off = ls;
            empty = false;
        }
    }
    const int sh = aligned ? (int)((reinterpret_cast<uintptr_t>(z) % 16) / sizeof(T)) : 0;
    auto one = [&](float v, int64_t c) {
        const float lp = fmaf(scale, v - ref, -off);
        // as a square: p below 2^-126, which ln p + H may lift above it, is not flushed
        const float root = __builtin_amdgcn_exp2f(lp * (0.5f * kLog2e)), pr = root * root;
        float g = -pr * (w + q * (fmaxf(lp, -1000.f) + h));  // p is 0 there, for any q below 1e35
        if (c == tok) g += w;
        return empty ? 0.f : scale * g;
    };
    for (int64_t c = (int64_t)t * V - sh; c < p.vocab; c += (int64_t)n * V) {
        if (c >= 0 && c + V <= p.vocab) {
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
    int waves, groups, nslice;
};
// A slice's waves: one up to these groups (16 a lane; four slices then share a
// workgroup: 10000 x 4000 bf16 27.5 us against 34.0 with four waves), else four, or
// sixteen where there are few rows (256 x 100000: 23.2 us against 28.1).
constexpr int kWaveGroups = 1024;
constexpr int64_t kFewRows = 256;
// Rows are cut only where they are so few and so long that most of the chip would
// idle: into about kItems slices altogether, joined by a second launch (16 x
// 100000 bf16, top 20: 20.9 us, whole 28.6; 64 x 32768: 21.8 us, whole 17.6).
constexpr int64_t kCutRows = 64, kCutBytes = 64 << 10, kItems = 1024;

// Whole rows fit a slice up to 256 KiB with four waves, 1 MiB with sixteen (the
// maxima take an eighth of it in LDS).
SlicePlan slice_plan(int64_t vocab, int64_t count, int bytes) {
    const int64_t all = (vocab + kGroup - 1) / kGroup;
    SlicePlan p;
    const bool cut = count <= kCutRows && vocab * bytes > kCutBytes && all > kWaveGroups;
    p.waves = all <= kWaveGroups ? 1 : count <= kFewRows && !cut ? 16 : 4;
    const int64_t fit = (p.waves == 16 ? 4 : 1) * (int64_t)kMaxSlice / bytes / kGroup;
    int64_t n = (all + fit - 1) / fit;
    if (cut) n = std::max(n, std::min((kItems + count - 1) / count, (all + 255) / 256));
    if (n > kMaxSlices) n = kMaxSlices;  // kMaxVocab columns fit that many
    p.groups = (int)((all + n - 1) / n);
    p.nslice = (int)((all + p.groups - 1) / p.groups);
    return p;
}

template <class T>
hipError_t logprobs_run(const LogprobArgs& a, hipStream_t st) {
    const RowOut o{a.tokens, a.token_type, a.logp, a.entropy, a.lse, a.top_logp, a.top_ids};
    if (short_row(a.vocab, a.top, sizeof(T))) {
        // as few lanes a row as hold it with 32 columns each (24 columns: one lane)
        int lg = 0;
        while ((int64_t)32 << lg < a.vocab) ++lg;
        const int ng = (int)((a.vocab + (kGroup << lg) - 1) / (kGroup << lg));
        const int64_t per = 256 >> lg;
        auto* kern = ng <= 1   ? logprob_short_kernel<T, 1>
                     : ng <= 2 ? logprob_short_kernel<T, 2>
                     : ng <= 3 ? logprob_short_kernel<T, 3>
                               : logprob_short_kernel<T, 4>;
        return in_launches((a.count + per - 1) / per, [&](int64_t first, unsigned n) {
            hipLaunchKernelGGL(kern, dim3(n), dim3(256), 0, st, (const T*)a.logits, a.count,
                               (int)a.vocab, a.ld, a.scale, lg, a.top, o, first);
        });
    }
    const SlicePlan p = slice_plan(a.vocab, a.count, sizeof(T));
    Stat* part = (Stat*)a.ws;
    Cand* cand =
        (Cand*)((char*)a.ws + ((size_t)a.count * p.nslice * sizeof(Stat) + 255) / 256 * 256);
    const int64_t items = a.count * p.nslice;
    const size_t lds = a.top ? (size_t)p.groups * sizeof(T) : 0;
    auto* kern = p.waves == 1   ? logprob_slice_kernel<T, 1>
                 : p.waves == 4 ? logprob_slice_kernel<T, 4>
                                : logprob_slice_kernel<T, 16>;
    const int slots = p.waves == 1 ? 4 : 1, threads = p.waves == 16 ? 1024 : 256;
    const hipError_t e =
        in_launches((items + slots - 1) / slots, [&](int64_t first, unsigned n) {
            hipLaunchKernelGGL(kern, dim3(n), dim3(threads), slots * lds, st, (const T*)a.logits,
                               items, a.vocab, a.ld, a.scale, p.groups, p.nslice, a.top, part,
                               cand, o, first);
        });
    if (e != hipSuccess || p.nslice == 1) return e;
    return in_launches(a.count, [&](int64_t first, unsigned n) {
        hipLaunchKernelGGL((logprob_join_kernel<T>), dim3(n), dim3(64), 0, st, (const T*)a.logits,
                           a.vocab, a.ld, a.scale, p.nslice, a.top, part, cand, o, first);
    });
}

template <class T>
hipError_t grad_run(const LogprobArgs& a, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int aligned =
        reinterpret_cast<uintptr_t>(a.logits) % 16 == reinterpret_cast<uintptr_t>(a.dlogits) % 16 &&
        (a.ld - a.ldd) % V == 0;
    const int64_t vecs = (a.vocab + V - 1 + V - 1) / V;  // whatever the row's alignment
    int lx = 0;
    while (lx < 8 && ((int64_t)1 << lx) < vecs) ++lx;
    const int64_t tiles = (vecs + 1023) / 1024, rows = (a.count + (256 >> lx) - 1) >> (8 - lx);
    // rows in a grid dimension of at most 65535: the rest in further launches
    for (int64_t r = 0; r < rows; r += 65535) {
        LogprobArgs q = a;
        const int64_t skip = r << (8 - lx);
        q.count -= skip;
        q.logits = (const T*)a.logits + skip * a.ld;
        q.dlogits = (T*)a.dlogits + skip * a.ldd;
        q.tokens = (const char*)a.tokens + skip * (a.token_type == kI32 ? 4 : 8);
        q.lse += skip;
        if (q.entropy) q.entropy += skip;
        q.dlogp += skip;
        if (q.dentropy) q.dentropy += skip;
        const int64_t n = rows - r < 65535 ? rows - r : 65535;
        hipLaunchKernelGGL((logprob_grad_kernel<T>), dim3((unsigned)tiles, (unsigned)n), dim3(256),
                           0, st, q, aligned, lx);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t logprob_ws_bytes(int64_t vocab, int top, int64_t count) {
    if (count == 0 || short_row(vocab, top, 4)) return 256;  // 4: any type
    const int64_t n = std::max(slice_plan(vocab, count, 2).nslice, slice_plan(vocab, count, 4).nslice);
    if (n < 2) return 256;
    return ((size_t)(count * n) * sizeof(Stat) + 255) / 256 * 256 +
           (size_t)(count * n) * (size_t)top * sizeof(Cand) + 256;
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
