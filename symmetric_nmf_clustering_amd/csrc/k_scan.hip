// Gated linear recurrence over time, per batch row and channel:
//   a_t = sigmoid(gate_t), c_t = 1 - a_t = sigmoid(-gate_t)
//   h_t = a_t h_{t-1} + c_t x_t,  h_{-1} = h0,
// and its gradient. A step is the affine map h -> a h + b; maps compose as
// (A1, B1) then (A2, B2) = (A1 A2, A2 B1 + B2), so time is scanned in parallel.
//
// One workgroup owns a tile of channels and walks its time segment in tiles of
// TG x R steps: a thread composes R consecutive steps of V channels, the
// thread groups' maps are scanned across lanes and waves, and every thread
// then runs its R steps again from its carry in. Inputs are read once, kept in
// registers between the two. Where batch x channels gives too few workgroups,
// time is cut into segments: a first launch composes each segment's map, the
// second starts each segment from the maps before it.
//
// Masked steps (t >= length) are the identity map; they are not read.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "seq.h"

namespace symnmf {
namespace {

// a = sigmoid(g) and c = sigmoid(-g), each to (8 + 2 |g|) 2^-24 relative: the
// exponential's argument is rounded once, its factor log2(e) is a float (1 - a
// would lose c where a is near 1). Below 2^-126 either may be 0, and a is 0 at
// g = -inf, where e is infinite and c is 1 by choice (NaN fails the comparison).
__device__ __forceinline__ void gates(float g, float& a, float& c) {
    const float e = __expf(-g);
    a = __builtin_amdgcn_rcpf(1.f + e);
    c = e > 1.2676506e30f ? 1.f : e * a;  // 2^100: 1 + e is e there
}

constexpr int kTileCh = 64;  // channels of a tile, unless the steps are few
constexpr int kTileT = 32;   // elements of a thread: R steps of V channels

struct Tile {       // how a workgroup's 256 threads lie over channels and time
    int cl_log2;    // threads over channels
    int nct;        // channel tiles
    int nseg;       // time segments
    int seg;        // steps per segment (a multiple of the tile's and of kScanChunk)
    int64_t items;  // nct x nseg x batch
    int64_t first;  // of this launch
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_or_zero(const T* p, bool on) {
    Vec<T, V> v;
    if (on) {
        v = load_vec<T, V>(p);
    } else {
#pragma unroll
        for (int u = 0; u < V; ++u) v.e[u] = from_f32<T>(0.f);
    }
    return v;
}

// Composition over the time groups of a workgroup. In: the thread's own map
// (A, B). Out: `in` the state before the thread's first step (h: the state
// before the tile's first step) and `next` the state after the tile. tot: the
// waves' maps, 2 x 4 x 64 V floats. DIR 1: groups in order of time; -1: from
// the last group to the first (the backward pass). Holds one barrier.
template <int V, int DIR>
__device__ __forceinline__ void scan_groups(float (&A)[V], float (&B)[V], const float (&h)[V],
                                            float (&in)[V], float (&next)[V], int cl_log2,
                                            float* tot) {
    constexpr int S = 64 * V;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int cl = cl_log2 < 6 ? 1 << cl_log2 : 64;   // lanes over channels
    const int wide = cl_log2 < 6 ? 1 : 1 << (cl_log2 - 6);  // waves over channels
    auto from = [&](float v, int o) {
        return DIR > 0 ? __shfl_up(v, o, 64) : __shfl_down(v, o, 64);
    };
    // lanes that have an earlier group `o` lanes away
    auto has = [&](int o) { return DIR > 0 ? lane >= o : lane + o < 64; };
    for (int o = cl; o < 64; o <<= 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const float pa = from(A[u], o), pb = from(B[u], o);
            if (has(o)) {
                B[u] = fmaf(A[u], pb, B[u]);
                A[u] *= pa;
            }
        }
    }
    const int ch = (lane & (cl - 1)) * V;
    float* ta = tot;  // [wave][channel]
    float* tb = tot + 4 * S;
    if (DIR > 0 ? lane >= 64 - cl : lane < cl) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            ta[w * S + ch + u] = A[u];
            tb[w * S + ch + u] = B[u];
        }
    }
    float ea[V], eb[V];  // the map of the wave's earlier groups
#pragma unroll
    for (int u = 0; u < V; ++u) {
        ea[u] = 1.f;
        eb[u] = 0.f;
        if (cl < 64) {
            const float pa = from(A[u], cl), pb = from(B[u], cl);
            if (has(cl)) {
                ea[u] = pa;
                eb[u] = pb;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < V; ++u) next[u] = in[u] = h[u];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = DIR > 0 ? i : 3 - i;
        if ((k ^ w) & (wide - 1)) continue;  // other channels
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if (k == w) in[u] = fmaf(ea[u], next[u], eb[u]);
            next[u] = fmaf(ta[k * S + ch + u], next[u], tb[k * S + ch + u]);
        }
    }
}

// The state a segment starts from: h0 through the maps of the segments before
// it (after it, for DIR -1), which the time groups compose between them.
template <int V, int DIR>
__device__ __forceinline__ void segment_start(float (&h)[V], const float* __restrict__ agg,
                                              int64_t lanes, int64_t at, bool on, int seg,
                                              const Tile& tl, int grp, float* tot) {
    const int tg = 256 >> tl.cl_log2;
    const int per = (tl.nseg + tg - 1) / tg;
    float A[V], B[V], in[V], next[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        A[u] = 1.f;
        B[u] = 0.f;
    }
    for (int i = 0; i < per; ++i) {
        const int s = DIR > 0 ? grp * per + i : grp * per + per - 1 - i;
        if (on && s < tl.nseg && (DIR > 0 ? s < seg : s > seg)) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const float a = agg[2 * s * lanes + at + u];
                B[u] = fmaf(a, B[u], agg[(2 * s + 1) * lanes + at + u]);
                A[u] *= a;
            }
        }
    }
    scan_groups<V, DIR>(A, B, h, in, next, tl.cl_log2, tot);
#pragma unroll
    for (int u = 0; u < V; ++u) h[u] = next[u];
}

// p + stride, kept from being rewritten as one of R multiples of the stride,
// which would take more scalar registers than there are.
template <class T>
__device__ __forceinline__ T* next_step(T* p, int64_t stride) {
    asm("" : "+s"(stride));
    return p + stride;
}

// R steps of V channels from `p` on, `stride` apart; ALL: every step is there,
// else those at and past `lim` (the first step being ts) are zeros. The addresses
// are one pointer per thread, moved on by a stride that the workgroup shares.
template <class T, int V, int R, bool ALL>
__device__ __forceinline__ void load_steps(Vec<T, V> (&v)[R], const T* p, int64_t stride, int ts,
                                           int lim) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = ALL ? load_vec<T, V>(p) : load_or_zero<T, V>(p, ts + r < lim);
        p = next_step(p, stride);
    }
}

// Where a workgroup works, for the kernels below. `back`: from the last item to
// the first, so that the second launch of a scan cut in time begins with what
// the first has just read (the last 256 MB of it may still be in the cache).
struct Place {
    int seg, c0, grp, t_lo, t_hi, lim;  // lim: the first step that is not taken
    int64_t b, at, lanes;
    bool on;
};
template <int V>
__device__ __forceinline__ Place place(const ScanArgs& p, const Tile& tl, bool back) {
    Place q;
    const int64_t nth = tl.first + (int64_t)blockIdx.x;
    const int64_t item = back ? tl.items - 1 - nth : nth;
    const int cl = 1 << tl.cl_log2;
    const int ct = (int)(item % tl.nct);
    q.seg = (int)(item / tl.nct % tl.nseg);
    q.b = item / tl.nct / tl.nseg;
    q.c0 = (ct * cl + (threadIdx.x & (cl - 1))) * V;
    q.grp = threadIdx.x >> tl.cl_log2;
    q.on = q.c0 < p.width;
    // a row's last lane ends with the row: the channels that it shares with the
    // lane before it come out the same from both
    q.c0 = min(q.c0, (int)p.width - V);
    q.t_lo = q.seg * tl.seg;
    q.t_hi = min((int)p.steps, q.t_lo + tl.seg);
    const int len = p.lengths ? min(max(p.lengths[q.b], 0), (int)p.steps) : (int)p.steps;
    q.lim = min(len, q.t_hi);
    q.lanes = p.batch * p.width;
    q.at = q.b * p.width + q.c0;
    return q;
}

// MODE 0: the outputs; 1: only the segment's map, to agg (per segment A, then
// B, batch x width each). CG: the gate does not change over time (stride 0), so
// it is read, and its sigmoid taken, once.
//
// Four waves per SIMD are asked of the compiler where it misses them by little: it
// then keeps two registers of the fp32 outputs' kernel in scratch, 12 bytes a lane
// (250 x 100000 fp32, one decay a channel: 42.0 us against 43.9). Elsewhere it would
// spill far more.
template <class T, int V, int MODE, bool CG>
__global__ __launch_bounds__(256, CG && sizeof(T) == 4 && V > 1 ? 4 : 1) void scan_kernel(ScanArgs p, Tile tl, float* __restrict__ agg) {
    constexpr int R = kTileT / V;
    __shared__ float tot[2][2 * 4 * 64 * V];
    const Place q = place<V>(p, tl, MODE == 0 && tl.nseg > 1);
    const int tt = (256 >> tl.cl_log2) * R;
    const bool on = q.on;
    const T* x = (const T*)p.x + q.b * p.x_b + q.c0;
    const T* g = (const T*)p.gate + q.b * p.g_b + q.c0;
    float h[V], prodA[V], ca[V], cc[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        h[u] = MODE == 0 && on && p.h0 ? p.h0[q.at + u] : 0.f;
        prodA[u] = 1.f;
        ca[u] = cc[u] = 0.f;
    }
    if (CG && on && q.lim > q.t_lo) {
        const Vec<T, V> v = load_vec<T, V>(g);
#pragma unroll
        for (int u = 0; u < V; ++u) gates(to_f32(v.e[u]), ca[u], cc[u]);
    }
    if (MODE == 0 && q.seg > 0)
        segment_start<V, 1>(h, agg, q.lanes, q.at, on, q.seg, tl, q.grp, tot[1]);

    // lanes past the width read what the last one reads, and write nothing
    Vec<T, V> xv[R], gv[CG ? 1 : R];
    const T* px = x + (int64_t)(q.t_lo + q.grp * R) * p.x_t;
    const T* pg = g + (int64_t)(q.t_lo + q.grp * R) * p.g_t;
    T* po = (T*)p.h + (q.b * p.steps + q.t_lo + q.grp * R) * p.width + q.c0;
    auto fetch = [&](int t0) {
        const int ts = t0 + q.grp * R;
        if (t0 + tt <= q.lim) {
            load_steps<T, V, R, true>(xv, px, p.x_t, ts, q.lim);
            if constexpr (!CG) load_steps<T, V, R, true>(gv, pg, p.g_t, ts, q.lim);
        } else {
            load_steps<T, V, R, false>(xv, px, p.x_t, ts, q.lim);
            if constexpr (!CG) load_steps<T, V, R, false>(gv, pg, p.g_t, ts, q.lim);
        }
        px += tt * p.x_t;
        pg += tt * p.g_t;
    };
    int buf = 0;
    fetch(q.t_lo);
    for (int t0 = q.t_lo; t0 < q.t_hi; t0 += tt, buf ^= 1) {
        const int ts = t0 + q.grp * R;
        float a[R][V], bb[R][V], A[V], B[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            A[u] = 1.f;
            B[u] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < V; ++u) {
                float c = cc[u];
                a[r][u] = ca[u];
                if (!CG) gates(to_f32(gv[CG ? 0 : r].e[u]), a[r][u], c);
                bb[r][u] = c * to_f32(xv[r].e[u]);
            }
        fetch(t0 + tt);  // the next tile's, while this one is composed
        if (t0 + tt > q.lim) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < V; ++u)
                    if (ts + r >= q.lim) {
                        a[r][u] = 1.f;
                        bb[r][u] = 0.f;
                    }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < V; ++u) {
                A[u] *= a[r][u];
                B[u] = fmaf(a[r][u], B[u], bb[r][u]);
            }
        float in[V], next[V];
        scan_groups<V, 1>(A, B, h, in, next, tl.cl_log2, tot[buf]);
        if (MODE == 1) {
            // (a scan cut in time has all four waves on the same channels)
            const int ch = (threadIdx.x & ((1 << tl.cl_log2) - 1)) * V;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int u = 0; u < V; ++u) prodA[u] *= tot[buf][k * 64 * V + ch + u];
        } else if (on) {
            if (p.states && ts % kScanChunk == 0 && ts < p.steps) {
                const int64_t nst = (p.steps + kScanChunk - 1) / kScanChunk;
                float* s = p.states + (q.b * nst + ts / kScanChunk) * p.width + q.c0;
#pragma unroll
                for (int u = 0; u < V; ++u) s[u] = in[u];
            }
            auto put = [&](auto masked) {
                T* o = po;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Vec<T, V> v;
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        in[u] = fmaf(a[r][u], in[u], bb[r][u]);
                        v.e[u] = from_f32<T>(!masked || ts + r < q.lim ? in[u] : 0.f);
                    }
                    if (!masked || ts + r < q.t_hi) store_vec<T, V>(o, v);
                    o = next_step(o, p.width);
                }
            };
            if (t0 + tt <= q.lim)
                put(std::false_type{});
            else
                put(std::true_type{});
            po += tt * p.width;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) h[u] = next[u];
    }
    if (!on || q.grp != 0) return;
    if (MODE == 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            agg[2 * q.seg * q.lanes + q.at + u] = prodA[u];
            agg[(2 * q.seg + 1) * q.lanes + q.at + u] = h[u];
        }
    } else if (p.last && q.seg == tl.nseg - 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) p.last[q.at + u] = h[u];
    }
}

// A few steps of many channels (live streams): a thread walks the steps of V
// channels one after another, all reads of kWalk steps on their way first.
constexpr int kWalk = 4;
template <class T, int V>
__global__ __launch_bounds__(256) void scan_walk_kernel(ScanArgs p, int64_t first) {
    const int64_t nv = p.width / V;  // V divides the width: the state may be updated in place
    const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.batch * nv) return;
    const int64_t b = i / nv, c0 = (i - b * nv) * V, at = b * p.width + c0;
    const T* x = (const T*)p.x + b * p.x_b + c0;
    const T* g = (const T*)p.gate + b * p.g_b + c0;
    T* o = (T*)p.h + b * p.steps * p.width + c0;
    const int steps = (int)p.steps;
    const int len = p.lengths ? min(max(p.lengths[b], 0), steps) : steps;
    const int64_t nst = (p.steps + kScanChunk - 1) / kScanChunk;
    float h[V];
#pragma unroll
    for (int u = 0; u < V; ++u) h[u] = p.h0 ? p.h0[at + u] : 0.f;
    for (int t0 = 0; t0 < steps; t0 += kWalk) {
        Vec<T, V> xv[kWalk], gv[kWalk];
#pragma unroll
        for (int r = 0; r < kWalk; ++r) {
            xv[r] = load_or_zero<T, V>(x + (int64_t)(t0 + r) * p.x_t, t0 + r < len);
            gv[r] = load_or_zero<T, V>(g + (int64_t)(t0 + r) * p.g_t, t0 + r < len);
        }
        if (p.states && t0 % kScanChunk == 0)
#pragma unroll
            for (int u = 0; u < V; ++u)
                p.states[(b * nst + t0 / kScanChunk) * p.width + c0 + u] = h[u];
#pragma unroll
        for (int r = 0; r < kWalk; ++r) {
            const bool in = t0 + r < len;
            Vec<T, V> v;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                float a, c;
                gates(to_f32(gv[r].e[u]), a, c);
                if (in) h[u] = fmaf(a, h[u], c * to_f32(xv[r].e[u]));
                v.e[u] = from_f32<T>(in ? h[u] : 0.f);
            }
            if (t0 + r < steps) store_vec<T, V>(o + (int64_t)(t0 + r) * p.width, v);
        }
    }
    if (p.last)
#pragma unroll
        for (int u = 0; u < V; ++u) p.last[at + u] = h[u];
}

// Backward. With lam_t the gradient at h_t from everything after step t's
// output, m_t = a_t lam_t flows to h_{t-1}:
//   lam_t = dh_t + m_{t+1} (m past the end: dlast), m_t = a_t (dh_t + m_{t+1})
//   dx_t = lam_t c_t, dgate_t = lam_t (h_{t-1} - x_t) a_t c_t, dh0 = m_0.
// A segment is walked from its end, tile by tile; h_{t-1} is rebuilt in fp32
// from the state kept at the tile's first step (a multiple of kScanChunk), so
// the forward's rounded output is neither read nor trusted.
template <class T, int V, int MODE>
__global__ __launch_bounds__(256) void scan_grad_kernel(ScanArgs p, Tile tl,
                                                        float* __restrict__ agg) {
    constexpr int R = kTileT / V;
    __shared__ float tot[2][2 * 4 * 64 * V];
    __shared__ float rtot[2][2 * 4 * 64 * V];
    const Place q = place<V>(p, tl, MODE == 0 && tl.nseg > 1);
    const int tt = (256 >> tl.cl_log2) * R;
    const bool on = q.on;
    const int64_t nst = (p.steps + kScanChunk - 1) / kScanChunk;
    const T* x = (const T*)p.x + q.b * p.x_b + q.c0;
    const T* g = (const T*)p.gate + q.b * p.g_b + q.c0;
    const T* d = (const T*)p.dh + q.b * p.d_b + q.c0;
    float m[V], prodA[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        m[u] = MODE == 0 && on && p.dlast ? p.dlast[q.at + u] : 0.f;
        prodA[u] = 1.f;
    }
    if (MODE == 0 && q.seg < tl.nseg - 1)
        segment_start<V, -1>(m, agg, q.lanes, q.at, on, q.seg, tl, q.grp, rtot[1]);

    Vec<T, V> xv[R], gv[R], dv[R];
    float hs[V];
    // The tiles that hold a step that counts; those after them are zeros, and m
    // passes them (8 x 2048 x 2048 bf16, ragged: 72.5 us, walked like the others 82.0).
    const int ntile = q.lim > q.t_lo ? (q.lim - q.t_lo + tt - 1) / tt : 0;
    if (MODE == 0 && on) {
        Vec<T, V> zero;
#pragma unroll
        for (int u = 0; u < V; ++u) zero.e[u] = from_f32<T>(0.f);
        for (int t = q.t_lo + ntile * tt + q.grp; t < q.t_hi; t += 256 >> tl.cl_log2) {
            const int64_t to = (q.b * p.steps + t) * p.width + q.c0;
            store_vec<T, V>((T*)p.dx + to, zero);
            store_vec<T, V>((T*)p.dgate + to, zero);
        }
    }
    const int64_t t_end = q.t_lo + (ntile - 1) * (int64_t)tt + q.grp * R;  // in the last tile
    const T* px = x + t_end * p.x_t;
    const T* pg = g + t_end * p.g_t;
    const T* pd = d + t_end * p.d_t;
    T* ox = (T*)p.dx + (q.b * p.steps + t_end) * p.width + q.c0;
    T* og = (T*)p.dgate + (q.b * p.steps + t_end) * p.width + q.c0;
    auto fetch = [&](int t0) {
        const int ts = t0 + q.grp * R;
        if (t0 < q.t_lo) return;
        if (t0 + tt <= q.lim) {
            load_steps<T, V, R, true>(gv, pg, p.g_t, ts, q.lim);
            load_steps<T, V, R, true>(dv, pd, p.d_t, ts, q.lim);
            if (MODE == 0) load_steps<T, V, R, true>(xv, px, p.x_t, ts, q.lim);
        } else {
            load_steps<T, V, R, false>(gv, pg, p.g_t, ts, q.lim);
            load_steps<T, V, R, false>(dv, pd, p.d_t, ts, q.lim);
            if (MODE == 0) load_steps<T, V, R, false>(xv, px, p.x_t, ts, q.lim);
        }
        if (MODE == 0)
#pragma unroll
            for (int u = 0; u < V; ++u)
                hs[u] = p.states[(q.b * nst + t0 / kScanChunk) * p.width + q.c0 + u];
        px -= tt * p.x_t;
        pg -= tt * p.g_t;
        pd -= tt * p.d_t;
    };
    int buf = 0;
    fetch(q.t_lo + (ntile - 1) * tt);
    for (int k = ntile - 1; k >= 0; --k, buf ^= 1) {
        const int t0 = q.t_lo + k * tt, ts = t0 + q.grp * R;
        float a[R][V], c[R][V], xf[R][V], df[R][V], A[V], B[V], D[V], h0[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            A[u] = 1.f;
            B[u] = D[u] = 0.f;
            h0[u] = hs[u];
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < V; ++u) {
                gates(to_f32(gv[r].e[u]), a[r][u], c[r][u]);
                df[r][u] = to_f32(dv[r].e[u]);
                if (MODE == 0) xf[r][u] = to_f32(xv[r].e[u]);
            }
        fetch(t0 - tt);  // the tile before, while this one is worked on
        if (t0 + tt > q.lim) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < V; ++u)
                    if (ts + r >= q.lim) {
                        a[r][u] = 1.f;
                        c[r][u] = 0.f;
                    }
        }
        // from the last step to the first: A is the product of the later a's when
        // it meets a step's c x
#pragma unroll
        for (int r = R - 1; r >= 0; --r)
#pragma unroll
            for (int u = 0; u < V; ++u) {
                if (MODE == 0) B[u] = fmaf(A[u], c[r][u] * xf[r][u], B[u]);
                D[u] = a[r][u] * (D[u] + df[r][u]);
                A[u] *= a[r][u];
            }
        float hin[V], hn[V], min_[V], mn[V], RA[V];
#pragma unroll
        for (int u = 0; u < V; ++u) RA[u] = A[u];
        if (MODE == 0) scan_groups<V, 1>(A, B, h0, hin, hn, tl.cl_log2, tot[buf]);
        scan_groups<V, -1>(RA, D, m, min_, mn, tl.cl_log2, rtot[buf]);
        if (MODE == 1) {
            const int ch = (threadIdx.x & ((1 << tl.cl_log2) - 1)) * V;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < V; ++u) prodA[u] *= rtot[buf][i * 64 * V + ch + u];
        } else if (on) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float before = hin[u] - xf[r][u];  // h_{t-1} - x_t
                    hin[u] = fmaf(a[r][u], hin[u], c[r][u] * xf[r][u]);
                    xf[r][u] = before;
                }
            auto put = [&](auto masked) {
                T* wx = ox + (R - 1) * p.width;
                T* wg = og + (R - 1) * p.width;
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    Vec<T, V> vx, vg;
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        const float lam = min_[u] + df[r][u];
                        const float lc = lam * c[r][u];
                        // by the step, not by its c of 0: what passes a masked
                        // step may be infinite or NaN
                        const bool in = !masked || ts + r < q.lim;
                        vx.e[u] = from_f32<T>(in ? lc : 0.f);
                        vg.e[u] = from_f32<T>(in ? lc * a[r][u] * xf[r][u] : 0.f);
                        min_[u] = a[r][u] * lam;
                    }
                    if (!masked || ts + r < q.t_hi) {
                        store_vec<T, V>(wx, vx);
                        store_vec<T, V>(wg, vg);
                    }
                    wx = next_step(wx, -p.width);
                    wg = next_step(wg, -p.width);
                }
            };
            if (t0 + tt <= q.lim)
                put(std::false_type{});
            else
                put(std::true_type{});
            ox -= tt * p.width;
            og -= tt * p.width;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) m[u] = mn[u];
    }
    if (!on || q.grp != 0) return;
    if (MODE == 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            agg[2 * q.seg * q.lanes + q.at + u] = prodA[u];
            agg[(2 * q.seg + 1) * q.lanes + q.at + u] = m[u];
        }
    } else if (p.dh0 && q.seg == 0) {
#pragma unroll
        for (int u = 0; u < V; ++u) p.dh0[q.at + u] = m[u];
    }
}

constexpr int kMaxSeg = 256;
// Workgroups below which a scan is cut in time, and as many as it is cut into. Cut,
// it reads its inputs twice but fills the chip (1 x 4096 steps, us uncut and cut:
// bf16 128 workgroups 86.6 and 66.7, 192 106.6 and 93.6, 224 112 and 115, 255 108 and
// 124; fp32 128 132 and 115, 192 142 and 184, 255 156 and 239). The backward reads
// three arrays and writes two, in fp32 with half the waves (bf16 128 135 and 89, 192
// 153 and 155, 255 141 and 175, fp32 64 154 and 91, 128 175 and 184, 255 252 and 344;
// 8 x 2048 x 2048 bf16 as 256: 80.2 us, cut into 512 86.0, into 1024 88.6).
constexpr int kCut = 192, kFill = 2048, kFillGrad = 1024;
constexpr int cut_grad(int bytes) { return bytes == 4 ? 128 : 192; }
constexpr int kWalkSteps = 8;  // up to these, steps are walked one by one

// Channels over threads: 64 channels to a tile, fewer where the width is smaller
// (the threads go to time instead), more where the steps are so few that the
// threads would have none.
Tile plan(int64_t batch, int64_t steps, int64_t width, int V, int cut, int fill) {
    Tile t;
    const int R = kTileT / V;
    t.cl_log2 = 0;
    while (t.cl_log2 < 8 && ((int64_t)V << t.cl_log2) < width &&
           ((V << t.cl_log2) < kTileCh || (int64_t)(128 >> t.cl_log2) * R >= steps))
        ++t.cl_log2;
    const int64_t cw = (int64_t)V << t.cl_log2;
    t.nct = (int)((width + cw - 1) / cw);
    const int64_t wg = batch * t.nct;
    const int64_t unit = (int64_t)(256 >> t.cl_log2) * R;  // a tile's steps
    const int64_t units = steps > 0 ? (steps + unit - 1) / unit : 1;
    // a cut costs a launch, about what two tiles take one after the other
    int64_t nseg = wg >= cut || units < 4 ? 1 : (fill + wg - 1) / wg;
    if (nseg > kMaxSeg) nseg = kMaxSeg;
    if (nseg > units) nseg = units;
    const int64_t per = (units + nseg - 1) / nseg;
    t.nseg = (int)((units + per - 1) / per);
    t.seg = (int)(per * unit);
    t.items = batch * t.nct * t.nseg;
    t.first = 0;
    return t;
}
// A tile has 256 x 32 elements. With 64 channels or fewer that is 128 steps or
// more and a multiple of 128; wider tiles hold all steps there are.
static_assert(256 * kTileT / kTileCh % kScanChunk == 0, "tiles start at kept states");

// kernel<<<items>>> of the plan, in as many launches as it takes.
template <class K>
hipError_t run_plan(K* kernel, const ScanArgs& a, Tile tl, hipStream_t st) {
    return in_launches(tl.items, [&](int64_t first, unsigned n) {
        tl.first = first;
        hipLaunchKernelGGL(kernel, dim3(n), dim3(256), 0, st, a, tl, (float*)a.ws);
    });
}
template <class T, int V, bool CG>
hipError_t scan_run(const ScanArgs& a, hipStream_t st) {
    const Tile tl = plan(a.batch, a.steps, a.width, V, kCut, kFill);
    if (tl.nseg > 1) {
        const hipError_t e = run_plan(scan_kernel<T, V, 1, CG>, a, tl, st);
        if (e != hipSuccess) return e;
    }
    return run_plan(scan_kernel<T, V, 0, CG>, a, tl, st);
}
template <class T, int V>
hipError_t walk_run(const ScanArgs& a, hipStream_t st) {
    return in_launches((a.batch * (a.width / V) + 255) / 256, [&](int64_t first, unsigned n) {
        hipLaunchKernelGGL((scan_walk_kernel<T, V>), dim3(n), dim3(256), 0, st, a, first);
    });
}
template <class T, int V>
hipError_t grad_run(const ScanArgs& a, hipStream_t st) {
    const Tile tl = plan(a.batch, a.steps, a.width, V, cut_grad(sizeof(T)), kFillGrad);
    if (tl.nseg > 1) {
        const hipError_t e = run_plan(scan_grad_kernel<T, V, 1>, a, tl, st);
        if (e != hipSuccess) return e;
    }
    return run_plan(scan_grad_kernel<T, V, 0>, a, tl, st);
}

// Channels to a lane, 8 bytes of them. 16 bytes put fewer steps into a thread and
// more maps into the scan across lanes, 4 bytes take more loads: 250 x 100000 fp32
// in 47.7 us, with 16 bytes in 68.5, with 4 in 50.5; 2 x 32768 x 1024 bf16 in 141.6,
// with 4 in 142.5. The backward holds more per element: 8 x 2048 x 2048 bf16 with 4
// bytes in 80.2 us, with 8 in 93.0.
template <class T>
hipError_t scan_vec(const ScanArgs& a, hipStream_t st) {
    constexpr int W = 16 / sizeof(T), V = 8 / sizeof(T);
    if (a.steps <= kWalkSteps) return a.width % W ? walk_run<T, 1>(a, st) : walk_run<T, W>(a, st);
    if (a.width >= V) return a.g_t ? scan_run<T, V, false>(a, st) : scan_run<T, V, true>(a, st);
    return a.g_t ? scan_run<T, 1, false>(a, st) : scan_run<T, 1, true>(a, st);
}
template <class T>
hipError_t grad_vec(const ScanArgs& a, hipStream_t st) {
    constexpr int V = 4 / sizeof(T);
    return a.width >= V ? grad_run<T, V>(a, st) : grad_run<T, 1>(a, st);
}

}  // namespace

// Two numbers per channel and time segment of the plan that has most (a plan that is
// cut has as many segments whatever it is cut below).
size_t scan_ws_bytes(int64_t batch, int64_t steps, int64_t width) {
    int64_t nseg = 1;
    for (int v : {1, 2, 4}) {
        nseg = std::max<int64_t>(nseg, plan(batch, steps, width, v, kCut, kFill).nseg);
        nseg = std::max<int64_t>(nseg, plan(batch, steps, width, v, cut_grad(2), kFillGrad).nseg);
    }
    return nseg > 1 ? 8 * (size_t)nseg * (size_t)batch * (size_t)width : 256;
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t st) {
    return a.type == kF32    ? scan_vec<float>(a, st)
           : a.type == kBF16 ? scan_vec<bf16_t>(a, st)
                             : scan_vec<f16_t>(a, st);
}
hipError_t launch_scan_grad(const ScanArgs& a, hipStream_t st) {
    return a.type == kF32    ? grad_vec<float>(a, st)
           : a.type == kBF16 ? grad_vec<bf16_t>(a, st)
                             : grad_vec<f16_t>(a, st);
}

}  // namespace symnmf
