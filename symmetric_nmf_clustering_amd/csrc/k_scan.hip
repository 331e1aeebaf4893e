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
#include "common.h"
#include "seq.h"

namespace symnmf {
namespace {

// a = sigmoid(g) and c = sigmoid(-g), each with full relative accuracy
// (1 - a would lose c's where a is near 1). exp(-g) is held below 2^100 so that
// c stays 1 where a underflows.
__device__ __forceinline__ void gates(float g, float& a, float& c) {
    const float e = fminf(__expf(-g), 1.2676506e30f);
    a = __builtin_amdgcn_rcpf(1.f + e);
    c = e * a;
}

constexpr int kTileCh = 64;  // most channels of a tile

struct Tile {       // how a workgroup's 256 threads lie over channels and time
    int cl_log2;    // lanes over channels (<= 64)
    int nct;        // channel tiles
    int nseg;       // time segments
    int seg;        // steps per segment (a multiple of the tile's and of kScanChunk)
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
// (A, B). Out: `h` becomes the state before the thread's first step (h: the
// state before the tile's first step) and `next` the state after the tile.
// tot: the waves' maps, 2 x 4 x kTileCh floats.
template <int V>
__device__ __forceinline__ void scan_groups(float (&A)[V], float (&B)[V], const float (&h)[V],
                                            float (&in)[V], float (&next)[V], int cl_log2,
                                            float* tot) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, cl = 1 << cl_log2;
    for (int o = cl; o < 64; o <<= 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const float pa = __shfl_up(A[u], o, 64), pb = __shfl_up(B[u], o, 64);
            if (lane >= o) {
                B[u] = fmaf(A[u], pb, B[u]);
                A[u] *= pa;
            }
        }
    }
    const int ch = (lane & (cl - 1)) * V;
    float* ta = tot;                 // [wave][channel]
    float* tb = tot + 4 * kTileCh;
    if (lane >= 64 - cl) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            ta[w * kTileCh + ch + u] = A[u];
            tb[w * kTileCh + ch + u] = B[u];
        }
    }
    float ea[V], eb[V];  // the map of the wave's earlier groups
#pragma unroll
    for (int u = 0; u < V; ++u) {
        ea[u] = cl < 64 ? __shfl_up(A[u], cl, 64) : 1.f;
        eb[u] = cl < 64 ? __shfl_up(B[u], cl, 64) : 0.f;
        if (lane < cl) {
            ea[u] = 1.f;
            eb[u] = 0.f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < V; ++u) next[u] = in[u] = h[u];
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if (k == w) in[u] = fmaf(ea[u], next[u], eb[u]);
            next[u] = fmaf(ta[k * kTileCh + ch + u], next[u], tb[k * kTileCh + ch + u]);
        }
    }
}

// MODE 0: the outputs; 1: only the segment's map, to agg (A at 0, B at `lane`
// stride batch x width, per segment).
template <class T, int V, int R, int MODE>
__global__ __launch_bounds__(256) void scan_kernel(ScanArgs p, Tile tl, float* __restrict__ agg) {
    __shared__ float tot[2][2 * 4 * kTileCh];
    const int cl = 1 << tl.cl_log2, tg = 256 >> tl.cl_log2;
    const int ct = blockIdx.x % tl.nct, seg = blockIdx.x / tl.nct, b = blockIdx.y;
    const int c0 = (ct * cl + (threadIdx.x & (cl - 1))) * V;
    const int grp = threadIdx.x >> tl.cl_log2;
    const bool on = c0 < p.width;  // V divides the width (or is 1)
    const int tt = tg * R;
    const int t_lo = seg * tl.seg;
    const int t_hi = min((int)p.steps, t_lo + tl.seg);
    const int len = p.lengths ? min(max(p.lengths[b], 0), (int)p.steps) : (int)p.steps;
    const int64_t lanes = p.batch * p.width, at = (int64_t)b * p.width + c0;
    const T* x = (const T*)p.x + b * p.x_b + c0;
    const T* g = (const T*)p.gate + b * p.g_b + c0;
    float h[V], prodA[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        h[u] = MODE == 0 && on && p.h0 ? p.h0[at + u] : 0.f;
        prodA[u] = 1.f;
    }
    if (MODE == 0 && on)
        for (int s = 0; s < seg; ++s)
#pragma unroll
            for (int u = 0; u < V; ++u)
                h[u] = fmaf(agg[(2 * (int64_t)s) * lanes + at + u], h[u],
                            agg[(2 * (int64_t)s + 1) * lanes + at + u]);
    int buf = 0;
    for (int t0 = t_lo; t0 < t_hi; t0 += tt, buf ^= 1) {
        const int ts = t0 + grp * R;
        float a[R][V], bb[R][V], A[V], B[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            A[u] = 1.f;
            B[u] = 0.f;
        }
        Vec<T, V> xv[R], gv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = on && ts + r < len && ts + r < t_hi;
            xv[r] = load_or_zero<T, V>(x + (int64_t)(ts + r) * p.x_t, in);
            gv[r] = load_or_zero<T, V>(g + (int64_t)(ts + r) * p.g_t, in);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = ts + r < len && ts + r < t_hi;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                float c;
                gates(to_f32(gv[r].e[u]), a[r][u], c);
                bb[r][u] = c * to_f32(xv[r].e[u]);
                if (!in) {
                    a[r][u] = 1.f;
                    bb[r][u] = 0.f;
                }
                A[u] *= a[r][u];
                B[u] = fmaf(a[r][u], B[u], bb[r][u]);
            }
        }
        float in0[V], next[V];
        scan_groups<V>(A, B, h, in0, next, tl.cl_log2, tot[buf]);
        if (MODE == 1) {
            const int ch = (threadIdx.x & (cl - 1)) * V;
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int u = 0; u < V; ++u) prodA[u] *= tot[buf][k * kTileCh + ch + u];
        } else if (on) {
            if (p.states && ts % kScanChunk == 0 && ts < p.steps) {
                const int64_t nst = (p.steps + kScanChunk - 1) / kScanChunk;
                float* s = p.states + ((int64_t)b * nst + ts / kScanChunk) * p.width + c0;
#pragma unroll
                for (int u = 0; u < V; ++u) s[u] = in0[u];
            }
            T* o = (T*)p.h + ((int64_t)b * p.steps + ts) * p.width + c0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (ts + r >= t_hi) break;
                Vec<T, V> v;
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    in0[u] = fmaf(a[r][u], in0[u], bb[r][u]);
                    v.e[u] = from_f32<T>(ts + r < len ? in0[u] : 0.f);
                }
                store_vec<T, V>(o + (int64_t)r * p.width, v);
            }
        }
#pragma unroll
        for (int u = 0; u < V; ++u) h[u] = next[u];
    }
    if (!on || grp != 0) return;
    if (MODE == 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            agg[(2 * (int64_t)seg) * lanes + at + u] = prodA[u];
            agg[(2 * (int64_t)seg + 1) * lanes + at + u] = h[u];
        }
    } else if (p.last && seg == tl.nseg - 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) p.last[at + u] = h[u];
    }
}

// Backward. With lam_t the gradient at h_t from everything after step t's
// output, m_t = a_t lam_t flows to h_{t-1}:
//   lam_t = dh_t + m_{t+1} (m past the end: dlast), m_t = a_t (dh_t + m_{t+1})
//   dx_t = lam_t c_t, dgate_t = lam_t (h_{t-1} - x_t) a_t c_t, dh0 = m_0.
// A segment is walked from its end, tile by tile; h_{t-1} is rebuilt in fp32
// from the state kept at the tile's first step (a multiple of kScanChunk), so
// the forward's rounded output is neither read nor trusted.
template <class T, int V, int R, int MODE>
__global__ __launch_bounds__(256) void scan_grad_kernel(ScanArgs p, Tile tl,
                                                        float* __restrict__ agg) {
    __shared__ float tot[2][2 * 4 * kTileCh];
    __shared__ float rtot[2][2 * 4 * kTileCh];
    const int cl = 1 << tl.cl_log2, tg = 256 >> tl.cl_log2;
    const int ct = blockIdx.x % tl.nct, seg = blockIdx.x / tl.nct, b = blockIdx.y;
    const int c0 = (ct * cl + (threadIdx.x & (cl - 1))) * V;
    const int grp = threadIdx.x >> tl.cl_log2;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int ch = (lane & (cl - 1)) * V;
    const bool on = c0 < p.width;
    const int tt = tg * R;
    const int t_lo = seg * tl.seg;
    const int t_hi = min((int)p.steps, t_lo + tl.seg);
    const int len = p.lengths ? min(max(p.lengths[b], 0), (int)p.steps) : (int)p.steps;
    const int64_t lanes = p.batch * p.width, at = (int64_t)b * p.width + c0;
    const int64_t nst = (p.steps + kScanChunk - 1) / kScanChunk;
    const T* x = (const T*)p.x + b * p.x_b + c0;
    const T* g = (const T*)p.gate + b * p.g_b + c0;
    const T* d = (const T*)p.dh + b * p.d_b + c0;
    float m[V], prodA[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        m[u] = MODE == 0 && on && p.dlast ? p.dlast[at + u] : 0.f;
        prodA[u] = 1.f;
    }
    if (MODE == 0 && on)
        for (int s = tl.nseg - 1; s > seg; --s)
#pragma unroll
            for (int u = 0; u < V; ++u)
                m[u] = fmaf(agg[(2 * (int64_t)s) * lanes + at + u], m[u],
                            agg[(2 * (int64_t)s + 1) * lanes + at + u]);
    const int ntile = (t_hi - t_lo + tt - 1) / tt;
    int buf = 0;
    for (int k = ntile - 1; k >= 0; --k, buf ^= 1) {
        const int t0 = t_lo + k * tt, ts = t0 + grp * R;
        Vec<T, V> xv[R], gv[R], dv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = on && ts + r < len && ts + r < t_hi;
            gv[r] = load_or_zero<T, V>(g + (int64_t)(ts + r) * p.g_t, in);
            dv[r] = load_or_zero<T, V>(d + (int64_t)(ts + r) * p.d_t, in);
            if (MODE == 0) xv[r] = load_or_zero<T, V>(x + (int64_t)(ts + r) * p.x_t, in);
        }
        float a[R][V], c[R][V], A[V], B[V], D[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            A[u] = 1.f;
            B[u] = D[u] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = ts + r < len && ts + r < t_hi;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                gates(to_f32(gv[r].e[u]), a[r][u], c[r][u]);
                if (!in) {
                    a[r][u] = 1.f;
                    c[r][u] = 0.f;
                }
                A[u] *= a[r][u];
                if (MODE == 0) B[u] = fmaf(a[r][u], B[u], c[r][u] * to_f32(xv[r].e[u]));
            }
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r)
#pragma unroll
            for (int u = 0; u < V; ++u) D[u] = a[r][u] * (D[u] + to_f32(dv[r].e[u]));
        // reverse composition over the groups: suffix maps across lanes, then waves
        float RA[V], RD[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            RA[u] = A[u];
            RD[u] = D[u];
        }
        for (int o = cl; o < 64; o <<= 1) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const float pa = __shfl_down(RA[u], o, 64), pd = __shfl_down(RD[u], o, 64);
                if (lane + o < 64) {
                    RD[u] = fmaf(RA[u], pd, RD[u]);
                    RA[u] *= pa;
                }
            }
        }
        float* ra = rtot[buf];
        float* rd = rtot[buf] + 4 * kTileCh;
        if (lane < cl) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                ra[w * kTileCh + ch + u] = RA[u];
                rd[w * kTileCh + ch + u] = RD[u];
            }
        }
        float ea[V], ed[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            ea[u] = cl < 64 ? __shfl_down(RA[u], cl, 64) : 1.f;
            ed[u] = cl < 64 ? __shfl_down(RD[u], cl, 64) : 0.f;
            if (lane >= 64 - cl) {
                ea[u] = 1.f;
                ed[u] = 0.f;
            }
        }
        float hs[V], hin[V], hn[V];
        if (MODE == 0) {
#pragma unroll
            for (int u = 0; u < V; ++u)
                hs[u] = on ? p.states[((int64_t)b * nst + t0 / kScanChunk) * p.width + c0 + u]
                           : 0.f;
            scan_groups<V>(A, B, hs, hin, hn, tl.cl_log2, tot[buf]);  // holds the barrier
        } else {
            __syncthreads();
        }
        float min_[V];
#pragma unroll
        for (int u = 0; u < V; ++u) min_[u] = m[u];
        for (int q = 3; q >= 0; --q) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                if (q == w) min_[u] = fmaf(ea[u], m[u], ed[u]);
                m[u] = fmaf(ra[q * kTileCh + ch + u], m[u], rd[q * kTileCh + ch + u]);
                if (MODE == 1) prodA[u] *= ra[q * kTileCh + ch + u];
            }
        }
        if (MODE == 0 && on) {
            float hp[R][V];  // h_{t-1}
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    hp[r][u] = hin[u];
                    hin[u] = fmaf(a[r][u], hin[u], c[r][u] * to_f32(xv[r].e[u]));
                }
            T* ox = (T*)p.dx + ((int64_t)b * p.steps + ts) * p.width + c0;
            T* og = (T*)p.dgate + ((int64_t)b * p.steps + ts) * p.width + c0;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                Vec<T, V> vx, vg;
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float lam = min_[u] + to_f32(dv[r].e[u]);
                    const float lc = lam * c[r][u];
                    vx.e[u] = from_f32<T>(lc);
                    vg.e[u] = from_f32<T>(lc * a[r][u] * (hp[r][u] - to_f32(xv[r].e[u])));
                    min_[u] = a[r][u] * lam;
                }
                if (ts + r < t_hi) {
                    store_vec<T, V>(ox + (int64_t)r * p.width, vx);
                    store_vec<T, V>(og + (int64_t)r * p.width, vg);
                }
            }
        }
    }
    if (!on || grp != 0) return;
    if (MODE == 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            agg[(2 * (int64_t)seg) * lanes + at + u] = prodA[u];
            agg[(2 * (int64_t)seg + 1) * lanes + at + u] = m[u];
        }
    } else if (p.dh0 && seg == 0) {
#pragma unroll
        for (int u = 0; u < V; ++u) p.dh0[at + u] = m[u];
    }
}

constexpr int kMaxSeg = 64;
constexpr int kFill = 512;  // workgroups that fill the chip

// Channels over lanes: 64 channels to a tile, fewer where the width is smaller
// (the lanes go to time instead).
Tile plan(int64_t batch, int64_t steps, int64_t width, int V, int R) {
    Tile t;
    const int most = V == 1 ? 4 : (V == 4 ? 4 : 3);
    t.cl_log2 = 0;
    while (t.cl_log2 < most && ((int64_t)V << t.cl_log2) < width) ++t.cl_log2;
    const int64_t cw = (int64_t)V << t.cl_log2;
    t.nct = (int)((width + cw - 1) / cw);
    const int64_t wg = batch * t.nct;
    int64_t unit = (int64_t)(256 >> t.cl_log2) * R;
    while (unit % kScanChunk) unit *= 2;
    const int64_t units = steps > 0 ? (steps + unit - 1) / unit : 1;
    int64_t nseg = wg >= kFill ? 1 : (kFill + wg - 1) / wg;
    if (nseg > kMaxSeg) nseg = kMaxSeg;
    if (nseg > units / 2) nseg = units / 2 > 0 ? units / 2 : 1;
    const int64_t per = (units + nseg - 1) / nseg;
    t.nseg = (int)((units + per - 1) / per);
    t.seg = (int)(per * unit);
    return t;
}

template <class T, int V, int R>
hipError_t scan_run(const ScanArgs& a, hipStream_t st) {
    const Tile tl = plan(a.batch, a.steps, a.width, V, R);
    const dim3 g((unsigned)(tl.nct * tl.nseg), (unsigned)a.batch);
    if (tl.nseg > 1) {
        hipLaunchKernelGGL((scan_kernel<T, V, R, 1>), g, dim3(256), 0, st, a, tl, (float*)a.ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((scan_kernel<T, V, R, 0>), g, dim3(256), 0, st, a, tl, (float*)a.ws);
    return hipGetLastError();
}
template <class T, int V, int R>
hipError_t grad_run(const ScanArgs& a, hipStream_t st) {
    const Tile tl = plan(a.batch, a.steps, a.width, V, R);
    const dim3 g((unsigned)(tl.nct * tl.nseg), (unsigned)a.batch);
    if (tl.nseg > 1) {
        hipLaunchKernelGGL((scan_grad_kernel<T, V, R, 1>), g, dim3(256), 0, st, a, tl,
                           (float*)a.ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((scan_grad_kernel<T, V, R, 0>), g, dim3(256), 0, st, a, tl, (float*)a.ws);
    return hipGetLastError();
}

bool vec_ok(const void* p, int64_t sb, int64_t st, int bytes, int v) {
    return reinterpret_cast<uintptr_t>(p) % (size_t)(bytes * v) == 0 && sb % v == 0 && st % v == 0;
}

template <class T>
hipError_t scan_vec(const ScanArgs& a, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (a.width % V == 0 && vec_ok(a.x, a.x_b, a.x_t, sizeof(T), V) &&
        vec_ok(a.gate, a.g_b, a.g_t, sizeof(T), V) && vec_ok(a.h, 0, 0, sizeof(T), V))
        return scan_run<T, V, 8>(a, st);
    return scan_run<T, 1, 8>(a, st);
}
template <class T>
hipError_t grad_vec(const ScanArgs& a, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (a.width % V == 0 && vec_ok(a.x, a.x_b, a.x_t, sizeof(T), V) &&
        vec_ok(a.gate, a.g_b, a.g_t, sizeof(T), V) && vec_ok(a.dh, a.d_b, a.d_t, sizeof(T), V) &&
        vec_ok(a.dx, 0, 0, sizeof(T), V) && vec_ok(a.dgate, 0, 0, sizeof(T), V))
        return grad_run<T, V, V == 8 ? 4 : 8>(a, st);
    return grad_run<T, 1, 8>(a, st);
}

}  // namespace

// Two numbers per channel and time segment, for as many segments as plan() can
// make: each holds two units or more, a unit kScanChunk steps or more.
size_t scan_ws_bytes(int64_t batch, int64_t steps, int64_t width) {
    int64_t nseg = (steps + kScanChunk - 1) / kScanChunk / 2;
    if (nseg > kMaxSeg) nseg = kMaxSeg;
    if (nseg < 2) return 256;
    return (size_t)(2 * nseg) * 4 * (size_t)batch * (size_t)width;
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
