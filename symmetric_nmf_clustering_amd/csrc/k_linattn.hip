// Linear attention with a decay for each head: plans of the walks (linattn.h), the
// join of time segments, sums over shared heads, and the step of a live stream.
#include "layers.h"
#include "linattn.h"

namespace symnmf {

namespace {

// ---- segments ------------------------------------------------------------------

// Few heads are cut in time: every segment's own state first (maps), then their
// join, then all segments walk at once, each from its state. That reads y and z
// twice, so time is cut only where heads and column tiles make less than 192
// workgroups, and into no more segments than two workgroups a CU, which run at once
// (192 workgroups of 2048 steps: 156 us whole, 197 cut in two; 160: 148 us whole or in
// three; 128: 125 us in four, 147 whole). Two segments do not pay for the launches (2 x 512
// steps of 8 heads of 64: 26 us whole, 30 in two, 23 in four), nor do short ones.
constexpr int kEnough = 192, kMost = 512;       // workgroups
constexpr int64_t kLeast = 128, kFewest = 3;    // steps of a segment, segments

int64_t plan_segments(const AttendDesc& d, int runs, int64_t* seg_len) {
    const int wide = d.dk > d.dv ? d.dk : d.dv;
    const int cols = wide > 64 && wide <= 128 && d.type != kF32 ? 128 : 64;
    const int64_t items = d.batch * d.heads * ((wide + cols - 1) / cols) * runs;
    int64_t n = items >= kEnough ? 1 : kMost / items;
    const int64_t most = d.steps / kLeast;
    if (n > most) n = most;
    if (n < kFewest) n = 1;
    int64_t len = (d.steps + n - 1) / n;
    len = (len + 63) / 64 * 64;
    if (len < 64) len = 64;
    *seg_len = len;
    n = (d.steps + len - 1) / len;
    return n < 1 ? 1 : n;
}

// Slot i of a head's segments holds the state that segment i makes from nothing, and
// receives the state it starts from: X_0 = s0, X_{i+1} = a^n_i X_i + L_i. A thread
// takes V neighbouring elements; sixteen segments' are asked for together (32 segments of
// 16 heads of 128 x 128, 67 MB: 14.2 us).
template <int V>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int64_t first,
                                                          int tiles) {
    const AttendRun& R = a.run[blockIdx.y];
    const int64_t id = first + blockIdx.x, bh = id / tiles, b = bh / a.heads;
    const int D = R.dx * R.dz, e = ((int)(id % tiles) * 256 + threadIdx.x) * V;
    if (e >= D) return;
    int64_t len = a.steps;
    if (a.lengths) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < len ? n : len);
    }
    const double gd = ln_decay(a.decay, (int)(bh % a.heads));
    const int whole = (int)(len / a.seg_len);  // segments without masked steps
    const float af = (float)exp(gd * (double)a.seg_len);
    const float ap = (float)exp(gd * (double)(len - whole * a.seg_len));
    float* p = R.seg + bh * a.nseg * D + e;
    Vec<float, V> X{};
    if (R.s0) {
        const float* s = R.s0 + bh * D;
#pragma unroll
        for (int j = 0; j < V; ++j)  // the slots' order is i dz + j
            X.e[j] = s[(e + j) / R.dz * R.s0_i + (e + j) % R.dz * R.s0_j];
    }
    for (int i0 = 0; i0 < a.nseg; i0 += 16) {
        Vec<float, V> L[16] = {};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (i0 + k < a.nseg - 1 && (i0 + k) * a.seg_len < len)
                L[k] = load_vec<float, V>(p + (int64_t)(i0 + k) * D);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int i = i0 + k;
            if (i >= a.nseg) break;
            store_vec<float, V>(p + (int64_t)i * D, X);
            const float keep = i < whole ? af : (i * a.seg_len < len ? ap : 1.f);
#pragma unroll
            for (int j = 0; j < V; ++j) X.e[j] = keep * X.e[j] + L[k].e[j];
        }
    }
}

// out[r, :] = sum of the `shared` rows of part that follow r * shared, in order; dk's and
// dv's rows in one launch (blockIdx.y).
struct SumArgs {
    const float* part[2];
    void* out[2];
    int32_t d[2];
    int32_t shared;
    int64_t rows;
};
template <class T>
__global__ __launch_bounds__(256) void attend_sum_kernel(SumArgs a, int64_t first) {
    const int d = a.d[blockIdx.y];
    const int64_t e = (first + blockIdx.x) * 256 + threadIdx.x;
    if (e >= a.rows * d) return;
    const int64_t row = e / d;
    const float* p = a.part[blockIdx.y] + row * a.shared * d + (e - row * d);
    float s = 0.f;
    for (int j = 0; j < a.shared; ++j) s += p[(int64_t)j * d];
    static_cast<T*>(a.out[blockIdx.y])[e] = from_f32<T>(s);
}

template <class T>
hipError_t sum_shared(const SumArgs& a, hipStream_t st) {
    const int64_t cells = a.rows * (a.d[0] > a.d[1] ? a.d[0] : a.d[1]);
    return in_launches((cells + 255) / 256, [&](int64_t first, unsigned n) {
        attend_sum_kernel<T><<<dim3(n, 2), 256, 0, st>>>(a, first);
    });
}

hipError_t walk(const AttendArgs& a, bool maps, hipStream_t st) {
    switch (a.type) {
        case kBF16: return launch_attend_walk<bf16_t>(a, maps, st);
        case kF16: return launch_attend_walk<f16_t>(a, maps, st);
        default: return launch_attend_walk<float>(a, maps, st);
    }
}

// `maps`: the first runs, whose segments' states are made (the others read one of theirs).
hipError_t run_all(AttendArgs a, int maps, hipStream_t st) {
    if (a.nseg > 1) {
        const int runs = a.nrun;
        a.nrun = maps;
        hipError_t e = walk(a, true, st);
        if (e != hipSuccess) return e;
        const int D = a.run[0].dx * a.run[0].dz;  // the same in all
        const int v = D % 4 == 0 ? 4 : 1, tiles = (D + 256 * v - 1) / (256 * v);
        e = in_launches(a.batch * a.heads * tiles, [&](int64_t first, unsigned n) {
            const dim3 grid(n, (unsigned)maps);
            if (v == 4)
                attend_join_kernel<4><<<grid, 256, 0, st>>>(a, first, tiles);
            else
                attend_join_kernel<1><<<grid, 256, 0, st>>>(a, first, tiles);
        });
        if (e != hipSuccess) return e;
        a.nrun = runs;
    }
    return walk(a, false, st);
}

AttendArgs common(const AttendCall& c, int runs) {
    AttendArgs a{};
    a.nrun = runs;
    a.decay = c.decay;
    a.lengths = c.lengths;
    a.type = c.d.type;
    a.heads = c.d.heads;
    a.group = c.d.heads / c.d.kv_heads;
    a.batch = c.d.batch;
    a.steps = c.d.steps;
    a.nseg = (int32_t)plan_segments(c.d, runs, &a.seg_len);
    return a;
}

struct Operand {
    const void* p;
    const int64_t* s;
    int32_t group;
    int32_t d;
};
void set_run(AttendRun& r, const Operand& x, const Operand& y, const Operand& z) {
    r.x = x.p, r.xb = x.s[0], r.xt = x.s[1], r.xh = x.s[2], r.xg = x.group;
    r.y = y.p, r.yb = y.s[0], r.yt = y.s[1], r.yh = y.s[2], r.yg = y.group;
    r.z = z.p, r.zb = z.s[0], r.zt = z.s[1], r.zh = z.s[2], r.zg = z.group;
    r.dx = x.d;
    r.dz = z.d;
    r.seg_i = z.d, r.seg_j = 1;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t seg_bytes(const AttendDesc& d, int runs) {
    int64_t len;
    const int64_t n = plan_segments(d, runs, &len);
    return n > 1 ? round256((size_t)d.batch * d.heads * n * d.dk * d.dv * 4) : 0;
}
size_t part_bytes(const AttendDesc& d, int width) {
    return d.heads == d.kv_heads ? 0 : round256((size_t)d.batch * d.steps * d.heads * width * 4);
}

}  // namespace

// 256 says that the workspace is not touched (callers share one for all such calls), so a call
// that does use it asks for more.
size_t attend_ws_bytes(const AttendDesc& d, bool gradient) {
    const size_t n = gradient ? 2 * seg_bytes(d, 3) + part_bytes(d, d.dk) + part_bytes(d, d.dv)
                              : seg_bytes(d, 1);
    return n == 0 ? 256 : (n < 512 ? 512 : n);
}

hipError_t launch_attend(const AttendCall& c, hipStream_t st) {
    AttendArgs a = common(c, 1);
    const int g = c.d.heads / c.d.kv_heads;
    AttendRun& r = a.run[0];
    set_run(r, {c.q, c.d.q, 1, c.d.dk}, {c.k, c.d.k, g, c.d.dk}, {c.v, c.d.v, g, c.d.dv});
    r.in_pow = 1;
    r.p_scale = r.in_scale = c.d.scale;
    r.st_scale = 1.f;
    r.s0 = c.state;
    r.s0_i = c.d.dv, r.s0_j = 1;
    r.s1 = c.last;
    r.s1_i = c.d.dv, r.s1_j = 1;
    r.out = c.o;
    r.seg = static_cast<float*>(c.ws);
    return run_all(a, 1, st);
}

// dq runs forward with the transposed state, dk and dv backward in time:
//   dq_t = scale sum_{s <= t} a^(t - s) (do_t . v_s) k_s + scale a^(t + 1) S do_t
//   dv_s = scale sum_{t >= s} a^(t - s) (k_s . q_t) do_t + a^(T - 1 - s) dlast^T k_s
//   dk_s = scale sum_{t >= s} a^(t - s) (v_s . do_t) q_t + a^(T - 1 - s) dlast v_s
// and dstate is what the backward walk of dv's state arrives with.
hipError_t launch_attend_grad(const AttendCall& c, hipStream_t st) {
    AttendArgs a = common(c, 3);
    const int g = c.d.heads / c.d.kv_heads, dk = c.d.dk, dv = c.d.dv;
    const Operand q{c.q, c.d.q, 1, dk}, k{c.k, c.d.k, g, dk}, v{c.v, c.d.v, g, dv},
        d{c.dout, c.d.d, 1, dv};
    char* ws = static_cast<char*>(c.ws);
    const size_t seg = seg_bytes(c.d, 3), pk = part_bytes(c.d, dk);
    float* part_k = reinterpret_cast<float*>(ws + 2 * seg);
    float* part_v = reinterpret_cast<float*>(ws + 2 * seg + pk);

    AttendRun& rq = a.run[0];
    set_run(rq, d, v, k);
    rq.in_pow = 1;
    rq.p_scale = rq.in_scale = c.d.scale;
    rq.st_scale = 1.f;
    rq.s0 = c.state;
    rq.s0_i = 1, rq.s0_j = dv;
    rq.out = c.dq;

    AttendRun& rv = a.run[1];
    set_run(rv, k, q, d);
    rv.reverse = 1;
    rv.p_scale = rv.st_scale = c.d.scale;
    rv.in_scale = 1.f;
    rv.s0 = c.dlast;
    rv.s0_i = dv, rv.s0_j = 1;
    rv.s1 = c.dstate;
    rv.s1_i = dv, rv.s1_j = 1;
    rv.out = g > 1 ? static_cast<void*>(part_v) : c.dv;
    rv.out32 = g > 1;

    AttendRun& rk = a.run[2];
    set_run(rk, v, d, q);
    rk.reverse = 1;
    rk.p_scale = rk.st_scale = c.d.scale;
    rk.in_scale = 1.f;
    rk.s0 = c.dlast;
    rk.s0_i = 1, rk.s0_j = dv;
    rk.out = g > 1 ? static_cast<void*>(part_k) : c.dk;
    rk.out32 = g > 1;

    rq.seg = reinterpret_cast<float*>(ws);
    rv.seg = rk.seg = reinterpret_cast<float*>(ws + seg);  // the one state, and transposed
    rk.seg_i = 1, rk.seg_j = dv;
    hipError_t e = run_all(a, 2, st);
    if (e != hipSuccess || g == 1) return e;
    const SumArgs sums{{part_k, part_v}, {c.dk, c.dv}, {dk, dv}, g,
                       c.d.batch * c.d.steps * c.d.kv_heads};
    switch (c.d.type) {
        case kBF16: return sum_shared<bf16_t>(sums, st);
        case kF16: return sum_shared<f16_t>(sums, st);
        default: return sum_shared<float>(sums, st);
    }
}

// ---- one live step ---------------------------------------------------------------

namespace {

struct StepArgs {
    const void *q, *k, *v;
    int64_t qb, qh, kb, kh, vb, vh;
    const float* decay;
    const float* s0;
    float* s1;
    void* o;
    int32_t heads, group, dk, dv;
    float scale;
};

// S' = a S + k v^T, o = scale q S'. The state is read and written once: 16 lanes take
// V columns each, 16 such groups the rows, every thread with R rows in flight. Bound by
// memory: 128 streams of 32 heads of 128 x 128 in 106.5 us (5.1 TB/s, the copy's rate). Where
// dv is no multiple of 4 a lane takes one column: 2048 x 16 heads of 50 x 50 in 296 us, of
// 50 x 52 in 145.
template <class T, int V>
__global__ __launch_bounds__(256) void attend_step_kernel(StepArgs a, int64_t first, int tiles) {
    constexpr int R = 8;
    __shared__ float qs[kMaxHeadDim], ks[kMaxHeadDim];
    __shared__ float part[4][16 * V];
    const int64_t id = first + blockIdx.x, bh = id / tiles, b = bh / a.heads;
    const int head = (int)(bh % a.heads), kv = head / a.group;
    const T* q = static_cast<const T*>(a.q) + b * a.qb + head * a.qh;
    const T* k = static_cast<const T*>(a.k) + b * a.kb + kv * a.kh;
    const T* v = static_cast<const T*>(a.v) + b * a.vb + kv * a.vh;
    const int c = (int)(id % tiles) * 16 * V + (threadIdx.x & 15) * V, r0 = threadIdx.x >> 4;
    const bool in = c < a.dv;  // V divides dv
    if (threadIdx.x < a.dk) {
        qs[threadIdx.x] = to_f32(q[threadIdx.x]);
        ks[threadIdx.x] = to_f32(k[threadIdx.x]);
    }
    // (as two numbers: the rounding of one would be made again at every step of a stream)
    const double kept = exp(ln_decay(a.decay, head));
    const float decay = (float)kept, decay_rest = (float)(kept - decay);
    float vc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) vc[j] = in ? to_f32(v[c + j]) : 0.f;
    __syncthreads();
    const float* s0 = a.s0 + bh * a.dk * a.dv + c;
    float* s1 = a.s1 + bh * a.dk * a.dv + c;
    float acc[V] = {};
    for (int i0 = r0; i0 < a.dk; i0 += 16 * R) {
        Vec<float, V> s[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (in && i0 + 16 * r < a.dk) s[r] = load_vec<float, V>(s0 + (i0 + 16 * r) * a.dv);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = i0 + 16 * r;
            if (!in || i >= a.dk) break;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[r].e[j] = fmaf(decay, s[r].e[j], fmaf(decay_rest, s[r].e[j], ks[i] * vc[j]));
                acc[j] += qs[i] * s[r].e[j];
            }
            store_vec<float, V>(s1 + i * a.dv, s[r]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        acc[j] += __shfl_xor(acc[j], 16, 64);
        acc[j] += __shfl_xor(acc[j], 32, 64);
    }
    const int lane = threadIdx.x & 63;
    if (lane < 16)
#pragma unroll
        for (int j = 0; j < V; ++j) part[threadIdx.x >> 6][lane * V + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < 16 * V) {
        const int z = (int)(id % tiles) * 16 * V + threadIdx.x;
        const float s = (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                        (part[2][threadIdx.x] + part[3][threadIdx.x]);
        if (z < a.dv) static_cast<T*>(a.o)[bh * a.dv + z] = from_f32<T>(s * a.scale);
    }
}

template <class T>
hipError_t step_as(const StepArgs& a, int64_t bh, hipStream_t st) {
    const int v = a.dv % 4 == 0 ? 4 : 1;
    const int tiles = (a.dv + 16 * v - 1) / (16 * v);
    return in_launches(bh * tiles, [&](int64_t first, unsigned n) {
        if (v == 4)
            attend_step_kernel<T, 4><<<n, 256, 0, st>>>(a, first, tiles);
        else
            attend_step_kernel<T, 1><<<n, 256, 0, st>>>(a, first, tiles);
    });
}

}  // namespace

hipError_t launch_attend_step(const AttendCall& c, hipStream_t st) {
    StepArgs a{};
    a.q = c.q, a.k = c.k, a.v = c.v;
    a.qb = c.d.q[0], a.qh = c.d.q[2], a.kb = c.d.k[0], a.kh = c.d.k[2];
    a.vb = c.d.v[0], a.vh = c.d.v[2];
    a.decay = c.decay;
    a.s0 = c.state;
    a.s1 = c.last;
    a.o = c.o;
    a.heads = c.d.heads;
    a.group = c.d.heads / c.d.kv_heads;
    a.dk = c.d.dk;
    a.dv = c.d.dv;
    a.scale = c.d.scale;
    const int64_t bh = c.d.batch * c.d.heads;
    switch (c.d.type) {
        case kBF16: return step_as<bf16_t>(a, bh, st);
        case kF16: return step_as<f16_t>(a, bh, st);
        default: return step_as<float>(a, bh, st);
    }
}

}  // namespace symnmf
