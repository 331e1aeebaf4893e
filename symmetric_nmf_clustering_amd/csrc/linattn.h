// The walk of decayed linear attention over time (see AttendRun in layers.h),
// instantiated for each element type by k_linattn_*.hip.
//
// Steps are taken in chunks of C. With W = a^(u - w) for w <= u inside a chunk,
//   P = (X Y^T) . W,   out = P Z + diag(a^(u + in_pow)) X S,
//   S <- a^n S + Y^T diag(a^(n - in_pow - w)) Z,
// four matrix products a chunk. A workgroup of NW waves walks one head (and one
// segment of its time) for 16 NW columns of z; wave i holds the dx x 16 block of
// S of its own columns in accumulators, so S is never stored: as the product's
// result a lane has S[4g + r][l % 16] (g = l / 16), which is also what the A
// operand of the next product wants of S^T if the depth index runs through the
// rows 4g + r and 16 + 4g + r. Every operand here takes its depth in that order.
// Results come out transposed (a lane has 4 columns of one step): 8 or 16 bytes a
// store. P alone passes through LDS, in the order its reader's lanes want it.
//
// bf16: products on the bf16 matrix cores. P and, in X S, the state are rounded to
// bf16 (as the inputs and the output are: each costs the output at most what its
// own rounding does). The state itself stays at float32's precision: the weights
// go to z, and w z is split exactly into three bf16 parts, three products each.
// fp32: 16x16x4 float32 products. fp16: widened to float32 as it is loaded.
#pragma once

#include <type_traits>

#include "bf16split.h"
#include "layers.h"

namespace symnmf {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// LDS of one wave is in order; across waves: their LDS writes are done before the
// barrier. Global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <class T>
struct InLds {  // how a tile is held
    using type = float;
};
template <>
struct InLds<bf16_t> {
    using type = bf16_t;
};

// 32 deep operands of a product: 8 values a lane. rows(p): depth 8g + j, p at the
// lane's own row; split(p): depth 4g + j and 16 + 4g + j (see above); column(t,
// stride): the same depth order down the rows of a tile, lane l % 16's column.
template <class LT>
struct Op;

template <>
struct Op<bf16_t> {
    using F = u32x4;
    static __device__ __forceinline__ F rows(const bf16_t* p, int g) {
        return *reinterpret_cast<const u32x4*>(p + 8 * g);
    }
    static __device__ __forceinline__ F split(const bf16_t* p, int g) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + 4 * g);
        const uint2 b = *reinterpret_cast<const uint2*>(p + 16 + 4 * g);
        return F{a.x, a.y, b.x, b.y};
    }
    static __device__ __forceinline__ F column(const bf16_t* t, int stride, int lane) {
        // a 4 x 16 block for each 16 lanes, read transposed: lane i asks for 4 elements of row
        // i / 4 and receives column i
        const bf16_t* p = t + (4 * (lane >> 4) + ((lane & 15) >> 2)) * stride + 4 * (lane & 3);
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 16 * stride));
        const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
        return F{ua.x, ua.y, ub.x, ub.y};
    }
    // the lane's values of two 16-deep blocks of a result
    static __device__ __forceinline__ F of(const floatx4& a, const floatx4& b) {
        return F{pack(a[0], a[1]), pack(a[2], a[3]), pack(b[0], b[1]), pack(b[2], b[3])};
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const f32x2 v = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    static __device__ __forceinline__ floatx4 mma(const F& a, const F& b, floatx4 c) {
        return mfma_bf16(a, b, c);
    }
    // a times (w . b) to float32's precision
    struct W {
        F p[3];
    };
    static __device__ __forceinline__ W weigh(const F& b, const float (&w)[8]) {
        W o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p1, p2, p3;
            split3_pair(__uint_as_float(b[i] << 16) * w[2 * i],
                        __uint_as_float(b[i] & 0xffff0000u) * w[2 * i + 1], p1, p2, p3);
            o.p[0][i] = p1;
            o.p[1][i] = p2;
            o.p[2][i] = p3;
        }
        return o;
    }
    static __device__ __forceinline__ floatx4 mma(const F& a, const W& b, floatx4 c) {
        c = mfma_bf16(a, b.p[2], c);
        c = mfma_bf16(a, b.p[1], c);
        return mfma_bf16(a, b.p[0], c);
    }
    static __device__ __forceinline__ void put4(bf16_t* p, const floatx4& v) {
        *reinterpret_cast<uint2*>(p) = uint2{pack(v[0], v[1]), pack(v[2], v[3])};
    }
};

template <>
struct Op<float> {
    struct F {
        float v[8];
    };
    static __device__ __forceinline__ F two(const float* p, const float* q) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(q);
        return F{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    static __device__ __forceinline__ F rows(const float* p, int g) {
        return two(p + 8 * g, p + 8 * g + 4);
    }
    static __device__ __forceinline__ F split(const float* p, int g) {
        return two(p + 4 * g, p + 16 + 4 * g);
    }
    static __device__ __forceinline__ F column(const float* t, int stride, int lane) {
        F o;
        const float* p = t + 4 * (lane >> 4) * stride + (lane & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = p[((j & 3) + (j >> 2) * 16) * stride];
        return o;
    }
    static __device__ __forceinline__ F of(const floatx4& a, const floatx4& b) {
        return F{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    static __device__ __forceinline__ floatx4 mma(const F& a, const F& b, floatx4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = mfma16x16x4(a.v[j], b.v[j], c);
        return c;
    }
    static __device__ __forceinline__ F weigh(const F& b, const float (&w)[8]) {
        F o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = b.v[j] * w[j];
        return o;
    }
    static __device__ __forceinline__ void put4(float* p, const floatx4& v) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    }
};

// The rows of one operand of a head, in the order of the walk.
template <class T>
struct Rows {
    const T* p;       // the first step's row
    int64_t stride;   // of a step, not negative
    int32_t reverse;
    int32_t d;        // columns
};
// WIDE tiles count a chunk's elements from its lowest row in 32 bits.
constexpr int64_t kNearStride = int64_t(1) << 24;

// A chunk's C x COLS tile on its way from memory through registers to LDS, by NT
// threads. Rows past n (at least 1) and columns past d are zeros. No access is
// behind a lane's branch, so that all of them are in flight together: those past the
// rows or columns read the last one, and store() clears them. (A branch around each
// costs a wait for each: 2.4 times the time of the whole walk.) WIDE: 16 bytes a
// lane, for d a multiple of that; otherwise one element a lane, neighbours together.
template <class T, class LT, int C, int COLS, int NT, bool WIDE>
struct Tile {
    static constexpr int V = WIDE ? 16 / sizeof(T) : 1, G = COLS / V, N = (C * G + NT - 1) / NT;
    static constexpr int STRIDE = COLS + 16 / (int)sizeof(LT);
    Vec<T, V> r[N];

    __device__ __forceinline__ void load(const Rows<T>& m, int64_t u0, int n, int c0) {
        const T* low = m.p + (m.reverse ? -(u0 + n - 1) : u0) * m.stride;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * NT, c = min(c0 + at % G * V, m.d - V);
            int row = min(at / G, n - 1);
            if (m.reverse) row = n - 1 - row;
            if constexpr (WIDE)
                r[i] = load_vec<T, V>(low + (uint32_t)(__mul24(row, (int)m.stride) + c));
            else
                r[i] = load_vec<T, V>(low + row * m.stride + c);
        }
    }
    // n: rows that count (C: all); d: columns that count, from c0 on
    template <bool FULL>
    __device__ __forceinline__ void store(LT* t, int d, int n, int c0) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * NT, row = at / G, c = at % G * V;
            if (C * G % NT && row >= C) continue;
            const bool in = c0 + c < d && (FULL || row < n);
            if constexpr (sizeof(T) == sizeof(LT) && WIDE) {
                u32x4 v = __builtin_bit_cast(u32x4, r[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = in ? v[j] : 0u;
                *reinterpret_cast<u32x4*>(t + row * STRIDE + c) = v;
            } else if constexpr (sizeof(T) == sizeof(LT)) {
                t[row * STRIDE + c] = in ? r[i].e[0] : LT{};
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) t[row * STRIDE + c + j] = in ? to_f32(r[i].e[j]) : 0.f;
            }
        }
    }
};

template <class T, int DX, int NW, int WN, bool OUT, bool WIDE>
struct WalkSizes {
    using LT = typename InLds<T>::type;
    static constexpr int C = sizeof(LT) == 2 ? 64 : 32;
    static constexpr int NT = 64 * NW, ZC = 16 * WN * NW;
    using TX = Tile<T, LT, C, DX, NT, WIDE>;
    using TZ = Tile<T, LT, C, ZC, NT, WIDE>;
    struct Lds {
        LT x[OUT ? C * TX::STRIDE : 8];
        LT y[C * TX::STRIDE];
        LT z[C * TZ::STRIDE];
        LT p[OUT ? C * C : 8];  // 16 x 16 blocks (u, w): a lane's 4 values of w together
        float wz[C];            // st_scale a^(C - in_pow - w): the weights of a whole chunk
        float wx[OUT ? C : 4];  // in_scale a^(u + in_pow)
        float wp[OUT ? C * 16 : 4];  // p_scale a^(u - w), as a lane holds a block, by bu - bw
        float pw[C + 1];        // a^0 ... a^C
    };
};

__device__ __forceinline__ double ln_decay(const float* decay, int head) {
    const double g = decay[head];
    return g < -200.0 ? -200.0 : g;  // exp(-200) is 0 in float32, and a^0 stays 1
}

// Four neighbouring columns of one step's result, of which `cols` are there (WIDE: all or
// none).
template <bool WIDE, class O>
__device__ __forceinline__ void put_out(O* p, const floatx4& v, int cols) {
    if (cols >= 4) {
        store_vec<O, 4>(p, {{from_f32<O>(v[0]), from_f32<O>(v[1]), from_f32<O>(v[2]),
                             from_f32<O>(v[3])}});
    } else if (!WIDE) {
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (r < cols) p[r] = from_f32<O>(v[r]);
    }
}

// blockIdx.x (+ first): column tile, segment and head; blockIdx.y: the run.
template <class T, int DX, int NW, int WN, bool OUT, bool WIDE>
__global__ __launch_bounds__(64 * NW, DX > 128 ? 1 : 2) void attend_walk_kernel(
    AttendArgs a, int64_t first, int64_t items, int ztiles) {
    using Z = WalkSizes<T, DX, NW, WN, OUT, WIDE>;
    using LT = typename Z::LT;
    using O = Op<LT>;
    constexpr int C = Z::C, NX = DX / 16, NB = C / 16, XS = Z::TX::STRIDE, ZS = Z::TZ::STRIDE;
    __shared__ alignas(16) typename Z::Lds lds;

    // items go round the XCDs; the column tiles of one item to the same XCD, whose L2
    // then has x and y for all of them
    const int64_t id = first + blockIdx.x;
    const int64_t grp = id >> 3;
    const int zt = (int)(grp % ztiles);
    const int64_t item = (grp / ztiles) + (id & 7) * ((items + 7) >> 3);
    if (grp / ztiles >= ((items + 7) >> 3) || item >= items) return;
    const AttendRun R = a.run[blockIdx.y];
    const int seg = (int)(item % a.nseg);
    const int64_t bh = item / a.nseg;
    const int64_t b = bh / a.heads;
    const int head = (int)(bh % a.heads);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
    const int z0 = zt * Z::ZC, zw = z0 + wave * 16 * WN;
    if (z0 >= R.dz) return;  // the whole workgroup

    int64_t len = a.steps;
    if (a.lengths) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < len ? n : len);
    }
    const int64_t u_begin = seg * a.seg_len;
    int64_t u_end = u_begin + a.seg_len;
    if (u_end > a.steps) u_end = a.steps;
    const int64_t u_stop = len < u_end ? len : u_end;  // of the segment's valid steps
    if (!OUT && (u_begin >= len || seg == a.nseg - 1)) return;  // the join does not read these

    const double gd = ln_decay(a.decay, head);
    for (int i = threadIdx.x; i <= C; i += Z::NT) lds.pw[i] = (float)exp(gd * i);
    for (int i = threadIdx.x; i < C; i += Z::NT)
        lds.wz[i] = R.st_scale * (float)exp(gd * (C - R.in_pow - i));
    if constexpr (OUT) {  // blocks above the diagonal that a 32-deep step reads
        for (int i = threadIdx.x; i < C * C; i += Z::NT) lds.p[i] = LT{};
    }

    const int64_t dir = R.reverse ? -1 : 1, from = R.reverse ? len - 1 : 0;
    auto rows_of = [&](const void* p, int64_t sb, int64_t st, int64_t sh, int grp_, int d) {
        return Rows<T>{static_cast<const T*>(p) + b * sb + from * st + (head / grp_) * sh, st,
                       R.reverse, d};
    };
    const Rows<T> mx = rows_of(R.x, R.xb, R.xt, R.xh, R.xg, R.dx);
    const Rows<T> my = rows_of(R.y, R.yb, R.yt, R.yh, R.yg, R.dx);
    const Rows<T> mz = rows_of(R.z, R.zb, R.zt, R.zh, R.zg, R.dz);

    // the state at the segment's start
    floatx4 S[NX][WN];
    auto element = [&](int i, int m, int r, int si, int sj) __attribute__((always_inline)) {  // where S[i][m][r] is, or -1
        const int row = 16 * i + 4 * g + r, j = zw + 16 * m + l16;
        return row < R.dx && j < R.dz ? row * si + j * sj : -1;
    };
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int m = 0; m < WN; ++m) S[i][m] = floatx4{0.f, 0.f, 0.f, 0.f};
    if constexpr (OUT) {
        const int64_t D = (int64_t)R.dx * R.dz;
        const float keep = (float)exp(gd * (double)a.seg_len);
        // S = what is joined, or s0 (m = -1) and then the segments before this one
        const int last = a.joined ? -1 : seg - 1;
        for (int m = -1; m <= last; ++m) {
            const float* s = m >= 0 ? R.seg + (bh * a.nseg + m) * D
                                    : (a.joined ? R.seg + (bh * a.nseg + seg) * D
                                                : (R.s0 ? R.s0 + bh * D : nullptr));
            if (!s) continue;
            const int64_t left = len - m * a.seg_len;
            if (m >= 0 && left <= 0) break;
            const bool slot = m >= 0 || a.joined;
            const int si = slot ? R.seg_i : R.s0_i, sj = slot ? R.seg_j : R.s0_j;
            const float k = m < 0 ? 0.f
                                  : (left >= a.seg_len ? keep : (float)exp(gd * (double)left));
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                float v[4 * WN];  // (asked for without branches: all in flight)
#pragma unroll
                for (int q = 0; q < 4 * WN; ++q)
                    v[q] = s[(uint32_t)max(element(i, q >> 2, q & 3, si, sj), 0)];
#pragma unroll
                for (int q = 0; q < 4 * WN; ++q) {
                    asm volatile("" : "+v"(v[q]));
                    const float to = k * S[i][q >> 2][q & 3] + v[q];
                    S[i][q >> 2][q & 3] = element(i, q >> 2, q & 3, si, sj) >= 0 ? to : 0.f;
                }
            }
        }
    }

    if constexpr (OUT) {
        for (int i = threadIdx.x; i < C; i += Z::NT)
            lds.wx[i] = R.in_scale * (float)exp(gd * (i + R.in_pow));
        for (int i = threadIdx.x; i < C * 16; i += Z::NT) {
            const int gap = 16 * (i >> 8) + (i >> 2 & 15) - (4 * (i >> 6 & 3) + (i & 3));
            lds.wp[i] = gap >= 0 ? R.p_scale * (float)exp(gd * gap) : 0.f;
        }
    }

    typename Z::TX rx, ry;
    typename Z::TZ rz;
    auto fetch = [&](int64_t u0) __attribute__((always_inline)) {
        const int n = (int)min(u_stop - u0, (int64_t)C);
        if (OUT) rx.load(mx, u0, n, 0);
        ry.load(my, u0, n, 0);
        rz.load(mz, u0, n, z0);
    };
    // A chunk of n steps from u0; FULL: n = C.
    auto chunk = [&](auto full, int64_t u0, int n) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        if (!WIDE) fetch(u0);  // (many registers: not kept through a chunk)
        lds_barrier();         // the tiles of the last chunk are read
        if (OUT) rx.template store<FULL>(lds.x, R.dx, n, 0);
        ry.template store<FULL>(lds.y, R.dx, n, 0);
        rz.template store<FULL>(lds.z, R.dz, n, z0);
        lds_barrier();

        if constexpr (OUT) {
            // P^T in 16 x 16 blocks on and below the diagonal, shared out among the waves
            constexpr int BLOCKS = NB * (NB + 1) / 2, MINE = (BLOCKS + NW - 1) / NW;
#pragma unroll
            for (int q = 0; q < MINE; ++q) {
                const int at = wave + q * NW;
                if (at >= BLOCKS) break;
                const int bu = (at >= 1) + (at >= 3) + (at >= 6), bw = at - bu * (bu + 1) / 2;
                floatx4 acc = {0.f, 0.f, 0.f, 0.f};
                const LT* py = lds.y + (16 * bw + l16) * XS;
                const LT* px = lds.x + (16 * bu + l16) * XS;
#pragma unroll
                for (int k = 0; k < DX / 32; ++k)
                    acc = O::mma(O::rows(py + 32 * k, g), O::rows(px + 32 * k, g), acc);
                const f32x4 wp = *reinterpret_cast<const f32x4*>(lds.wp + ((bu - bw) * 64 + lane) * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = wp[r] != 0.f ? acc[r] * wp[r] : 0.f;
                O::put4(lds.p + ((bu * NB + bw) * 64 + lane) * 4, acc);
            }
            lds_barrier();
        }

        typename O::F zf[C / 32][WN];
#pragma unroll
        for (int k = 0; k < C / 32; ++k)
#pragma unroll
            for (int m = 0; m < WN; ++m)
                zf[k][m] = O::column(lds.z + 32 * k * ZS + 16 * (WN * wave + m), ZS, lane);

        if constexpr (OUT) {
            typename O::F sf[DX / 32][WN];
#pragma unroll
            for (int k = 0; k < DX / 32; ++k)
#pragma unroll
                for (int m = 0; m < WN; ++m) sf[k][m] = O::of(S[2 * k][m], S[2 * k + 1][m]);
            const int64_t e0 = ((b * a.steps + from + dir * (u0 + l16)) * a.heads + head) * R.dz + zw + 4 * g;
            const int64_t es = dir * 16 * a.heads * R.dz;
#pragma unroll
            for (int bu = 0; bu < NB; ++bu) {
                floatx4 acc[WN] = {};
                const LT* px = lds.x + (16 * bu + l16) * XS;
#pragma unroll
                for (int k = 0; k < DX / 32; ++k) {
                    const auto xf = O::split(px + 32 * k, g);
#pragma unroll
                    for (int m = 0; m < WN; ++m) acc[m] = O::mma(sf[k][m], xf, acc[m]);
                }
                const float wx = lds.wx[16 * bu + l16];
#pragma unroll
                for (int m = 0; m < WN; ++m) acc[m] *= wx;
#pragma unroll
                for (int k = 0; k <= bu / 2; ++k) {
                    typename O::F pf;
                    const LT* pp = lds.p + ((bu * NB + 2 * k) * 64 + lane) * 4;
                    if constexpr (sizeof(LT) == 2) {
                        const uint2 p0 = *reinterpret_cast<const uint2*>(pp);
                        const uint2 p1 = *reinterpret_cast<const uint2*>(pp + 256);
                        pf = typename O::F{p0.x, p0.y, p1.x, p1.y};
                    } else {
                        pf = O::two(pp, pp + 256);
                    }
#pragma unroll
                    for (int m = 0; m < WN; ++m) acc[m] = O::mma(zf[k][m], pf, acc[m]);
                }
                if (FULL || 16 * bu + l16 < n) {
                    const int64_t e = e0 + bu * es;
                    if (R.out32) {
#pragma unroll
                        for (int m = 0; m < WN; ++m)
                            put_out<WIDE>(static_cast<float*>(R.out) + e + 16 * m, acc[m],
                                          R.dz - zw - 16 * m - 4 * g);
                    } else {
#pragma unroll
                        for (int m = 0; m < WN; ++m)
                            put_out<WIDE>(static_cast<T*>(R.out) + e + 16 * m, acc[m],
                                          R.dz - zw - 16 * m - 4 * g);
                    }
                }
            }
        }

        if (WIDE && u0 + C < u_stop) fetch(u0 + C);  // (earlier, its registers are wanted above)
        // S <- a^n S + Y^T (w Z); rows of z past n are zeros
        const float an = FULL ? lds.pw[C] : lds.pw[n];
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int m = 0; m < WN; ++m) S[i][m] *= an;
#pragma unroll
        for (int k = 0; k < C / 32; ++k) {
            float w[8];
            if constexpr (FULL) {
                const f32x4 a0 = *reinterpret_cast<const f32x4*>(lds.wz + 32 * k + 4 * g);
                const f32x4 a1 = *reinterpret_cast<const f32x4*>(lds.wz + 32 * k + 16 + 4 * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = a0[j];
                    w[4 + j] = a1[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = n - R.in_pow - (32 * k + 4 * g + (j & 3) + (j >> 2) * 16);
                    w[j] = R.st_scale * lds.pw[at < 0 ? 0 : at];
                }
            }
            decltype(O::weigh(zf[0][0], w)) zw8[WN];
#pragma unroll
            for (int m = 0; m < WN; ++m) zw8[m] = O::weigh(zf[k][m], w);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const auto yf = O::column(lds.y + 32 * k * XS + 16 * i, XS, lane);
#pragma unroll
                for (int m = 0; m < WN; ++m) S[i][m] = O::mma(yf, zw8[m], S[i][m]);
            }
        }
    };
    if (WIDE && u_begin < u_stop) fetch(u_begin);
    int64_t u0 = u_begin;
    for (; u0 + C <= u_stop; u0 += C) chunk(std::true_type{}, u0, C);
    if (u0 < u_stop) chunk(std::false_type{}, u0, (int)(u_stop - u0));

    // steps past the length
    if constexpr (OUT) {
        const int64_t lo = u_begin > len ? u_begin : len;
        const int64_t cells = u_end > lo ? (u_end - lo) * Z::ZC : 0;
        for (int64_t i = threadIdx.x; i < cells; i += Z::NT) {
            const int z = z0 + (int)(i % Z::ZC);
            if (z >= R.dz) continue;
            const int64_t e = ((b * a.steps + lo + i / Z::ZC) * a.heads + head) * R.dz + z;
            if (R.out32)
                static_cast<float*>(R.out)[e] = 0.f;
            else
                static_cast<T*>(R.out)[e] = from_f32<T>(0.f);
        }
    }

    float* s = nullptr;
    int si = R.seg_i, sj = R.seg_j;
    if (!OUT) {
        s = R.seg + (bh * a.nseg + seg) * ((int64_t)R.dx * R.dz);
    } else if (seg == a.nseg - 1 && R.s1) {
        s = R.s1 + bh * ((int64_t)R.dx * R.dz);
        si = R.s1_i;
        sj = R.s1_j;
    }
    if (s) {
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int m = 0; m < WN; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = element(i, m, r, si, sj);
                    if (at >= 0) s[(uint32_t)at] = S[i][m][r];
                }
    }
}

template <class T, int DX, int NW, int WN, bool OUT>
hipError_t attend_walk_as(const AttendArgs& a, hipStream_t st) {
    constexpr int ZC = 16 * NW * WN, V = 16 / sizeof(T);
    int dz = 0;
    bool wide = true;
    for (int r = 0; r < a.nrun; ++r) {
        dz = a.run[r].dz > dz ? a.run[r].dz : dz;
        const AttendRun& q = a.run[r];
        wide = wide && q.dx % V == 0 && q.dz % V == 0 && q.xt < kNearStride && q.yt < kNearStride &&
               q.zt < kNearStride;
    }
    const int ztiles = (dz + ZC - 1) / ZC;
    const int64_t items = a.batch * a.heads * a.nseg;
    const int64_t blocks = (items + 7) / 8 * 8 * ztiles;
    return in_launches(blocks, [&](int64_t first, unsigned n) {
        const dim3 grid(n, (unsigned)a.nrun);
        if (wide)
            attend_walk_kernel<T, DX, NW, WN, OUT, true>
                <<<grid, 64 * NW, 0, st>>>(a, first, items, ztiles);
        else
            attend_walk_kernel<T, DX, NW, WN, OUT, false>
                <<<grid, 64 * NW, 0, st>>>(a, first, items, ztiles);
    });
}

template <class T>
hipError_t launch_attend_walk(const AttendArgs& a, bool maps, hipStream_t st) {
    int dx = 0, dz = 0;
    for (int r = 0; r < a.nrun; ++r) {
        dx = a.run[r].dx > dx ? a.run[r].dx : dx;
        dz = a.run[r].dz > dz ? a.run[r].dz : dz;
    }
    // small heads: two waves hold all columns of z; wide ones: two column tiles a wave, which
    // share what it reads of x and y
#define SYMNMF_WALK(DX, NW, WN) \
    return maps ? attend_walk_as<T, DX, NW, WN, false>(a, st) \
                : attend_walk_as<T, DX, NW, WN, true>(a, st)
    if (dx <= 32 && dz <= 32) SYMNMF_WALK(32, 2, 1);
    if (dx <= 32) SYMNMF_WALK(32, 4, 1);
    if (dx <= 64 && dz <= 32) SYMNMF_WALK(64, 2, 1);
    if (dx <= 64) SYMNMF_WALK(64, 4, 1);
    if (dx <= 128 && dz <= 64) SYMNMF_WALK(128, 4, 1);
    if (dx <= 128) SYMNMF_WALK(128, 4, 2);
    SYMNMF_WALK(256, 4, 1);
#undef SYMNMF_WALK
}

}  // namespace symnmf
