// The walk of decayed linear attention over time (see AttendRun in layers.h),
// instantiated for each element type by k_linattn_*.hip.
//
// Steps are taken in chunks of C. With W = a^(u - w) for w <= u inside a chunk,
//   P = (X Y^T) . W,   out = P Z + diag(a^(u + in_pow)) X S,
//   S <- a^n S + Y^T diag(a^(n - in_pow - w)) Z,
// four matrix products a chunk. No power of a is negative, so strong decays only underflow.
// A workgroup of NW waves walks one head (and one segment of its time) for 16 WN NW columns
// of z; a wave holds the dx x 16 WN block of S of its own columns in accumulators, so S is
// never stored: as the product's result a lane has S[4g + r][l % 16] (g = l / 16), which is
// also what the A operand of the next product wants of S^T if the depth index runs through
// the rows 4g + r and 16 + 4g + r. Every operand here takes its depth in that order. Results
// come out transposed (a lane has 4 columns of one step): 8 or 16 bytes a store. P alone
// passes through LDS, in the order its reader's lanes want it. Whole chunks and a last,
// shorter one are two copies of the loop's body: bounds in the common one cost registers
// that spill. The next chunk's rows are asked for as soon as this one's are in LDS.
//
// What bounds it (bf16, heads of 128): with two workgroups a CU, issue. Of a SIMD's cycles
// matrix products take 34% and other vector operations 51% (548 for 32 steps and a wave), and
// waves wait for LDS and barriers in 29% of theirs. 32 x 2048 steps of 16 heads: 286 us,
// 4.0 TB/s; alone on its CU a workgroup takes 5 us for 64 steps (16 x 2048: 168 us).
//
// All products run on the bf16 matrix cores, on bf16 parts ("planes") of their operands
// whose products are summed in float32:
//   bf16: one plane; P and, in X S, the state are two, which hold them to 2^-16 (in one, o's error
//     against float64 is 2.35e-3 of its size, not the 1.66e-3 of its own rounding, for 8% of the time:
//     1 x 32768 x 16 heads 230 us against 212), two products.
//   fp16: two planes hold an element exactly; P and S, in two, lose 2^-16; three products.
//   fp32: three planes (bf16split.h), six products, which is float32's precision; 16x16x4
//     float32 products would take 2.7 times their cycles.
// The state itself stays at float32's precision in every type: the weights go to z, and w z
// is split into three planes (3, 5 and 6 products).
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

// Planes of an element, of P and the state as an operand, and steps of a chunk (at most).
template <class T>
struct Planes {
    static constexpr int N = 3, S = 3, C = 32;
};
template <>
struct Planes<f16_t> {
    static constexpr int N = 2, S = 2, C = 32;
};
template <>
struct Planes<bf16_t> {
    static constexpr int N = 1, S = 2, C = 64;
};

// 32 deep operands of a product: a lane's 8 values, as N planes of bf16.
template <int N>
struct Frag {
    u32x4 p[N];
};

// (a, b) -> the packed pairs of their first N planes
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[N]) {
    f32x2 v = {a, b};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bf16x2 h = __builtin_convertvector(v, bf16x2);
        p[i] = __builtin_bit_cast(uint32_t, h);
        if (i + 1 < N) v = v - __builtin_convertvector(h, f32x2);
    }
}
template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&v)[8]) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[N];
        split_pair<N>(v[2 * i], v[2 * i + 1], p);
#pragma unroll
        for (int j = 0; j < N; ++j) f.p[j][i] = p[j];
    }
    return f;
}
// the lane's values of two 16-deep blocks of a result
template <int N>
__device__ __forceinline__ Frag<N> frag_of(const floatx4& a, const floatx4& b) {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split8<N>(v);
}
// w . f to float32's precision
template <int N>
__device__ __forceinline__ Frag<3> weigh(const Frag<N>& f, const float (&w)[8]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = v[2 * i + 1] = 0.f;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) {
            v[2 * i] += __uint_as_float(f.p[j][i] << 16);
            v[2 * i + 1] += __uint_as_float(f.p[j][i] & 0xffff0000u);
        }
        v[2 * i] *= w[2 * i];
        v[2 * i + 1] *= w[2 * i + 1];
    }
    return split8<3>(v);
}
// The products of planes i and j with i + j < K, smallest first.
template <int K, int NA, int NB>
__device__ __forceinline__ floatx4 mma(const Frag<NA>& a, const Frag<NB>& b, floatx4 c) {
#pragma unroll
    for (int s = K - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB) c = mfma_bf16(a.p[i], b.p[s - i], c);
    return c;
}

// Reads of a tile (N planes, `plane` elements apart). rows: depth 8g + j of the lane's own
// row p; split: depth 4g + j and 16 + 4g + j (see above); column: the same order down
// the rows of a tile, lane l % 16's column.
template <int N>
__device__ __forceinline__ Frag<N> read_rows(const bf16_t* p, int plane, int g) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        f.p[i] = *reinterpret_cast<const u32x4*>(p + i * plane + 8 * g);
    return f;
}
template <int N>
__device__ __forceinline__ Frag<N> read_split(const bf16_t* p, int plane, int next, int g) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + i * plane + 4 * g);
        const uint2 b = *reinterpret_cast<const uint2*>(p + i * plane + next + 4 * g);
        f.p[i] = u32x4{a.x, a.y, b.x, b.y};
    }
    return f;
}
template <int N>
__device__ __forceinline__ Frag<N> read_column(const bf16_t* t, int plane, int stride, int lane) {
    // a 4 x 16 block for each 16 lanes, read transposed: lane i asks for 4 elements of row
    // i / 4 and receives column i
    const bf16_t* p = t + (4 * (lane >> 4) + ((lane & 15) >> 2)) * stride + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) s16x4 lds4;
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + i * plane));
        const s16x4 b =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + i * plane + 16 * stride));
        const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
        f.p[i] = u32x4{ua.x, ua.y, ub.x, ub.y};
    }
    return f;
}

// The rows of one operand of a head, in the order of the walk.
template <class T>
struct Rows {
    const T* p;       // the first step's row
    int64_t stride;   // of a step, not negative
    int32_t reverse;
    int32_t d;        // columns
};
// WIDE tiles count a chunk's elements from its lowest row in 32 bits, with a product of signed
// 24-bit factors.
constexpr int64_t kNearStride = int64_t(1) << 23;

// A chunk's C x COLS tile on its way from memory through registers to LDS, by NT
// threads. Rows past n (at least 1) and columns past d are zeros. No access is
// behind a lane's branch, so that all of them are in flight together: those past the
// rows or columns read the last one, and store() clears them. (A branch around each
// costs a wait for each: 2.4 times the time of the whole walk.) WIDE: 16 bytes a
// lane, for d a multiple of that; otherwise one element a lane, neighbours together.
template <class T, int C, int COLS, int NT, bool WIDE, int PAD>
struct Tile {
    static constexpr int V = WIDE ? 16 / sizeof(T) : 1, G = COLS / V, N = (C * G + NT - 1) / NT;
    static constexpr int STRIDE = COLS + PAD, PLANE = C * STRIDE, NP = Planes<T>::N;
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
    __device__ __forceinline__ void store(bf16_t* t, int d, int n, int c0) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * NT, row = at / G, c = at % G * V;
            if (C * G % NT && row >= C) continue;
            const bool in = c0 + c < d && (FULL || row < n);
            bf16_t* q = t + row * STRIDE + c;
            if constexpr (V == 1) {
                float v = in ? to_f32(r[i].e[0]) : 0.f;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    q[j * PLANE] = from_f32<bf16_t>(v);
                    v -= to_f32(q[j * PLANE]);
                }
            } else if constexpr (NP == 1) {
                u32x4 v = __builtin_bit_cast(u32x4, r[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = in ? v[j] : 0u;
                *reinterpret_cast<u32x4*>(q) = v;
            } else {
                Vec<uint32_t, V / 2> w[NP];
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    uint32_t p[NP];
                    split_pair<NP>(in ? to_f32(r[i].e[2 * j]) : 0.f,
                                   in ? to_f32(r[i].e[2 * j + 1]) : 0.f, p);
#pragma unroll
                    for (int k = 0; k < NP; ++k) w[k].e[j] = p[k];
                }
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    *reinterpret_cast<Vec<uint32_t, V / 2>*>(q + k * PLANE) = w[k];
            }
        }
    }
};

template <class T, int DX, int NW, int WN, bool OUT, bool WIDE>
struct WalkSizes {
    // 64 steps of two column tiles a wave leave no registers to ask for the next chunk's rows
    // early; 32 do (4 x 4096 x 32 heads of 128 bf16: 203 us against 271). Element loads of 64
    // steps spill (2 x 2048 x 8 heads of 33 and 24: 79 us, of 32 steps 32).
    static constexpr int C = WN == 2 || !WIDE ? 32 : Planes<T>::C;
    static constexpr int NP = Planes<T>::N, NS = Planes<T>::S;
    static constexpr int NT = 64 * NW, ZC = 16 * WN * NW;
    // pads of 16 bytes keep reads of rows off one another's banks, of 32 those down columns
    using TX = Tile<T, C, DX, NT, WIDE, 8>;
    using TY = Tile<T, C, DX, NT, WIDE, 16>;
    using TZ = Tile<T, C, ZC, NT, WIDE, 16>;
    struct Lds {
        bf16_t x[OUT ? NP * TX::PLANE : 8];
        bf16_t y[NP * TY::PLANE];
        bf16_t z[NP * TZ::PLANE];
        bf16_t p[OUT ? NS * C * C : 8];  // 16 x 16 blocks (u, w): a lane's 4 values of w together
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
    AttendArgs a, int64_t first, int64_t units, int ztiles) {
    using Z = WalkSizes<T, DX, NW, WN, OUT, WIDE>;
    constexpr int C = Z::C, NP = Z::NP, NS = Z::NS, NX = DX / 16, NB = C / 16;
    constexpr int XS = Z::TX::STRIDE, YS = Z::TY::STRIDE, ZS = Z::TZ::STRIDE;
    constexpr int XP = Z::TX::PLANE, YP = Z::TY::PLANE, ZP = Z::TZ::PLANE;
    __shared__ alignas(16) typename Z::Lds lds;

    // Workgroups go round the XCDs. An XCD takes whole units, the column tiles and the heads
    // that share rows of one segment, whose L2 then serves them all: neighbouring units, or,
    // where batch rows have lengths, every eighth one, so that the XCDs are loaded alike.
    const int64_t id = first + blockIdx.x, mine = id >> 3, each = (units + 7) >> 3;
    const int zt = (int)(mine % ztiles);
    const int64_t at_head = mine / ztiles, nth = at_head / a.group;
    const int64_t unit = a.lengths ? nth * 8 + (id & 7) : (id & 7) * each + nth;
    if (nth >= each || unit >= units) return;
    const AttendRun R = a.run[blockIdx.y];
    const int shared = a.heads / a.group;
    const int64_t row = unit / a.nseg, b = row / shared;
    const int head = (int)(row % shared) * a.group + (int)(at_head % a.group);
    // Workgroups 256 apart meet on a CU. Every other 256 take their segments from the last to
    // the first: short batch rows have no steps in their last ones.
    const bool turn = row * a.nseg * a.group * ztiles >> 8 & 1;
    const int seg = turn ? a.nseg - 1 - (int)(unit % a.nseg) : (int)(unit % a.nseg);
    const int64_t bh = b * a.heads + head;
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
    const int64_t dir = R.reverse ? -1 : 1, from = R.reverse ? len - 1 : 0;
    auto rows_of = [&](const void* p, int64_t sb, int64_t st, int64_t sh, int grp_, int d) {
        return Rows<T>{static_cast<const T*>(p) + b * sb + from * st + (head / grp_) * sh, st,
                       R.reverse, d};
    };
    const Rows<T> mx = rows_of(R.x, R.xb, R.xt, R.xh, R.xg, R.dx);
    const Rows<T> my = rows_of(R.y, R.yb, R.yt, R.yh, R.yg, R.dx);
    const Rows<T> mz = rows_of(R.z, R.zb, R.zt, R.zh, R.zg, R.dz);

    typename Z::TX rx;
    typename Z::TY ry;
    typename Z::TZ rz;
    auto fetch = [&](int64_t u0) __attribute__((always_inline)) {
        const int n = (int)min(u_stop - u0, (int64_t)C);
        if (OUT) rx.load(mx, u0, n, 0);
        ry.load(my, u0, n, 0);
        rz.load(mz, u0, n, z0);
    };
    // the state at the segment's start
    floatx4 S[NX][WN];
    // where S[i][m][r] is, or -1
    auto element = [&](int i, int m, int r, int si, int sj) __attribute__((always_inline)) {
        const int row = 16 * i + 4 * g + r, j = zw + 16 * m + l16;
        return row < R.dx && j < R.dz ? row * si + j * sj : -1;
    };
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int m = 0; m < WN; ++m) S[i][m] = floatx4{0.f, 0.f, 0.f, 0.f};
    const bool last = seg == a.nseg - 1;
    if (OUT && (u_begin < len || last)) {  // (others clear their steps alone)
        const int64_t D = (int64_t)R.dx * R.dz;
        const bool cut = a.nseg > 1;  // the join has left the segment's state in its slot
        const float* s = cut ? R.seg + (bh * a.nseg + seg) * D : (R.s0 ? R.s0 + bh * D : nullptr);
        const int si = cut ? R.seg_i : R.s0_i, sj = cut ? R.seg_j : R.s0_j;
        if (s) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                float v[4 * WN];  // (asked for without branches: all in flight)
#pragma unroll
                for (int q = 0; q < 4 * WN; ++q)
                    v[q] = s[(uint32_t)max(element(i, q >> 2, q & 3, si, sj), 0)];
#pragma unroll
                for (int q = 0; q < 4 * WN; ++q) {
                    asm volatile("" : "+v"(v[q]));
                    S[i][q >> 2][q & 3] = element(i, q >> 2, q & 3, si, sj) >= 0 ? v[q] : 0.f;
                }
            }
        }
    }

    if (WIDE && u_begin < u_stop) fetch(u_begin);
    // the tables of weights, from one table of powers
    if (u_begin < u_stop)
        for (int i = threadIdx.x; i <= C; i += Z::NT) lds.pw[i] = (float)exp(gd * i);
    lds_barrier();
    for (int i = threadIdx.x; i < C; i += Z::NT) {
        lds.wz[i] = R.st_scale * lds.pw[C - R.in_pow - i];
        if (OUT) lds.wx[i] = R.in_scale * lds.pw[i + R.in_pow];
    }
    if constexpr (OUT) {
        for (int i = threadIdx.x; i < C * 16; i += Z::NT) {
            const int gap = 16 * (i >> 8) + (i >> 2 & 15) - (4 * (i >> 6 & 3) + (i & 3));
            lds.wp[i] = gap >= 0 ? R.p_scale * lds.pw[gap] : 0.f;
        }
        // blocks above the diagonal that a 32-deep step reads
        for (int i = threadIdx.x; i < NS * C * C / 2; i += Z::NT)
            reinterpret_cast<uint32_t*>(lds.p)[i] = 0;
    }

    constexpr int BLOCKS = NB * (NB + 1) / 2, MINE = (BLOCKS + NW - 1) / NW;
    // of a lane's 4 values of its blocks of P, two by two: all bits of those on and below the
    // diagonal
    uint32_t keep[OUT ? MINE : 1][2];
    if constexpr (OUT)
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int at = wave + q * NW, row = l16 - 4 * g;
            const bool below = at != 0 && at != 2 && at != 5 && at != 9;
            keep[q][0] = below || row > 0 ? ~0u : (row == 0 ? 0xffffu : 0u);
            keep[q][1] = below || row > 2 ? ~0u : (row == 2 ? 0xffffu : 0u);
        }

    // A chunk of n steps from u0; FULL: n = C.
    auto chunk = [&](auto full, int64_t u0, int n) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        if (!WIDE) fetch(u0);  // (an element a register: they would spill if kept for a chunk)
        lds_barrier();         // the tiles of the last chunk are read
        if (OUT) rx.template store<FULL>(lds.x, R.dx, n, 0);
        ry.template store<FULL>(lds.y, R.dx, n, 0);
        rz.template store<FULL>(lds.z, R.dz, n, z0);
        lds_barrier();
        if (WIDE && u0 + C < u_stop) fetch(u0 + C);

        if constexpr (OUT) {
            // P^T in 16 x 16 blocks on and below the diagonal, shared out among the waves
#pragma unroll
            for (int q = 0; q < MINE; ++q) {
                const int at = wave + q * NW;
                if (at >= BLOCKS) break;
                const int bu = (at >= 1) + (at >= 3) + (at >= 6), bw = at - bu * (bu + 1) / 2;
                floatx4 acc = {0.f, 0.f, 0.f, 0.f};
                const bf16_t* py = lds.y + (16 * bw + l16) * YS;
                const bf16_t* px = lds.x + (16 * bu + l16) * XS;
#pragma unroll
                for (int k = 0; k < DX / 32; ++k)
                    acc = mma<NP>(read_rows<NP>(py + 32 * k, YP, g),
                                  read_rows<NP>(px + 32 * k, XP, g), acc);
                const f32x4 wp = *reinterpret_cast<const f32x4*>(lds.wp + ((bu - bw) * 64 + lane) * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r] *= wp[r];
                    if (!FULL) acc[r] = wp[r] == 0.f ? 0.f : acc[r];
                }
                uint32_t p0[NS], p1[NS];
                split_pair<NS>(acc[0], acc[1], p0);
                split_pair<NS>(acc[2], acc[3], p1);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    *reinterpret_cast<uint2*>(lds.p + j * C * C + ((bu * NB + bw) * 64 + lane) * 4) =
                        uint2{p0[j] & keep[q][0], p1[j] & keep[q][1]};
            }
            lds_barrier();
        }

        Frag<NP> zf[C / 32][WN];
#pragma unroll
        for (int k = 0; k < C / 32; ++k)
#pragma unroll
            for (int m = 0; m < WN; ++m)
                zf[k][m] = read_column<NP>(lds.z + 32 * k * ZS + 16 * (WN * wave + m), ZP, ZS, lane);

        if constexpr (OUT) {
            Frag<NS> sf[DX / 32][WN];
#pragma unroll
            for (int k = 0; k < DX / 32; ++k)
#pragma unroll
                for (int m = 0; m < WN; ++m) sf[k][m] = frag_of<NS>(S[2 * k][m], S[2 * k + 1][m]);
            const int64_t e0 = ((b * a.steps + from + dir * (u0 + l16)) * a.heads + head) * R.dz + zw + 4 * g;
            const int64_t es = dir * 16 * a.heads * R.dz;
#pragma unroll
            for (int bu = 0; bu < NB; ++bu) {
                floatx4 acc[WN] = {};
                const bf16_t* px = lds.x + (16 * bu + l16) * XS;
#pragma unroll
                for (int k = 0; k < DX / 32; ++k) {
                    const auto xf = read_split<NP>(px + 32 * k, XP, 16, g);
#pragma unroll
                    for (int m = 0; m < WN; ++m) acc[m] = mma<NS>(sf[k][m], xf, acc[m]);
                }
                const float wx = lds.wx[16 * bu + l16];
#pragma unroll
                for (int m = 0; m < WN; ++m) acc[m] *= wx;
                if (!FULL && wx == 0.f)
#pragma unroll
                    for (int m = 0; m < WN; ++m) acc[m] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k <= bu / 2; ++k) {
                    // (a lane's 4 values of a block lie at lane * 4; those of the next block
                    // down 256 further)
                    const auto pf = read_split<NS>(
                        lds.p + ((bu * NB + 2 * k) * 64 + l16) * 4 + 60 * g, C * C, 256, g);
#pragma unroll
                    for (int m = 0; m < WN; ++m) acc[m] = mma<NS>(zf[k][m], pf, acc[m]);
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
            Frag<3> zw8[WN];
#pragma unroll
            for (int m = 0; m < WN; ++m) zw8[m] = weigh(zf[k][m], w);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const auto yf = read_column<NP>(lds.y + 32 * k * YS + 16 * i, YP, YS, lane);
#pragma unroll
                for (int m = 0; m < WN; ++m) S[i][m] = mma<3>(yf, zw8[m], S[i][m]);
            }
        }
    };
    // Steps without weight for one another (the later of a pair, or far apart under a strong
    // decay) may overflow in their product, which is cleared, not multiplied by 0. Below the
    // diagonal a weight is 0 only where the least one is: such a head takes the copy with bounds
    // for all chunks, which looks at each weight.
    bool faint = false;
    if (OUT && u_begin < u_stop) {
        const float least = fminf(lds.pw[C], 1.f);
        faint = R.p_scale * least == 0.f || R.in_scale * least == 0.f;
    }
    int64_t u0 = u_begin;
    if (!faint)
        for (; u0 + C <= u_stop; u0 += C) chunk(std::true_type{}, u0, C);
    for (; u0 < u_stop; u0 += C) chunk(std::false_type{}, u0, (int)min(u_stop - u0, (int64_t)C));

    // steps past the length
    if constexpr (OUT) {
        const int64_t lo = u_begin > len ? u_begin : len;
        constexpr int V = WIDE ? 16 / sizeof(T) : 1, G = Z::ZC / V;
        const int rows = u_end > lo ? (int)(u_end - lo) : 0;
        const int z = z0 + threadIdx.x % G * V;  // (G divides the workgroup's threads)
        if (z < R.dz) {
            const int64_t e = ((b * a.steps + lo) * a.heads + head) * R.dz + z;
            const int64_t es = (int64_t)a.heads * R.dz;
            for (int row = threadIdx.x / G; row < rows; row += Z::NT / G) {
                if (R.out32)
                    store_vec<float, V>(static_cast<float*>(R.out) + e + row * es, Vec<float, V>{});
                else
                    store_vec<T, V>(static_cast<T*>(R.out) + e + row * es, Vec<T, V>{});
            }
        }
    }

    float* s = nullptr;
    int si = R.seg_i, sj = R.seg_j;
    if (!OUT) {
        s = R.seg + (bh * a.nseg + seg) * ((int64_t)R.dx * R.dz);
    } else if (last && R.s1) {
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
    const int64_t units = a.batch * (a.heads / a.group) * a.nseg;
    const int64_t blocks = (units + 7) / 8 * 8 * a.group * ztiles;
    return in_launches(blocks, [&](int64_t first, unsigned n) {
        const dim3 grid(n, (unsigned)a.nrun);
        if (wide)
            attend_walk_kernel<T, DX, NW, WN, OUT, true>
                <<<grid, 64 * NW, 0, st>>>(a, first, units, ztiles);
        else
            attend_walk_kernel<T, DX, NW, WN, OUT, false>
                <<<grid, 64 * NW, 0, st>>>(a, first, units, ztiles);
    });
}

template <class T>
hipError_t launch_attend_walk(const AttendArgs& a, bool maps, hipStream_t st) {
    int dx = 0, dz = 0;
    for (int r = 0; r < a.nrun; ++r) {
        dx = a.run[r].dx > dx ? a.run[r].dx : dx;
        dz = a.run[r].dz > dz ? a.run[r].dz : dz;
    }
    // a CU with one workgroup alone: eight waves with one column tile each rather than four
    // with two (gradient of 4 x 2048 steps of 16 heads, 192 workgroups: 146 us against 163; two
    // workgroups a CU, 512 for 32768 steps of 16 heads: 252 against 233)
    const bool few = a.batch * a.heads * a.nseg * a.nrun <= 256;
    // small heads: two waves hold all columns of z; wide ones: two column tiles a wave, which
    // share what it reads of x and y
#define SYMNMF_WALK(DX, NW, WN) \
    return maps ? attend_walk_as<T, DX, NW, WN, false>(a, st) \
                : attend_walk_as<T, DX, NW, WN, true>(a, st)
    if (dx <= 32 && dz <= 32) SYMNMF_WALK(32, 2, 1);
    if (dx <= 32) SYMNMF_WALK(32, 4, 1);
    if (dx <= 64 && dz <= 32) SYMNMF_WALK(64, 2, 1);
    if (dx <= 64) SYMNMF_WALK(64, 4, 1);
    // (fp32's planes leave LDS for two workgroups a CU only with one column tile)
    constexpr int W = Planes<T>::N < 3 ? 2 : 1;
    if (dx <= 96 && dz <= 64) SYMNMF_WALK(96, 4, 1);
    if (dx <= 96) SYMNMF_WALK(96, 4, W);
    if (dx <= 128 && dz <= 64) SYMNMF_WALK(128, 4, 1);
    if constexpr (W == 2)
        if (dx <= 128 && few) SYMNMF_WALK(128, 8, 1);
    if (dx <= 128) SYMNMF_WALK(128, 4, W);
    SYMNMF_WALK(256, 4, 1);
#undef SYMNMF_WALK
}

}  // namespace symnmf
