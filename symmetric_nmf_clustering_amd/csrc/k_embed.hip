// Event embedding: out[i] = scale * table[ids[i]], and its gradient
//   dtable[v] = scale * sum_{i : ids[i] = v} dout[i].
//
// The gradient sorts the tokens by id (stable, so a row's terms stay in the
// order of the tokens), cuts the sorted list into chunks and lets one group
// of threads add each chunk's rows in order in fp32. A row whose terms lie in
// one chunk is written at once; the others leave one partial per chunk, which
// a second kernel adds in chunk order. No floating-point atomics: the result
// is the same on every run.
#include <algorithm>

#include "common.h"
#include "seq.h"

namespace symnmf {
namespace {

// ---- lookup ------------------------------------------------------------------

// One row per group of `lx` lanes (a power of two <= 256), V elements a lane
// and step. An id < 0 is an empty slot (zeros); one past the table gives NaN.
template <class TI, class TO, class ID, int V>
__global__ __launch_bounds__(256) void embed_kernel(const TI* __restrict__ table, int64_t rows,
                                                    int width, int64_t ldt,
                                                    const ID* __restrict__ ids, int64_t count,
                                                    float scale, TO* __restrict__ out, int64_t ldo,
                                                    int lx_log2, int64_t first) {
    const int lx = 1 << lx_log2;
    const int lane = threadIdx.x & (lx - 1);
    const int64_t i = (first + blockIdx.x) * (256 >> lx_log2) + (threadIdx.x >> lx_log2);
    if (i >= count) return;
    const int64_t id = (int64_t)ids[i];
    const bool in = id >= 0 && id < rows;
    const float fill = id < 0 ? 0.f : __builtin_nanf("");
    const TI* src = table + (in ? id : 0) * ldt;
    TO* dst = out + i * ldo;
    if (width < V) {
        for (int c = lane; c < width; c += lx) dst[c] = from_f32<TO>(in ? to_f32(src[c]) * scale : fill);
        return;
    }
    for (int c0 = lane * V; c0 < width; c0 += lx * V) {
        const int c = min(c0, width - V);  // the last access of a row ends with it
        Vec<TO, V> o;
        if (in) {
            const Vec<TI, V> v = load_vec<TI, V>(src + c);
#pragma unroll
            for (int u = 0; u < V; ++u) o.e[u] = from_f32<TO>(to_f32(v.e[u]) * scale);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) o.e[u] = from_f32<TO>(fill);
        }
        store_vec<TO, V>(dst + c, o);
    }
}

// ---- gradient ------------------------------------------------------------------

constexpr int kSortMaxBits = 9;              // digit of one sort pass
constexpr int kSortMaxBins = 1 << kSortMaxBits;
constexpr int kSortMaxBlocks = 128;

// How a list of `count` ids below `rows` is sorted: passes of `bits` bits from
// the lowest, `nblk` blocks of `tile` tokens.
struct SortPlan {
    int bits, passes, nblk, tile;
};
SortPlan sort_plan(int64_t rows, int64_t count) {
    SortPlan p;
    int need = 1;
    while (need < 32 && (rows >> need) > 0) ++need;  // the key `rows` (no row) included
    p.passes = (need + kSortMaxBits - 1) / kSortMaxBits;
    p.bits = (need + p.passes - 1) / p.passes;
    int64_t tile = 1024;
    while ((count + tile - 1) / tile > kSortMaxBlocks) tile *= 2;
    p.tile = (int)tile;
    p.nblk = (int)((count + tile - 1) / tile);
    return p;
}

template <class ID>
__device__ __forceinline__ uint32_t key_of(ID id, int64_t rows) {
    return id >= 0 && (int64_t)id < rows ? (uint32_t)id : (uint32_t)rows;
}

// First pass's keys come from the ids, later ones from the previous pass.
template <class ID>
struct FirstKeys {
    const ID* ids;
    int64_t rows;
    __device__ uint32_t key(int64_t i) const { return key_of(ids[i], rows); }
    __device__ int32_t pos(int64_t i) const { return (int32_t)i; }
};
struct NextKeys {
    const uint32_t* keys;
    const int32_t* at;
    __device__ uint32_t key(int64_t i) const { return keys[i]; }
    __device__ int32_t pos(int64_t i) const { return at[i]; }
};

// The next place of a digit's token in the wave's table `at` (digit -> next
// place), for 64 tokens at once and in lane order: equal digits find each other
// by one ballot per bit, the first of them moves the table on.
__device__ __forceinline__ int wave_place(int32_t* at, uint32_t digits, int bits, bool on) {
    const int d = (int)(digits & ((1u << bits) - 1u));
    uint64_t same = __ballot(on);
#pragma unroll
    for (int b = 0; b < kSortMaxBits; ++b)
        if (b < bits) {  // uniform
            const uint64_t one = __ballot((d >> b) & 1);
            same &= ~(one ^ (uint64_t)(int64_t)-((d >> b) & 1));
        }
    const int rank = __popcll(same & ((1ull << (threadIdx.x & 63)) - 1ull));
    const int place = on ? at[d] + rank : 0;
    wave_lds_sync();
    if (on && rank == 0) at[d] += __popcll(same);
    wave_lds_sync();
    return place;
}

// Zeros over a table of `rows` rows of `row_words` 4-byte words, `ld_words`
// apart (any type: zero is all bits clear), or of 2-byte elements where the
// layout is not one of whole words.
struct ZeroFill {
    void* p;
    int64_t rows, width, ld;  // in units of `unit` bytes
    int unit;                 // 16, 4 or 2
    template <class W>
    __device__ void put(int64_t part, int64_t parts) const {
        W zero{};
        W* q = static_cast<W*>(p);
        const int64_t step = parts * blockDim.x;
        int64_t e = part * blockDim.x + threadIdx.x;
        if (ld == width) {
            for (; e < rows * width; e += step) q[e] = zero;
        } else {
            for (; e < rows * width; e += step) q[e / width * ld + e % width] = zero;
        }
    }
    __device__ void run(int64_t part, int64_t parts) const {
        if (unit == 16)
            put<uint4>(part, parts);
        else if (unit == 4)
            put<uint32_t>(part, parts);
        else
            put<uint16_t>(part, parts);
    }
};

constexpr int kFillRows = 8;  // rows a thread clears, their flags read together

// Zeros over the rows that no token names, as 2^lx lanes a row; `words` of `unit`
// bytes to a row.
struct AbsentFill {
    void* p;
    const uint8_t* present;
    int64_t words, ld;
    int unit, lx;
    int64_t rows;
    __host__ __device__ int64_t per_block() const { return (int64_t)(256 >> lx) * kFillRows; }
    __host__ __device__ int64_t blocks() const { return (rows + per_block() - 1) / per_block(); }
    template <class W>
    __device__ void put(int64_t part) const {
        const int lane = threadIdx.x & ((1 << lx) - 1), groups = 256 >> lx;
        const int64_t v0 = part * per_block() + (threadIdx.x >> lx);
        uint8_t is[kFillRows];
#pragma unroll
        for (int u = 0; u < kFillRows; ++u)
            is[u] = v0 + u * groups < rows ? present[v0 + u * groups] : 1;
        W zero{};
#pragma unroll
        for (int u = 0; u < kFillRows; ++u)
            if (!is[u]) {
                W* q = static_cast<W*>(p) + (v0 + u * groups) * ld;
                for (int64_t c = lane; c < words; c += 1 << lx) q[c] = zero;
            }
    }
    __device__ void run(int64_t part, int64_t parts) const {
        for (; part < blocks(); part += parts) {
            if (unit == 16)
                put<uint4>(part);
            else if (unit == 4)
                put<uint32_t>(part);
            else
                put<uint16_t>(part);
        }
    }
};

// hist[b][digit] of block b's tile. The first pass also clears the table's presence flags, which its scatter sets.
template <class SRC>
__global__ __launch_bounds__(256) void sort_hist_kernel(SRC src, int64_t count, int tile, int shift,
                                                        int bins, int32_t* __restrict__ hist,
                                                        uint8_t* __restrict__ present,
                                                        int64_t rows) {
    __shared__ int32_t h[kSortMaxBins];
    for (int b = threadIdx.x; b < bins; b += 256) h[b] = 0;
    if (present)
        for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < rows;
             v += (int64_t)gridDim.x * 256)
            present[v] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * tile;
    const int64_t hi = lo + tile < count ? lo + tile : count;
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256)
        atomicAdd(&h[(src.key(i) >> shift) & (bins - 1)], 1);  // counts: order-free
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += 256) hist[(int64_t)blockIdx.x * bins + b] = h[b];
}

// Moves a tile's tokens to their places, in order: the place of a token is the
// number of tokens with a smaller digit, plus those with its digit in earlier
// blocks, earlier waves' quarters of the tile and earlier lanes of its wave.
template <class SRC>
__global__ __launch_bounds__(256) void sort_scatter_kernel(
    SRC src, int64_t count, int tile, int shift, int bits, const int32_t* __restrict__ hist,
    uint32_t* __restrict__ keys_out, int32_t* __restrict__ pos_out, uint8_t* __restrict__ present,
    int64_t rows) {
    __shared__ int32_t at[4][kSortMaxBins];  // counts, then next place, by wave and digit
    __shared__ int32_t wtot[4];
    const int bins = 1 << bits, t = threadIdx.x, lane = t & 63, w = t >> 6;
    const int nblk = gridDim.x, blk = blockIdx.x;
    for (int b = t; b < 4 * kSortMaxBins; b += 256) (&at[0][0])[b] = 0;
    // this block's first place for each digit: thread t owns the digits 2t, 2t + 1
    // (bins is even); sixteen blocks' counts in flight
    int before[2] = {0, 0}, total[2] = {0, 0};
    if (2 * t < bins) {
        const int2* h2 = reinterpret_cast<const int2*>(hist) + t;
        for (int k0 = 0; k0 < nblk; k0 += 16) {
            int2 v[16];
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] = k0 + u < nblk ? h2[(int64_t)(k0 + u) * (bins / 2)] : make_int2(0, 0);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                total[0] += v[u].x;
                total[1] += v[u].y;
                if (k0 + u < blk) {
                    before[0] += v[u].x;
                    before[1] += v[u].y;
                }
            }
        }
    }
    int incl = total[0] + total[1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o, 64);
        if (lane >= o) incl += v;
    }
    if (lane == 63) wtot[w] = incl;
    __syncthreads();
    int base = incl - total[0] - total[1];
    for (int k = 0; k < w; ++k) base += wtot[k];
    const int first0 = base + before[0], first1 = base + total[0] + before[1];
    // counts of each wave's quarter
    const int quarter = tile / 4;
    const int64_t lo = (int64_t)blk * tile + (int64_t)w * quarter;
    int64_t hi = lo + quarter;
    if (hi > count) hi = count;
    constexpr int K = 4;  // rounds of 64 tokens whose keys are loaded together
    for (int64_t r = lo; r < hi; r += 64 * K) {
        uint32_t key[K];
#pragma unroll
        for (int u = 0; u < K; ++u) key[u] = r + 64 * u + lane < hi ? src.key(r + 64 * u + lane) : 0u;
#pragma unroll
        for (int u = 0; u < K; ++u)
            if (r + 64 * u + lane < hi) atomicAdd(&at[w][(key[u] >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int b = 2 * t + u;
        if (b < bins) {
            int p = u ? first1 : first0;
            for (int k = 0; k < 4; ++k) {
                const int n = at[k][b];
                at[k][b] = p;
                p += n;
            }
        }
    }
    __syncthreads();
    for (int64_t r = lo; r < hi; r += 64 * K) {  // uniform over the wave
        uint32_t key[K];
        int32_t pos[K];
#pragma unroll
        for (int u = 0; u < K; ++u) {
            const int64_t i = r + 64 * u + lane;
            key[u] = i < hi ? src.key(i) : 0u;
            pos[u] = i < hi ? src.pos(i) : 0;
        }
#pragma unroll
        for (int u = 0; u < K; ++u) {
            const bool on = r + 64 * u + lane < hi;
            const int place = wave_place(at[w], key[u] >> shift, bits, on);
            if (on) {
                keys_out[place] = key[u];
                pos_out[place] = pos[u];
                if (present && (int64_t)key[u] < rows) present[key[u]] = 1;
            }
        }
    }
}

// Short lists: a token's place is the number of tokens that go before it, counted
// directly: 16 tokens per workgroup, 16 threads to a token, every id in LDS.
// One launch, quadratic but wide: 5000 tokens take 9.6 us, where one workgroup's
// passes in LDS took 16.3 and the four launches of the long lists' sort 23.6. The
// launch's other workgroups clear the table.
constexpr int64_t kSmallCount = 8192;
constexpr int kRankTokens = 16;

template <class ID>
__global__ __launch_bounds__(256) void sort_small_kernel(const ID* __restrict__ ids, int64_t rows,
                                                         int count, int nblk,
                                                         uint32_t* __restrict__ keys_out,
                                                         int32_t* __restrict__ pos_out,
                                                         ZeroFill zf) {
    __shared__ __align__(16) uint32_t key[kSmallCount];
    const int t = threadIdx.x;
    if ((int)blockIdx.x >= nblk) {
        zf.run((int)blockIdx.x - nblk, (int)gridDim.x - nblk);
        return;
    }
    const int padded = (count + 63) / 64 * 64;  // 16 threads x 4 ids
    // 16 bytes of ids a load, all of a thread's on their way together
    constexpr int P = 16 / sizeof(ID), L = (int)kSmallCount / (256 * P);
    Vec<ID, P> id[L];
#pragma unroll
    for (int q = 0; q < L; ++q) {
        const int i0 = (t + 256 * q) * P;
        if (i0 + P <= count) {
            id[q] = load_vec<ID, P>(ids + i0);
        } else {
#pragma unroll
            for (int u = 0; u < P; ++u) id[q].e[u] = i0 + u < count ? ids[i0 + u] : 0;
        }
    }
#pragma unroll
    for (int q = 0; q < L; ++q)
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int i0 = (t + 256 * q) * P + u;
            if (i0 < padded) key[i0] = i0 < count ? key_of(id[q].e[u], rows) : 0xffffffffu;
        }
    __syncthreads();
    const int i = min((int)blockIdx.x * kRankTokens + (t >> 4), count - 1);
    const bool on = (int)blockIdx.x * kRankTokens + (t >> 4) < count;
    const uint32_t mine = key[i];
    // equal ids stay in token order: before the four that hold i, up to `mine`
    // counts, from there on only what is smaller (and the few between)
    int n = 0;
#pragma unroll 4
    for (int j = 4 * (t & 15); j < padded; j += 64) {
        const uint4 k = *reinterpret_cast<const uint4*>(key + j);
        const uint32_t below = mine + (j + 4 <= i ? 1u : 0u);
        n += (k.x < below) + (k.y < below) + (k.z < below) + (k.w < below);
    }
    if ((t & 15) == 0)
        for (int j = i & ~3; j < i; ++j) n += key[j] == mine;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
    if ((t & 15) == 0 && on) {
        keys_out[n] = mine;
        pos_out[n] = i;
    }
}

inline int log2_up(int64_t v, int most) {
    int l = 0;
    while (l < most && (int64_t(1) << l) < v) ++l;
    return l;
}

// Sorted tokens per chunk of the sum: as few as leave the launch at about 4096
// waves, 8 to 128. Finer chunks hide more latency but leave more partials
// (32768 rows of 1024: 32 tokens 125 us, 16 tokens 137; 65536 rows of 24: 8 tokens
// 48 us, 32 tokens 55).
int chunk_len(int64_t count, int64_t width) {
    const int64_t lanes = int64_t(1) << log2_up((width + 3) / 4, 8);
    int c = 8;
    while (c < 128 && count * lanes > (int64_t)c * 64 * 4096) c *= 2;
    return c;
}

constexpr int kSumRows = 8;  // tokens whose rows a thread has in flight

template <class TO, int V>
__device__ __forceinline__ void put_row(TO* dst, int c, int width, const float (&acc)[V],
                                        float scale, int accumulate) {
    if (c + V <= width) {
        Vec<TO, V> o;
        if (accumulate) {
            const Vec<TO, V> old = load_vec<TO, V>(dst + c);
#pragma unroll
            for (int u = 0; u < V; ++u)
                o.e[u] = from_f32<TO>(to_f32(old.e[u]) + scale * acc[u]);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) o.e[u] = from_f32<TO>(scale * acc[u]);
        }
        store_vec<TO, V>(dst + c, o);
    } else {
        for (int u = 0; u < V; ++u)
            if (c + u < width) {
                const float old = accumulate ? to_f32(dst[c + u]) : 0.f;
                dst[c + u] = from_f32<TO>(old + scale * acc[u]);
            }
    }
}

// Group of lx lanes per chunk and column tile (blockIdx.y). Blocks past the
// chunks clear the rest of the rows no token names.
template <class TD, class TO, int V>
__global__ __launch_bounds__(256) void embed_grad_sum_kernel(
    const TD* __restrict__ dout, int64_t ldd, int width, const uint32_t* __restrict__ keys,
    const int32_t* __restrict__ pos, int64_t count, int clen, int64_t nchunks, int sum_blocks,
    float scale, int accumulate, TO* __restrict__ dtable, int64_t ldt, int64_t rows,
    AbsentFill af, float* __restrict__ part, int ldpart, int lx_log2) {
    const int lx = 1 << lx_log2, groups = 256 >> lx_log2;
    const int lane = threadIdx.x & (lx - 1), grp = threadIdx.x >> lx_log2;
    const int c = ((int)blockIdx.y * lx + lane) * V;
    if ((int)blockIdx.x >= sum_blocks) {
        if (blockIdx.y == 0) af.run((int)blockIdx.x - sum_blocks, (int)gridDim.x - sum_blocks);
        return;
    }
    const int64_t chunk = (int64_t)blockIdx.x * groups + grp;
    if (chunk >= nchunks || c >= width) return;
    const int64_t lo = chunk * clen;
    const int64_t hi = lo + clen < count ? lo + clen : count;
    const bool whole = c + V <= width;
    float acc[V] = {};
    uint32_t cur = keys[lo];
    bool head = lo > 0 && keys[lo - 1] == cur;  // the first row began in an earlier chunk
    for (int64_t e0 = lo; e0 < hi; e0 += kSumRows) {
        // the rows of kSumRows tokens on their way together
        uint32_t key[kSumRows];
        int32_t at[kSumRows];
        Vec<TD, V> v[kSumRows];
#pragma unroll
        for (int q = 0; q < kSumRows; ++q) {
            key[q] = e0 + q < hi ? keys[e0 + q] : (uint32_t)rows;
            at[q] = e0 + q < hi ? pos[e0 + q] : 0;
        }
#pragma unroll
        for (int q = 0; q < kSumRows; ++q) {
#pragma unroll
            for (int u = 0; u < V; ++u) v[q].e[u] = from_f32<TD>(0.f);
            if ((int64_t)key[q] < rows) {
                const TD* src = dout + (int64_t)at[q] * ldd + c;
                if (whole) {
                    v[q] = load_vec<TD, V>(src);
                } else {
                    for (int u = 0; u < V; ++u)
                        if (c + u < width) v[q].e[u] = src[u];
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kSumRows; ++q) {
            if (e0 + q >= hi) break;
            if (key[q] != cur) {
                if (head) {
#pragma unroll
                    for (int u = 0; u < V; ++u)
                        if (c + u < width) part[2 * chunk * ldpart + c + u] = acc[u];
                } else if ((int64_t)cur < rows) {
                    put_row<TO, V>(dtable + (int64_t)cur * ldt, c, width, acc, scale, accumulate);
                }
                head = false;
                cur = key[q];
#pragma unroll
                for (int u = 0; u < V; ++u) acc[u] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < V; ++u) acc[u] += to_f32(v[q].e[u]);
        }
    }
    if ((int64_t)cur >= rows) return;
    const bool tail = hi < count && keys[hi] == cur;
    if (head || tail) {
        const int64_t slot = 2 * chunk + (head ? 0 : 1);
#pragma unroll
        for (int u = 0; u < V; ++u)
            if (c + u < width) part[slot * ldpart + c + u] = acc[u];
    } else {
        put_row<TO, V>(dtable + (int64_t)cur * ldt, c, width, acc, scale, accumulate);
    }
}

// A row that began in this chunk and goes on: its tail partial here, then the
// head partials of the chunks that follow, in order.
template <class TO>
__global__ __launch_bounds__(256) void embed_grad_fold_kernel(
    const uint32_t* __restrict__ keys, int64_t count, int clen, int64_t nchunks, float scale,
    int accumulate, TO* __restrict__ dtable, int64_t ldt, int64_t rows, int width,
    const float* __restrict__ part, int ldpart, int lx) {
    const int64_t chunk = blockIdx.x;
    const int64_t lo = chunk * clen, hi = lo + clen;
    if (hi >= count) return;
    const uint32_t key = keys[hi];
    if ((int64_t)key >= rows || keys[hi - 1] != key) return;   // no row goes on
    if (keys[lo] == key && lo > 0 && keys[lo - 1] == key) return;  // it began earlier
    // the chunks after this one that hold terms of it begin with its key
    int64_t more = 0;
    for (;;) {
        const int64_t j = chunk + 1 + more + threadIdx.x;
        const int n = __syncthreads_count(j < nchunks && keys[j * clen] == key);
        more += n;
        if (n < 256) break;
    }
    // The partials are shared out over groups of 2^lx lanes, each of which adds a
    // run of them in order, 16 in flight; then the groups' sums in order. Rows of
    // partials are padded to a multiple of 4 (what the padding holds is not stored).
    __shared__ float4 sums[256];
    const int lane = threadIdx.x & ((1 << lx) - 1), grp = threadIdx.x >> lx, groups = 256 >> lx;
    const int64_t per = (more + groups) / groups, j0 = grp * per;  // the tail partial is the first
    const int64_t j1 = j0 + per < more + 1 ? j0 + per : more + 1;
    const int64_t step = 2 * (int64_t)ldpart;
    const int c = (int)((blockIdx.y << lx) + lane) * 4;
    float4 s = {0.f, 0.f, 0.f, 0.f};
    if (c < width) {
        const float* p = part + 2 * chunk * (int64_t)ldpart + c;
        for (int64_t j = j0; j < j1; j += 16) {
            float4 v[16];
#pragma unroll
            for (int u = 0; u < 16; ++u)
                if (j + u < j1)
                    v[u] = *reinterpret_cast<const float4*>(p + (j + u) * step +
                                                            (j + u == 0 ? ldpart : 0));
#pragma unroll
            for (int u = 0; u < 16; ++u)
                if (j + u < j1) {
                    s.x += v[u].x;
                    s.y += v[u].y;
                    s.z += v[u].z;
                    s.w += v[u].w;
                }
        }
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (grp != 0 || c >= width) return;
    for (int q = 1; q < groups; ++q) {
        const float4 o = sums[(q << lx) + lane];
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
    }
    const float r[4] = {s.x, s.y, s.z, s.w};
    put_row<TO, 4>(dtable + (int64_t)key * ldt, c, width, r, scale, accumulate);
}

// Short lists whose rows have few terms, in one launch: a workgroup takes the rows
// whose terms begin in its window of the sorted tokens. Rows of up to kRowTokens
// terms are added by one group of 2^lx lanes each, all terms on their way
// together; longer ones after that by all groups, each a run of the terms, and
// then the groups' sums in order. One workgroup per row is too little where a row
// takes thousands of terms, which the sizes cannot tell but do suggest: 5000
// tokens into 20000 x 24 take 17.4 us so, against 19.7 with partials and a fold;
// 2000 into 5000 x 257 16.8 against 22.0; but 8192 into 50 x 24 29.6 against 23.5
// and 8192 into 5000 x 1024 53 against 34. Column tiles (128 columns) are the grid's
// second dimension, of at most 65535.
bool by_rows(int64_t rows, int64_t width, int64_t count) {
    if (width > 65535 * 128) return false;
    return count <= 1024 || (count <= kSmallCount && count <= rows && count * width <= 1 << 19);
}
constexpr int kRowTokens = 16;

template <class TD, class TO>
__global__ __launch_bounds__(256) void embed_grad_rows_kernel(
    const TD* __restrict__ dout, int64_t ldd, int width, const uint32_t* __restrict__ keys,
    const int32_t* __restrict__ pos, int count, int window, float scale, int accumulate,
    TO* __restrict__ dtable, int64_t ldt, int64_t rows, int lx) {
    constexpr int V = 4, K = kRowTokens;
    __shared__ int longs[256];
    __shared__ int nlong;
    __shared__ float4 sums[256];
    const int lane = threadIdx.x & ((1 << lx) - 1), grp = threadIdx.x >> lx, groups = 256 >> lx;
    const int c = (int)((blockIdx.y << lx) + lane) * V;
    const bool whole = c + V <= width;
    // acc += the terms [p, p + n) of the sorted list, n <= K, in order
    auto add = [&](float(&acc)[V], int p, int n) {
        int32_t at[K];
        Vec<TD, V> v[K];
#pragma unroll
        for (int q = 0; q < K; ++q) at[q] = q < n ? pos[p + q] : 0;
#pragma unroll
        for (int q = 0; q < K; ++q) {
#pragma unroll
            for (int u = 0; u < V; ++u) v[q].e[u] = from_f32<TD>(0.f);
            if (q < n) {
                const TD* src = dout + (int64_t)at[q] * ldd + c;
                if (whole) {
                    v[q] = load_vec<TD, V>(src);
                } else {
                    for (int u = 0; u < V; ++u)
                        if (c + u < width) v[q].e[u] = src[u];
                }
            }
        }
#pragma unroll
        for (int q = 0; q < K; ++q)
            if (q < n)
#pragma unroll
                for (int u = 0; u < V; ++u) acc[u] += to_f32(v[q].e[u]);
    };
    if (threadIdx.x == 0) nlong = 0;
    __syncthreads();
    const int w0 = (int)blockIdx.x * window;
    for (int p = w0 + grp; p < min(w0 + window, count); p += groups) {
        const uint32_t key = keys[p];
        if ((int64_t)key >= rows || (p > 0 && keys[p - 1] == key)) continue;  // begins no row
        int n = 1;
#pragma unroll
        for (int q = 1; q <= K; ++q) n += p + q < count && keys[p + q] == key ? 1 : 0;
        if (n > K) {
            if (lane == 0) longs[atomicAdd(&nlong, 1)] = p;  // rows, in any order
        } else if (c < width) {
            float acc[V] = {};
            add(acc, p, n);
            put_row<TO, V>(dtable + (int64_t)key * ldt, c, width, acc, scale, accumulate);
        }
    }
    __syncthreads();
    for (int i = 0; i < nlong; ++i) {
        const int p = longs[i];
        const uint32_t key = keys[p];
        int n = 0;
        for (;;) {
            const int j = p + n + (int)threadIdx.x;
            const int m = __syncthreads_count(j < count && keys[j] == key);
            n += m;
            if (m < 256) break;
        }
        const int per = (n + groups - 1) / groups, end = p + min(n, (grp + 1) * per);
        float acc[V] = {};
        if (c < width)
            for (int q = p + grp * per; q < end; q += K) add(acc, q, min(K, end - q));
        sums[threadIdx.x] = float4{acc[0], acc[1], acc[2], acc[3]};
        __syncthreads();
        if (grp == 0 && c < width) {
            for (int g = 1; g < groups; ++g) {
                const float4 o = sums[(g << lx) + lane];
                acc[0] += o.x;
                acc[1] += o.y;
                acc[2] += o.z;
                acc[3] += o.w;
            }
            put_row<TO, V>(dtable + (int64_t)key * ldt, c, width, acc, scale, accumulate);
        }
        __syncthreads();
    }
}

template <class TI, class TO, class ID>
hipError_t embed_run(const EmbedArgs& a, hipStream_t st) {
    constexpr int V = sizeof(TI) == 4 || sizeof(TO) == 4 ? 4 : 8;
    const int lg = log2_up((a.width + V - 1) / V, 8);
    const int64_t per = 256 >> lg;
    return in_launches((a.count + per - 1) / per, [&](int64_t first, unsigned n) {
        hipLaunchKernelGGL((embed_kernel<TI, TO, ID, V>), dim3(n), dim3(256), 0, st,
                           (const TI*)a.table, a.rows, (int)a.width, a.ldt, (const ID*)a.ids,
                           a.count, a.scale, (TO*)a.out, a.ldo, lg, first);
    });
}
template <class TI, class TO>
hipError_t embed_id(const EmbedArgs& a, hipStream_t st) {
    return a.id_type == kI32 ? embed_run<TI, TO, int32_t>(a, st)
                             : embed_run<TI, TO, int64_t>(a, st);
}
template <class TI>
hipError_t embed_out(const EmbedArgs& a, hipStream_t st) {
    return a.out_type == kF32    ? embed_id<TI, float>(a, st)
           : a.out_type == kBF16 ? embed_id<TI, bf16_t>(a, st)
                                 : embed_id<TI, f16_t>(a, st);
}

struct GradLayout {
    uint32_t *k0, *k1;
    int32_t *p0, *p1, *hist;
    uint8_t* present;
    float* part;
    int ldpart;
    size_t bytes;
};
GradLayout grad_layout(void* ws, int64_t rows, int64_t width, int64_t count) {
    GradLayout L;
    const SortPlan p = sort_plan(rows, count);
    const int64_t nchunks = (count + chunk_len(count, width) - 1) / chunk_len(count, width);
    L.ldpart = (int)((width + 3) / 4 * 4);
    size_t off = 0;
    auto take = [&](size_t n) {
        char* q = ws ? static_cast<char*>(ws) + off : nullptr;
        off += (n + 255) / 256 * 256;
        return (void*)q;
    };
    L.k0 = (uint32_t*)take(4 * (size_t)count);
    L.k1 = (uint32_t*)take(4 * (size_t)count);
    L.p0 = (int32_t*)take(4 * (size_t)count);
    L.p1 = (int32_t*)take(4 * (size_t)count);
    const bool small = count <= kSmallCount;
    L.hist = (int32_t*)take(small ? 0 : 4 * (size_t)p.nblk << p.bits);
    L.present = (uint8_t*)take(small ? 0 : (size_t)rows);
    L.part = (float*)take(by_rows(rows, width, count) ? 0
                                                      : 8 * (size_t)nchunks * (size_t)L.ldpart);
    L.bytes = off;
    return L;
}

ZeroFill zero_fill(const EmbedGradArgs& a) {
    const int eb = dtype_bytes(a.dtable_type);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.dtable);
    ZeroFill z{a.dtable, a.rows, a.width, a.ldt, eb};
    if (a.ldt == a.width && a.rows * a.width * eb % 16 == 0) {  // one run of memory
        z.width = a.rows * a.width;
        z.rows = 1;
        z.ld = z.width;
    }
    for (int u = 16; u > eb; u /= 2)
        if (u != 8 && at % u == 0 && z.width * eb % u == 0 && (z.rows == 1 || z.ld * eb % u == 0)) {
            z.width = z.width * eb / u;
            z.ld = z.ld * eb / u;
            z.unit = u;
            break;
        }
    return z;
}

// The rows to clear one by one (none when adding, or where a short list's sort
// clears the whole table).
AbsentFill absent_fill(const EmbedGradArgs& a, const uint8_t* present) {
    const int eb = dtype_bytes(a.dtable_type);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.dtable);
    int unit = eb;
    for (int u : {4, 16})
        if (u > eb && at % u == 0 && a.width * eb % u == 0 && a.ldt * eb % u == 0) unit = u;
    AbsentFill f{a.dtable, present, a.width * eb / unit, a.ldt * eb / unit, unit, 0, 0};
    f.lx = log2_up(f.words, 8);
    f.rows = a.accumulate || a.count <= kSmallCount ? 0 : a.rows;
    return f;
}

template <class ID>
hipError_t sort_ids(const EmbedGradArgs& a, const GradLayout& L, const uint32_t** keys,
                    const int32_t** pos, hipStream_t st) {
    const SortPlan p = sort_plan(a.rows, a.count);
    if (a.count <= kSmallCount) {
        const ZeroFill zf = zero_fill(a);
        const int nblk = (int)((a.count + kRankTokens - 1) / kRankTokens);
        // a workgroup per 16 KiB to clear, up to sixteen per CU
        int64_t fill = a.accumulate ? 0 : (zf.rows * zf.width * zf.unit + 16383) / 16384;
        if (fill > 4096) fill = 4096;
        hipLaunchKernelGGL((sort_small_kernel<ID>), dim3((unsigned)(nblk + fill)), dim3(256), 0, st,
                           (const ID*)a.ids, a.rows, (int)a.count, nblk, L.k0, L.p0, zf);
        *keys = L.k0;
        *pos = L.p0;
        return hipGetLastError();
    }
    uint32_t* ko[2] = {L.k0, L.k1};
    int32_t* po[2] = {L.p0, L.p1};
    for (int s = 0; s < p.passes; ++s) {
        uint32_t* kd = ko[s & 1];
        int32_t* pd = po[s & 1];
        const int shift = s * p.bits;
        uint8_t* first = s == 0 ? L.present : nullptr;
        const dim3 g((unsigned)p.nblk), b(256);
        if (s == 0) {
            FirstKeys<ID> src{(const ID*)a.ids, a.rows};
            hipLaunchKernelGGL((sort_hist_kernel<FirstKeys<ID>>), g, b, 0, st, src, a.count, p.tile,
                               shift, 1 << p.bits, L.hist, first, a.rows);
            hipLaunchKernelGGL((sort_scatter_kernel<FirstKeys<ID>>), g, b, 0, st, src, a.count,
                               p.tile, shift, p.bits, L.hist, kd, pd, first, a.rows);
        } else {
            NextKeys src{ko[(s - 1) & 1], po[(s - 1) & 1]};
            hipLaunchKernelGGL((sort_hist_kernel<NextKeys>), g, b, 0, st, src, a.count, p.tile,
                               shift, 1 << p.bits, L.hist, first, a.rows);
            hipLaunchKernelGGL((sort_scatter_kernel<NextKeys>), g, b, 0, st, src, a.count, p.tile,
                               shift, p.bits, L.hist, kd, pd, first, a.rows);
        }
        *keys = kd;
        *pos = pd;
    }
    return hipGetLastError();
}

template <class TD, class TO>
hipError_t grad_run(const EmbedGradArgs& a, const GradLayout& L, const uint32_t* keys,
                    const int32_t* pos, const AbsentFill& af, hipStream_t st) {
    // 4 elements a thread, so many threads share a row's reads (bf16 rows of 1024
    // into a float32 table: 125 us against 136 with 8; rows of 1000 into a bf16
    // table: 45 against 60)
    constexpr int V = 4;
    if (by_rows(a.rows, a.width, a.count)) {
        // at most 32 lanes to a row: the groups share long rows between them
        const int lx = log2_up((a.width + V - 1) / V, 5), window = 256 >> lx;
        const dim3 g((unsigned)((a.count + window - 1) / window),
                     (unsigned)(((a.width + V - 1) / V + (1 << lx) - 1) >> lx));
        hipLaunchKernelGGL((embed_grad_rows_kernel<TD, TO>), g, dim3(256), 0, st,
                           (const TD*)a.dout, a.ldd, (int)a.width, keys, pos, (int)a.count, window,
                           a.scale, a.accumulate, (TO*)a.dtable, a.ldt, a.rows, lx);
        return hipGetLastError();
    }
    const int clen = chunk_len(a.count, a.width);
    const int64_t nchunks = (a.count + clen - 1) / clen;
    const int64_t nv = (a.width + V - 1) / V;
    const int lg = log2_up(nv, 8);
    const int64_t groups = 256 >> lg;
    const int64_t sum_blocks = (nchunks + groups - 1) / groups;
    // with at most 2^23 workgroups for the sum (128 tokens a chunk by then) the grid
    // stays below 2^24
    const int64_t fill = std::min<int64_t>(af.blocks(), 1 << 16);
    const unsigned cols = (unsigned)((nv + (1 << lg) - 1) >> lg);
    hipLaunchKernelGGL((embed_grad_sum_kernel<TD, TO, V>),
                       dim3((unsigned)(sum_blocks + fill), cols), dim3(256), 0, st,
                       (const TD*)a.dout, a.ldd, (int)a.width, keys, pos, a.count, clen, nchunks,
                       (int)sum_blocks, a.scale, a.accumulate, (TO*)a.dtable, a.ldt, a.rows,
                       af, L.part, L.ldpart, lg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || nchunks < 2) return e;
    const int fx = log2_up((a.width + 3) / 4, 8);
    const unsigned fy = (unsigned)(((a.width + 3) / 4 + (1 << fx) - 1) >> fx);
    hipLaunchKernelGGL((embed_grad_fold_kernel<TO>), dim3((unsigned)nchunks, fy), dim3(256), 0, st,
                       keys, a.count, clen, nchunks, a.scale, a.accumulate, (TO*)a.dtable, a.ldt,
                       a.rows, (int)a.width, L.part, L.ldpart, fx);
    return hipGetLastError();
}
template <class TD>
hipError_t grad_out(const EmbedGradArgs& a, const GradLayout& L, const uint32_t* keys,
                    const int32_t* pos, const AbsentFill& af, hipStream_t st) {
    return a.dtable_type == kF32    ? grad_run<TD, float>(a, L, keys, pos, af, st)
           : a.dtable_type == kBF16 ? grad_run<TD, bf16_t>(a, L, keys, pos, af, st)
                                    : grad_run<TD, f16_t>(a, L, keys, pos, af, st);
}

// dtable = 0 where there are no tokens at all.
__global__ __launch_bounds__(256) void zero_kernel(ZeroFill zf) { zf.run(blockIdx.x, gridDim.x); }

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t st) {
    return a.table_type == kF32    ? embed_out<float>(a, st)
           : a.table_type == kBF16 ? embed_out<bf16_t>(a, st)
                                   : embed_out<f16_t>(a, st);
}

size_t embed_grad_ws_bytes(int64_t rows, int64_t width, int64_t count) {
    if (count == 0) return 256;
    return grad_layout(nullptr, rows, width, count).bytes;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t st) {
    if (a.count == 0) {
        if (a.accumulate) return hipSuccess;
        hipLaunchKernelGGL(zero_kernel, dim3(1024), dim3(256), 0, st, zero_fill(a));
        return hipGetLastError();
    }
    const GradLayout L = grad_layout(a.ws, a.rows, a.width, a.count);
    const uint32_t* keys = nullptr;
    const int32_t* pos = nullptr;
    AbsentFill af = absent_fill(a, L.present);
    hipError_t e = a.id_type == kI32 ? sort_ids<int32_t>(a, L, &keys, &pos, st)
                                     : sort_ids<int64_t>(a, L, &keys, &pos, st);
    if (e != hipSuccess) return e;
    return a.dout_type == kF32    ? grad_out<float>(a, L, keys, pos, af, st)
           : a.dout_type == kBF16 ? grad_out<bf16_t>(a, L, keys, pos, af, st)
                                  : grad_out<f16_t>(a, L, keys, pos, af, st);
}

}  // namespace symnmf
