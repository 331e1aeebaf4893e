// Shared by the sequence operators (k_embed.hip, k_scan.hip, k_logprob.hip and
// their host side seq.cpp): element types, vector loads and the launchers.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace symnmf {

// Element types of the C ABI (enum symnmf_dtype, enum symnmf_index).
enum : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
enum : int { kI32 = 0, kI64 = 1 };
inline int dtype_bytes(int t) { return t == kF32 ? 4 : 2; }

struct bf16_t {
    uint16_t bits;
};
struct f16_t {
    _Float16 v;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) {
    return __uint_as_float((uint32_t)v.bits << 16);
}
__device__ __forceinline__ float to_f32(f16_t v) { return (float)v.v; }

// One rounding to nearest even (the conversion instruction; NaN stays NaN).
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
    return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)v)};
}
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float v) {
    return f16_t{(_Float16)v};
}

// V consecutive elements, moved as one access of up to 16 bytes at any element's
// address: global loads and stores need no more alignment than that here, so
// rows of odd length keep their wide accesses (the compiler picks the widest
// access the target allows for the copy).
template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};
template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
    Vec<T, V> v;
    __builtin_memcpy(&v, p, sizeof(T) * V);
    return v;
}
template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& v) {
    __builtin_memcpy(p, &v, sizeof(T) * V);
}

// A launch takes fewer than 2^32 threads along a grid's first dimension. Work of
// `blocks` workgroups goes out as launches of at most kMaxBlocks, which stay below
// that with 1024 threads each; every one fills the chip for a millisecond or so.
// launch(first, n): the workgroups first ... first + n - 1.
constexpr int64_t kMaxBlocks = int64_t(1) << 20;
template <class F>
hipError_t in_launches(int64_t blocks, F&& launch) {
    for (int64_t first = 0; first < blocks; first += kMaxBlocks) {
        launch(first, (unsigned)(blocks - first < kMaxBlocks ? blocks - first : kMaxBlocks));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// symnmf_workspace_bytes for the sequence operators; 0 for invalid sizes (seq.cpp).
size_t seq_workspace_bytes(int op, int64_t n, int32_t k, int64_t T);

// ---- launchers (seq.cpp checks the arguments) ------------------------------

struct EmbedArgs {
    const void* table;
    int table_type;
    int64_t rows, width, ldt;
    const void* ids;
    int id_type;
    int64_t count;
    float scale;
    void* out;
    int out_type;
    int64_t ldo;
};
hipError_t launch_embed(const EmbedArgs& a, hipStream_t st);

struct EmbedGradArgs {
    const void* dout;
    int dout_type;
    int64_t count, width, ldd;
    const void* ids;
    int id_type;
    float scale;
    int accumulate;
    void* dtable;
    int dtable_type;
    int64_t rows, ldt;
    void* ws;
};
size_t embed_grad_ws_bytes(int64_t rows, int64_t width, int64_t count);
hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t st);

constexpr int kScanChunk = 128;  // steps between the states a forward scan keeps

struct ScanArgs {
    int type;
    int64_t batch, steps, width;
    const void* x;
    int64_t x_b, x_t;  // strides of batch and time in elements
    const void* gate;
    int64_t g_b, g_t;
    const int32_t* lengths;  // nullable
    const float* h0;         // nullable, batch x width
    // forward
    void* h;  // batch x steps x width, dense
    float* last;    // nullable
    float* states;  // forward: nullable, written; backward: read
    // backward
    const void* dh;
    int64_t d_b, d_t;
    const float* dlast;  // nullable
    void* dx;            // dense
    void* dgate;         // dense
    float* dh0;          // nullable
    void* ws;
};
size_t scan_ws_bytes(int64_t batch, int64_t steps, int64_t width);
hipError_t launch_scan(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_grad(const ScanArgs& a, hipStream_t st);

constexpr int kMaxTop = 32;  // most alternatives a row can be asked for
constexpr int64_t kMaxVocab = 4000000;  // 64 slices of 256 KiB hold a float32 row

struct LogprobArgs {
    int type;
    int64_t count, vocab, ld;
    const void* logits;
    const void* tokens;
    int token_type;
    float scale;
    float* logp;
    float* entropy;
    float* lse;
    int top;
    float* top_logp;
    int32_t* top_ids;
    // gradient
    const float* dlogp;
    const float* dentropy;  // nullable
    void* dlogits;
    int64_t ldd;
    void* ws;
};
size_t logprob_ws_bytes(int64_t vocab, int top, int64_t count);
hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t st);
hipError_t launch_logprobs_grad(const LogprobArgs& a, hipStream_t st);

}  // namespace symnmf
