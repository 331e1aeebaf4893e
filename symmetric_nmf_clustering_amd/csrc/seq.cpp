// Host side of the sequence operators of include/symnmf.h: event embedding,
// gated scan, token log probabilities. Argument checks, then one launcher per
// call (k_embed.hip, k_scan.hip, k_logprob.hip). Every call is asynchronous.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "seq.h"
#include "symnmf.h"

using namespace symnmf;

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 30;

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
inline bool type_ok(int t) { return t == SYMNMF_F32 || t == SYMNMF_BF16 || t == SYMNMF_F16; }
inline bool index_ok(int t) { return t == SYMNMF_I32 || t == SYMNMF_I64; }
// A device array of elements of `bytes` bytes: not null, and aligned to them.
inline bool arr(const void* p, int bytes) {
    return p && reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}
inline bool arr_or_null(const void* p, int bytes) { return !p || arr(p, bytes); }
inline int index_bytes(int t) { return t == SYMNMF_I32 ? 4 : 8; }
inline bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
inline bool ws_fits(const void* ws, size_t got, size_t need) {
    return ws && reinterpret_cast<uintptr_t>(ws) % 256 == 0 && got >= need;
}
inline int done(hipError_t e) { return e == hipSuccess ? SYMNMF_OK : SYMNMF_E_HIP; }

// Sizes the scan's kernels index with: steps and channels of a row in 32 bits. Its
// workgroups (batch rows x channel tiles) are counted in 64 and sent out in several
// launches where one does not take them.
bool scan_sizes_ok(int64_t batch, int64_t steps, int64_t width) {
    return in(batch, 1, 65535) && in(steps, 0, kMaxCount) && in(width, 1, 1 << 24) &&
           batch * width <= int64_t(1) << 36;
}

}  // namespace

namespace symnmf {

size_t seq_workspace_bytes(int op, int64_t n, int32_t k, int64_t T) {
    switch (op) {
        case SYMNMF_OP_EMBED_GRAD:
            if (n < 1 || n > kMaxCount || k < 1 || k > (1 << 24) || T < 0 || T > kMaxCount)
                return 0;
            return embed_grad_ws_bytes(n, k, T);
        case SYMNMF_OP_GATED_SCAN:
            if (!scan_sizes_ok(k, T, n)) return 0;
            return scan_ws_bytes(k, T, n);
        case SYMNMF_OP_TOKEN_LOGPROBS:
            if (n < 1 || n > kMaxVocab || k < 0 || k > kMaxTop || T < 0 || T > kMaxCount) return 0;
            return logprob_ws_bytes(n, k, T);
        default: return 0;
    }
}

}  // namespace symnmf

extern "C" {

int symnmf_embed(const void* table, int table_type, int64_t rows, int64_t width, int64_t ldt,
                 const void* ids, int id_type, int64_t count, float scale, void* out, int out_type,
                 int64_t ldo, void* hip_stream) {
    if (!type_ok(table_type) || !type_ok(out_type) || !index_ok(id_type) ||
        !in(rows, 1, kMaxCount) || !in(width, 1, 1 << 24) || ldt < width || ldo < width ||
        !in(count, 0, kMaxCount) || !arr(table, dtype_bytes(table_type)))
        return SYMNMF_E_INVALID;
    if (count == 0) return SYMNMF_OK;
    if (!arr(ids, index_bytes(id_type)) || !arr(out, dtype_bytes(out_type)))
        return SYMNMF_E_INVALID;
    return done(launch_embed({table, table_type, rows, width, ldt, ids, id_type, count, scale, out,
                              out_type, ldo},
                             as_stream(hip_stream)));
}

int symnmf_embed_grad(const void* dout, int dout_type, int64_t count, int64_t width, int64_t ldd,
                      const void* ids, int id_type, float scale, int accumulate, void* dtable,
                      int dtable_type, int64_t rows, int64_t ldt, void* ws, size_t ws_bytes,
                      void* hip_stream) {
    if (!type_ok(dout_type) || !type_ok(dtable_type) || !index_ok(id_type) ||
        !in(rows, 1, kMaxCount) || !in(width, 1, 1 << 24) || ldd < width || ldt < width ||
        !in(count, 0, kMaxCount) || !arr(dtable, dtype_bytes(dtable_type)) ||
        (accumulate != 0 && accumulate != 1))
        return SYMNMF_E_INVALID;
    if (count && (!arr(dout, dtype_bytes(dout_type)) || !arr(ids, index_bytes(id_type))))
        return SYMNMF_E_INVALID;
    if (!ws_fits(ws, ws_bytes, embed_grad_ws_bytes(rows, width, count))) return SYMNMF_E_WORKSPACE;
    return done(launch_embed_grad({dout, dout_type, count, width, ldd, ids, id_type, scale,
                                   accumulate, dtable, dtable_type, rows, ldt, ws},
                                  as_stream(hip_stream)));
}

int symnmf_gated_scan(int type, int64_t batch, int64_t steps, int64_t width, const void* x,
                      int64_t x_batch, int64_t x_step, const void* gate, int64_t gate_batch,
                      int64_t gate_step, const int32_t* lengths, const float* h0, void* h,
                      float* h_last, float* states, void* ws, size_t ws_bytes, void* hip_stream) {
    if (!type_ok(type) || !scan_sizes_ok(batch, steps, width) || x_batch < 0 || x_step < 0 ||
        gate_batch < 0 || gate_step < 0 || !arr_or_null(lengths, 4) || !arr_or_null(h0, 4) ||
        !arr_or_null(h_last, 4) || !arr_or_null(states, 4))
        return SYMNMF_E_INVALID;
    const int eb = dtype_bytes(type);
    if (steps && (!arr(x, eb) || !arr(gate, eb) || !arr(h, eb))) return SYMNMF_E_INVALID;
    if (!ws_fits(ws, ws_bytes, scan_ws_bytes(batch, steps, width))) return SYMNMF_E_WORKSPACE;
    ScanArgs a{};
    a.type = type;
    a.batch = batch;
    a.steps = steps;
    a.width = width;
    a.x = x;
    a.x_b = x_batch;
    a.x_t = x_step;
    a.gate = gate;
    a.g_b = gate_batch;
    a.g_t = gate_step;
    a.lengths = lengths;
    a.h0 = h0;
    a.h = h;
    a.last = h_last;
    a.states = states;
    a.ws = ws;
    return done(launch_scan(a, as_stream(hip_stream)));
}

int symnmf_gated_scan_grad(int type, int64_t batch, int64_t steps, int64_t width, const void* x,
                           int64_t x_batch, int64_t x_step, const void* gate, int64_t gate_batch,
                           int64_t gate_step, const int32_t* lengths, const float* states,
                           const void* dh, int64_t dh_batch, int64_t dh_step,
                           const float* dh_last, void* dx, void* dgate, float* dh0, void* ws,
                           size_t ws_bytes, void* hip_stream) {
    if (!type_ok(type) || !scan_sizes_ok(batch, steps, width) || x_batch < 0 || x_step < 0 ||
        gate_batch < 0 || gate_step < 0 || dh_batch < 0 || dh_step < 0 ||
        !arr_or_null(lengths, 4) || !arr_or_null(dh_last, 4) || !arr_or_null(dh0, 4))
        return SYMNMF_E_INVALID;
    const int eb = dtype_bytes(type);
    if (steps && (!arr(x, eb) || !arr(gate, eb) || !arr(dh, eb) || !arr(dx, eb) ||
                  !arr(dgate, eb) || !arr(states, 4)))
        return SYMNMF_E_INVALID;
    if (!ws_fits(ws, ws_bytes, scan_ws_bytes(batch, steps, width))) return SYMNMF_E_WORKSPACE;
    ScanArgs a{};
    a.type = type;
    a.batch = batch;
    a.steps = steps;
    a.width = width;
    a.x = x;
    a.x_b = x_batch;
    a.x_t = x_step;
    a.gate = gate;
    a.g_b = gate_batch;
    a.g_t = gate_step;
    a.lengths = lengths;
    a.states = const_cast<float*>(states);
    a.dh = dh;
    a.d_b = dh_batch;
    a.d_t = dh_step;
    a.dlast = dh_last;
    a.dx = dx;
    a.dgate = dgate;
    a.dh0 = dh0;
    a.ws = ws;
    return done(launch_scan_grad(a, as_stream(hip_stream)));
}

int symnmf_token_logprobs(const void* logits, int type, int64_t count, int64_t vocab, int64_t ld,
                          const void* tokens, int token_type, float scale, float* logp,
                          float* entropy, float* lse, int32_t top, float* top_logp,
                          int32_t* top_ids, void* ws, size_t ws_bytes, void* hip_stream) {
    if (!type_ok(type) || !index_ok(token_type) || !in(count, 0, kMaxCount) ||
        !in(vocab, 1, kMaxVocab) || ld < vocab || !(scale > 0.f) || !std::isfinite(scale) ||
        !in(top, 0, kMaxTop))
        return SYMNMF_E_INVALID;
    if (count == 0) return SYMNMF_OK;
    if (!arr(logits, dtype_bytes(type)) || !arr(tokens, index_bytes(token_type)) || !arr(logp, 4) ||
        !arr_or_null(entropy, 4) || !arr_or_null(lse, 4) ||
        (top && (!arr(top_logp, 4) || !arr(top_ids, 4))))
        return SYMNMF_E_INVALID;
    if (!ws_fits(ws, ws_bytes, logprob_ws_bytes(vocab, top, count))) return SYMNMF_E_WORKSPACE;
    LogprobArgs a{};
    a.type = type;
    a.count = count;
    a.vocab = vocab;
    a.ld = ld;
    a.logits = logits;
    a.tokens = tokens;
    a.token_type = token_type;
    a.scale = scale;
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.top = top;
    a.top_logp = top_logp;
    a.top_ids = top_ids;
    a.ws = ws;
    return done(launch_logprobs(a, as_stream(hip_stream)));
}

int symnmf_token_logprobs_grad(const void* logits, int type, int64_t count, int64_t vocab,
                               int64_t ld, const void* tokens, int token_type, float scale,
                               const float* lse, const float* entropy, const float* dlogp,
                               const float* dentropy, void* dlogits, int64_t ldd,
                               void* hip_stream) {
    if (!type_ok(type) || !index_ok(token_type) || !in(count, 0, kMaxCount) ||
        !in(vocab, 1, kMaxVocab) || ld < vocab || ldd < vocab || !(scale > 0.f) ||
        !std::isfinite(scale))
        return SYMNMF_E_INVALID;
    if (count == 0) return SYMNMF_OK;
    if (!arr(logits, dtype_bytes(type)) || !arr(tokens, index_bytes(token_type)) || !arr(lse, 4) ||
        !arr_or_null(entropy, 4) || !arr(dlogp, 4) || !arr_or_null(dentropy, 4) ||
        (dentropy && !entropy) || !arr(dlogits, dtype_bytes(type)))
        return SYMNMF_E_INVALID;
    LogprobArgs a{};
    a.type = type;
    a.count = count;
    a.vocab = vocab;
    a.ld = ld;
    a.logits = logits;
    a.tokens = tokens;
    a.token_type = token_type;
    a.scale = scale;
    a.lse = const_cast<float*>(lse);
    a.entropy = const_cast<float*>(entropy);
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    a.ldd = ldd;
    return done(launch_logprobs_grad(a, as_stream(hip_stream)));
}

}  // extern "C"
