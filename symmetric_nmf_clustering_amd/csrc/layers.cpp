// Host side of the layer operators of include/symnmf.h: linear attention, rotary
// positions, the AdamW step. Argument checks, then one launcher per call
// (k_linattn*.hip, k_rotary.hip, k_adamw.hip). Every call is asynchronous.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "layers.h"
#include "symnmf.h"

using namespace symnmf;

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 30;

inline bool type_ok(int t) { return t == SYMNMF_F32 || t == SYMNMF_BF16 || t == SYMNMF_F16; }
inline bool arr(const void* p, int bytes) {
    return p && reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}
inline bool arr_or_null(const void* p, int bytes) { return !p || arr(p, bytes); }
inline bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
inline int done(hipError_t e) { return e == hipSuccess ? SYMNMF_OK : SYMNMF_E_HIP; }

// The descriptor's sizes; products of them are counted in 64 bits by the kernels.
bool attend_ok(const symnmf_attend_desc* d) {
    if (!d || !type_ok(d->type) || !in(d->heads, 1, 65536) || !in(d->kv_heads, 1, d->heads) ||
        d->heads % d->kv_heads || !in(d->dk, 1, kMaxHeadDim) || !in(d->dv, 1, kMaxHeadDim) ||
        !in(d->batch, 1, kMaxCount) || !in(d->steps, 0, kMaxCount) || !std::isfinite(d->scale) ||
        d->batch * d->heads > kMaxCount || (d->steps && d->batch * d->heads > (int64_t(1) << 44) / d->steps))
        return false;
    for (int i = 0; i < 3; ++i)
        if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0 || d->do_stride[i] < 0)
            return false;
    return true;
}

AttendCall call_of(const symnmf_attend_desc* d, const void* q, const void* k, const void* v,
                   const float* decay) {
    AttendCall c{};
    c.d.type = d->type;
    c.d.heads = d->heads;
    c.d.kv_heads = d->kv_heads;
    c.d.dk = d->dk;
    c.d.dv = d->dv;
    c.d.scale = d->scale;
    c.d.batch = d->batch;
    c.d.steps = d->steps;
    std::memcpy(c.d.q, d->q_stride, sizeof c.d.q);
    std::memcpy(c.d.k, d->k_stride, sizeof c.d.k);
    std::memcpy(c.d.v, d->v_stride, sizeof c.d.v);
    std::memcpy(c.d.d, d->do_stride, sizeof c.d.d);
    c.q = q;
    c.k = k;
    c.v = v;
    c.decay = decay;
    return c;
}

bool ws_fits(const void* ws, size_t got, size_t need) {
    return ws && reinterpret_cast<uintptr_t>(ws) % 256 == 0 && got >= need;
}

}  // namespace

extern "C" {

size_t symnmf_linear_attention_ws_bytes(const symnmf_attend_desc* d, int gradient) {
    if (!attend_ok(d) || (gradient != 0 && gradient != 1)) return 0;
    return attend_ws_bytes(call_of(d, nullptr, nullptr, nullptr, nullptr).d, gradient != 0);
}

int symnmf_linear_attention(const symnmf_attend_desc* d, const void* q, const void* k,
                            const void* v, const float* decay, const int32_t* lengths,
                            const float* state, void* o, float* last, void* ws, size_t ws_bytes,
                            void* hip_stream) {
    if (!attend_ok(d) || !arr(decay, 4) || !arr_or_null(lengths, 4) || !arr_or_null(state, 4) ||
        !arr_or_null(last, 4))
        return SYMNMF_E_INVALID;
    const int eb = dtype_bytes(d->type);
    if (d->steps && (!arr(q, eb) || !arr(k, eb) || !arr(v, eb) || !arr(o, eb)))
        return SYMNMF_E_INVALID;
    AttendCall c = call_of(d, q, k, v, decay);
    if (!ws_fits(ws, ws_bytes, attend_ws_bytes(c.d, false))) return SYMNMF_E_WORKSPACE;
    c.lengths = lengths;
    c.state = state;
    c.o = o;
    c.last = last;
    c.ws = ws;
    return done(launch_attend(c, static_cast<hipStream_t>(hip_stream)));
}

int symnmf_linear_attention_grad(const symnmf_attend_desc* d, const void* q, const void* k,
                                 const void* v, const float* decay, const int32_t* lengths,
                                 const float* state, const void* dout, const float* dlast, void* dq,
                                 void* dk, void* dv, float* dstate, void* ws, size_t ws_bytes,
                                 void* hip_stream) {
    if (!attend_ok(d) || !arr(decay, 4) || !arr_or_null(lengths, 4) || !arr_or_null(state, 4) ||
        !arr_or_null(dlast, 4) || !arr_or_null(dstate, 4))
        return SYMNMF_E_INVALID;
    const int eb = dtype_bytes(d->type);
    if (d->steps && (!arr(q, eb) || !arr(k, eb) || !arr(v, eb) || !arr(dout, eb) || !arr(dq, eb) ||
                     !arr(dk, eb) || !arr(dv, eb)))
        return SYMNMF_E_INVALID;
    AttendCall c = call_of(d, q, k, v, decay);
    if (!ws_fits(ws, ws_bytes, attend_ws_bytes(c.d, true))) return SYMNMF_E_WORKSPACE;
    c.lengths = lengths;
    c.state = state;
    c.dout = dout;
    c.dlast = dlast;
    c.dq = dq;
    c.dk = dk;
    c.dv = dv;
    c.dstate = dstate;
    c.ws = ws;
    return done(launch_attend_grad(c, static_cast<hipStream_t>(hip_stream)));
}

int symnmf_linear_attention_step(const symnmf_attend_desc* d, const void* q, const void* k,
                                 const void* v, const float* decay, const float* state, void* o,
                                 float* new_state, void* hip_stream) {
    if (!attend_ok(d) || d->steps != 1 || !arr(decay, 4) || !arr(state, 4) || !arr(new_state, 4))
        return SYMNMF_E_INVALID;
    const int eb = dtype_bytes(d->type);
    if (!arr(q, eb) || !arr(k, eb) || !arr(v, eb) || !arr(o, eb)) return SYMNMF_E_INVALID;
    AttendCall c = call_of(d, q, k, v, decay);
    c.state = state;
    c.o = o;
    c.last = new_state;
    return done(launch_attend_step(c, static_cast<hipStream_t>(hip_stream)));
}

int symnmf_rotary(int type, int64_t batch, int64_t steps, int32_t heads, int32_t width,
                  int32_t dims, int interleaved, int inverse, float amplitude, const void* x,
                  int64_t x_batch, int64_t x_step, int64_t x_head, const void* positions,
                  int position_type, int64_t pos_batch, int64_t pos_step, const double* freqs,
                  void* out, int64_t out_batch, int64_t out_step, int64_t out_head,
                  void* hip_stream) {
    if (!type_ok(type) || !in(batch, 0, kMaxCount) || !in(steps, 0, kMaxCount) ||
        !in(heads, 1, 65536) || !in(width, 1, 65536) || !in(dims, 0, width) || dims % 2 ||
        (interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) ||
        !std::isfinite(amplitude) || x_batch < 0 || x_step < 0 || x_head < 0 || pos_batch < 0 ||
        pos_step < 0 || out_batch < 0 || out_step < 0 || out_head < 0 ||
        (position_type != SYMNMF_I32 && position_type != SYMNMF_I64) ||
        (steps && batch > (int64_t(1) << 40) / steps))
        return SYMNMF_E_INVALID;
    if (batch == 0 || steps == 0) return SYMNMF_OK;
    const int eb = dtype_bytes(type);
    if (!arr(x, eb) || !arr(out, eb) || !arr(positions, position_type == SYMNMF_I32 ? 4 : 8) ||
        (dims && !arr(freqs, 8)))
        return SYMNMF_E_INVALID;
    return done(launch_rotary({type, batch, steps, heads, width, dims, interleaved, inverse,
                               amplitude, x, x_batch, x_step, x_head, positions, position_type,
                               pos_batch, pos_step, freqs, out, out_batch, out_step, out_head},
                              static_cast<hipStream_t>(hip_stream)));
}

int symnmf_adamw(int param_type, int grad_type, int state_bits, const symnmf_adamw_tensor* tensors,
                 int32_t count, double lr, double beta1, double beta2, double eps,
                 double weight_decay, int64_t step, float grad_scale, const int64_t* step_dev,
                 const float* lr_dev, const float* grad_scale_dev, void* hip_stream) {
    if (!type_ok(param_type) || !type_ok(grad_type) || (state_bits != 32 && state_bits != 8) ||
        count < 0 || (count && !tensors) || !std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        !std::isfinite(weight_decay) || (!step_dev && step < 1) || !std::isfinite(grad_scale) ||
        !arr_or_null(step_dev, 8) || !arr_or_null(lr_dev, 4) || !arr_or_null(grad_scale_dev, 4))
        return SYMNMF_E_INVALID;
    static_assert(sizeof(symnmf_adamw_tensor) == sizeof(AdamTensor), "one layout");
    const int sb = state_bits == 32 ? 4 : 1;
    for (int32_t i = 0; i < count; ++i) {
        const symnmf_adamw_tensor& t = tensors[i];
        if (!in(t.n, 0, int64_t(1) << 40)) return SYMNMF_E_INVALID;
        if (t.n == 0) continue;
        if (!arr(t.param, dtype_bytes(param_type)) || !arr(t.grad, dtype_bytes(grad_type)) ||
            !arr(t.m, sb) || !arr(t.v, sb) || !arr_or_null(t.master, 4) ||
            (state_bits == 8 && (!arr(t.m_scale, 4) || !arr(t.v_scale, 4))))
            return SYMNMF_E_INVALID;
    }
    AdamArgs a{};
    a.param_type = param_type;
    a.grad_type = grad_type;
    a.bits = state_bits;
    a.tensors = reinterpret_cast<const AdamTensor*>(tensors);
    a.count = count;
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    a.weight_decay = weight_decay;
    a.step = (double)(step_dev ? 1 : step);
    a.grad_scale = grad_scale;
    a.step_dev = step_dev;
    a.lr_dev = lr_dev;
    a.grad_scale_dev = grad_scale_dev;
    return done(launch_adamw(a, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
