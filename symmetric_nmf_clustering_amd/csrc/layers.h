// Shared by the layer operators (linear attention, rotary positions, the AdamW
// step) and their host side layers.cpp: the launchers' arguments.
#pragma once

#include "seq.h"

namespace symnmf {

// ---- linear attention --------------------------------------------------------

constexpr int kMaxHeadDim = 256;

// One evaluation of a decayed linear attention: rows x (queries), y (keys), z
// (values) of a head, a state dx by dz,
//   out_u = p_scale sum_{w <= u} a^(u - w) (x_u . y_w) z_w + in_scale a^(u + in_pow) x_u S_in
//   S_out = a^n S_in + st_scale sum_w a^(n - in_pow - w) y_w z_w^T,
// where u counts the head's n valid steps from the first, or from the last
// (reverse). in_pow is 1 or 0: whether the incoming state is decayed once more
// before the first step reads it.
struct AttendRun {
    const void *x, *y, *z;
    int64_t xb, xt, xh, yb, yt, yh, zb, zt, zh;  // strides of batch, step, head
    int32_t xg, yg, zg;                          // query heads that share a head of it
    int32_t dx, dz;
    int32_t reverse, in_pow;
    float p_scale, in_scale, st_scale;
    const float* s0;      // nullable (zeros): batch x heads x (dx dz), element (i, j) at
    int32_t s0_i, s0_j;   // i s0_i + j s0_j
    float* s1;            // nullable: the state after the last step
    int32_t s1_i, s1_j;
    void* out;            // batch x steps x heads x dz, dense
    int32_t out32;        // out is float32 whatever the type
    float* seg;           // nseg > 1: batch x heads x nseg x (dx dz), element (i, j) at
    int32_t seg_i, seg_j;  // i seg_i + j seg_j
};

struct AttendArgs {
    AttendRun run[3];
    int32_t nrun;
    const float* decay;      // heads: ln a
    const int32_t* lengths;  // nullable
    int32_t type, heads, nseg;
    int32_t group;  // neighbouring heads that read the same rows: walked on one XCD
    int64_t batch, steps, seg_len;
};

// Kernels of one element type (k_linattn_*.hip): out = the walk itself, or the
// segments' own states (maps).
template <class T>
hipError_t launch_attend_walk(const AttendArgs& a, bool maps, hipStream_t st);

struct AttendDesc {
    int32_t type, heads, kv_heads, dk, dv;
    float scale;
    int64_t batch, steps;
    int64_t q[3], k[3], v[3], d[3];  // strides of batch, step, head
};
struct AttendCall {
    AttendDesc d;
    const void *q, *k, *v, *dout;
    const float* decay;
    const int32_t* lengths;
    const float *state, *dlast;
    void *o, *dq, *dk, *dv;
    float *last, *dstate;
    void* ws;
};
size_t attend_ws_bytes(const AttendDesc& d, bool gradient);
hipError_t launch_attend(const AttendCall& c, hipStream_t st);
hipError_t launch_attend_grad(const AttendCall& c, hipStream_t st);
hipError_t launch_attend_step(const AttendCall& c, hipStream_t st);  // state -> last

// ---- rotary positions ----------------------------------------------------------

struct RotaryArgs {
    int type;
    int64_t batch, steps;
    int32_t heads, width, dims;
    int interleaved, inverse;
    float amplitude;
    const void* x;
    int64_t x_b, x_t, x_h;
    const void* pos;
    int pos_type;
    int64_t pos_b, pos_t;
    const double* freqs;  // dims / 2
    void* out;
    int64_t o_b, o_t, o_h;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st);

// ---- AdamW -----------------------------------------------------------------------

constexpr int kAdamBlock = 256;  // elements of an 8-bit state that share a scale

struct AdamTensor {
    void* param;
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    int64_t n;
};
struct AdamArgs {
    int param_type, grad_type, bits;
    const AdamTensor* tensors;  // host
    int32_t count;
    double lr, beta1, beta2, eps, weight_decay;
    double step;
    float grad_scale;
    const int64_t* step_dev;        // nullable: overrides step
    const float* lr_dev;            // nullable: overrides lr
    const float* grad_scale_dev;    // nullable: multiplies grad_scale
};
hipError_t launch_adamw(const AdamArgs& a, hipStream_t st);

}  // namespace symnmf
