// Internal launch interface of the gated linear recurrence and the root-mean-square
// norm; not part of the C ABI.
#pragma once

#include <algorithm>

#include "attn_internal.cuh"

namespace gdn {

// How a channel's decay and input weight come about (gdn_linear_recurrence_args).
enum { RECUR_PRECOMPUTED = 0, RECUR_RAW = 1, RECUR_RAW_UNIT = 2 };

struct RecurrenceParams {
    int B, T, C, num_slots;
    int S;  // cu null: tokens of every sequence
    long long x_stride, a_stride, b_stride, dy_stride;
    const void *x, *a, *b;  // b null: an input weight of 1
    const float *A_log, *dt_bias;
    const int32_t *cu, *slots;
    const float *init;
    int32_t *status;
    // forward
    float *final_state;
    void *y;
    float *checkpoints;
    // backward
    const void *dy;
    const float *states;  // the forward call's checkpoints
    const float *dfinal;
    void *dx, *da, *db;
    float *dA_log, *ddt_bias, *dinit;
    void *workspace;
};

size_t recurrence_workspace_bytes(int T, int C, int longest);
size_t recurrence_backward_workspace_bytes(int B, int T, int C);
// longest: an upper bound on the longest sequence (a hint)
cudaError_t launch_recurrence(const RecurrenceParams &p, int io_dtype, int mode, int longest, cudaStream_t stream);
cudaError_t launch_recurrence_backward(const RecurrenceParams &p, int io_dtype, int mode, cudaStream_t stream);

struct RmsNormParams {
    int T, H, d, group;
    float eps, offset;
    long long x_stride, r_stride, z_stride, dy_stride;
    const void *x, *r, *z;
    const float *w;
    void *s_out, *y;
    float *scale;
    // backward (x: what was normalised, r: the gradient that reaches it from elsewhere)
    const void *dy;
    void *dx, *dz;
    float *dw;
    float *partials;
};

size_t rms_norm_backward_workspace_bytes(int T, int H, int d);
cudaError_t launch_rms_norm(const RmsNormParams &p, int io_dtype, int out_dtype, cudaStream_t stream);
cudaError_t launch_rms_norm_backward(const RmsNormParams &p, int io_dtype, cudaStream_t stream);

// ---------------------------------------------------------------- device helpers

// The type of the gate inputs: the I/O type if they are raw, FP32 if they are decays and weights.
template <typename T, int MODE>
struct GateType {
    using type = T;
};
template <typename T>
struct GateType<T, RECUR_PRECOMPUTED> {
    using type = float;
};

// What the gates of one (token, channel) come to.
struct Gate {
    float g, w;           // decay, input weight
    float lg, sig_a;      // log g; sigmoid(a + dt_bias)
    float sig_b, factor;  // sigmoid(b); sqrt(1 - g^2) (1 without unit_input)
};

// rate = exp(A_log); b absent: has_b 0.
template <int MODE>
__device__ __forceinline__ Gate gate_of(float a, float b, float rate, float dt_bias, bool has_b) {
    Gate r;
    if constexpr (MODE == RECUR_PRECOMPUTED) {
        r.g = a;
        r.w = has_b ? b : 1.f;
        r.lg = r.sig_a = r.sig_b = r.factor = 0.f;
    } else {
        const float v = a + dt_bias;
        const float e = expf(-fabsf(v));
        r.lg = -rate * (fmaxf(v, 0.f) + log1pf(e));
        r.g = expf(r.lg);
        r.sig_a = (v >= 0.f ? 1.f : e) / (1.f + e);
        r.sig_b = has_b ? 1.f / (1.f + expf(-b)) : 1.f;
        r.factor = MODE == RECUR_RAW_UNIT ? sqrtf(-expm1f(2.f * r.lg)) : 1.f;
        r.w = r.sig_b * r.factor;
    }
    return r;
}

// The gradients of a and b (and their parameters) from those of g and w.
struct GateGrad {
    float da, db, dA;  // dA: that of A_log; dt_bias has a's
};

template <int MODE>
__device__ __forceinline__ GateGrad gate_grad(const Gate &r, float dg, float dw, float rate) {
    GateGrad o;
    if constexpr (MODE == RECUR_PRECOMPUTED) {
        o.da = dg;
        o.db = dw;
        o.dA = 0.f;
    } else {
        float dlg = dg * r.g;
        if (MODE == RECUR_RAW_UNIT && r.factor > 0.f) dlg -= dw * r.sig_b * (r.g * r.g / r.factor);
        o.da = -dlg * rate * r.sig_a;
        o.dA = dlg * r.lg;
        o.db = dw * r.factor * (r.sig_b * (1.f - r.sig_b));
    }
    return o;
}

// Sequence b's tokens [start, end) as cu_seqlens has them, or of S tokens each.
__device__ __forceinline__ int recurrence_start(const RecurrenceParams &p, int b) { return p.cu ? p.cu[b] : b * p.S; }

}  // namespace gdn
