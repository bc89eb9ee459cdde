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
};

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
    float g;              // decay
    float sig_b, factor;  // sigmoid(b); sqrt(1 - g^2) (1 without unit_input)
    __device__ __forceinline__ float w() const { return sig_b * factor; }  // the input's weight
};

// The gates' arithmetic is FP32 in the fewest instructions: the recurrence moves 8 bytes a channel of a token at 16 bits, which
// leaves an SM time for 44.  With u = 2^-24, relative: e^-|v| is good to (2 |v| + 4) u, a sigmoid of b to (|b| + 8) u
// (the exponent is rounded: 3e-6 at |b| = 50), since the special functions are the approximate ones.
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718056f;
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e) / e for e in [0, 1]: a least-maximum fit in Chebyshev polynomials, 1.6e-7 off at most in FP32.
// (A logarithm of 1 + e would lose the digits of a small e, and with them the memory of a slow decay.)
#define GDN_LOG1P(FMA, K)                                    \
    y = FMA(K(0.00523227453f), e, K(-0.029503556f));         \
    y = FMA(y, e, K(0.0782232136f));                         \
    y = FMA(y, e, K(-0.136630133f));                         \
    y = FMA(y, e, K(0.191058978f));                          \
    y = FMA(y, e, K(-0.248429537f));                         \
    y = FMA(y, e, K(0.333190948f));                          \
    y = FMA(y, e, K(-0.499994934f));                         \
    y = FMA(y, e, K(0.99999994f));
__device__ __forceinline__ float log1p_over(float e) {
    float y;
    GDN_LOG1P(fmaf, float)
    return y;
}

// 1 - g^2 for g = e^-t: for small t 2 g sinh(t), whose series keeps its digits (t^6 / 5040 off); beyond, g^2 is 0.67 at
// most, and the relative error of 1 - g^2 is four times g's (2 x 0.67 / 0.33), that of its root twice.
constexpr float SMALL_T = 0.2f;
__device__ __forceinline__ float one_minus_square(float g, float t) {
    const float q = t * t, s = fmaf(fmaf(q, 1.f / 120.f, 1.f / 6.f), q, 1.f);
    return t < SMALL_T ? 2.f * g * t * s : fmaf(-g, g, 1.f);
}

// A decay from its base-2 logarithm x.  For results next to 1 the approximate exponential lies 0.22 to 0.35 units of 2^-24
// low on average (65,536 logarithms in each of three ranges), which a memory of 1000 tokens adds up to 2e-5; its
// argument makes up for 0.27 of them.  (It is fitted there: decays near 0.06 come out 0.06 units of their own high on average.)
constexpr float DECAY_UP = 0.27f * 0x1p-24f * LOG2E;

// rate = exp(A_log); b absent: has_b 0.
template <int MODE>
__device__ __forceinline__ Gate gate_of(float a, float b, float rate, float dt_bias, bool has_b) {
    Gate r;
    if constexpr (MODE == RECUR_PRECOMPUTED) {
        r.g = a;
        r.sig_b = has_b ? b : 1.f;
        r.factor = 1.f;
    } else {
        const float v = a + dt_bias;
        const float e = exp2_approx(-LOG2E * fabsf(v));
        const float t = rate * fmaf(log1p_over(e), e, fmaxf(v, 0.f));
        r.g = exp2_approx(fmaf(-LOG2E, t, DECAY_UP));
        r.sig_b = has_b ? rcp_approx(1.f + exp2_approx(-LOG2E * b)) : 1.f;
        r.factor = MODE == RECUR_RAW_UNIT ? sqrt_approx(one_minus_square(r.g, t)) : 1.f;
    }
    return r;
}

// ---------------------------------------------------------------- two channels at once

// Two FP32 numbers in one register pair, for the instructions that take two at a time.
struct F2 {
    unsigned long long u;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(x), "f"(y)); }
    __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
    __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(u)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
    return d;
}

__device__ __forceinline__ F2 exp2_approx(F2 a) {
    float x, y;
    a.get(x, y);
    return F2(exp2_approx(x), exp2_approx(y));
}
__device__ __forceinline__ F2 rcp_approx(F2 a) {
    float x, y;
    a.get(x, y);
    return F2(rcp_approx(x), rcp_approx(y));
}
// e^-|a|
__device__ __forceinline__ F2 exp_minus_abs(F2 a) {
    float x, y;
    a.get(x, y);
    return F2(exp2_approx(-LOG2E * fabsf(x)), exp2_approx(-LOG2E * fabsf(y)));
}
__device__ __forceinline__ F2 log1p_over(F2 e) {
    F2 y;
    GDN_LOG1P(fma2, F2)
    return y;
}

// gate_of for two channels, up to roundings (log2(e) is multiplied into the rate first); exponent: the base-2 logarithm of g;
// minus_rate: -log2(e) exp(A_log).
struct GatePair {
    F2 g, exponent;
    F2 b;  // e^-b (0 without b); RECUR_PRECOMPUTED: the input's weight
};
template <int MODE>
__device__ __forceinline__ GatePair gate_pair(F2 a, F2 b, F2 minus_rate, F2 dt_bias, bool has_b) {
    GatePair r;
    if constexpr (MODE == RECUR_PRECOMPUTED) {
        r.g = a;
        r.b = has_b ? b : F2(1.f);
    } else {
        float x, y;
        const F2 v = add2(a, dt_bias), e = exp_minus_abs(v);
        v.get(x, y);
        r.exponent = mul2(minus_rate, fma2(log1p_over(e), e, F2(fmaxf(x, 0.f), fmaxf(y, 0.f))));
        r.g = exp2_approx(add2(r.exponent, F2(DECAY_UP)));
        r.b = has_b ? exp2_approx(mul2(b, F2(-LOG2E))) : F2(0.f);
    }
    return r;
}
// sqrt(1 - g^2) (RECUR_RAW_UNIT)
__device__ __forceinline__ F2 factor_pair(const GatePair &q) {
    // as one_minus_square
    const F2 t = mul2(q.exponent, F2(-LN2)), t2 = mul2(t, t);
    const F2 s = mul2(fma2(fma2(t2, F2(1.f / 120.f), F2(1.f / 6.f)), t2, F2(1.f)), mul2(t, add2(q.g, q.g)));
    float g1, g2, t1, t2s, s1, s2;
    q.g.get(g1, g2);
    t.get(t1, t2s);
    s.get(s1, s2);
    s1 = t1 < SMALL_T ? s1 : fmaf(-g1, g1, 1.f);
    s2 = t2s < SMALL_T ? s2 : fmaf(-g2, g2, 1.f);
    return F2(sqrt_approx(s1), sqrt_approx(s2));
}
// sigmoid(b), or the weight itself.  has_b only spares the arithmetic without b (e^-b is 0, its sigmoid 1): forwards the
// branch pays (16,384 BF16 tokens of 2048 channels 66 instead of 69 us, 4096 without b 130 instead of 136), in the backward
// kernel's unrolled gradients it costs (4096 channels 257 without it, 274 with it).
template <int MODE>
__device__ __forceinline__ F2 input_gate(const GatePair &q, bool has_b = true) {
    if constexpr (MODE == RECUR_PRECOMPUTED) return q.b;
    else return has_b ? rcp_approx(add2(q.b, F2(1.f))) : F2(1.f);
}
template <int MODE>
__device__ __forceinline__ F2 weight_of(const GatePair &q, bool has_b = true) {
    const F2 sig_b = input_gate<MODE>(q, has_b);
    return MODE == RECUR_RAW_UNIT ? mul2(sig_b, factor_pair(q)) : sig_b;
}

// The gradients of a, b and A_log (dA up to a factor of ln 2) from those of g and w; dt_bias has a's.
struct GradPair {
    F2 da, db, dA, w;  // w: the input's weight
};
template <int MODE>
__device__ __forceinline__ GradPair grad_pair(const GatePair &q, F2 a, F2 dg, F2 dw, F2 minus_rate, F2 dt_bias) {
    GradPair o;
    const F2 sig_b = input_gate<MODE>(q);
    o.w = sig_b;
    if constexpr (MODE == RECUR_PRECOMPUTED) {
        o.da = dg;
        o.db = dw;
    } else {
        // (1 / (1 + e^-v) is good to a few units relative for either sign: nothing here takes it from 1)
        float x, y;
        const F2 sig_a = rcp_approx(add2(exp2_approx(mul2(add2(a, dt_bias), F2(-LOG2E))), F2(1.f)));
        F2 dlg = mul2(dg, q.g), di = mul2(dw, sig_b);
        if constexpr (MODE == RECUR_RAW_UNIT) {
            // -g^2 / factor, 0 where the factor is
            float f1, f2;
            const F2 factor = factor_pair(q);
            factor.get(f1, f2);
            const F2 k = mul2(mul2(q.g, q.g), F2(f1 > 0.f ? -rcp_approx(f1) : 0.f, f2 > 0.f ? -rcp_approx(f2) : 0.f));
            dlg = fma2(di, k, dlg);
            di = mul2(di, factor);
            o.w = mul2(sig_b, factor);
        }
        o.da = mul2(mul2(dlg, sig_a), mul2(minus_rate, F2(LN2)));
        // (an infinite gate's exponent too is multiplied by a dlg of 0)
        q.exponent.get(x, y);
        o.dA = mul2(dlg, F2(fmaxf(x, -3.402823466e38f), fmaxf(y, -3.402823466e38f)));
        // 1 - sigmoid(b) = e^-b sigmoid(b), which keeps its digits where the sigmoid is next to 1 (where e^-b is infinite,
        // the sigmoid is 0, and so is this)
        q.b.get(x, y);
        o.db = mul2(di, mul2(F2(fminf(x, 3.402823466e38f), fminf(y, 3.402823466e38f)), sig_b));
    }
    return o;
}

// Sequence b's tokens [start, end) as cu_seqlens has them, or of S tokens each.
__device__ __forceinline__ int recurrence_start(const RecurrenceParams &p, int b) { return p.cu ? p.cu[b] : b * p.S; }

}  // namespace gdn
