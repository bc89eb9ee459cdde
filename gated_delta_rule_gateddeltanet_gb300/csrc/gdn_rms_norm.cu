// Root-mean-square norm of rows, with the residual's addition before it, a gate after
// it and an output in 8 bits; forward and backward.
//
//   s = x (+ r),  y = s / sqrt(mean s^2 + eps) * (w + offset) * silu(z)
//
// Both directions are HBM streams: a row is read once, 8 channels a thread and piece, and
// everything about it is worked out in registers.  What a row needs of other threads is one
// sum (two backwards) and, for 8 bits, a maximum.
//   forward   a CTA a token (whole-token norms and scales), four pieces a thread so that
//             enough loads are on their way; heads of 32 to 256 channels without any
//             barrier, their sums being shuffles of a few lanes.  8192 BF16 tokens of 4096,
//             residual added, to e4m3: 39.5 us (5.9 TB/s, 0.88 of a copy's rate; a piece a thread
//             55 us).  4099 FP16 tokens of 48 gated heads of 128 to e4m3, a scale a head: 26.0 us
//             (4.9 TB/s; 29 instructions a channel, gate and scales among them, fill 74% of the issue slots).
//             One token of 2048: 1.5 us, a launch.
//   backward  CTAs walk over the tokens behind a ring of bulk copies, so that a channel's part
//             of dweight stays in one thread.  8192 BF16 tokens of 4096: 45 us (5.9 TB/s),
//             FP32 70 us (7.7 TB/s: part of it comes from L2); 8192 FP16 tokens of 40 gated heads of 128:
//             97 us (4.3 TB/s, 0.64: 34 instructions a channel).
#include <type_traits>

#include "layer_internal.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The larger of two or three numbers, NaN if one is.
__device__ __forceinline__ float max_or_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// 8-bit values stand for y = t f with f a factor of the whole row (the norm's, or 1), which does not enter the quotients:
// they are t times the one number `times`, with fewer roundings than y / scale has.  scale: max|y| / 448 (or 127), with a
// normal reciprocal.
struct Scale {
    float scale, times;
};
__device__ __forceinline__ Scale scale_of(float top, float factor, float most) {
    const float largest = top * factor;
    if (!(largest <= 3.402823466e38f)) return {__int_as_float(0x7fc00000), __int_as_float(0x7fc00000)};
    if (largest == 0.f) return {1.f, factor};
    const float scale = largest * (1.f / most);
    if (scale < 0x1p-120f || top < 0x1p-100f || top > 0x1p100f) return {fmaxf(scale, 0x1p-120f), __fdiv_rn(factor, fmaxf(scale, 0x1p-120f))};
    // most / top: the approximate quotient and its remainder's share, one step of Markstein's refinement of a quotient (IBM
    // J. Res. Develop. 34, 1990); both numbers are far from the ends of the range
    const float r = rcp_approx(top), q = most * r;
    return {scale, fmaf(fmaf(-q, top, most), r, q)};
}

// (0 for z below -88, where e^-z is infinite)
__device__ __forceinline__ float sigmoid(float z) { return rcp_approx(1.f + exp2_approx(-LOG2E * z)); }
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
__device__ __forceinline__ F2 silu(F2 z) {
    float a, b;
    mul2(z, F2(-LOG2E)).get(a, b);
    add2(F2(exp2_approx(a), exp2_approx(b)), F2(1.f)).get(a, b);
    return mul2(z, F2(rcp_approx(a), rcp_approx(b)));
}

constexpr int V = 8;  // channels of a piece

// A piece as it is loaded, so that all of a thread's loads can be on their way before the first is used.
template <typename T>
struct Piece {
    static constexpr int N = Vec16<T>::N;
    Vec16<T> v[V / N];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int k = 0; k < V / N; ++k) v[k].load(p + k * N);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < V / N; ++k) v[k].u = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int k = 0; k < V / N; ++k) v[k].store(p + k * N);
    }
    __device__ __forceinline__ void from(const float (&f)[V]) {
#pragma unroll
        for (int k = 0; k < V / N; ++k) {
            float g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = f[k * N + i];
            v[k].from(g);
        }
    }
    __device__ __forceinline__ void to(F2 (&f)[V / 2]) const {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) f[k] = F2(to_f32(v[2 * k / N].e[2 * k % N]), to_f32(v[2 * k / N].e[2 * k % N + 1]));
    }
    __device__ __forceinline__ void from(const F2 (&f)[V / 2]) {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            float a, b;
            f[k].get(a, b);
            if constexpr (N == 8) {
                uint32_t two;
                if constexpr (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(two) : "f"(b), "f"(a));
                else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(two) : "f"(b), "f"(a));
                (k == 0 ? v[0].u.x : k == 1 ? v[0].u.y : k == 2 ? v[0].u.z : v[0].u.w) = two;
            } else {
                v[2 * k / N].e[2 * k % N] = from_f32<T>(a);
                v[2 * k / N].e[2 * k % N + 1] = from_f32<T>(b);
            }
        }
    }
    __device__ __forceinline__ void to(float (&f)[V]) const {
#pragma unroll
        for (int k = 0; k < V / N; ++k) {
            float g[N];
            v[k].to(g);
#pragma unroll
            for (int i = 0; i < N; ++i) f[k * N + i] = g[i];
        }
    }
};
template <typename T, typename F, int M>
__device__ __forceinline__ void write8(T *p, const F (&f)[M]) {
    Piece<T> v;
    v.from(f);
    v.store(p);
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}
__device__ __forceinline__ int int8_of(float q) { return min(127, max(-127, __float2int_rn(q))); }
template <int OUT>
__device__ __forceinline__ void quantise8(uint8_t *p, const F2 (&f)[V / 2], float times) {
    float q[V];
    const F2 m(times);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) mul2(f[i], m).get(q[2 * i], q[2 * i + 1]);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float *r = q + 4 * k;
        if constexpr (OUT == GDN_INT8) {
            w[k] = __byte_perm(__byte_perm(int8_of(r[0]), int8_of(r[1]), 0x0040), __byte_perm(int8_of(r[2]), int8_of(r[3]), 0x0040), 0x5410);
        } else {
            w[k] = (uint32_t)e4m3x2(r[0], r[1]) | (uint32_t)e4m3x2(r[2], r[3]) << 16;
        }
    }
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint8_t quantise1(float y, float times, int out) {
    const float q = y * times;
    return out == GDN_INT8 ? (uint8_t)int8_of(q) : (uint8_t)e4m3x2(q, 0.f);
}

// The sum of the squares, and the largest magnitude.
__device__ __forceinline__ float squares(const F2 (&f)[V / 2]) {
    F2 sum = mul2(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < V / 2; ++i) sum = fma2(f[i], f[i], sum);
    float a, b;
    sum.get(a, b);
    return a + b;
}
__device__ __forceinline__ float largest(const F2 (&f)[V / 2], float top) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        float a, b;
        f[i].get(a, b);
        top = max_or_nan(top, fabsf(a), fabsf(b));
    }
    return top;
}

// The sum (or maximum) over `lanes` neighbouring lanes, a power of two.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) v = max_or_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// Over the CTA; buf: 32 floats that no one else uses until the next barrier but one.
__device__ __forceinline__ float cta_sum(float v, float *buf) {
    v = lanes_sum(v, 32);
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    return lanes_sum(lane < warps ? buf[lane] : 0.f, 32);
}
__device__ __forceinline__ float cta_max(float v, float *buf) {
    v = lanes_max(v, 32);
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    return lanes_max(lane < warps ? buf[lane] : 0.f, 32);
}

// OUT: GDN_F32 stands for the I/O type.
constexpr int SAME = GDN_F32;

// ---------------------------------------------------------------- forward

// Threads of a CTA of it at most: four pieces of FP32 a thread take more registers than 1024 threads have.
template <typename T>
constexpr int token_limit(int U) { return sizeof(T) == 4 && U > 1 ? 512 : 1024; }

// A CTA takes one token; a row's sum is over `lanes` neighbouring threads (heads of 8 to 256 channels), or over the
// CTA (lanes 0: one head).  Thread i holds pieces i, i + threads, .. of it (U at most).
template <typename T, int OUT, int U>
__global__ void __launch_bounds__(token_limit<T>(U)) norm_token_kernel(const RmsNormParams p, int lanes) {
    dependent_prologue();
    __shared__ float buf[3][32];
    const int n = p.H * p.d, pieces = n / V, threads = blockDim.x;
    const long long t = blockIdx.x;
    Piece<T> x[U], r[U], z[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int i = threadIdx.x + k * threads;
        x[k].zero();
        if (i >= pieces) continue;
        x[k].load(static_cast<const T *>(p.x) + t * p.x_stride + i * V);
        if (p.r) r[k].load(static_cast<const T *>(p.r) + t * p.r_stride + i * V);
        if (p.z) z[k].load(static_cast<const T *>(p.z) + t * p.z_stride + i * V);
    }
    Piece<float> weight;  // (of one piece, ahead of its use; of four it would take too many registers)
    if (U == 1 && p.w && threadIdx.x < pieces) weight.load(p.w + (lanes ? threadIdx.x * V % p.d : threadIdx.x * V));
    float sum[U], all = 0.f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int i = threadIdx.x + k * threads;
        F2 s[V / 2];
        x[k].to(s);
        if (p.r && i < pieces) {
            F2 add[V / 2];
            r[k].to(add);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[v] = add2(s[v], add[v]);
            x[k].from(s);
            x[k].to(s);  // what is normalised is the sum as it is stored
            x[k].store(static_cast<T *>(p.s_out) + t * n + i * V);
        }
        sum[k] = squares(s);
        all += sum[k];
    }
    if (lanes) {
#pragma unroll
        for (int k = 0; k < U; ++k) sum[k] = lanes_sum(sum[k], lanes);
    } else {
        all = cta_sum(all, buf[0]);
#pragma unroll
        for (int k = 0; k < U; ++k) sum[k] = all;
    }
    float top = 0.f;
    F2 s[U][V / 2];
    const float mean = 1.f / (float)p.d;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int i = threadIdx.x + k * threads;
        const float rs = rsqrtf(sum[k] * mean + p.eps);
        const F2 rstd(OUT != SAME && !lanes ? 1.f : rs), offset(p.offset);  // (8 bits of one row: the factor goes to the scale)
        x[k].to(s[k]);
        if (i >= pieces) continue;
        if (p.w) {
            F2 w[V / 2];
            if (U > 1) weight.load(p.w + (lanes ? i * V % p.d : i * V));
            weight.to(w);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[k][v] = mul2(s[k][v], mul2(rstd, add2(w[v], offset)));
        } else {
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[k][v] = mul2(s[k][v], rstd);
        }
        if (p.z) {
            F2 gate[V / 2];
            z[k].to(gate);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[k][v] = mul2(s[k][v], silu(gate[v]));
        }
        if constexpr (OUT == SAME) write8(static_cast<T *>(p.y) + t * n + i * V, s[k]);
        else top = largest(s[k], top);
    }
    if constexpr (OUT != SAME) {
        constexpr float MOST = OUT == GDN_INT8 ? 127.f : 448.f;
        const float factor = lanes ? 1.f : rsqrtf(all * mean + p.eps);
        Scale scale;
        if (p.group == 0) {
            scale = scale_of(cta_max(top, buf[1]), factor, MOST);
            if (threadIdx.x == 0) p.scale[t] = scale.scale;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = threadIdx.x + k * threads;
            if (p.group) {  // (whole groups of lanes are past the end together)
                scale = scale_of(lanes_max(largest(s[k], 0.f), p.group / V), factor, MOST);
                if (i < pieces && (i & (p.group / V - 1)) == 0) p.scale[(t * n + i * V) >> (31 - __clz(p.group))] = scale.scale;
            }
            if (i < pieces) quantise8<OUT>(static_cast<uint8_t *>(p.y) + t * n + i * V, s[k], scale.times);
        }
    }
}

// Heads of 32 to 256 channels (a power of two), no scale over whole tokens.  A CTA's threads lie side by side over the
// pieces of `rows` tokens (blockIdx.x: over the parts of a long token; y and z: over the tokens); each takes its piece of U tokens, `rows` apart.
constexpr int HEAD_NT = 128, HEAD_U = 4;

template <typename T, int OUT, int LANES>
__global__ void __launch_bounds__(HEAD_NT) norm_head_kernel(const RmsNormParams p, int rows) {
    dependent_prologue();
    constexpr int U = HEAD_U;
    const int n = p.H * p.d, pieces = n / V;
    const int j = blockIdx.x * blockDim.x + threadIdx.x, row = j / pieces, c = (j - row * pieces) * V;
    const long long t0 = ((long long)blockIdx.z * gridDim.y + blockIdx.y) * (rows * U) + row;
    const bool column = row < rows;
    auto in = [&](int k) { return column && t0 + k * rows < p.T; };
    Piece<T> x[U], z[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        x[k].zero();
        z[k].zero();
        if (!in(k)) continue;
        x[k].load(static_cast<const T *>(p.x) + (t0 + k * rows) * p.x_stride + c);
        if (p.z) z[k].load(static_cast<const T *>(p.z) + (t0 + k * rows) * p.z_stride + c);
    }
    const int group = p.group / V, shift = 31 - __clz(p.group);  // (a power of two)
    F2 w[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) w[v] = F2(1.f);
    if (p.w) {  // (a multiple of the lanes stands before each CTA's threads)
        Piece<float> pw;
        pw.load(p.w + j % LANES * V);
        pw.to(w);
#pragma unroll
        for (int v = 0; v < V / 2; ++v) w[v] = add2(w[v], F2(p.offset));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const long long at = (t0 + k * rows) * n + c;
        F2 s[V / 2];
        x[k].to(s);
        if (p.r && in(k)) {
            Piece<T> r;
            F2 add[V / 2];
            r.load(static_cast<const T *>(p.r) + (t0 + k * rows) * p.r_stride + c);
            r.to(add);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[v] = add2(s[v], add[v]);
            x[k].from(s);
            x[k].to(s);
            x[k].store(static_cast<T *>(p.s_out) + at);
        }
        const float rs = rsqrtf(lanes_sum(squares(s), LANES) * (1.f / (LANES * V)) + p.eps);
        const F2 rstd(rs);
#pragma unroll
        for (int v = 0; v < V / 2; ++v) s[v] = mul2(s[v], OUT == SAME ? mul2(rstd, w[v]) : w[v]);
        if (p.z) {
            F2 gate[V / 2];
            z[k].to(gate);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) s[v] = mul2(s[v], silu(gate[v]));
        }
        if constexpr (OUT == SAME) {
            if (in(k)) write8(static_cast<T *>(p.y) + at, s);
        } else {
            const Scale scale = scale_of(lanes_max(largest(s, 0.f), group), rs, OUT == GDN_INT8 ? 127.f : 448.f);
            if (in(k)) {
                if ((j & (group - 1)) == 0) p.scale[at >> shift] = scale.scale;
                quantise8<OUT>(static_cast<uint8_t *>(p.y) + at, s, scale.times);
            }
        }
    }
}

// Any sizes, alignment and types: a CTA a token, whose rows are read again for every step.
constexpr int ANY_NT = 128;

template <typename T>
__global__ void __launch_bounds__(ANY_NT) norm_any_kernel(const RmsNormParams p, int out_dtype) {
    dependent_prologue();
    __shared__ float buf[2][32];
    const long long t = blockIdx.x, n = (long long)p.H * p.d;
    const T *x = static_cast<const T *>(p.x) + t * p.x_stride;
    const T *r = p.r ? static_cast<const T *>(p.r) + t * p.r_stride : nullptr;
    const T *z = p.z ? static_cast<const T *>(p.z) + t * p.z_stride : nullptr;
    T *s_out = r ? static_cast<T *>(p.s_out) + t * n : nullptr;
    const bool eight = out_dtype == GDN_FP8_E4M3 || out_dtype == GDN_INT8;
    const float most = out_dtype == GDN_INT8 ? 127.f : 448.f;
    const T *s = r ? s_out : x;
    float top = 0.f;
    int turn = 0;
    // pass 0: 16 or 32 bits are written, or a token's largest magnitude found; pass 1: 8 bits
    for (int pass = 0; pass < (eight ? 2 : 1); ++pass) {
        Scale token_scale = {};
        if (pass && p.group == 0) {
            token_scale = scale_of(cta_max(top, buf[turn ^= 1]), 1.f, most);
            if (threadIdx.x == 0) p.scale[t] = token_scale.scale;
        }
        for (int h = 0; h < p.H; ++h) {
            const long long at = (long long)h * p.d;
            float sum = 0.f;
            for (int i = threadIdx.x; i < p.d; i += ANY_NT) {
                if (r && pass == 0) s_out[at + i] = from_f32<T>(to_f32(x[at + i]) + to_f32(r[at + i]));
                const float v = to_f32(s[at + i]);
                sum += v * v;
            }
            const float rstd = rsqrtf(cta_sum(sum, buf[turn ^= 1]) / (float)p.d + p.eps);
            auto value = [&](int i) {
                float v = to_f32(s[at + i]);
                v *= p.w ? rstd * (p.w[i] + p.offset) : rstd;
                if (z) v *= silu(to_f32(z[at + i]));
                return v;
            };
            if (!eight) {
                for (int i = threadIdx.x; i < p.d; i += ANY_NT) static_cast<T *>(p.y)[t * n + at + i] = from_f32<T>(value(i));
            } else if (pass == 0) {
                if (p.group == 0)
                    for (int i = threadIdx.x; i < p.d; i += ANY_NT) top = max_or_nan(top, fabsf(value(i)));
            } else {
                // (a thread's channels of s are its own: what it added, it reads)
                uint8_t *y = static_cast<uint8_t *>(p.y) + t * n + at;
                if (p.group == 0) {
                    for (int i = threadIdx.x; i < p.d; i += ANY_NT) y[i] = quantise1(value(i), token_scale.times, out_dtype);
                } else {
                    for (int g0 = threadIdx.x / 32 * 32; g0 < p.d; g0 += ANY_NT) {
                        // a warp's 32 channels; groups of 64 and 128 look at those of the other warps as well
                        const int start = g0 / p.group * p.group;
                        float m = 0.f;
                        for (int i = start + threadIdx.x % 32; i < start + p.group; i += 32) m = max_or_nan(m, fabsf(value(i)));
                        const Scale scale = scale_of(lanes_max(m, 32), 1.f, most);
                        if (g0 == start && threadIdx.x % 32 == 0) p.scale[(t * n + at + start) / p.group] = scale.scale;
                        y[g0 + threadIdx.x % 32] = quantise1(value(g0 + threadIdx.x % 32), scale.times, out_dtype);
                    }
                }
            }
        }
        __syncthreads();  // pass 1 reads sums that other threads stored
    }
}

// ---------------------------------------------------------------- backward

// With e = dy silu(z): dx = rstd (e w - n mean(e w n)) + dr, dw = sum e n, dz = dy n w silu'(z), n = s rstd.
// The CTAs' parts of dw are summed by a second kernel in order.

// Rows arrive in a ring of stages in shared memory, a bulk copy a row of each input, as far ahead as there is room; a
// CTA takes `cols` channels of every gridDim.x-th token (whole tokens, or whole heads of them: blockIdx.y), thread i the
// pieces i, i + threads, .. of them (U at most).
constexpr int RING_NT = 256, MAX_STAGES = 8;
constexpr size_t RING_BYTES = 200 * 1024;  // of an SM
// CTAs of RING_NT threads that share an SM (three of two pieces a thread would not have the registers).
constexpr int ring_blocks(int U) { return U == 1 ? 3 : 2; }

template <typename T, int U, int NT>
__global__ void __launch_bounds__(NT, ring_blocks(U) * RING_NT / NT) norm_ring_backward_kernel(const RmsNormParams p, int lanes, int cols, int stages) {
    dependent_prologue();
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ float2 buf[2][32];
    __shared__ uint64_t full[MAX_STAGES];
    const int all_cols = p.H * p.d, c0 = blockIdx.y * cols, n = min(cols, all_cols - c0), pieces = n / V;
    const int threads = blockDim.x, arrays = 2 + (p.r != nullptr) + (p.z != nullptr);
    const uint32_t row_bytes = (uint32_t)n * sizeof(T);
    T *ring = reinterpret_cast<T *>(raw);
    auto fetch = [&](int stage, long long t) {
        T *dst = ring + (long long)stage * arrays * n;
        ptx::mbar_arrive_expect_tx(&full[stage], row_bytes * arrays);
        ptx::bulk_g2s(dst, static_cast<const T *>(p.x) + t * p.x_stride + c0, row_bytes, &full[stage]);
        ptx::bulk_g2s(dst += n, static_cast<const T *>(p.dy) + t * p.dy_stride + c0, row_bytes, &full[stage]);
        if (p.r) ptx::bulk_g2s(dst += n, static_cast<const T *>(p.r) + t * p.r_stride + c0, row_bytes, &full[stage]);
        if (p.z) ptx::bulk_g2s(dst += n, static_cast<const T *>(p.z) + t * p.z_stride + c0, row_bytes, &full[stage]);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
        ptx::fence_mbar_init();
        for (int s = 0; s < stages; ++s) {
            const long long t = blockIdx.x + (long long)s * gridDim.x;
            if (t < p.T) fetch(s, t);
        }
    }
    F2 part[U][V / 2], w[U][V / 2];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int i = threadIdx.x + k * threads;
#pragma unroll
        for (int v = 0; v < V / 2; ++v) part[k][v] = F2(0.f), w[k][v] = F2(1.f);
        if (p.w && i < pieces) {
            Piece<float> pw;
            pw.load(p.w + i * V % p.d);
            pw.to(w[k]);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) w[k][v] = add2(w[k][v], F2(p.offset));
        }
    }
    __syncthreads();
    const float mean = 1.f / (float)p.d;
    int stage = 0, turn = 0;
    uint32_t parity = 0;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
        ptx::mbar_wait_bounded(&full[stage], parity, 2000000000ll);
        const T *src = ring + (long long)stage * arrays * n;
        Piece<T> x[U], dy[U], r[U], z[U];
        float2 sum[U], all = make_float2(0.f, 0.f);  // of s^2 and of e w s: mean(e w n) = rstd mean(e w s)
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = threadIdx.x + k * threads;
            sum[k] = make_float2(0.f, 0.f);
            if (i < pieces) {
                const T *at = src + i * V;
                F2 xf[V / 2], e[V / 2];
                x[k].load(at);
                dy[k].load(at += n);
                if (p.r) r[k].load(at += n);
                x[k].to(xf);
                dy[k].to(e);
                if (p.z) {
                    F2 zf[V / 2];
                    z[k].load(at += n);
                    z[k].to(zf);
#pragma unroll
                    for (int v = 0; v < V / 2; ++v) e[v] = mul2(e[v], silu(zf[v]));
                }
                F2 dot(0.f);
#pragma unroll
                for (int v = 0; v < V / 2; ++v) dot = fma2(mul2(e[v], w[k][v]), xf[v], dot);
                float a, b;
                dot.get(a, b);
                sum[k] = make_float2(squares(xf), a + b);
            }
            all.x += sum[k].x;
            all.y += sum[k].y;
        }
        if (lanes) {
#pragma unroll
            for (int k = 0; k < U; ++k) sum[k] = make_float2(lanes_sum(sum[k].x, lanes), lanes_sum(sum[k].y, lanes));
        } else {
            all = make_float2(lanes_sum(all.x, 32), lanes_sum(all.y, 32));
            turn ^= 1;
            if (threadIdx.x % 32 == 0) buf[turn][threadIdx.x / 32] = all;
        }
        __syncthreads();  // every thread has its pieces: the stage can be filled again
        if (threadIdx.x == 0 && t + (long long)stages * gridDim.x < p.T) fetch(stage, t + (long long)stages * gridDim.x);
        if (++stage == stages) stage = 0, parity ^= 1;
        if (!lanes) {
            const int lane = threadIdx.x % 32;
            all = lane < threads / 32 ? buf[turn][lane] : make_float2(0.f, 0.f);
            all = make_float2(lanes_sum(all.x, 32), lanes_sum(all.y, 32));
#pragma unroll
            for (int k = 0; k < U; ++k) sum[k] = all;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = threadIdx.x + k * threads;
            if (i >= pieces) continue;
            const float rs = rsqrtf(sum[k].x * mean + p.eps);
            const F2 rstd(rs), minus_dot(-sum[k].y * rs * mean);
            F2 xf[V / 2], e[V / 2], add[V / 2];
            x[k].to(xf);
            dy[k].to(e);
            if (p.r) r[k].to(add);
            if (p.z) {
                F2 zf[V / 2];
                z[k].to(zf);
#pragma unroll
                for (int v = 0; v < V / 2; ++v) {
                    // silu = z sig, silu' = sig (1 + z (1 - sig))
                    float a, b;
                    zf[v].get(a, b);
                    const F2 sig(sigmoid(a), sigmoid(b));
                    const F2 slope = mul2(sig, fma2(zf[v], fma2(sig, F2(-1.f), F2(1.f)), F2(1.f)));
                    const F2 dyn = mul2(e[v], mul2(xf[v], rstd));
                    e[v] = mul2(e[v], mul2(zf[v], sig));
                    zf[v] = mul2(mul2(dyn, w[k][v]), slope);
                }
                write8(static_cast<T *>(p.dz) + t * all_cols + c0 + i * V, zf);
            }
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                const F2 nx = mul2(xf[v], rstd);
                part[k][v] = fma2(e[v], nx, part[k][v]);
                xf[v] = mul2(rstd, fma2(nx, minus_dot, mul2(e[v], w[k][v])));
                if (p.r) xf[v] = add2(xf[v], add[v]);
            }
            write8(static_cast<T *>(p.dx) + t * all_cols + c0 + i * V, xf);
        }
    }
    if (!p.dw) return;
    float *out = p.partials + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * p.d;
    if (p.H == 1) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = threadIdx.x + k * threads;
            if (i < pieces) write8(out + i * V, part[k]);
        }
        return;
    }
    // the heads' parts are summed in order; the ring has room for them, and no copy is on its way any more
    float *heads = reinterpret_cast<float *>(raw);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int i = threadIdx.x + k * threads;
        if (i < pieces) write8(heads + i * V, part[k]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += threads) {
        float sum = 0.f;
        for (int h = 0; h < n; h += p.d) sum += heads[h + c];
        out[c] = sum;
    }
}

template <typename T>
__global__ void __launch_bounds__(ANY_NT) norm_any_backward_kernel(const RmsNormParams p) {
    dependent_prologue();
    __shared__ float buf[2][32];
    const long long n = (long long)p.H * p.d;
    float *part = p.dw ? p.partials + (long long)blockIdx.x * p.d : nullptr;
    if (part)
        for (int i = threadIdx.x; i < p.d; i += ANY_NT) part[i] = 0.f;
    int turn = 0;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
        for (int h = 0; h < p.H; ++h) {
            const long long at = (long long)h * p.d;
            const T *x = static_cast<const T *>(p.x) + t * p.x_stride + at;
            const T *dy = static_cast<const T *>(p.dy) + t * p.dy_stride + at;
            const T *r = p.r ? static_cast<const T *>(p.r) + t * p.r_stride + at : nullptr;
            const T *z = p.z ? static_cast<const T *>(p.z) + t * p.z_stride + at : nullptr;
            auto weight = [&](int i) { return p.w ? p.w[i] + p.offset : 1.f; };
            auto gated = [&](int i) { return to_f32(dy[i]) * (z ? silu(to_f32(z[i])) : 1.f); };
            float sum = 0.f, dot = 0.f;
            for (int i = threadIdx.x; i < p.d; i += ANY_NT) {
                const float v = to_f32(x[i]);
                sum = fmaf(v, v, sum);
                dot = fmaf(gated(i) * weight(i), v, dot);
            }
            const float rstd = rsqrtf(cta_sum(sum, buf[turn ^= 1]) / (float)p.d + p.eps);
            dot = cta_sum(dot, buf[turn ^= 1]) * rstd / (float)p.d;
            for (int i = threadIdx.x; i < p.d; i += ANY_NT) {
                const float nx = to_f32(x[i]) * rstd, e = gated(i);
                float dx = rstd * fmaf(-nx, dot, e * weight(i));
                if (r) dx += to_f32(r[i]);
                static_cast<T *>(p.dx)[t * n + at + i] = from_f32<T>(dx);
                if (part) part[i] += e * nx;
                if (z) {
                    const float zv = to_f32(z[i]), sig = sigmoid(zv);
                    static_cast<T *>(p.dz)[t * n + at + i] = from_f32<T>(to_f32(dy[i]) * nx * weight(i) * (sig * fmaf(zv, 1.f - sig, 1.f)));
                }
            }
        }
    }
}

// dw of 32 channels a CTA: warps take rows of the parts in turn, their sums are joined in order.
constexpr int SUM_WARPS = 16;
__global__ void __launch_bounds__(32 * SUM_WARPS) norm_sums_kernel(const RmsNormParams p, int parts) {
    dependent_prologue();
    __shared__ float buf[SUM_WARPS][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < p.d) {
#pragma unroll 8
        for (int k = warp; k < parts; k += SUM_WARPS) sum += p.partials[(long long)k * p.d + c];
    }
    buf[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < p.d) {
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < SUM_WARPS; ++k) sum += buf[k][lane];
        p.dw[c] = sum;
    }
}

// ---------------------------------------------------------------- launches

bool whole(const void *ptr, long long stride, size_t elem) {
    return ((reinterpret_cast<uintptr_t>(ptr) | (unsigned long long)stride * elem) & 15u) == 0;
}
bool power_of_two(int n) { return (n & (n - 1)) == 0; }

// Lanes that a head's sum is taken over if it is a few lanes', else 0.
int head_lanes(int d) { return d % V == 0 && d / V <= 32 && power_of_two(d / V) ? d / V : 0; }

// Threads of a CTA that takes a token of `pieces`, U each: whole warps, as even as can be.
int token_threads(int pieces, int U) { return ((pieces + U - 1) / U + 31) / 32 * 32; }

// How the backward pass is cut: CTAs over the tokens (what is resident at once, or one a token) and over the channels.
struct Cut {
    int cols, threads, tokens, parts;  // parts: of the channels
};
Cut backward_cut(int T, int H, int d) {
    const long long n = (long long)H * d;
    Cut c;
    // heads of a few lanes need nothing of one another: as many of them a CTA as its threads have a piece each of
    const bool heads = H > 1 && head_lanes(d);
    c.cols = (int)(heads ? std::min<long long>(n, RING_NT * V) : n);
    c.parts = (int)((n + c.cols - 1) / c.cols);
    const long long pieces = (c.cols + V - 1) / V;
    // (up to two pieces a thread; twice the threads beyond)
    c.threads = pieces > 2 * RING_NT ? 2 * RING_NT : (int)std::min<long long>(RING_NT, (pieces + 31) / 32 * 32);
    const int slots = std::min(8, ring_blocks(pieces > RING_NT ? 2 : 1) * RING_NT / c.threads) * current_device_sms();
    c.tokens = std::min(T, std::max(1, slots / c.parts));
    return c;
}

template <typename T, int OUT>
cudaError_t forward_typed(const RmsNormParams &p, int out_dtype, cudaStream_t stream) {
    const long long n = (long long)p.H * p.d;
    const int lanes = head_lanes(p.d);
    const bool vec = n % V == 0 && p.d % V == 0 && whole(p.x, p.x_stride, sizeof(T)) && whole(p.r, p.r_stride, sizeof(T)) &&
                     whole(p.z, p.z_stride, sizeof(T)) && whole(p.w, 0, 4) && whole(p.s_out, n, sizeof(T)) &&
                     (OUT == SAME ? whole(p.y, n, sizeof(T)) : reinterpret_cast<uintptr_t>(p.y) % 8 == 0);
    const long long pieces = n / V;
    if (vec && lanes >= 4 && (OUT == SAME || p.group)) {
        const int rows = (int)std::max<long long>(1, HEAD_NT / pieces), parts = (int)((pieces * rows + HEAD_NT - 1) / HEAD_NT);
        const int threads = (int)((pieces * rows + parts * 32 - 1) / (parts * 32)) * 32;
        const long long runs = ((long long)p.T + rows * HEAD_U - 1) / (rows * HEAD_U);
        const long long deep = (runs + 65534) / 65535;
        const dim3 grid((unsigned)parts, (unsigned)((runs + deep - 1) / deep), (unsigned)deep), block((unsigned)threads);
        switch (lanes) {
            case 4: return launch_dependent(norm_head_kernel<T, OUT, 4>, grid, block, 0, stream, p, rows);
            case 8: return launch_dependent(norm_head_kernel<T, OUT, 8>, grid, block, 0, stream, p, rows);
            case 16: return launch_dependent(norm_head_kernel<T, OUT, 16>, grid, block, 0, stream, p, rows);
            default: return launch_dependent(norm_head_kernel<T, OUT, 32>, grid, block, 0, stream, p, rows);
        }
    }
    if (vec && (p.H == 1 || lanes) && pieces <= 4 * token_limit<T>(4)) {
        // Few tokens: as many threads as there are pieces, for latency.  Many: four pieces a thread, whose loads are all
        // on their way at once, and fewer threads to wait for one another.
        const dim3 grid((unsigned)p.T);
        const int few = p.H > 1 ? lanes : 0;
        if (pieces <= 512 && p.T < 8 * current_device_sms())
            return launch_dependent(norm_token_kernel<T, OUT, 1>, grid, dim3(token_threads((int)pieces, 1)), 0, stream, p, few);
        return launch_dependent(norm_token_kernel<T, OUT, 4>, grid, dim3(token_threads((int)pieces, 4)), 0, stream, p, few);
    }
    return launch_dependent(norm_any_kernel<T>, dim3((unsigned)p.T), dim3(ANY_NT), 0, stream, p, out_dtype);
}

template <typename T>
cudaError_t forward_out(const RmsNormParams &p, int out_dtype, cudaStream_t stream) {
    switch (out_dtype) {
        case GDN_FP8_E4M3: return forward_typed<T, GDN_FP8_E4M3>(p, out_dtype, stream);
        case GDN_INT8: return forward_typed<T, GDN_INT8>(p, out_dtype, stream);
        default: return forward_typed<T, SAME>(p, out_dtype, stream);
    }
}

template <typename T, int U, int NT>
cudaError_t launch_ring(const RmsNormParams &p, const Cut &cut, int lanes, size_t stage, cudaStream_t stream) {
    // (smaller CTAs share an SM with more)
    const size_t room = std::max(stage * 2, RING_BYTES / ring_blocks(U) * (size_t)cut.threads / RING_NT);
    const int stages = (int)std::min<size_t>(MAX_STAGES, room / stage);
    auto kernel = norm_ring_backward_kernel<T, U, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RING_BYTES);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3((unsigned)cut.tokens, (unsigned)cut.parts), dim3((unsigned)cut.threads), stages * stage, stream,
                            p, lanes, cut.cols, stages);
}

template <typename T>
cudaError_t backward_typed(const RmsNormParams &p, cudaStream_t stream) {
    const long long n = (long long)p.H * p.d;
    const int lanes = p.H > 1 ? head_lanes(p.d) : 0;
    const Cut cut = backward_cut(p.T, p.H, p.d);
    const size_t stage = (size_t)(2 + (p.r != nullptr) + (p.z != nullptr)) * cut.cols * sizeof(T);
    int parts = cut.tokens * cut.parts;
    cudaError_t e = cudaSuccess;
    if (p.T > 0) {
        const bool vec = p.d % V == 0 && whole(p.x, p.x_stride, sizeof(T)) && whole(p.dy, p.dy_stride, sizeof(T)) &&
                         whole(p.r, p.r_stride, sizeof(T)) && whole(p.z, p.z_stride, sizeof(T)) && whole(p.w, 0, 4) &&
                         whole(p.dx, n, sizeof(T)) && whole(p.dz, n, sizeof(T));
        const int pieces = cut.cols / V;
        if (vec && (p.H == 1 || lanes) && pieces <= 4 * RING_NT && stage * 2 <= RING_BYTES && cut.parts <= 65535) {
            if (pieces <= RING_NT) e = launch_ring<T, 1, RING_NT>(p, cut, lanes, stage, stream);
            else if (pieces <= 2 * RING_NT) e = launch_ring<T, 2, RING_NT>(p, cut, lanes, stage, stream);
            else e = launch_ring<T, 2, 2 * RING_NT>(p, cut, lanes, stage, stream);
        } else {
            parts = cut.tokens;
            e = launch_dependent(norm_any_backward_kernel<T>, dim3((unsigned)parts), dim3(ANY_NT), 0, stream, p);
        }
    }
    if (e != cudaSuccess || !p.dw) return e;
    return launch_dependent(norm_sums_kernel, dim3((unsigned)((p.d + 31) / 32)), dim3(32 * SUM_WARPS), 0, stream, p, parts);
}

}  // namespace

size_t rms_norm_backward_workspace_bytes(int T, int H, int d) {
    const Cut cut = backward_cut(T, H, d);
    return 4 * (size_t)cut.tokens * cut.parts * d;
}

cudaError_t launch_rms_norm(const RmsNormParams &p, int io_dtype, int out_dtype, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return forward_out<__half>(p, out_dtype, stream);
        case GDN_BF16: return forward_out<__nv_bfloat16>(p, out_dtype, stream);
        default: return forward_out<float>(p, out_dtype, stream);
    }
}

cudaError_t launch_rms_norm_backward(const RmsNormParams &p, int io_dtype, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return backward_typed<__half>(p, stream);
        case GDN_BF16: return backward_typed<__nv_bfloat16>(p, stream);
        default: return backward_typed<float>(p, stream);
    }
}

}  // namespace gdn
