// Root-mean-square norm of rows, with the residual's addition before it, a gate after
// it and an output in 8 bits; forward and backward.
#include "layer_internal.cuh"

namespace gdn {
namespace {

constexpr int NT = 128;

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float cta_sum(float v, float *buf) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s += buf[i];
    return s;
}

__device__ __forceinline__ float cta_max(float v, float *buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max_or_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s = max_or_nan(s, buf[i]);
    return s;
}

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }

// The scale of 8-bit values whose largest magnitude is top.
__device__ __forceinline__ float scale_of(float top, float most) {
    if (!(top <= 3.402823466e38f)) return __int_as_float(0x7fc00000);
    return top == 0.f ? 1.f : __fdiv_rn(top, most);
}

__device__ __forceinline__ uint8_t to_e4m3(float q) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(0.f), "f"(q));
    return (uint8_t)v;
}
__device__ __forceinline__ int8_t to_int8(float q) { return (int8_t)min(127, max(-127, __float2int_rn(q))); }

// A CTA a token; any sizes, alignment and types.  Rows are read again for every step.
template <typename T>
__global__ void __launch_bounds__(NT) norm_any_kernel(const RmsNormParams p, int out_dtype) {
    dependent_prologue();
    __shared__ float buf[NT / 32];
    const long long t = blockIdx.x, n = (long long)p.H * p.d;
    const T *x = static_cast<const T *>(p.x) + t * p.x_stride;
    const T *r = p.r ? static_cast<const T *>(p.r) + t * p.r_stride : nullptr;
    const T *z = p.z ? static_cast<const T *>(p.z) + t * p.z_stride : nullptr;
    T *s_out = r ? static_cast<T *>(p.s_out) + t * n : nullptr;
    const bool eight = out_dtype == GDN_FP8_E4M3 || out_dtype == GDN_INT8;
    const float most = out_dtype == GDN_INT8 ? 127.f : 448.f;
    const T *s = r ? s_out : x;
    float top = 0.f;
    // pass 0: 16 or 32 bits are written, or a token's largest magnitude found; pass 1: 8 bits
    for (int pass = 0; pass < (eight ? 2 : 1); ++pass) {
        const float token_scale = pass ? scale_of(cta_max(top, buf), most) : 0.f;
        if (pass && p.group == 0 && threadIdx.x == 0) p.scale[t] = token_scale;
        for (int h = 0; h < p.H; ++h) {
            const long long at = (long long)h * p.d;
            float sum = 0.f;
            for (int i = threadIdx.x; i < p.d; i += NT) {
                if (r && pass == 0) s_out[at + i] = from_f32<T>(to_f32(x[at + i]) + to_f32(r[at + i]));
                const float v = to_f32(s[at + i]);
                sum += v * v;
            }
            const float rstd = rsqrtf(cta_sum(sum, buf) / (float)p.d + p.eps);
            auto value = [&](int i) {
                float v = to_f32(s[at + i]) * rstd;
                if (p.w) v *= p.w[i] + p.offset;
                if (z) v *= silu(to_f32(z[at + i]));
                return v;
            };
            if (!eight) {
                for (int i = threadIdx.x; i < p.d; i += NT) static_cast<T *>(p.y)[t * n + at + i] = from_f32<T>(value(i));
            } else if (pass == 0) {
                if (p.group == 0)
                    for (int i = threadIdx.x; i < p.d; i += NT) top = max_or_nan(top, fabsf(value(i)));
            } else {
                // a warp takes whole groups; without groups a thread takes channels as before
                const int step = p.group ? p.group : 32;
                for (int g0 = threadIdx.x / 32 * step; g0 < p.d; g0 += NT / 32 * step) {
                    float scale = token_scale;
                    if (p.group) {
                        float m = 0.f;
                        for (int i = g0 + threadIdx.x % 32; i < g0 + step; i += 32) m = max_or_nan(m, fabsf(value(i)));
                        for (int o = 16; o; o >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                        scale = scale_of(m, most);
                        if (threadIdx.x % 32 == 0) p.scale[(t * n + at + g0) / p.group] = scale;
                    }
                    for (int i = g0 + threadIdx.x % 32; i < min(g0 + step, p.d); i += 32) {
                        const float q = __fdiv_rn(value(i), scale);
                        uint8_t *dst = static_cast<uint8_t *>(p.y) + t * n + at + i;
                        *dst = out_dtype == GDN_INT8 ? (uint8_t)to_int8(q) : to_e4m3(q);
                    }
                }
            }
        }
    }
}

// Backward, a CTA for every PART_TOKENS-th token; its rows' part of dweight.
constexpr int PART_CTAS = 592;

template <typename T>
__global__ void __launch_bounds__(NT) norm_any_backward_kernel(const RmsNormParams p) {
    dependent_prologue();
    __shared__ float buf[NT / 32];
    const long long n = (long long)p.H * p.d;
    float *part = p.dw ? p.partials + (long long)blockIdx.x * p.d : nullptr;
    if (part)
        for (int i = threadIdx.x; i < p.d; i += NT) part[i] = 0.f;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
        for (int h = 0; h < p.H; ++h) {
            const long long at = (long long)h * p.d;
            const T *x = static_cast<const T *>(p.x) + t * p.x_stride + at;
            const T *dy = static_cast<const T *>(p.dy) + t * p.dy_stride + at;
            const T *r = p.r ? static_cast<const T *>(p.r) + t * p.r_stride + at : nullptr;
            const T *z = p.z ? static_cast<const T *>(p.z) + t * p.z_stride + at : nullptr;
            auto weight = [&](int i) { return p.w ? p.w[i] + p.offset : 1.f; };
            auto gated = [&](int i) { return to_f32(dy[i]) * (z ? silu(to_f32(z[i])) : 1.f); };
            float sum = 0.f;
            for (int i = threadIdx.x; i < p.d; i += NT) sum += to_f32(x[i]) * to_f32(x[i]);
            const float rstd = rsqrtf(cta_sum(sum, buf) / (float)p.d + p.eps);
            float dot = 0.f;
            for (int i = threadIdx.x; i < p.d; i += NT) dot += gated(i) * weight(i) * (to_f32(x[i]) * rstd);
            dot = cta_sum(dot, buf) / (float)p.d;
            for (int i = threadIdx.x; i < p.d; i += NT) {
                const float nx = to_f32(x[i]) * rstd, e = gated(i);
                float dx = rstd * (e * weight(i) - nx * dot);
                if (r) dx += to_f32(r[i]);
                static_cast<T *>(p.dx)[t * n + at + i] = from_f32<T>(dx);
                if (part) part[i] += e * nx;
                if (z) {
                    const float zv = to_f32(z[i]), sig = 1.f / (1.f + expf(-zv));
                    static_cast<T *>(p.dz)[t * n + at + i] =
                        from_f32<T>(to_f32(dy[i]) * nx * weight(i) * (sig * (1.f + zv * (1.f - sig))));
                }
            }
        }
    }
}

__global__ void __launch_bounds__(NT) norm_sums_kernel(const RmsNormParams p, int parts) {
    dependent_prologue();
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i >= p.d) return;
    float sum = 0.f;
    for (int k = 0; k < parts; ++k) sum += p.partials[(long long)k * p.d + i];
    p.dw[i] = sum;
}

int parts_of(int T) { return T < PART_CTAS ? T : PART_CTAS; }

template <typename T>
cudaError_t backward_typed(const RmsNormParams &p, cudaStream_t stream) {
    cudaError_t e = p.T == 0 ? cudaSuccess : launch_dependent(norm_any_backward_kernel<T>, dim3((unsigned)parts_of(p.T)), dim3(NT), 0, stream, p);
    if (e != cudaSuccess || !p.dw) return e;
    return launch_dependent(norm_sums_kernel, dim3((unsigned)((p.d + NT - 1) / NT)), dim3(NT), 0, stream, p, parts_of(p.T));
}

}  // namespace

size_t rms_norm_backward_workspace_bytes(int T, int, int d) { return 4 * (size_t)parts_of(T) * d; }

cudaError_t launch_rms_norm(const RmsNormParams &p, int io_dtype, int out_dtype, cudaStream_t stream) {
    const dim3 grid((unsigned)p.T), block(NT);
    switch (io_dtype) {
        case GDN_F16: return launch_dependent(norm_any_kernel<__half>, grid, block, 0, stream, p, out_dtype);
        case GDN_BF16: return launch_dependent(norm_any_kernel<__nv_bfloat16>, grid, block, 0, stream, p, out_dtype);
        default: return launch_dependent(norm_any_kernel<float>, grid, block, 0, stream, p, out_dtype);
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
