// The gated linear recurrence, backward: l_t = dy_t + g_(t+1) l_(t+1) a channel, and the
// gradients of the inputs from it.
#include "layer_internal.cuh"

namespace gdn {
namespace {

constexpr int NT = 128;
constexpr int BLOCK = GDN_RECURRENCE_CHECKPOINT;

// A thread carries one channel backwards through a sequence, a block of tokens between
// checkpoints at a time, whose states it computes again.
template <typename T, int MODE>
__global__ void __launch_bounds__(NT) recurrence_serial_backward_kernel(const RecurrenceParams p) {
    dependent_prologue();
    using G = typename GateType<T, MODE>::type;
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y;
    if (c == 0 && b == 0 && p.cu && (p.cu[0] != 0 || p.cu[p.B] != p.T)) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    if (c >= p.C) return;
    float *sums = static_cast<float *>(p.workspace);
    float sum_A = 0.f, sum_dt = 0.f;
    const int begin = recurrence_start(p, b), end = recurrence_start(p, b + 1);
    const int slot = p.slots ? p.slots[b] : b;
    if (begin < 0 || end < begin || end > p.T) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    } else if (slot < 0 || slot >= p.num_slots) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
    } else {
        const float rate = MODE ? expf(p.A_log[c]) : 0.f, dt = MODE ? p.dt_bias[c] : 0.f;
        auto gate = [&](long long t) {
            const float a = to_f32(static_cast<const G *>(p.a)[t * p.a_stride + c]);
            const float bv = p.b ? to_f32(static_cast<const G *>(p.b)[t * p.b_stride + c]) : 0.f;
            return gate_of<MODE>(a, bv, rate, dt, p.b != nullptr);
        };
        float m = p.dfinal ? p.dfinal[(long long)slot * p.C + c] : 0.f;  // what reaches the state after token t
        float before[BLOCK];
        for (int top = end; top > begin;) {
            const int low = max(begin, (top - 1) / BLOCK * BLOCK);
            float h = low == begin ? (p.init ? p.init[(long long)slot * p.C + c] : 0.f)
                                   : p.states[(long long)(low / BLOCK) * p.C + c];
            for (int t = low; t < top; ++t) {
                before[t - low] = h;
                const Gate g = gate(t);
                h = g.g * h + g.w * to_f32(static_cast<const T *>(p.x)[t * p.x_stride + c]);
            }
            for (long long t = top - 1; t >= low; --t) {
                const Gate g = gate(t);
                const float l = m + to_f32(static_cast<const T *>(p.dy)[t * p.dy_stride + c]);
                const float x = to_f32(static_cast<const T *>(p.x)[t * p.x_stride + c]);
                const GateGrad d = gate_grad<MODE>(g, l * before[t - low], l * x, rate);
                static_cast<T *>(p.dx)[t * p.C + c] = from_f32<T>(l * g.w);
                static_cast<G *>(p.da)[t * p.C + c] = from_f32<G>(d.da);
                if (p.b) static_cast<G *>(p.db)[t * p.C + c] = from_f32<G>(d.db);
                sum_A += d.dA;
                sum_dt += d.da;
                m = g.g * l;
            }
            top = low;
        }
        if (p.dinit) p.dinit[(long long)slot * p.C + c] = m;
    }
    if constexpr (MODE != RECUR_PRECOMPUTED) {
        sums[2 * (long long)b * p.C + c] = sum_A;
        sums[(2 * (long long)b + 1) * p.C + c] = sum_dt;
    }
}

__global__ void __launch_bounds__(NT) recurrence_sums_kernel(const RecurrenceParams p) {
    dependent_prologue();
    const int c = blockIdx.x * NT + threadIdx.x;
    if (c >= p.C) return;
    const float *sums = static_cast<const float *>(p.workspace);
    float A = 0.f, dt = 0.f;
    for (long long b = 0; b < p.B; ++b) {
        A += sums[2 * b * p.C + c];
        dt += sums[(2 * b + 1) * p.C + c];
    }
    if (p.dA_log) p.dA_log[c] = A;
    if (p.ddt_bias) p.ddt_bias[c] = dt;
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, cudaStream_t stream) {
    const unsigned gx = (unsigned)((p.C + NT - 1) / NT);
    cudaError_t e = p.B == 0 ? cudaSuccess : launch_dependent(recurrence_serial_backward_kernel<T, MODE>, dim3(gx, (unsigned)p.B), dim3(NT), 0, stream, p);
    if (e != cudaSuccess || MODE == RECUR_PRECOMPUTED || (!p.dA_log && !p.ddt_bias)) return e;
    return launch_dependent(recurrence_sums_kernel, dim3(gx), dim3(NT), 0, stream, p);
}

template <typename T>
cudaError_t launch_mode(const RecurrenceParams &p, int mode, cudaStream_t stream) {
    switch (mode) {
        case RECUR_PRECOMPUTED: return launch_typed<T, RECUR_PRECOMPUTED>(p, stream);
        case RECUR_RAW: return launch_typed<T, RECUR_RAW>(p, stream);
        default: return launch_typed<T, RECUR_RAW_UNIT>(p, stream);
    }
}

}  // namespace

size_t recurrence_backward_workspace_bytes(int B, int, int C) { return 8 * (size_t)B * C; }

cudaError_t launch_recurrence_backward(const RecurrenceParams &p, int io_dtype, int mode, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return launch_mode<__half>(p, mode, stream);
        case GDN_BF16: return launch_mode<__nv_bfloat16>(p, mode, stream);
        default: return launch_mode<float>(p, mode, stream);
    }
}

}  // namespace gdn
