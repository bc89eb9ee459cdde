// The gated linear recurrence, forward: h_t = g_t h_(t-1) + w_t x_t a channel.
#include "layer_internal.cuh"

namespace gdn {
namespace {

constexpr int NT = 128;

// A thread carries one channel through a sequence's tokens.
template <typename T, int MODE>
__global__ void __launch_bounds__(NT) recurrence_serial_kernel(const RecurrenceParams p) {
    dependent_prologue();
    using G = typename GateType<T, MODE>::type;
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y;
    if (c == 0 && b == 0 && p.cu && (p.cu[0] != 0 || p.cu[p.B] != p.T)) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    if (c >= p.C) return;
    const int begin = recurrence_start(p, b), end = recurrence_start(p, b + 1);
    if (begin < 0 || end < begin || end > p.T) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
        return;
    }
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.num_slots) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
        return;
    }
    float h = p.init ? p.init[(long long)slot * p.C + c] : 0.f;
    const float rate = MODE ? expf(p.A_log[c]) : 0.f, dt = MODE ? p.dt_bias[c] : 0.f;
    for (long long t = begin; t < end; ++t) {
        if (p.checkpoints && t % GDN_RECURRENCE_CHECKPOINT == 0)
            p.checkpoints[t / GDN_RECURRENCE_CHECKPOINT * p.C + c] = t == begin ? 0.f : h;
        const float a = to_f32(static_cast<const G *>(p.a)[t * p.a_stride + c]);
        const float bv = p.b ? to_f32(static_cast<const G *>(p.b)[t * p.b_stride + c]) : 0.f;
        const Gate g = gate_of<MODE>(a, bv, rate, dt, p.b != nullptr);
        h = g.g * h + g.w * to_f32(static_cast<const T *>(p.x)[t * p.x_stride + c]);
        static_cast<T *>(p.y)[t * p.C + c] = from_f32<T>(h);
    }
    if (p.final_state) p.final_state[(long long)slot * p.C + c] = h;
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, int longest, cudaStream_t stream) {
    return launch_dependent(recurrence_serial_kernel<T, MODE>, dim3((unsigned)((p.C + NT - 1) / NT), (unsigned)p.B),
                            dim3(NT), 0, stream, p);
}

template <typename T>
cudaError_t launch_mode(const RecurrenceParams &p, int mode, int longest, cudaStream_t stream) {
    switch (mode) {
        case RECUR_PRECOMPUTED: return launch_typed<T, RECUR_PRECOMPUTED>(p, longest, stream);
        case RECUR_RAW: return launch_typed<T, RECUR_RAW>(p, longest, stream);
        default: return launch_typed<T, RECUR_RAW_UNIT>(p, longest, stream);
    }
}

}  // namespace

size_t recurrence_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_recurrence(const RecurrenceParams &p, int io_dtype, int mode, int longest, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return launch_mode<__half>(p, mode, longest, stream);
        case GDN_BF16: return launch_mode<__nv_bfloat16>(p, mode, longest, stream);
        default: return launch_mode<float>(p, mode, longest, stream);
    }
}

}  // namespace gdn
