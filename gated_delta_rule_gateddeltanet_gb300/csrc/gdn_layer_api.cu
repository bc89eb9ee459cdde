// The C ABI of the gated linear recurrence and the root-mean-square norm: argument
// checks and dispatch.  Everything that the host can check is checked here, before
// any launch; data-dependent checks happen in the kernels.
#include <math.h>
#include <stdint.h>

#include "layer_internal.cuh"

namespace {

bool valid_io(int t) { return t == GDN_F32 || t == GDN_F16 || t == GDN_BF16; }
size_t io_bytes(int t) { return t == GDN_F32 ? 4 : 2; }
bool eight_bit(int t) { return t == GDN_FP8_E4M3 || t == GDN_INT8; }
bool aligned(const void *ptr, size_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; }
// The stride to use for one given as 0, or -1 for a stride below `least`.
long long stride_or(int64_t given, int64_t least) { return given == 0 ? least : given < least ? -1 : given; }
cudaStream_t cuda_stream(gdn_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
gdn_status of(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Sizes and modes, of a forward call's arguments or a backward call's.
template <typename Args>
gdn_status check_recurrence_sizes(const Args *a) {
    if (!a) return GDN_ERR_NULL;
    if (!valid_io(a->io_dtype)) return GDN_ERR_DTYPE;
    if (a->gate_mode != GDN_GATES_RAW && a->gate_mode != GDN_GATES_PRECOMPUTED) return GDN_ERR_ARG;
    if ((a->unit_input != 0 && a->unit_input != 1) || (a->unit_input && a->gate_mode != GDN_GATES_RAW)) return GDN_ERR_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->total_tokens < 0 || a->total_tokens > (1 << 30) || a->channels < 1 || a->channels > (1 << 24)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// What both directions have: gates, packing, states.
template <typename Args>
gdn_status resolve_recurrence(const Args *a, gdn::RecurrenceParams *p, int *mode) {
    if (a->num_seqs > 0 && (a->num_state_slots < 1 || (!a->state_slots && a->num_state_slots < a->num_seqs))) return GDN_ERR_SHAPE;
    if (!a->cu_seqlens && a->num_seqs > 0 && a->total_tokens % a->num_seqs != 0) return GDN_ERR_SHAPE;
    p->x_stride = stride_or(a->x_stride, a->channels);
    p->a_stride = stride_or(a->a_stride, a->channels);
    p->b_stride = stride_or(a->b_stride, a->channels);
    if (p->x_stride < 0 || p->a_stride < 0 || p->b_stride < 0) return GDN_ERR_SHAPE;
    const bool raw = a->gate_mode == GDN_GATES_RAW;
    if (a->total_tokens > 0 && (!a->x || !a->a)) return GDN_ERR_NULL;
    if (raw && (!a->A_log || !a->dt_bias)) return GDN_ERR_NULL;
    const size_t gate = raw ? io_bytes(a->io_dtype) : 4;
    if (!aligned(a->x, io_bytes(a->io_dtype)) || !aligned(a->a, gate) || !aligned(a->b, gate) || !aligned(a->A_log, 4) ||
        !aligned(a->dt_bias, 4) || !aligned(a->initial_state, 4))
        return GDN_ERR_ALIGN;
    p->B = a->num_seqs;
    p->T = a->total_tokens;
    p->C = a->channels;
    p->num_slots = a->num_state_slots;
    p->S = a->num_seqs > 0 ? a->total_tokens / a->num_seqs : 0;
    p->x = a->x;
    p->a = a->a;
    p->b = a->b;
    p->A_log = raw ? a->A_log : nullptr;
    p->dt_bias = raw ? a->dt_bias : nullptr;
    p->cu = a->cu_seqlens;
    p->slots = a->state_slots;
    p->init = a->initial_state;
    p->status = a->status;
    *mode = !raw ? gdn::RECUR_PRECOMPUTED : a->unit_input ? gdn::RECUR_RAW_UNIT : gdn::RECUR_RAW;
    return GDN_OK;
}

gdn_status check_workspace(const void *workspace, size_t has, size_t needs) {
    if (needs == 0) return GDN_OK;
    if (!workspace || has < needs) return GDN_ERR_WORKSPACE;
    return aligned(workspace, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

gdn_status check_forward_sizes(const gdn_linear_recurrence_args *a) {
    const gdn_status st = check_recurrence_sizes(a);
    if (st != GDN_OK) return st;
    return a->max_seqlen < 0 ? GDN_ERR_SHAPE : GDN_OK;
}

// The longest sequence, as far as the host knows (num_seqs > 0).
int longest(const gdn_linear_recurrence_args *a) {
    if (!a->cu_seqlens) return a->total_tokens / a->num_seqs;
    int n = a->total_tokens;
    if (a->max_seqlen > 0 && a->max_seqlen < n) n = a->max_seqlen;
    return n;
}

gdn_status check_norm_sizes(int T, int H, int d, int io, float eps, float offset) {
    if (!valid_io(io)) return GDN_ERR_DTYPE;
    // (the kernels count a row's channels in steps of up to 128 with 32-bit counters)
    if (T < 0 || H < 1 || d < 1 || (int64_t)H * d > INT32_MAX - 255) return GDN_ERR_SHAPE;
    if (!(eps > 0.f) || isinf(eps) || !isfinite(offset)) return GDN_ERR_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_linear_recurrence(const gdn_linear_recurrence_args *a, gdn_stream_t stream) {
    gdn_status st = check_forward_sizes(a);
    if (st != GDN_OK) return st;
    gdn::RecurrenceParams p{};
    int mode;
    if ((st = resolve_recurrence(a, &p, &mode)) != GDN_OK) return st;
    if (a->num_seqs == 0) return GDN_OK;
    if (a->total_tokens > 0 && !a->output) return GDN_ERR_NULL;
    if (!aligned(a->output, io_bytes(a->io_dtype)) || !aligned(a->final_state, 4) || !aligned(a->checkpoints, 4))
        return GDN_ERR_ALIGN;
    p.y = a->output;
    p.final_state = a->final_state;
    p.checkpoints = a->checkpoints;
    cudaStream_t s = cuda_stream(stream);
#ifdef GDN_DEBUG_CHECKS
    if (p.final_state && gdn::debug_check_distinct_slots(p.slots, nullptr, p.B, p.num_slots, p.status, s) != cudaSuccess)
        return GDN_ERR_CUDA;
#endif
    return of(gdn::launch_recurrence(p, a->io_dtype, mode, longest(a), s));
}

gdn_status gdn_linear_recurrence_backward(const gdn_linear_recurrence_backward_args *a, gdn_stream_t stream) {
    gdn_status st = check_recurrence_sizes(a);
    if (st != GDN_OK) return st;
    gdn::RecurrenceParams p{};
    int mode;
    if ((st = resolve_recurrence(a, &p, &mode)) != GDN_OK) return st;
    p.dy_stride = stride_or(a->dy_stride, a->channels);
    if (p.dy_stride < 0) return GDN_ERR_SHAPE;
    const bool raw = mode != gdn::RECUR_PRECOMPUTED;
    if (!raw && (a->dA_log || a->ddt_bias)) return GDN_ERR_ARG;
    if (a->db && !a->b) return GDN_ERR_ARG;
    if (a->total_tokens > 0 && (!a->dy || !a->checkpoints || !a->dx || !a->da || (a->b && !a->db))) return GDN_ERR_NULL;
    const size_t io = io_bytes(a->io_dtype), gate = raw ? io : 4;
    if (!aligned(a->dy, io) || !aligned(a->dx, io) || !aligned(a->da, gate) || !aligned(a->db, gate) ||
        !aligned(a->checkpoints, 4) || !aligned(a->d_final_state, 4) || !aligned(a->d_initial_state, 4) ||
        !aligned(a->dA_log, 4) || !aligned(a->ddt_bias, 4))
        return GDN_ERR_ALIGN;
    if (a->d_initial_state && a->d_initial_state == a->d_final_state) return GDN_ERR_ARG;
    p.dy = a->dy;
    p.states = a->checkpoints;
    p.dfinal = a->d_final_state;
    p.dx = a->dx;
    p.da = a->da;
    p.db = a->db;
    p.dA_log = a->dA_log;
    p.ddt_bias = a->ddt_bias;
    p.dinit = a->d_initial_state;
    cudaStream_t s = cuda_stream(stream);
#ifdef GDN_DEBUG_CHECKS
    if (p.dinit && gdn::debug_check_distinct_slots(p.slots, nullptr, p.B, p.num_slots, p.status, s) != cudaSuccess)
        return GDN_ERR_CUDA;
#endif
    return of(gdn::launch_recurrence_backward(p, a->io_dtype, mode, s));
}

gdn_status gdn_rms_norm(const gdn_rms_norm_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    gdn_status st = check_norm_sizes(a->total_tokens, a->num_heads, a->head_dim, a->io_dtype, a->eps, a->weight_offset);
    if (st != GDN_OK) return st;
    const bool eight = eight_bit(a->out_dtype);
    if (!eight && a->out_dtype != a->io_dtype) return GDN_ERR_DTYPE;
    const int G = a->scale_group;
    if (G != 0 && (!eight || (G != 32 && G != 64 && G != 128))) return GDN_ERR_ARG;
    if (G != 0 && a->head_dim % G != 0) return GDN_ERR_SHAPE;
    const int64_t n = (int64_t)a->num_heads * a->head_dim;
    gdn::RmsNormParams p{};
    p.x_stride = stride_or(a->x_stride, n);
    p.r_stride = stride_or(a->residual_stride, n);
    p.z_stride = stride_or(a->gate_stride, n);
    if (p.x_stride < 0 || p.r_stride < 0 || p.z_stride < 0) return GDN_ERR_SHAPE;
    if (!a->residual && a->residual_out) return GDN_ERR_ARG;
    if (a->scale && !eight) return GDN_ERR_ARG;
    if (a->total_tokens == 0) return GDN_OK;
    if (!a->x || !a->output || (a->residual && !a->residual_out) || (eight && !a->scale)) return GDN_ERR_NULL;
    const size_t io = io_bytes(a->io_dtype);
    if (!aligned(a->x, io) || !aligned(a->residual, io) || !aligned(a->gate, io) || !aligned(a->residual_out, io) ||
        !aligned(a->output, eight ? 1 : io) || !aligned(a->weight, 4) || !aligned(a->scale, 4))
        return GDN_ERR_ALIGN;
    // in place: a thread writes only what it has read itself, at the same stride; two outputs are never one
    if ((a->residual_out && ((a->residual_out == a->x && p.x_stride != n) || (a->residual_out == a->residual && p.r_stride != n))) ||
        (a->output == a->x && (eight || p.x_stride != n)) || (a->output == a->gate && (eight || p.z_stride != n)) ||
        a->output == a->residual || a->output == a->residual_out || (a->residual_out && a->residual_out == a->gate))
        return GDN_ERR_ARG;
    p.T = a->total_tokens;
    p.H = a->num_heads;
    p.d = a->head_dim;
    p.group = G;
    p.eps = a->eps;
    p.offset = a->weight_offset;
    p.x = a->x;
    p.r = a->residual;
    p.z = a->gate;
    p.w = a->weight;
    p.s_out = a->residual_out;
    p.y = a->output;
    p.scale = a->scale;
    return of(gdn::launch_rms_norm(p, a->io_dtype, a->out_dtype, cuda_stream(stream)));
}

gdn_status gdn_rms_norm_backward_workspace_size(const gdn_rms_norm_backward_args *a, size_t *bytes) {
    if (!a || !bytes) return GDN_ERR_NULL;
    const gdn_status st = check_norm_sizes(a->total_tokens, a->num_heads, a->head_dim, a->io_dtype, a->eps, a->weight_offset);
    if (st != GDN_OK) return st;
    *bytes = gdn::rms_norm_backward_workspace_bytes(a->total_tokens, a->num_heads, a->head_dim);
    return GDN_OK;
}

gdn_status gdn_rms_norm_backward(const gdn_rms_norm_backward_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    gdn_status st = check_norm_sizes(a->total_tokens, a->num_heads, a->head_dim, a->io_dtype, a->eps, a->weight_offset);
    if (st != GDN_OK) return st;
    const int64_t n = (int64_t)a->num_heads * a->head_dim;
    gdn::RmsNormParams p{};
    p.x_stride = stride_or(a->x_stride, n);
    p.dy_stride = stride_or(a->dy_stride, n);
    p.z_stride = stride_or(a->gate_stride, n);
    p.r_stride = stride_or(a->d_residual_stride, n);
    if (p.x_stride < 0 || p.dy_stride < 0 || p.z_stride < 0 || p.r_stride < 0) return GDN_ERR_SHAPE;
    if ((a->dgate && !a->gate) || (a->dweight && !a->weight)) return GDN_ERR_ARG;
    if (a->total_tokens > 0 && (!a->x || !a->dy || !a->dx || (a->gate && !a->dgate))) return GDN_ERR_NULL;
    const size_t io = io_bytes(a->io_dtype);
    if (!aligned(a->x, io) || !aligned(a->dy, io) || !aligned(a->gate, io) || !aligned(a->d_residual, io) ||
        !aligned(a->dx, io) || !aligned(a->dgate, io) || !aligned(a->weight, 4) || !aligned(a->dweight, 4))
        return GDN_ERR_ALIGN;
    if (a->dx && (a->dx == a->x || a->dx == a->dy || a->dx == a->gate || a->dx == a->d_residual || a->dx == a->dgate))
        return GDN_ERR_ARG;
    if (a->dgate && (a->dgate == a->x || a->dgate == a->dy || a->dgate == a->gate || a->dgate == a->d_residual))
        return GDN_ERR_ARG;
    const size_t needs = a->dweight ? gdn::rms_norm_backward_workspace_bytes(a->total_tokens, a->num_heads, a->head_dim) : 0;
    if ((st = check_workspace(a->workspace, a->workspace_bytes, needs)) != GDN_OK) return st;
    p.T = a->total_tokens;
    p.H = a->num_heads;
    p.d = a->head_dim;
    p.eps = a->eps;
    p.offset = a->weight_offset;
    p.x = a->x;
    p.dy = a->dy;
    p.z = a->gate;
    p.r = a->d_residual;
    p.w = a->weight;
    p.dx = a->dx;
    p.dz = a->dgate;
    p.dw = a->dweight;
    p.partials = static_cast<float *>(a->workspace);
    return of(gdn::launch_rms_norm_backward(p, a->io_dtype, cuda_stream(stream)));
}

}  // extern "C"
