// The C ABI of the softmax-attention operators: argument checks and dispatch.
// Everything that the host can check is checked here, before any launch;
// data-dependent checks happen in the kernels.
#include <math.h>
#include <stdint.h>

#include "attn_internal.cuh"

namespace {

bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

bool valid_io(int t) { return t == GDN_F32 || t == GDN_F16 || t == GDN_BF16; }
size_t io_bytes(int t) { return t == GDN_F32 ? 4 : 2; }
bool eight_bit(int t) { return t == GDN_FP8_E4M3 || t == GDN_INT8; }
size_t cache_bytes(int t) { return eight_bit(t) ? 1 : io_bytes(t); }

// The stride to use for one given as 0, or -1 for a stride below `least`.
long long stride_or(int64_t given, int64_t least) { return given == 0 ? least : given < least ? -1 : given; }

gdn_status check_cache_sizes(const gdn_kv_cache &c) {
    if (!valid_io(c.cache_dtype) && !eight_bit(c.cache_dtype)) return GDN_ERR_DTYPE;
    if (c.num_pages < 1 || c.page_size < 1 || (int64_t)c.num_pages * c.page_size > INT32_MAX) return GDN_ERR_SHAPE;
    if (c.num_kv_heads < 1 || c.num_kv_heads > 65535 || (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

gdn_status resolve_cache(const gdn_kv_cache &c, gdn::PagedCache *out) {
    const gdn_status st = check_cache_sizes(c);
    if (st != GDN_OK) return st;
    if (!c.k || !c.v || (eight_bit(c.cache_dtype) && (!c.k_scale || !c.v_scale))) return GDN_ERR_NULL;
    gdn::PagedCache p{};
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.H = c.num_kv_heads;
    p.d = c.head_dim;
    const bool packed = c.page_stride == 0 && c.token_stride == 0 && c.head_stride == 0;
    p.head_stride = packed ? c.head_dim : c.head_stride;
    p.token_stride = packed ? (int64_t)c.num_kv_heads * c.head_dim : c.token_stride;
    p.page_stride = packed ? (int64_t)c.page_size * p.token_stride : c.page_stride;
    const size_t esz = cache_bytes(c.cache_dtype);
    const int64_t most = (INT64_C(1) << 40) / (int64_t)esz - 1;  // what a tensor map takes
    auto bad = [&](int extent, int64_t stride) { return stride < 0 || (extent > 1 && (stride == 0 || stride > most)); };
    if (bad(c.num_kv_heads, p.head_stride) || bad(c.page_size, p.token_stride) || bad(c.num_pages, p.page_stride))
        return GDN_ERR_SHAPE;
    if (!aligned16(c.k) || !aligned16(c.v) || (p.head_stride * esz) % 16 || (p.token_stride * esz) % 16 ||
        (p.page_stride * esz) % 16)
        return GDN_ERR_ALIGN;
    if (eight_bit(c.cache_dtype)) {
        const bool spacked = c.scale_page_stride == 0 && c.scale_token_stride == 0 && c.scale_head_stride == 0;
        p.s_head_stride = spacked ? 1 : c.scale_head_stride;
        p.s_token_stride = spacked ? c.num_kv_heads : c.scale_token_stride;
        p.s_page_stride = spacked ? (int64_t)c.page_size * c.num_kv_heads : c.scale_page_stride;
        if (p.s_head_stride < 0 || p.s_token_stride < 0 || p.s_page_stride < 0 || p.s_head_stride > INT32_MAX ||
            p.s_token_stride > INT32_MAX || p.s_page_stride > INT32_MAX)
            return GDN_ERR_SHAPE;
        p.k_scale = c.k_scale;
        p.v_scale = c.v_scale;
    }
    p.k = c.k;
    p.v = c.v;
    *out = p;
    return GDN_OK;
}

gdn_status check_attention_sizes(const gdn_paged_attention_args *a) {
    if (!a) return GDN_ERR_NULL;
    const gdn_status st = check_cache_sizes(a->cache);
    if (st != GDN_OK) return st;
    const int ct = a->cache.cache_dtype;
    if (eight_bit(ct) ? a->io_dtype != GDN_F16 && a->io_dtype != GDN_BF16 : a->io_dtype != ct) return GDN_ERR_DTYPE;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->total_tokens < 0 || a->pages_per_seq < 0) return GDN_ERR_SHAPE;
    if (a->num_q_heads < 1 || a->num_q_heads % a->cache.num_kv_heads != 0) return GDN_ERR_SHAPE;
    if (a->window < 0 || a->max_seqlen < 0) return GDN_ERR_SHAPE;
    if (!(a->scale >= 0.f) || isinf(a->scale)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// Query rows of one key head that a sequence is expected to bring.
int rows_hint(const gdn_paged_attention_args *a) {
    const int64_t group = a->num_q_heads / a->cache.num_kv_heads;
    int64_t n = 1;
    if (a->max_seqlen > 0) n = a->max_seqlen;
    else if (a->num_seqs > 0) n = ((int64_t)a->total_tokens + a->num_seqs - 1) / a->num_seqs;
    if (n < 1) n = 1;
    return (int)(n * group > 64 ? 64 : n * group);
}

size_t attention_bytes(const gdn_paged_attention_args *a) {
    return 4 * gdn::attention_workspace_floats(a->cache.cache_dtype == GDN_F32, a->cache.head_dim, rows_hint(a));
}

cudaStream_t cuda_stream(gdn_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

gdn_status gdn_rotary_table(const gdn_rotary_table_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    if (a->scaling < GDN_ROPE_NONE || a->scaling > GDN_ROPE_YARN) return GDN_ERR_ARG;
    if (a->max_positions < 0 || a->rotary_dim < 2 || a->rotary_dim % 2 != 0) return GDN_ERR_SHAPE;
    if (!(a->base > 1.0) || isinf(a->base) || !(a->attention_factor >= 0.0) || isinf(a->attention_factor))
        return GDN_ERR_ARG;
    const bool scaled = a->scaling != GDN_ROPE_NONE;
    if (scaled && (!(a->factor >= 1.0) || isinf(a->factor))) return GDN_ERR_ARG;
    const bool ramp = a->scaling == GDN_ROPE_BY_PARTS || a->scaling == GDN_ROPE_YARN;
    if (ramp && (a->original_positions < 1 || !(a->beta_slow > 0.0) || !(a->beta_fast > a->beta_slow) ||
                 isinf(a->beta_fast)))
        return GDN_ERR_ARG;
    if (a->scaling == GDN_ROPE_NTK && a->rotary_dim <= 2) return GDN_ERR_SHAPE;
    if (a->max_positions == 0) return GDN_OK;
    if (!a->table) return GDN_ERR_NULL;
    const double two_pi = 6.283185307179586476925;
    gdn::RotaryTableParams p{};
    p.P = a->max_positions;
    p.pairs = a->rotary_dim / 2;
    p.scaling = a->scaling;
    p.base = a->base;
    p.inv_factor = scaled ? 1.0 / a->factor : 1.0;
    p.magnitude = a->attention_factor > 0.0 ? a->attention_factor : 1.0;
    if (a->scaling == GDN_ROPE_NTK) p.base *= pow(a->factor, a->rotary_dim / (a->rotary_dim - 2.0));
    if (a->scaling == GDN_ROPE_BY_PARTS) {
        p.ramp_lo = a->beta_slow;
        p.ramp_hi = a->beta_fast;
        p.turns_per_freq = a->original_positions / two_pi;
    }
    if (a->scaling == GDN_ROPE_YARN) {
        auto index = [&](double turns) {
            return a->rotary_dim * log(a->original_positions / (two_pi * turns)) / (2.0 * log(a->base));
        };
        p.ramp_lo = fmin(fmax(floor(index(a->beta_fast)), 0.0), a->rotary_dim - 1.0);
        p.ramp_hi = fmin(fmax(ceil(index(a->beta_slow)), 0.0), a->rotary_dim - 1.0);
        if (p.ramp_hi <= p.ramp_lo) p.ramp_hi = p.ramp_lo + 0.001;  // a step instead of a ramp
        if (a->attention_factor == 0.0) p.magnitude = 0.1 * log(a->factor) + 1.0;
    }
    p.table = a->table;
    return gdn::launch_rotary_table(p, cuda_stream(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_rotary(const gdn_rotary_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    if (!valid_io(a->io_dtype)) return GDN_ERR_DTYPE;
    if ((a->interleaved != 0 && a->interleaved != 1) || (a->inverse != 0 && a->inverse != 1)) return GDN_ERR_ARG;
    if (a->total_tokens < 0 || a->num_q_heads < 0 || a->num_k_heads < 0 || a->max_positions < 0) return GDN_ERR_SHAPE;
    if (a->head_dim < 2 || a->head_dim % 2 || a->rotary_dim < 2 || a->rotary_dim % 2 || a->rotary_dim > a->head_dim)
        return GDN_ERR_SHAPE;
    const int64_t qn = (int64_t)a->num_q_heads * a->head_dim, kn = (int64_t)a->num_k_heads * a->head_dim;
    gdn::RotaryParams p{};
    p.q_stride = stride_or(a->q_stride, qn);
    p.k_stride = stride_or(a->k_stride, kn);
    p.qo_stride = stride_or(a->q_out_stride, qn);
    p.ko_stride = stride_or(a->k_out_stride, kn);
    if (p.q_stride < 0 || p.k_stride < 0 || p.qo_stride < 0 || p.ko_stride < 0) return GDN_ERR_SHAPE;
    if (a->total_tokens == 0 || qn + kn == 0) return GDN_OK;
    if ((qn && (!a->q || !a->q_out)) || (kn && (!a->k || !a->k_out)) || !a->positions || !a->table) return GDN_ERR_NULL;
    // (a thread writes only what it read itself, which in-place calls rely on)
    if ((qn && a->q == a->q_out && p.q_stride != p.qo_stride) || (kn && a->k == a->k_out && p.k_stride != p.ko_stride))
        return GDN_ERR_ARG;
    const int64_t pairs = (int64_t)a->total_tokens * ((a->num_q_heads + a->num_k_heads) * (int64_t)a->head_dim / 2);
    if (pairs / gdn::ROTARY_THREADS >= INT32_MAX || a->num_q_heads + (int64_t)a->num_k_heads > 65535) return GDN_ERR_SHAPE;
    p.T = a->total_tokens;
    p.Hq = a->num_q_heads;
    p.Hk = a->num_k_heads;
    p.d = a->head_dim;
    p.rot = a->rotary_dim;
    p.P = a->max_positions;
    p.interleaved = a->interleaved;
    p.sign = a->inverse ? -1.f : 1.f;
    p.q = qn ? a->q : nullptr;
    p.k = kn ? a->k : nullptr;
    p.q_out = qn ? a->q_out : nullptr;
    p.k_out = kn ? a->k_out : nullptr;
    p.pos = a->positions;
    p.table = a->table;
    p.status = a->status;
    return gdn::launch_rotary(p, a->io_dtype, cuda_stream(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_cache_write(const gdn_kv_write_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    if (!valid_io(a->io_dtype)) return GDN_ERR_DTYPE;
    const gdn_status sizes = check_cache_sizes(a->cache);
    if (sizes != GDN_OK) return sizes;
    if (!eight_bit(a->cache.cache_dtype) && a->cache.cache_dtype != a->io_dtype) return GDN_ERR_DTYPE;
    if (a->interleaved != 0 && a->interleaved != 1) return GDN_ERR_ARG;
    if (a->total_tokens < 0 || a->num_q_heads < 0 || a->max_positions < 0) return GDN_ERR_SHAPE;
    const int d = a->cache.head_dim;
    if (a->table && (a->rotary_dim < 16 || a->rotary_dim % 16 || a->rotary_dim > d)) return GDN_ERR_SHAPE;
    if (a->num_q_heads > 0 && !a->table) return GDN_ERR_ARG;
    const int64_t kn = (int64_t)a->cache.num_kv_heads * d, qn = (int64_t)a->num_q_heads * d;
    gdn::KvWriteParams p{};
    p.k_stride = stride_or(a->k_stride, kn);
    p.v_stride = stride_or(a->v_stride, kn);
    p.q_stride = stride_or(a->q_stride, qn);
    p.qo_stride = stride_or(a->q_out_stride, qn);
    if (p.k_stride < 0 || p.v_stride < 0 || p.q_stride < 0 || p.qo_stride < 0) return GDN_ERR_SHAPE;
    const gdn_status st = resolve_cache(a->cache, &p.c);
    if (st != GDN_OK) return st;
    if (eight_bit(a->cache.cache_dtype) &&  // rows that share a scale can be read, not written
        ((p.c.num_pages > 1 && p.c.s_page_stride == 0) || (p.c.page_size > 1 && p.c.s_token_stride == 0) ||
         (p.c.H > 1 && p.c.s_head_stride == 0)))
        return GDN_ERR_SHAPE;
    if (a->total_tokens == 0) return GDN_OK;
    if (!a->k || !a->v || !a->slots || (a->table && !a->positions) || (qn && (!a->q || !a->q_out))) return GDN_ERR_NULL;
    const size_t esz = io_bytes(a->io_dtype);
    if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->table) || (p.k_stride * esz) % 16 || (p.v_stride * esz) % 16 ||
        (qn && (!aligned16(a->q) || !aligned16(a->q_out) || (p.q_stride * esz) % 16 || (p.qo_stride * esz) % 16)))
        return GDN_ERR_ALIGN;
    if (qn && a->q == a->q_out && p.q_stride != p.qo_stride) return GDN_ERR_ARG;
    if ((int64_t)a->total_tokens * (2 * kn + qn) / 64 >= INT32_MAX) return GDN_ERR_SHAPE;
    p.T = a->total_tokens;
    p.Hq = a->num_q_heads;
    p.rot = a->table ? a->rotary_dim : 0;
    p.P = a->max_positions;
    p.interleaved = a->interleaved;
    p.k = a->k;
    p.v = a->v;
    p.q = a->q;
    p.q_out = a->q_out;
    p.slots = a->slots;
    p.pos = a->positions;
    p.table = a->table;
    p.status = a->status;
    return gdn::launch_kv_write(p, a->io_dtype, a->cache.cache_dtype, cuda_stream(stream)) == cudaSuccess ? GDN_OK
                                                                                                          : GDN_ERR_CUDA;
}

gdn_status gdn_kv_cache_read(const gdn_kv_read_args *a, gdn_stream_t stream) {
    if (!a) return GDN_ERR_NULL;
    if (!valid_io(a->io_dtype)) return GDN_ERR_DTYPE;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->total_tokens < 0 || a->pages_per_seq < 0) return GDN_ERR_SHAPE;
    gdn::KvReadParams p{};
    p.bt_stride = stride_or(a->block_table_stride, a->pages_per_seq);
    if (p.bt_stride < 0) return GDN_ERR_SHAPE;
    const gdn_status st = resolve_cache(a->cache, &p.c);
    if (st != GDN_OK) return st;
    if (a->num_seqs == 0 || a->total_tokens == 0) return GDN_OK;
    if (!a->cu_seqlens || !a->k_out || !a->v_out || (a->pages_per_seq > 0 && !a->block_table)) return GDN_ERR_NULL;
    if (!aligned16(a->k_out) || !aligned16(a->v_out)) return GDN_ERR_ALIGN;
    p.B = a->num_seqs;
    p.T = a->total_tokens;
    p.pages_per_seq = a->pages_per_seq;
    p.block_table = a->block_table;
    p.cu = a->cu_seqlens;
    p.k_out = a->k_out;
    p.v_out = a->v_out;
    p.status = a->status;
    return gdn::launch_kv_read(p, a->io_dtype, a->cache.cache_dtype, cuda_stream(stream)) == cudaSuccess ? GDN_OK
                                                                                                         : GDN_ERR_CUDA;
}

gdn_status gdn_paged_attention_workspace_size(const gdn_paged_attention_args *a, size_t *bytes) {
    if (!bytes) return GDN_ERR_NULL;
    const gdn_status st = check_attention_sizes(a);
    if (st != GDN_OK) return st;
    *bytes = attention_bytes(a);
    return GDN_OK;
}

gdn_status gdn_paged_attention(const gdn_paged_attention_args *a, gdn_stream_t stream) {
    const gdn_status sizes = check_attention_sizes(a);
    if (sizes != GDN_OK) return sizes;
    gdn::PagedAttnParams p{};
    const int d = a->cache.head_dim;
    p.q_stride = stride_or(a->q_stride, (int64_t)a->num_q_heads * d);
    p.bt_stride = stride_or(a->block_table_stride, a->pages_per_seq);
    if (p.q_stride < 0 || p.bt_stride < 0) return GDN_ERR_SHAPE;
    if (!a->cu_seqlens && a->total_tokens != a->num_seqs) return GDN_ERR_SHAPE;
    const gdn_status st = resolve_cache(a->cache, &p.c);
    if (st != GDN_OK) return st;
    if (a->num_seqs == 0 || a->total_tokens == 0) return GDN_OK;
    if (!a->q || !a->output || !a->kv_lens || (a->pages_per_seq > 0 && !a->block_table)) return GDN_ERR_NULL;
    if (!aligned16(a->q) || !aligned16(a->output) || (p.q_stride * io_bytes(a->io_dtype)) % 16) return GDN_ERR_ALIGN;
    if (!a->workspace || a->workspace_bytes < attention_bytes(a)) return GDN_ERR_WORKSPACE;
    if (!aligned16(a->workspace)) return GDN_ERR_ALIGN;
    p.B = a->num_seqs;
    p.T = a->total_tokens;
    p.Hq = a->num_q_heads;
    p.G = a->num_q_heads / a->cache.num_kv_heads;
    p.pages_per_seq = a->pages_per_seq;
    p.window = a->window;
    p.rows_hint = rows_hint(a);
    p.io_bf16 = a->io_dtype == GDN_BF16;
    p.scale_log2 = (a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
    p.q = a->q;
    p.block_table = a->block_table;
    p.kv_lens = a->kv_lens;
    p.cu = a->cu_seqlens;
    p.out = a->output;
    p.lse = a->lse;
    p.status = a->status;
    p.partials = static_cast<float *>(a->workspace);
    p.s_page_stride32 = (int)p.c.s_page_stride;
    p.s_token_stride32 = (int)p.c.s_token_stride;
    p.s_head_stride32 = (int)p.c.s_head_stride;
    p.page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (p.c.page_size == 1 << s) p.page_shift = s;
    cudaError_t e;
    switch (a->cache.cache_dtype) {
        case GDN_F16: e = gdn::launch_paged_attention<GDN_F16>(p, cuda_stream(stream)); break;
        case GDN_BF16: e = gdn::launch_paged_attention<GDN_BF16>(p, cuda_stream(stream)); break;
        case GDN_FP8_E4M3: e = gdn::launch_paged_attention<GDN_FP8_E4M3>(p, cuda_stream(stream)); break;
        case GDN_INT8: e = gdn::launch_paged_attention<GDN_INT8>(p, cuda_stream(stream)); break;
        default: e = gdn::launch_paged_attention<GDN_F32>(p, cuda_stream(stream)); break;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
