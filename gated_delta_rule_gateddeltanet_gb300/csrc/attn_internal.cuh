// Internal launch interface of the softmax-attention operators (rotary
// positions, paged key-value cache, paged attention); not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {

// A frequency table's parameters, resolved on the host (see gdn_rotary_table_args).
struct RotaryTableParams {
    int P, pairs, scaling;
    double base;            // after GDN_ROPE_NTK's stretch
    double inv_factor;      // 1 / s
    double ramp_lo, ramp_hi;  // YARN: pair indices; BY_PARTS: turns
    double turns_per_freq;  // BY_PARTS: P0 / (2 pi)
    double magnitude;
    float *table;
};

constexpr int ROTARY_THREADS = 128;  // of a CTA; a thread rotates at least one pair

struct RotaryParams {
    int T, Hq, Hk, d, rot, P, interleaved;
    float sign;  // -1: the inverse rotation
    long long q_stride, k_stride, qo_stride, ko_stride;
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t *pos;
    const float *table;
    int32_t *status;
};

// A paged cache with its strides resolved (elements).
struct PagedCache {
    int num_pages, page_size, H, d;
    long long page_stride, token_stride, head_stride;
    long long s_page_stride, s_token_stride, s_head_stride;
    void *k, *v;
    float *k_scale, *v_scale;
};

struct KvWriteParams {
    PagedCache c;
    int T, Hq, rot, P, interleaved;
    long long k_stride, v_stride, q_stride, qo_stride;
    const void *k, *v, *q;
    void *q_out;
    const int32_t *slots, *pos;
    const float *table;  // null: no rotation
    int32_t *status;
};

struct KvReadParams {
    PagedCache c;
    int B, T, pages_per_seq;
    int tok;                 // tokens a warp, set by the launch
    unsigned per_token_inv;  // 2^32 / pieces of a token
    long long bt_stride;
    const int32_t *block_table, *cu;
    void *k_out, *v_out;
    int32_t *status;
};

struct PagedAttnParams {
    PagedCache c;
    int B, T, Hq, G, pages_per_seq, window, rows_hint;  // rows_hint: query rows (tokens x group) expected per key head
    int io_bf16;       // q and out are BF16 (8-bit caches; otherwise they have the cache's type)
    float scale_log2;  // softmax scale times log2(e)
    long long bt_stride, q_stride;
    const void *q;
    const int32_t *block_table, *kv_lens, *cu;  // cu null: one token per sequence
    void *out;
    float *lse;
    int32_t *status;
    float *partials;
    int page_shift;  // log2(page_size), -1 if it is not a power of two
    int s_page_stride32, s_token_stride32, s_head_stride32;  // the scale strides of the cache
};

cudaError_t launch_rotary_table(const RotaryTableParams &p, cudaStream_t stream);
cudaError_t launch_rotary(const RotaryParams &p, int io_dtype, cudaStream_t stream);
cudaError_t launch_kv_write(const KvWriteParams &p, int io_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadParams &p, int io_dtype, int cache_dtype, cudaStream_t stream);

// Tensor map over one half of a paged cache, strides in elements: rows are cut
// into spans of 128 bytes (a row, if that is less), dimensions are (element of
// a span, token, span, head, page).  A box of box_tokens tokens and box_spans
// spans lands in shared memory as box_spans tiles of box_tokens spans each,
// with the 16-byte pieces swizzled: piece x of the r-th span of a tile that
// starts on a 1024-byte boundary at x ^ (r % 8), for 64-byte spans at x ^ (r / 2 % 4).
bool encode_cache_rows(CUtensorMap *map, const void *base, int elem_bytes, int d, int heads, int page_size, int pages,
                       long long head_stride, long long token_stride, long long page_stride, int box_tokens, int box_spans);

// Attention kernels are instantiated per cache type, one translation unit each.
template <int CacheDtype>
cudaError_t launch_paged_attention(const PagedAttnParams &p, cudaStream_t stream);

// Query rows a kernel takes at a time, in groups of 8: two groups, or what the
// registers of a consumer hold of FP32 rows.  (Four groups read the cache half as
// often for 32 rows, but run 52 us against 45 us at 16 requests x 4 drafts x 8 heads a
// key head of 128, up to 8191 cached, 38 us against 30 us at 64, 47 us against 37 us at e4m3.)
constexpr int max_row_tiles(bool f32, int d) { return f32 && d > 64 ? 1 : 2; }
inline int row_tiles(bool f32, int d, int rows) { return rows <= 8 ? 1 : max_row_tiles(f32, d); }
// One CTA per SM: its ring of copies takes the whole shared memory.
inline int attention_ctas() { return current_device_sms(); }
// A CTA's record of a split unit (8 int32), and two unnormalised parts: rows x d
// outputs and each row's maximum and sum.
inline size_t attention_workspace_floats(bool f32, int d, int rows) {
    return (size_t)attention_ctas() * (8 + 2 * 8 * row_tiles(f32, d, rows) * (d + 2));
}

// ---------------------------------------------------------------- device helpers

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes of T as floats, and back (each rounded once).
template <typename T>
struct Vec16 {
    static constexpr int N = 16 / (int)sizeof(T);
    union {
        uint4 u;
        T e[N];
    };
    __device__ __forceinline__ Vec16() {}
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = u; }
    __device__ __forceinline__ void to(float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(e[i]);
    }
    __device__ __forceinline__ void from(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<T>(f[i]);
    }
};

// One channel pair turned by (c, s).  The products and the sum are rounded
// separately (no fused multiply-add), so that a value quantised after the
// rotation does not depend on which of the two products was fused.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float &ya, float &yb) {
    ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    yb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Two 16-byte groups of N channels turned: half layout pairs x1[i] with x2[i];
// interleaved pairs neighbours inside x1 and inside x2.  c, s: the N pairs' entries.
template <int N>
__device__ __forceinline__ void turn_groups(float (&x1)[N], float (&x2)[N], const float (&c)[N], const float (&s)[N],
                                            bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            turn(x1[i], x1[i + 1], c[i / 2], s[i / 2], x1[i], x1[i + 1]);
            turn(x2[i], x2[i + 1], c[N / 2 + i / 2], s[N / 2 + i / 2], x2[i], x2[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) turn(x1[i], x2[i], c[i], s[i], x1[i], x2[i]);
    }
}

// Channels of the two groups that item i of a row covers: a rotated item's
// two groups hold N whole pairs, later items are plain neighbours.
template <int N>
__device__ __forceinline__ void item_channels(int i, int rot, bool interleaved, int &c1, int &c2) {
    const int turned = rot / (2 * N);
    if (i < turned && !interleaved) {
        c1 = i * N;
        c2 = c1 + rot / 2;
    } else {
        c1 = i * 2 * N;
        c2 = c1 + N;
    }
}

template <int N>
__device__ __forceinline__ void load_floats(const float *p, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
}

}  // namespace gdn
