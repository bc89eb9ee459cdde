// The paged key-value cache: writing new tokens (rotated and quantised on the
// way) and reading contexts back.
//
// Both are HBM streams: a write reads a token's k, v (and q) once and writes
// its cache rows once; a read back reads cache rows once and writes them in
// the I/O type.  At decode sizes a write is a launch latency and three
// dependent loads (slot, row, table), so it takes the query rotation along.
//
// Write: a row (one token's channels of one head) belongs to a group of
// d * sizeof(T) / 32 lanes, each holding two 16-byte groups with whole channel
// pairs.  The rotation needs no exchange and the largest magnitude is a few
// shuffles inside the group; the quantised row leaves as one contiguous run.
#include "attn_internal.cuh"

namespace gdn {
namespace {

constexpr int NT = 256;

template <int CacheDtype>
struct Elem;
template <>
struct Elem<GDN_F32> { using type = float; };
template <>
struct Elem<GDN_F16> { using type = __half; };
template <>
struct Elem<GDN_BF16> { using type = __nv_bfloat16; };
template <>
struct Elem<GDN_FP8_E4M3> { using type = uint8_t; };
template <>
struct Elem<GDN_INT8> { using type = int8_t; };

// A row's scale for its largest magnitude (infinity marks a row with a
// non-finite channel).  e4m3 takes a power of two: with top = m 2^e, m in
// [1/2, 1), top <= 448 * 2^x = 0.875 * 2^(x+9) for x = e - 9 if m <= 0.875, else e - 8.
template <int CacheDtype>
__device__ __forceinline__ float row_scale(float top) {
    if (!(top <= 3.402823466e38f)) return __int_as_float(0x7fc00000);
    if (top == 0.f) return 1.f;
    if constexpr (CacheDtype == GDN_INT8) {
        return __fdiv_rn(top, 127.f);
    } else {
        int e;
        const float m = frexpf(top, &e);
        return __int_as_float((max(e - (m > 0.875f ? 8 : 9), -120) + 127) << 23);
    }
}

// N channels (a multiple of 4) as 8-bit values.
template <int CacheDtype, int N>
__device__ __forceinline__ void quantise(const float (&x)[N], float scale, uint32_t (&out)[N / 4]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if constexpr (CacheDtype == GDN_INT8) {
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = min(127, max(-127, __float2int_rn(__fdiv_rn(x[i + j], scale))));
                w |= (uint32_t)(q & 255) << (8 * j);
            }
            out[i / 4] = w;
        } else {
            const float inv = __fdiv_rn(1.f, scale);  // a power of two: exact
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[i + 1] * inv), "f"(x[i] * inv));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[i + 3] * inv), "f"(x[i + 2] * inv));
            out[i / 4] = (uint32_t)lo | (uint32_t)hi << 16;
        }
    }
}

template <typename T, int CacheDtype>
__global__ void __launch_bounds__(NT) kv_write_kernel(const KvWriteParams p) {
    dependent_prologue();
    using C = typename Elem<CacheDtype>::type;
    constexpr int N = Vec16<T>::N;
    constexpr bool Q8 = CacheDtype == GDN_FP8_E4M3 || CacheDtype == GDN_INT8;
    const int lanes = p.c.d / (2 * N);  // 4 to 32 lanes a row
    const int rows = 2 * p.c.H + p.Hq;  // rows a token: k heads, v heads, q heads
    const long long row = ((long long)blockIdx.x * NT + threadIdx.x) / lanes;
    const int item = threadIdx.x % lanes;
    const long long t = row / rows;
    const int which = (int)(row - t * rows);
    bool active = t < p.T;
    const bool is_k = which < p.c.H, is_q = which >= 2 * p.c.H;
    const int h = is_q ? which - 2 * p.c.H : is_k ? which : which - p.c.H;

    int slot = -1, pos = 0;
    if (active) {
        slot = p.slots[t];
        if (slot < -1 || slot >= p.c.num_pages * p.c.page_size) {
            if (which == 0 && item == 0) flag_error(p.status, GDN_DEVERR_CACHE_SLOT);
            active = false;
        }
        if (p.table) {
            pos = p.pos[t];
            if (pos < 0 || pos >= p.P) {
                if (which == 0 && item == 0) flag_error(p.status, GDN_DEVERR_POSITION);
                active = false;
            }
        }
        if (slot < 0 && !is_q) active = false;
    }

    const bool turned = active && p.table && (is_k || is_q) && item * 2 * N < p.rot;
    int c1, c2;
    item_channels<N>(item, p.table ? p.rot : 0, p.interleaved != 0, c1, c2);
    float x1[N] = {}, x2[N] = {};
    if (active) {
        const T *src = is_k ? static_cast<const T *>(p.k) + t * p.k_stride
                            : is_q ? static_cast<const T *>(p.q) + t * p.q_stride
                                   : static_cast<const T *>(p.v) + t * p.v_stride;
        src += (long long)h * p.c.d;
        Vec16<T> a, b;
        a.load(src + c1);
        b.load(src + c2);
        a.to(x1);
        b.to(x2);
    }
    if (turned) {
        float c[N], s[N];
        const float *tab = p.table + (long long)pos * p.rot + item * N;
        load_floats<N>(tab, c);
        load_floats<N>(tab + p.rot / 2, s);
        turn_groups<N>(x1, x2, c, s, p.interleaved != 0);
    }
    float scale = 1.f;
    if constexpr (Q8) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float a = fabsf(x1[i]), b = fabsf(x2[i]);
            top = fmaxf(top, a <= 3.402823466e38f ? a : __int_as_float(0x7f800000));
            top = fmaxf(top, b <= 3.402823466e38f ? b : __int_as_float(0x7f800000));
        }
        for (int m = 1; m < lanes; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        scale = row_scale<CacheDtype>(top);
    }
    if (!active) return;
    if (is_q) {
        T *dst = static_cast<T *>(p.q_out) + t * p.qo_stride + (long long)h * p.c.d;
        Vec16<T> a, b;
        a.from(x1);
        b.from(x2);
        a.store(dst + c1);
        b.store(dst + c2);
        return;
    }
    const long long page = slot / p.c.page_size, off = slot % p.c.page_size;
    C *dst = static_cast<C *>(is_k ? p.c.k : p.c.v) + page * p.c.page_stride + off * p.c.token_stride +
             h * p.c.head_stride;
    if constexpr (Q8) {
        uint32_t a[N / 4], b[N / 4];
        quantise<CacheDtype, N>(x1, scale, a);
        quantise<CacheDtype, N>(x2, scale, b);
        if constexpr (N == 8) {
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(a[0], a[1]);
            *reinterpret_cast<uint2 *>(dst + c2) = make_uint2(b[0], b[1]);
        } else {
            *reinterpret_cast<uint32_t *>(dst + c1) = a[0];
            *reinterpret_cast<uint32_t *>(dst + c2) = b[0];
        }
        if (item == 0)
            (is_k ? p.c.k_scale : p.c.v_scale)[page * p.c.s_page_stride + off * p.c.s_token_stride +
                                               h * p.c.s_head_stride] = scale;
    } else {
        Vec16<T> a, b;
        a.from(x1);
        b.from(x2);
        a.store(reinterpret_cast<T *>(dst) + c1);
        b.store(reinterpret_cast<T *>(dst) + c2);
    }
}

// ---------------------------------------------------------------- read back

constexpr int READ_TOKENS = 16;  // output tokens a CTA
constexpr int ITEM = 16;         // channels a thread moves at a time

template <int CacheDtype>
__device__ __forceinline__ void load_item(const typename Elem<CacheDtype>::type *src, float scale, float (&x)[ITEM]) {
    if constexpr (CacheDtype == GDN_FP8_E4M3 || CacheDtype == GDN_INT8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(src);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (CacheDtype == GDN_INT8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * i + j] = (float)(int8_t)(w[i] >> (8 * j)) * scale;
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t h2;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i] >> (16 * j))));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                    x[4 * i + 2 * j] = f.x * scale;
                    x[4 * i + 2 * j + 1] = f.y * scale;
                }
            }
        }
    } else {
        using T = typename Elem<CacheDtype>::type;
        constexpr int N = Vec16<T>::N;
#pragma unroll
        for (int i = 0; i < ITEM; i += N) {
            Vec16<T> v;
            v.load(src + i);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i + j] = to_f32(v.e[j]);
        }
    }
}

template <typename T, int CacheDtype>
__global__ void __launch_bounds__(NT) kv_read_kernel(const KvReadParams p) {
    dependent_prologue();
    using C = typename Elem<CacheDtype>::type;
    constexpr bool Q8 = CacheDtype == GDN_FP8_E4M3 || CacheDtype == GDN_INT8;
    __shared__ long long row_off[READ_TOKENS], scale_off[READ_TOKENS];  // -1: skipped, -2: zero row
    const int t0 = blockIdx.x * READ_TOKENS;
    if (threadIdx.x < READ_TOKENS) {
        const int t = t0 + threadIdx.x;
        long long off = -1, soff = 0;
        // the last sequence that starts at or before t
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int begin = p.cu[lo], end = p.cu[lo + 1];
        if (t < p.T) {
            if (begin < 0 || t < begin || t >= end || end > p.T ||
                (long long)(t - begin) >= (long long)p.pages_per_seq * p.c.page_size) {
                flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
            } else {
                const int pos = t - begin;
                const int page = p.block_table[lo * p.bt_stride + pos / p.c.page_size];
                const int in_page = pos % p.c.page_size;
                if (page < 0 || page >= p.c.num_pages) {
                    flag_error(p.status, GDN_DEVERR_PAGE);
                    off = -2;
                } else {
                    off = page * p.c.page_stride + in_page * p.c.token_stride;
                    soff = page * p.c.s_page_stride + in_page * p.c.s_token_stride;
                }
            }
        }
        row_off[threadIdx.x] = off;
        scale_off[threadIdx.x] = soff;
    }
    __syncthreads();
    const int per_head = p.c.d / ITEM, per_half = p.c.H * per_head;
    const int n = READ_TOKENS * 2 * per_half;
    for (int i = threadIdx.x; i < n; i += NT) {
        const int r = i / (2 * per_half), j = i - r * 2 * per_half;
        const bool is_v = j >= per_half;
        const int k = is_v ? j - per_half : j;
        const int h = k / per_head, ch = (k - h * per_head) * ITEM;
        const long long off = row_off[r];
        if (off == -1) continue;
        float x[ITEM] = {};
        if (off >= 0) {
            float scale = 1.f;
            if constexpr (Q8) scale = (is_v ? p.c.v_scale : p.c.k_scale)[scale_off[r] + h * p.c.s_head_stride];
            load_item<CacheDtype>(static_cast<const C *>(is_v ? p.c.v : p.c.k) + off + h * p.c.head_stride + ch, scale,
                                  x);
        }
        T *dst = static_cast<T *>(is_v ? p.v_out : p.k_out) + ((long long)(t0 + r) * p.c.H + h) * p.c.d + ch;
        constexpr int N = Vec16<T>::N;
#pragma unroll
        for (int e = 0; e < ITEM; e += N) {
            Vec16<T> v;
#pragma unroll
            for (int u = 0; u < N; ++u) v.e[u] = from_f32<T>(x[e + u]);
            v.store(dst + e);
        }
    }
}

template <typename T, int CacheDtype>
cudaError_t write_typed(const KvWriteParams &p, cudaStream_t stream) {
    const long long threads = (long long)p.T * (2 * p.c.H + p.Hq) * (p.c.d / (2 * Vec16<T>::N));
    return launch_dependent(kv_write_kernel<T, CacheDtype>, dim3((unsigned)((threads + NT - 1) / NT)), dim3(NT), 0,
                            stream, p);
}

template <typename T>
cudaError_t write_io(const KvWriteParams &p, int io_dtype, int cache_dtype, cudaStream_t stream) {
    if (cache_dtype == GDN_FP8_E4M3) return write_typed<T, GDN_FP8_E4M3>(p, stream);
    if (cache_dtype == GDN_INT8) return write_typed<T, GDN_INT8>(p, stream);
    constexpr int same = sizeof(T) == 4 ? GDN_F32 : GDN_F16;  // 16-bit rows are stored as T (the type's name is unused)
    return write_typed<T, same>(p, stream);
}

template <typename T>
cudaError_t read_io(const KvReadParams &p, int cache_dtype, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.T + READ_TOKENS - 1) / READ_TOKENS));
    switch (cache_dtype) {
        case GDN_F16: return launch_dependent(kv_read_kernel<T, GDN_F16>, grid, dim3(NT), 0, stream, p);
        case GDN_BF16: return launch_dependent(kv_read_kernel<T, GDN_BF16>, grid, dim3(NT), 0, stream, p);
        case GDN_FP8_E4M3: return launch_dependent(kv_read_kernel<T, GDN_FP8_E4M3>, grid, dim3(NT), 0, stream, p);
        case GDN_INT8: return launch_dependent(kv_read_kernel<T, GDN_INT8>, grid, dim3(NT), 0, stream, p);
        default: return launch_dependent(kv_read_kernel<T, GDN_F32>, grid, dim3(NT), 0, stream, p);
    }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteParams &p, int io_dtype, int cache_dtype, cudaStream_t stream) {
    if (p.T == 0) return cudaSuccess;
    switch (io_dtype) {
        case GDN_F16: return write_io<__half>(p, io_dtype, cache_dtype, stream);
        case GDN_BF16: return write_io<__nv_bfloat16>(p, io_dtype, cache_dtype, stream);
        default: return write_io<float>(p, io_dtype, cache_dtype, stream);
    }
}

cudaError_t launch_kv_read(const KvReadParams &p, int io_dtype, int cache_dtype, cudaStream_t stream) {
    if (p.T == 0 || p.B == 0) return cudaSuccess;
    switch (io_dtype) {
        case GDN_F16: return read_io<__half>(p, cache_dtype, stream);
        case GDN_BF16: return read_io<__nv_bfloat16>(p, cache_dtype, stream);
        default: return read_io<float>(p, cache_dtype, stream);
    }
}

}  // namespace gdn
