// The paged key-value cache: writing new tokens (rotated and quantised on the
// way) and reading contexts back.
//
// Both are HBM streams: a write reads a token's k, v (and q) once and writes
// its cache rows once; a read back reads cache rows once and writes them in
// the I/O type.  At decode sizes a write is a launch and two dependent loads
// (position, table), so it takes the query rotation along: 1.7 us for 64 tokens
// of 8 + 8 heads of 128.
//
// Write: a row (one token's channels of one head) belongs to a group of
// d * sizeof(T) / 32 lanes, each holding two 16-byte groups with whole channel
// pairs.  The rotation needs no exchange and the largest magnitude is a few
// shuffles inside the group; the quantised row leaves as one contiguous run.
// 8 x 512 BF16 tokens of 8 + 8 heads of 128: 7.4 us as they are (traffic: 5.3 us), 8.2
// us to e4m3, 9.3 us to int8 (4.1 us).  No one resource is full: over the int8 write's 2.7
// waves of CTAs the issue slots are 68% busy while the SMs are active (a launch's start and
// end are a quarter of the time), its ALU 51%, and warps wait for the row, then the table.
//
// Read back: a warp looks up its tokens' rows, a lane each, and then moves them
// in pieces of 16 output bytes, READ_UNROLL in flight a lane (with 2 45.5 us
// where 4 took 41.7 us for int8; 8: the same, 16-bit rows 19% slower).  Keys
// first, then values: the two in turn ran 20% slower at 16 bits.  39,000 tokens
// of 8 + 8 int8 heads of 128 to BF16: 40.1 us, 6.1 TB/s (0.90 of a copy's rate);
// 16-bit rows 51 us, 6.2 TB/s; four contexts of at most 77 tokens 2.0 us.
#include "attn_internal.cuh"

#include <string.h>

#include <algorithm>

namespace gdn {
namespace {

// (256: a write of 4096 int8 tokens 9.7 us instead of 9.4 us, four short ones with their read
// back 4.1 us instead of 4.0 us; 512: 10.3 and 4.8 us)
constexpr int NT = 128;

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

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A row's scale for its largest magnitude (infinity or NaN: the row has a
// non-finite channel).  e4m3 takes a power of two: with top = m 2^e, m in
// [1, 2), top <= 448 * 2^x = 1.75 * 2^(x+8) for x = e - 8 if m <= 1.75, else e - 7.
template <int CacheDtype>
__device__ __forceinline__ float row_scale(float top) {
    if (!(top <= 3.402823466e38f)) return __int_as_float(0x7fc00000);
    if (top == 0.f) return 1.f;
    if constexpr (CacheDtype == GDN_INT8) {
        return __fdiv_rn(top, 127.f);
    } else {
        const int bits = __float_as_int(top);
        const int e = (bits >> 23) - 127 - ((bits & 0x7fffff) > 0x600000 ? 7 : 8);
        return __int_as_float((max(e, -120) + 127) << 23);
    }
}

// N channels (a multiple of 4) as 8-bit values.  int8 is the correctly rounded
// quotient x / scale, rounded to the nearest integer, ties to even.  The
// product y with the reciprocal is within 2^-15 of it (at most 127, three
// roundings of 2^-24 or less), which decides unless y is that close to the middle of
// two integers: 0.5% of 16-bit inputs, whose scale is a short ratio.  h, the
// multiple of 1/2 next to y, is then that middle, x - h scale is exact, and
// z = h + (x - h scale) / scale, rounded once, lies on the quotient's side of h
// or on h: the reciprocal's error moves the second term by less than 2^-25 ulp
// of h where it reaches half an ulp, and a quotient of two floats is further
// than that from the middle between two floats.
template <int CacheDtype, int N>
__device__ __forceinline__ void quantise(const float (&x)[N], float scale, uint32_t (&out)[N / 4]) {
    if constexpr (CacheDtype == GDN_INT8) {
        int q[N];
        if (scale >= 0x1p-100f) {
            const float inv = __frcp_rn(scale);
            constexpr float HALVES = 6291456.f, WHOLES = 12582912.f;  // 1.5 * 2^22, 1.5 * 2^23: ulps of 1/2 and 1
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float h = __fsub_rn(__fmaf_rn(x[i], inv, HALVES), HALVES);
                const float z = __fmaf_rn(__fmaf_rn(-h, scale, x[i]), inv, h);
                q[i] = __float_as_int(__fadd_rn(z, WHOLES));  // its low byte is the integer
            }
        } else {  // subnormal remainders, and NaN
#pragma unroll
            for (int i = 0; i < N; ++i) q[i] = min(127, max(-127, __float2int_rn(__fdiv_rn(x[i], scale))));
        }
#pragma unroll
        for (int i = 0; i < N; i += 4)
            out[i / 4] = __byte_perm(__byte_perm(q[i], q[i + 1], 0x0040), __byte_perm(q[i + 2], q[i + 3], 0x0040), 0x5410);
    } else {
        // the reciprocal of a power of two is exact; a NaN stays one
        const float inv = scale == scale ? __int_as_float((254 << 23) - __float_as_int(scale)) : scale;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
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
    const int lane_bits = 31 - __clz(p.c.d / (2 * N)), lanes = 1 << lane_bits;  // 4 to 32 lanes a row
    const unsigned rows = 2 * p.c.H + p.Hq;  // rows a token: k heads, v heads, q heads
    // T * rows fits 32 bits (checked on the host)
    const unsigned row = blockIdx.x * (unsigned)(NT >> lane_bits) + (threadIdx.x >> lane_bits);
    const int item = threadIdx.x & (lanes - 1);
    const unsigned token = row / rows;
    const int which = (int)(row - token * rows);
    const long long t = token;
    bool active = t < p.T;
    const bool is_k = which < p.c.H, is_q = which >= 2 * p.c.H;
    const int h = is_q ? which - 2 * p.c.H : is_k ? which : which - p.c.H;
    int c1, c2;
    item_channels<N>(item, p.table ? p.rot : 0, p.interleaved != 0, c1, c2);

    // The row, its slot and its position are independent loads.
    int slot = -1, pos = 0;
    float x1[N] = {}, x2[N] = {};
    if (active) {
        const T *src = is_k ? static_cast<const T *>(p.k) + t * p.k_stride
                            : is_q ? static_cast<const T *>(p.q) + t * p.q_stride
                                   : static_cast<const T *>(p.v) + t * p.v_stride;
        src += (long long)h * p.c.d;
        Vec16<T> a, b;
        a.load(src + c1);
        b.load(src + c2);
        slot = p.slots[t];
        if (p.table) pos = p.pos[t];
        a.to(x1);
        b.to(x2);
        if (slot < -1 || slot >= p.c.num_pages * p.c.page_size) {
            if (which == 0 && item == 0) flag_error(p.status, GDN_DEVERR_CACHE_SLOT);
            active = false;
        }
        if (p.table && (pos < 0 || pos >= p.P)) {
            if (which == 0 && item == 0) flag_error(p.status, GDN_DEVERR_POSITION);
            active = false;
        }
        if (slot < 0 && !is_q) active = false;
    }

    const bool turned = active && p.table && (is_k || is_q) && item * 2 * N < p.rot;
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
        for (int i = 0; i < N; ++i) top = max_or_nan(max_or_nan(top, fabsf(x1[i])), fabsf(x2[i]));
        for (int m = 1; m < lanes; m <<= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
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
    const long long page = slot / p.c.page_size, off = slot - page * p.c.page_size;
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

constexpr int READ_UNROLL = 4;  // pieces in flight a lane

// N channels of a cache row, as loaded.
template <int CacheDtype, int N>
struct Raw {
    using C = typename Elem<CacheDtype>::type;
    static constexpr int WORDS = N * (int)sizeof(C) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const C *src) {
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(src + i * 4 / sizeof(C));
                w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
            }
        } else if constexpr (WORDS == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            w[0] = u.x, w[1] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(src);
        }
    }
    __device__ __forceinline__ void to(float scale, float (&x)[N]) const {
        if constexpr (CacheDtype == GDN_FP8_E4M3 || CacheDtype == GDN_INT8) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint32_t pair = w[i / 4] >> (8 * (i % 4));
                if constexpr (CacheDtype == GDN_INT8) {
                    x[i] = (float)(int8_t)pair * scale;
                    x[i + 1] = (float)(int8_t)(pair >> 8) * scale;
                } else {
                    uint32_t h2;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)pair));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                    x[i] = f.x * scale;
                    x[i + 1] = f.y * scale;
                }
            }
        } else {
            C e[N];
            memcpy(e, w, sizeof(w));
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
        }
    }
};

// blockIdx.y: keys, values.  A warp takes p.tok tokens (at most 32): a lane looks up each token's
// sequence, page and row, then all lanes move the rows' pieces of 16 output
// bytes, U of them in flight.
// SINGLE: it takes one.
template <typename T, int CacheDtype, bool SINGLE>
__global__ void __launch_bounds__(NT) kv_read_kernel(const KvReadParams p) {
    dependent_prologue();
    using C = typename Elem<CacheDtype>::type;
    constexpr bool Q8 = CacheDtype == GDN_FP8_E4M3 || CacheDtype == GDN_INT8;
    constexpr int N = Vec16<T>::N;
    constexpr int U = READ_UNROLL;
    // The look-ups below assume ascending entries; the value CTAs check them, some each.
    if (blockIdx.y == 1)
        for (long long b = (long long)blockIdx.x * NT + threadIdx.x; b < p.B; b += (long long)gridDim.x * NT)
            if (p.cu[b + 1] < p.cu[b] || (b == 0 && p.cu[0] != 0) || (b == p.B - 1 && p.cu[p.B] != p.T))
                flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    const int lane = threadIdx.x % 32;
    const long long t0 = ((long long)blockIdx.x * (NT / 32) + threadIdx.x / 32) * (SINGLE ? 1 : p.tok);
    if (t0 >= p.T) return;
    const int tokens = SINGLE ? 1 : (int)min((long long)p.tok, p.T - t0);

    // the last sequence that starts at or before t0, all lanes probing; then before the lane's own token
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, at < hi && p.cu[at] <= t0);
        const int k = before ? 31 - __clz(before) : 0;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    long long off = -1, soff = 0;  // -1: skipped, -2: a row of zeros
    if (lane < tokens) {
        const int t = (int)t0 + lane;
        int begin = p.cu[lo], end = p.cu[lo + 1];
        if (t >= end && lo + 1 < p.B) {
            hi = p.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            begin = p.cu[lo], end = p.cu[lo + 1];
        }
        const int pos = t - begin;
        if (begin < 0 || pos < 0 || t >= end || end > p.T ||
            (long long)pos >= (long long)p.pages_per_seq * p.c.page_size) {
            flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
        } else {
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

    const int head_shift = 31 - __clz(p.c.d / N);  // a head has 8 to 64 pieces
    const int per_token = p.c.H << head_shift, n = tokens * per_token;
    const C *src = static_cast<const C *>(blockIdx.y ? p.c.v : p.c.k);
    const float *scales = blockIdx.y ? p.c.v_scale : p.c.k_scale;
    T *out = static_cast<T *>(blockIdx.y ? p.v_out : p.k_out) + t0 * p.c.H * p.c.d;
    if constexpr (SINGLE) {
        off = __shfl_sync(0xffffffffu, off, 0);
        soff = __shfl_sync(0xffffffffu, soff, 0);
        if (off == -1) return;
    }
    for (int base = 0; base < n; base += 32 * U) {
        Raw<CacheDtype, N> raw[U];
        float scale[U];
        T *dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + 32 * u + lane;
            int k = i;
            long long o = off, so = soff;
            if constexpr (!SINGLE) {
                const int r = __umulhi((unsigned)i, p.per_token_inv);
                k = i - r * per_token;
                o = __shfl_sync(0xffffffffu, off, r);
                so = __shfl_sync(0xffffffffu, soff, r);
            }
            const int h = k >> head_shift, ch = (k & ((1 << head_shift) - 1)) * N;
            dst[u] = i < n && o != -1 ? out + (long long)i * N : nullptr;
            raw[u] = {};
            scale[u] = 0.f;
            if (i < n && o >= 0) {
                raw[u].load(src + o + h * p.c.head_stride + ch);
                if constexpr (Q8) scale[u] = scales[so + h * p.c.s_head_stride];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!dst[u]) continue;
            float x[N];
            raw[u].to(scale[u], x);
            Vec16<T> v;
            v.from(x);
            v.store(dst[u]);
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

template <typename T, bool SINGLE>
cudaError_t read_io(const KvReadParams &p, int cache_dtype, cudaStream_t stream) {
    const long long warps = (p.T + (long long)p.tok - 1) / p.tok;
    const dim3 grid((unsigned)((warps + NT / 32 - 1) / (NT / 32)), 2);
    switch (cache_dtype) {
        case GDN_F16: return launch_dependent(kv_read_kernel<T, GDN_F16, SINGLE>, grid, dim3(NT), 0, stream, p);
        case GDN_BF16: return launch_dependent(kv_read_kernel<T, GDN_BF16, SINGLE>, grid, dim3(NT), 0, stream, p);
        case GDN_FP8_E4M3: return launch_dependent(kv_read_kernel<T, GDN_FP8_E4M3, SINGLE>, grid, dim3(NT), 0, stream, p);
        case GDN_INT8: return launch_dependent(kv_read_kernel<T, GDN_INT8, SINGLE>, grid, dim3(NT), 0, stream, p);
        default: return launch_dependent(kv_read_kernel<T, GDN_F32, SINGLE>, grid, dim3(NT), 0, stream, p);
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

cudaError_t launch_kv_read(const KvReadParams &given, int io_dtype, int cache_dtype, cudaStream_t stream) {
    if (given.T == 0 || given.B == 0) return cudaSuccess;
    KvReadParams p = given;
    // A token a warp where that fills a pass of its lanes (or would leave warps out otherwise), else as many as
    // two passes hold.  (39,000 tokens of 8 int8 heads of 128: 40.1 us with one, 41.6 us with two.)
    const long long per_token = (long long)p.c.H * p.c.d * (io_dtype == GDN_F32 ? 4 : 2) / 16;
    const long long most = 2 * 32 * READ_UNROLL / per_token, share = p.T / (32LL * current_device_sms());
    p.tok = per_token >= 32 * READ_UNROLL ? 1 : (int)std::max(1LL, std::min(std::min(most, share), 32LL));
    p.per_token_inv = (unsigned)((1ULL << 32) / per_token + 1);  // exact below 2^32 / per_token (one token: not used)
    const bool single = p.tok == 1;
    auto launch = [&](auto t) {
        using T = decltype(t);
        return single ? read_io<T, true>(p, cache_dtype, stream) : read_io<T, false>(p, cache_dtype, stream);
    };
    switch (io_dtype) {
        case GDN_F16: return launch(__half());
        case GDN_BF16: return launch(__nv_bfloat16());
        default: return launch(0.f);
    }
}

}  // namespace gdn
