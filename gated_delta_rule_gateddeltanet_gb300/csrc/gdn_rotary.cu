// Rotary positions: the table of cosines and sines, and the rotation.
//
// The rotation turns each channel pair (a, b) of a head by its position's
// angle: (a c - b s, b c + a s).  It is HBM-bound: q and k are read and
// written once (4 bytes a channel at 16 bits) and a token's table row serves
// all its heads.  A thread owns an "item" of a head's row: two 16-byte groups
// that hold whole pairs (channels i.. and i + rot/2.. in the half layout, 32
// neighbouring bytes in the interleaved one and past the rotated part).  It
// loads the item's cosines and sines once and applies them to HEADS heads, so
// the table costs one read per HEADS heads and HEADS independent pairs of
// loads are in flight per thread.  8192 BF16 tokens of 18 heads of 256, a quarter
// rotated: 24.4 us, 6.3 TB/s (0.93 of a copy's rate); 4111 FP32 tokens of 16 heads
// of 64, interleaved, inverse: 6.1 us, 5.7 TB/s; 64 tokens of 40 heads: 1.7 us, a launch.
#include "attn_internal.cuh"

namespace gdn {
namespace {

// (256: 24.8 us instead of 24.4 us for the prompt above, 6.3 us instead of 6.1 us for the gradient; 512: 30.7 and
// 6.8 us; 64: 24.4 and 6.5 us.  Two heads a thread instead of four 25.3 us, six 26.9 us.)
constexpr int NT = ROTARY_THREADS;

// Table: a thread owns pair i and walks ROWS positions; its frequency is
// evaluated once, in 64 bits like the angles (an FP32 product of position and
// frequency would be off by 0.03 rad at position 10^6).  Bound by the sine and cosine
// in 64 bits: 262,144 positions x 64 take 572 us (writing them: 10 us), once a program.
constexpr int TABLE_ROWS = 16;

__global__ void __launch_bounds__(NT) table_kernel(const RotaryTableParams p) {
    dependent_prologue();
    const long long idx = (long long)blockIdx.x * NT + threadIdx.x;
    const int i = (int)(idx % p.pairs);
    const long long row0 = idx / p.pairs * TABLE_ROWS;
    if (row0 >= p.P) return;
    double w = pow(p.base, -(double)i / (double)p.pairs);
    if (p.scaling == GDN_ROPE_LINEAR) {
        w *= p.inv_factor;
    } else if (p.scaling == GDN_ROPE_BY_PARTS) {
        const double keep = fmin(fmax((p.turns_per_freq * w - p.ramp_lo) / (p.ramp_hi - p.ramp_lo), 0.0), 1.0);
        w *= keep + (1.0 - keep) * p.inv_factor;
    } else if (p.scaling == GDN_ROPE_YARN) {
        const double keep = 1.0 - fmin(fmax(((double)i - p.ramp_lo) / (p.ramp_hi - p.ramp_lo), 0.0), 1.0);
        w *= keep + (1.0 - keep) * p.inv_factor;
    }
    const long long end = min((long long)p.P, row0 + TABLE_ROWS);
    for (long long r = row0; r < end; ++r) {
        double s, c;
        sincos((double)r * w, &s, &c);
        float *row = p.table + r * 2 * p.pairs;
        row[i] = (float)(c * p.magnitude);
        row[p.pairs + i] = (float)(s * p.magnitude);
    }
}

// grid.x: (token, item) in flat order; grid.y: groups of HEADS heads (q's, then k's).
template <typename T, int HEADS>
__global__ void __launch_bounds__(NT) rotary_kernel(const RotaryParams p) {
    dependent_prologue();
    constexpr int N = Vec16<T>::N;
    const int items = p.d / (2 * N);
    const long long idx = (long long)blockIdx.x * NT + threadIdx.x;
    const long long t = idx / items;
    const int item = (int)(idx - t * items);
    if (t >= p.T) return;
    const int pos = p.pos[t];
    if (pos < 0 || pos >= p.P) {
        if (item == 0 && blockIdx.y == 0) flag_error(p.status, GDN_DEVERR_POSITION);
        return;
    }
    const bool turned = item * 2 * N < p.rot;
    int c1, c2;
    item_channels<N>(item, p.rot, p.interleaved != 0, c1, c2);
    const int h0 = blockIdx.y * HEADS;
    Vec16<T> x1[HEADS], x2[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        const int h = h0 + j;
        if (h >= p.Hq + p.Hk) break;
        const T *src = h < p.Hq ? static_cast<const T *>(p.q) + t * p.q_stride + (long long)h * p.d
                                : static_cast<const T *>(p.k) + t * p.k_stride + (long long)(h - p.Hq) * p.d;
        x1[j].load(src + c1);
        x2[j].load(src + c2);
    }
    float c[N], s[N];
    if (turned) {
        const float *row = p.table + (long long)pos * p.rot + item * N;
        load_floats<N>(row, c);
        load_floats<N>(row + p.rot / 2, s);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] *= p.sign;
    }
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        const int h = h0 + j;
        if (h >= p.Hq + p.Hk) break;
        T *dst = h < p.Hq ? static_cast<T *>(p.q_out) + t * p.qo_stride + (long long)h * p.d
                          : static_cast<T *>(p.k_out) + t * p.ko_stride + (long long)(h - p.Hq) * p.d;
        if (turned) {
            float f1[N], f2[N];
            x1[j].to(f1);
            x2[j].to(f2);
            turn_groups<N>(f1, f2, c, s, p.interleaved != 0);
            x1[j].from(f1);
            x2[j].from(f2);
        }
        x1[j].store(dst + c1);
        x2[j].store(dst + c2);
    }
}

// Any even sizes and any alignment: a thread per channel pair.
template <typename T>
__global__ void __launch_bounds__(NT) rotary_pair_kernel(const RotaryParams p) {
    dependent_prologue();
    const int pairs = p.d / 2, H = p.Hq + p.Hk;
    const long long idx = (long long)blockIdx.x * NT + threadIdx.x;
    if (idx >= (long long)p.T * H * pairs) return;
    const int i = (int)(idx % pairs);
    const int h = (int)(idx / pairs % H);
    const long long t = idx / pairs / H;
    const int pos = p.pos[t];
    if (pos < 0 || pos >= p.P) {
        if (i == 0 && h == 0) flag_error(p.status, GDN_DEVERR_POSITION);
        return;
    }
    const T *src = h < p.Hq ? static_cast<const T *>(p.q) + t * p.q_stride + (long long)h * p.d
                            : static_cast<const T *>(p.k) + t * p.k_stride + (long long)(h - p.Hq) * p.d;
    T *dst = h < p.Hq ? static_cast<T *>(p.q_out) + t * p.qo_stride + (long long)h * p.d
                      : static_cast<T *>(p.k_out) + t * p.ko_stride + (long long)(h - p.Hq) * p.d;
    const bool turned = 2 * i < p.rot;
    const int c1 = turned && !p.interleaved ? i : 2 * i;
    const int c2 = turned && !p.interleaved ? i + p.rot / 2 : 2 * i + 1;
    const T a = src[c1], b = src[c2];
    if (turned) {
        const float *row = p.table + (long long)pos * p.rot;
        float ya, yb;
        turn(to_f32(a), to_f32(b), row[i], p.sign * row[p.rot / 2 + i], ya, yb);
        dst[c1] = from_f32<T>(ya);
        dst[c2] = from_f32<T>(yb);
    } else {
        dst[c1] = a;
        dst[c2] = b;
    }
}

bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

template <typename T>
cudaError_t launch_typed(const RotaryParams &p, cudaStream_t stream) {
    constexpr int N = Vec16<T>::N;
    const int H = p.Hq + p.Hk;
    const long long strides = (p.Hq ? p.q_stride | p.qo_stride : 0) | (p.Hk ? p.k_stride | p.ko_stride : 0);
    const bool vec = p.d % (2 * N) == 0 && p.rot % (2 * N) == 0 && strides % N == 0 && aligned16(p.q) &&
                     aligned16(p.k) && aligned16(p.q_out) && aligned16(p.k_out) && aligned16(p.table);
    if (!vec) {
        const long long n = (long long)p.T * H * (p.d / 2);
        return launch_dependent(rotary_pair_kernel<T>, dim3((unsigned)((n + NT - 1) / NT)), dim3(NT), 0, stream, p);
    }
    const long long n = (long long)p.T * (p.d / (2 * N));
    const unsigned gx = (unsigned)((n + NT - 1) / NT);
    // four heads a thread once that still fills the GPU's threads
    if (n * H >= 4LL * 2048 * current_device_sms())
        return launch_dependent(rotary_kernel<T, 4>, dim3(gx, (unsigned)((H + 3) / 4)), dim3(NT), 0, stream, p);
    return launch_dependent(rotary_kernel<T, 1>, dim3(gx, (unsigned)H), dim3(NT), 0, stream, p);
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryTableParams &p, cudaStream_t stream) {
    if (p.P == 0) return cudaSuccess;
    const long long n = ((long long)p.P + TABLE_ROWS - 1) / TABLE_ROWS * p.pairs;
    return launch_dependent(table_kernel, dim3((unsigned)((n + NT - 1) / NT)), dim3(NT), 0, stream, p);
}

cudaError_t launch_rotary(const RotaryParams &p, int io_dtype, cudaStream_t stream) {
    if (p.T == 0 || p.Hq + p.Hk == 0) return cudaSuccess;
    switch (io_dtype) {
        case GDN_F16: return launch_typed<__half>(p, stream);
        case GDN_BF16: return launch_typed<__nv_bfloat16>(p, stream);
        default: return launch_typed<float>(p, stream);
    }
}

}  // namespace gdn
