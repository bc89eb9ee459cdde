// Attention of new tokens over a paged key-value cache.
//
//   o = sum_t softmax_t(scale q k_t) v_t
//
// Every cached row is read once and used for the few query rows of its head
// (G = query heads per key head, times the new tokens), 2 G flops a byte at 16
// bits, so the kernel is bound by HBM and everything below serves to keep the
// memory pipe full: the products run on warp-level tensor instructions, whose
// rate is several times what the stream needs; 128-row tcgen05 tiles would be
// nearly all padding at 1 to 64 query rows.
//
// Transposed products.  With cached tokens (then value channels) as the M = 16
// side of the instruction and query rows as its N = 8 side,
//   S^T = K Q^T,   O^T = V^T P^T,
// eight query rows cost no padding (as the M side they would pad to 16), and
// the running maximum and sum of a query row live in the lanes that hold its
// column of both S^T and O^T.  P^T changes from accumulator to operand layout
// with one 8 x 8 register transpose per 8 tokens.
//
// No layout work on the cache.  The order of channels along a contraction and
// of channels among the output rows is free as long as both operands agree, so
// a lane's 16 consecutive bytes of a key row serve as its k-slots of two
// (8-bit: four) instructions, and 16 consecutive bytes of a value row as its
// rows of four (eight).  Each lane therefore consumes exactly the 16-byte
// pieces that it copied itself: a warp's ring of cp.async slots is a private
// FIFO per lane, with no barrier, no bank conflict and no swizzle, and each
// of the CTA's warps streams on its own (tiles of 16 or 32 tokens).
//
// Work split.  The lengths are on the device, so the split is made there: all
// (sequence, key head, group of query rows) units are cut into chunks of
// W tiles, laid end to end, and CTA c of G takes chunks [c total / G, (c + 1)
// total / G).  A unit that spans several CTAs leaves unnormalised partial
// results with their maxima and sums, and the last of its CTAs to finish joins
// them in CTA order.  Copies run ahead across unit boundaries.
//
// Numerics.  Scores, maxima, sums and outputs are FP32.  The weights P are
// 32-bit numbers that go to the tensor cores as two 16-bit parts (hi + lo, about
// 22 bits for FP16 values and 16 for BF16), which leaves the rounding of the
// result as the only one that matters; the memory-bound stream hides the
// second product.  FP32 caches use three TF32 products for each (hi hi, hi lo,
// lo hi).  The running maximum is only raised when a score exceeds it by more
// than 2^8 (the exponent headroom of the weights), so most tiles need no
// reduction across lanes and no rescaling.  8-bit rows: key scales multiply
// scores and value scales multiply weights, so the maximum is taken over
// score + log2(value scale); query rows are scaled to [1, 2) by a power of
// two, because 8-bit caches use FP16 products whatever the I/O type.
#pragma once

#include "attn_internal.cuh"
#include "ptx.cuh"

namespace gdn {
namespace attn {

// ---------------------------------------------------------------- instructions

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int src_bytes) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(src_bytes)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int N>  // N 32-bit words (1, 2 or 4)
__device__ __forceinline__ void lds(uint32_t (&w)[N], uint32_t addr) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 8 x 8 matrix of 16-bit values, one packed pair a lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// x = hi + lo with hi a TF32 number (10 fraction bits kept).  A non-finite x stays in hi alone.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = x & 0xffffe000u;
    const float l = __uint_as_float(x) - __uint_as_float(hi);
    lo = (x & 0x7f800000u) == 0x7f800000u ? 0u : __float_as_uint(l);
    if ((x & 0x7f800000u) == 0x7f800000u) hi = x;
}
// D += A B for FP32 operands
__device__ __forceinline__ void mma_f32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&bh)[2],
                                        const uint32_t (&bl)[2]) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
    mma_tf32(d, al, bh);
    mma_tf32(d, ah, bl);
    mma_tf32(d, ah, bh);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Four 8-bit values of a word as two FP16 pairs (bytes 0, 1 and bytes 2, 3), exactly.
template <int CT>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &p01, uint32_t &p23) {
    if constexpr (CT == GDN_FP8_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(p01), "=r"(p23)
            : "r"(w));
    } else {
        // 0x64xx is 1024 + xx: the biased byte x + 128 below that exponent, less 1152
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
        const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
        p01 = *reinterpret_cast<const uint32_t *>(&x);
        p23 = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// Whether a 32-bit word of cache elements holds an infinity or NaN.
template <int CT>
__device__ __forceinline__ bool non_finite(uint32_t w) {
    if constexpr (CT == GDN_F32) return (w & 0x7f800000u) == 0x7f800000u;
    if constexpr (CT == GDN_F16) return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
    if constexpr (CT == GDN_BF16) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    if constexpr (CT == GDN_FP8_E4M3)
        return (w & 0x7fu) == 0x7fu || (w & 0x7f00u) == 0x7f00u || (w & 0x7f0000u) == 0x7f0000u ||
               (w & 0x7f000000u) == 0x7f000000u;
    return false;
}

// ---------------------------------------------------------------- configuration

constexpr int SMEM_LIMIT = 232448;
constexpr int ITEMS = 64;          // output channels joined at a time
constexpr int BUF_ROW = ITEMS + 4;  // floats a row of the join buffer

template <int CT, int D_, int NT_>
struct Cfg {
    static constexpr int D = D_, NT = NT_, ROWS = 8 * NT;
    static constexpr bool F32 = CT == GDN_F32, BF16 = CT == GDN_BF16;
    static constexpr bool Q8 = CT == GDN_FP8_E4M3 || CT == GDN_INT8;
    static constexpr int ESZ = F32 ? 4 : Q8 ? 1 : 2;
    static constexpr int RB = D * ESZ;                  // bytes a cache row
    static constexpr int CHK = RB / 4 < 16 ? RB / 4 : 16;  // a lane's piece of a key row
    static constexpr int CHV = RB / 8 < 16 ? RB / 8 : 16;  // and of a value row
    static constexpr int KB = RB / (4 * CHK), VB = RB / (8 * CHV);  // pieces a row and lane
    static constexpr int CPL = CHV / ESZ;               // channels of a value piece
    static constexpr int MT = D / 16;                   // 16-channel output tiles
    static constexpr int MPV = MT / VB;                 // of them per value piece (CPL / 2)
    static constexpr int TS = 32 * RB <= 4096 ? 2 : 1;  // 16-token subtiles a tile
    static constexpr int TT = 16 * TS;
    static constexpr int SLOT = TT * RB + (Q8 ? TT * 8 : 0);  // half a tile (its keys or its values), scales after the rows
    static constexpr int join_bytes(int w) { return w * ROWS * BUF_ROW * 4; }
    static constexpr int ml_bytes(int w) { return 2 * (w + 1) * ROWS * 2 * 4; }
    static constexpr int slots(int w) { return (SMEM_LIMIT - 1024 - join_bytes(w) - ml_bytes(w)) / (w * SLOT); }
    static constexpr int W = slots(8) >= 3 ? 8 : 4;     // warps
    static constexpr int S = slots(W) < 8 ? slots(W) : 8;  // ring slots a warp
    static constexpr int SMEM = 1024 + join_bytes(W) + ml_bytes(W) + W * S * SLOT;
    static constexpr int QR = F32 ? D / 4 : D / 8;      // query registers per 8 rows
    static constexpr int THREADS = 32 * W;
    static constexpr float BIAS = CT == GDN_F16 || Q8 ? 6.f : -8.f;  // weights are 2^(s - m + BIAS)
    static constexpr float HEADROOM = 8.f;  // a score may exceed the maximum by this: FP16 weights stay below 2^14
    static_assert(S >= 2, "a ring needs two slots");
};

// One sequence as the kernel sees it.
struct Seq {
    int b, len, n, cu0;
    int first;  // first cache position any query sees
    int t0;     // `first` rounded down to a tile
    int tiles, chunks, row_groups, units;
};

template <class C>
__device__ __forceinline__ Seq load_seq(const PagedAttnParams &p, int b, bool flag) {
    Seq s;
    s.b = b;
    s.len = p.kv_lens[b];
    s.cu0 = p.cu ? p.cu[b] : b;
    const int cu1 = p.cu ? p.cu[b + 1] : b + 1;
    s.n = cu1 - s.cu0;
    const bool bad_cu = s.cu0 < 0 || s.n < 0 || cu1 > p.T || (b == 0 && s.cu0 != 0);
    const bool bad_len = s.len < 0 || (long long)s.len > (long long)p.pages_per_seq * p.c.page_size;
    if (flag && bad_cu) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    if (flag && bad_len) flag_error(p.status, GDN_DEVERR_KV_LEN);
    if (bad_cu || bad_len) s.n = 0;
    s.first = p.window > 0 ? max(0, s.len - s.n - p.window + 1) : 0;
    s.t0 = s.first / C::TT * C::TT;
    s.tiles = s.len > s.t0 ? (s.len - s.t0 - 1) / C::TT + 1 : 0;
    s.chunks = s.tiles > 0 ? (s.tiles - 1) / C::W + 1 : 1;
    s.row_groups = (int)(((long long)s.n * p.G + C::ROWS - 1) / C::ROWS);
    s.units = p.c.H * s.row_groups;
    return s;
}

// A walk over a CTA's chunks, one segment (part of one unit) at a time.
struct Walk {
    Seq s;
    int unit, chunk;     // the current segment's unit and first chunk
    int seg_chunks;
    long long left;      // chunks of this CTA not yet behind the walk, this segment's included
    int tile, tile_end;  // the warp's next tile and the segment's end
};

template <class C>
__device__ __forceinline__ void open_segment(Walk &w, int warp) {
    w.seg_chunks = (int)min((long long)(w.s.chunks - w.chunk), w.left);
    w.tile = w.chunk * C::W + warp;
    w.tile_end = min((w.chunk + w.seg_chunks) * C::W, w.s.tiles);
}

template <class C>
__device__ __forceinline__ void next_segment(Walk &w, const PagedAttnParams &p, int warp) {
    w.left -= w.seg_chunks;
    if (w.left <= 0) return;
    w.chunk = 0;
    if (++w.unit == w.s.units) {
        int b = w.s.b;
        do {
            if (++b >= p.B) {  // (not reached: the chunks were counted from the same lengths)
                w.left = 0;
                return;
            }
            w.s = load_seq<C>(p, b, false);
        } while (w.s.units == 0);
        w.unit = 0;
    }
    open_segment<C>(w, warp);
}

// ---------------------------------------------------------------- the kernel

// Refills the ring slot that was just used: S copies are always in flight or
// waiting, keys and values in turn, so the next copy is of the kind just used
// when S is even and of the other kind when it is odd.
template <int S, class K, class V>
__device__ __forceinline__ void refill(K &issue_k, V &issue_v, bool used_k) {
    if (used_k == (S % 2 == 0)) issue_k();
    else issue_v();
}

template <int CT, class C>
__global__ void __launch_bounds__(C::THREADS, 1) paged_attention_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int NT = C::NT, ROWS = C::ROWS, D = C::D, TS = C::TS, TT = C::TT, W = C::W, S = C::S;
    constexpr int KB = C::KB, VB = C::VB, MT = C::MT, MPV = C::MPV, QR = C::QR;
    constexpr bool Q8 = C::Q8, F32 = C::F32, BF16 = C::BF16;
    constexpr uint32_t FULL = 0xffffffffu;
    const float NEG_INF = __int_as_float(0xff800000);

    extern __shared__ __align__(1024) uint8_t smem[];
    long long *scan = reinterpret_cast<long long *>(smem);             // [W] warp sums
    int *found = reinterpret_cast<int *>(smem + 512);                  // sequence, then the last-CTA flag
    long long *found_off = reinterpret_cast<long long *>(smem + 528);  // chunk offset in that sequence
    float *buf = reinterpret_cast<float *>(smem + 1024);               // [W][ROWS][BUF_ROW]
    float2 *ml = reinterpret_cast<float2 *>(smem + 1024 + C::join_bytes(W));  // [2][W + 1][ROWS]; row W: joined
    uint8_t *ring = smem + 1024 + C::join_bytes(W) + C::ml_bytes(W);

    dependent_prologue();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

    // ---- this CTA's share of the chunks
    long long total, start;
    {
        const int per = (p.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = load_seq<C>(p, b, blockIdx.x == 0);
            sum += (long long)s.units * s.chunks;
        }
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < warp) before += scan[i];
            total += scan[i];
        }
        const long long ctas = min((long long)gridDim.x, total);
        if ((long long)blockIdx.x >= ctas) return;
        start = total * blockIdx.x / ctas;
        long long excl = before + incl - sum;
        if (start >= excl && start < excl + sum) {
            for (int b = b0;; ++b) {
                const Seq s = load_seq<C>(p, b, false);
                const long long here = (long long)s.units * s.chunks;
                if (start < excl + here) {
                    *found = b;
                    *found_off = start - excl;
                    break;
                }
                excl += here;
            }
        }
        __syncthreads();
    }
    const long long ctas = min((long long)gridDim.x, total);  // those with work
    Walk use;  // what the products are at
    use.s = load_seq<C>(p, *found, false);
    use.unit = (int)(*found_off / use.s.chunks);
    use.chunk = (int)(*found_off - (long long)use.unit * use.s.chunks);
    use.left = total * (blockIdx.x + 1) / ctas - start;
    open_segment<C>(use, warp);
    Walk get = use;  // what the copies are at, some tiles ahead

    // ---- copies
    const uint32_t ring0 = ptx::smem_u32(ring) + warp * (S * C::SLOT);
    const uint8_t *kbase = static_cast<const uint8_t *>(p.c.k), *vbase = static_cast<const uint8_t *>(p.c.v);
    bool wanted = false;         // whether this lane's token of the tile at `get` is read at all
    int page = 0, in_page = 0;   // where it is
    long long row = -1;          // its byte offset in the cache (head included), -1: not read
    uint32_t put = 0, take = 0;  // ring positions in bytes

    auto look_up = [&]() {  // one tile ahead of its use, so that the table's latency is hidden
        while (get.left > 0 && get.tile >= get.tile_end) next_segment<C>(get, p, warp);
        wanted = false;
        if (get.left > 0) {
            const int t = get.s.t0 + get.tile * TT + (lane & (TT - 1));
            if (t >= get.s.first && t < get.s.len) {
                const int i = t / p.c.page_size;
                in_page = t - i * p.c.page_size;
                page = p.block_table[get.s.b * p.bt_stride + i];
                wanted = true;
            }
        }
    };
    auto issue_k = [&]() {
        if (get.left > 0) {
            row = -1;
            const int head = get.unit / get.s.row_groups;
            if (wanted) {
                if (page >= 0 && page < p.c.num_pages)
                    row = (page * p.c.page_stride + in_page * p.c.token_stride + head * p.c.head_stride) * C::ESZ;
                else
                    flag_error(p.status, GDN_DEVERR_PAGE);
            }
            const uint32_t dst = ring0 + put + lane * C::CHK;
#pragma unroll
            for (int r = 0; r < 2 * TS; ++r) {
                const long long o = __shfl_sync(FULL, row, r * 8 + g);
                const uint8_t *src = kbase + (o < 0 ? 0 : o) + c * C::CHK;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
                    copy_async<C::CHK>(dst + (r * KB + kb) * 32 * C::CHK, src + kb * 4 * C::CHK, o < 0 ? 0 : C::CHK);
            }
            if constexpr (Q8) {
                // lanes' tokens: TS == 2 one each, TS == 1 lanes 0-15 fetch key scales and 16-31 value scales
                const long long so = row < 0 ? 0
                                             : page * p.c.s_page_stride + in_page * p.c.s_token_stride +
                                                   head * p.c.s_head_stride;
                const uint32_t sdst = ring0 + put + TT * C::RB;
                const int bytes = row < 0 ? 0 : 4;
                if constexpr (TS == 2) {
                    copy_async<4>(sdst + lane * 4, p.c.k_scale + so, bytes);
                    copy_async<4>(sdst + 128 + lane * 4, p.c.v_scale + so, bytes);
                } else {
                    copy_async<4>(sdst + lane * 4, (lane < 16 ? p.c.k_scale : p.c.v_scale) + so, bytes);
                }
            }
        }
        copy_commit();
        put = put + C::SLOT == S * C::SLOT ? 0 : put + C::SLOT;
    };
    auto issue_v = [&]() {
        if (get.left > 0) {
            const uint32_t dst = ring0 + put + lane * C::CHV;
#pragma unroll
            for (int r = 0; r < 4 * TS; ++r) {
                const int tk = r & 3;
                const int token = (r >> 2) * 16 + (F32 ? c + 4 * tk : 2 * c + (tk & 1) + 8 * (tk >> 1));
                const long long o = __shfl_sync(FULL, row, token);
                const uint8_t *src = vbase + (o < 0 ? 0 : o) + g * C::CHV;
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
                    copy_async<C::CHV>(dst + (r * VB + vb) * 32 * C::CHV, src + vb * 8 * C::CHV, o < 0 ? 0 : C::CHV);
            }
            get.tile += W;
            look_up();
        }
        copy_commit();
        put = put + C::SLOT == S * C::SLOT ? 0 : put + C::SLOT;
    };
    look_up();
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (i % 2 == 0) issue_k();
        else issue_v();
    }

    // ---- one segment after another
    int parity = 0;
    while (true) {
        const int head = use.unit / use.s.row_groups;
        const int row0 = (use.unit - head * use.s.row_groups) * ROWS;   // first query row of the unit
        const int rows = min(ROWS, use.s.n * p.G - row0);               // query rows it has
        const int pos0 = use.s.len - use.s.n;                           // the first query's position

        // queries: lane (g, c) holds, of row 8 nt + g, the channels that its key pieces have
        uint32_t q[NT][QR];
        float col_scale[NT][2];  // scores' factor of the lane's two columns
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g;
            const int i = (row0 + r) / p.G, hq = (row0 + r) - i * p.G;
            const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                                 ((long long)(use.s.cu0 + i) * p.q_stride + ((long long)head * p.G + hq) * D) * (F32 ? 4 : 2);
            const bool real = r < rows;
            if constexpr (Q8) {
                // 16 channels a piece; scaled so that the row's largest magnitude is in [1, 2)
                uint32_t raw[KB][8];
                float top = 0.f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const uint4 *s4 = reinterpret_cast<const uint4 *>(src + (kb * 4 + c) * 32);
                    const uint4 x = real ? s4[0] : make_uint4(0, 0, 0, 0), y = real ? s4[1] : make_uint4(0, 0, 0, 0);
                    raw[kb][0] = x.x, raw[kb][1] = x.y, raw[kb][2] = x.z, raw[kb][3] = x.w;
                    raw[kb][4] = y.x, raw[kb][5] = y.y, raw[kb][6] = y.z, raw[kb][7] = y.w;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = p.io_bf16 ? unpack2<true>(raw[kb][j]) : unpack2<false>(raw[kb][j]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                // the exponent of top, kept in a range where both powers of two are normal
                int e = ((__float_as_uint(top) >> 23) & 255) - 127;
                e = top > 0.f && top <= 3.402823466e38f ? max(e, -100) : 0;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = p.io_bf16 ? unpack2<true>(raw[kb][j]) : unpack2<false>(raw[kb][j]);
                        q[nt][kb * 8 + j] = pack2<false>(f.x * down, f.y * down);
                    }
                col_scale[nt][0] = p.scale_log2 * __shfl_sync(FULL, up, 8 * c);
                col_scale[nt][1] = p.scale_log2 * __shfl_sync(FULL, up, 8 * c + 4);
            } else {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const uint4 x = real ? *reinterpret_cast<const uint4 *>(src + (kb * 4 + c) * 16) : make_uint4(0, 0, 0, 0);
                    q[nt][kb * 4] = x.x, q[nt][kb * 4 + 1] = x.y, q[nt][kb * 4 + 2] = x.z, q[nt][kb * 4 + 3] = x.w;
                }
                col_scale[nt][0] = col_scale[nt][1] = p.scale_log2;
            }
        }
        // positions that every query row of the unit sees: [all_lo, all_hi)
        const int all_hi = pos0 + row0 / p.G + 1;
        const int all_lo = p.window > 0 ? max(0, pos0 + (row0 + rows - 1) / p.G - p.window + 1) : 0;
        auto seen = [&](int r, int t) {  // whether row r of the unit sees position t
            const int pos = pos0 + (row0 + min(r, rows - 1)) / p.G;
            return t <= pos && (p.window == 0 || t > pos - p.window);
        };

        float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = NEG_INF;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
        }

        for (; use.tile < use.tile_end; use.tile += W) {
            const int tile_t = use.s.t0 + use.tile * TT;
            const bool edge = tile_t < all_lo || tile_t + TT > all_hi;

            // ---- scores: S^T = K Q^T
            copy_wait<S - 1>();
            float sc[TS][NT][4], sc2[TS][NT][4];
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[ts][nt][e] = sc2[ts][nt][e] = 0.f;
            const uint32_t ks = ring0 + take + lane * C::CHK;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int ts = 0; ts < TS; ++ts) {
                    uint32_t x[4], y[4];
                    lds<4>(x, ks + ((2 * ts) * KB + kb) * 32 * C::CHK);
                    lds<4>(y, ks + ((2 * ts + 1) * KB + kb) * 32 * C::CHK);
                    if constexpr (Q8) {
                        uint32_t u[8], v[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            widen<CT>(x[j], u[2 * j], u[2 * j + 1]);
                            widen<CT>(y[j], v[2 * j], v[2 * j + 1]);
                        }
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16<false>((j & 2) ? sc2[ts][nt] : sc[ts][nt], u[j], v[j], u[j + 1], v[j + 1],
                                             q[nt][kb * 8 + j], q[nt][kb * 8 + j + 1]);
                    } else if constexpr (F32) {
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const uint32_t a[4] = {x[j], y[j], x[j + 1], y[j + 1]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t bh[2], bl[2];
                                split_tf32(q[nt][kb * 4 + j], bh[0], bl[0]);
                                split_tf32(q[nt][kb * 4 + j + 1], bh[1], bl[1]);
                                mma_f32(j ? sc2[ts][nt] : sc[ts][nt], a, bh, bl);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j += 2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16<BF16>(j ? sc2[ts][nt] : sc[ts][nt], x[j], y[j], x[j + 1], y[j + 1],
                                            q[nt][kb * 4 + j], q[nt][kb * 4 + j + 1]);
                    }
                }
            // the lane's tokens are rows g and g + 8 of each subtile
            float vs[TS][2], lv[TS][2], ksc[TS][2];
            if constexpr (Q8) {
                __syncwarp();  // the scales were copied by other lanes
                const float *kscale = reinterpret_cast<const float *>(ring + warp * (S * C::SLOT) + take + TT * C::RB);
#pragma unroll
                for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = ts * 16 + g + 8 * e;
                        ksc[ts][e] = kscale[i];
                        vs[ts][e] = kscale[TT + i];
                        lv[ts][e] = log2_fast(fmaxf(fabsf(vs[ts][e]), 1e-30f));  // (rows of zeros may have scale 0)
                    }
                __syncwarp();
            }
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = NEG_INF;
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = (sc[ts][nt][e] + sc2[ts][nt][e]) * col_scale[nt][e & 1];
                        if constexpr (Q8) x *= ksc[ts][e >> 1];
                        if (edge && !seen(nt * 8 + 2 * c + (e & 1), tile_t + ts * 16 + g + 8 * (e >> 1))) x = NEG_INF;
                        sc[ts][nt][e] = x;
                        float y = x;
                        if constexpr (Q8) y = x == NEG_INF ? x : x + lv[ts][e >> 1];
                        top[nt][e & 1] = fmaxf(top[nt][e & 1], y);
                    }
            refill<S>(issue_k, issue_v, true);
            take = take + C::SLOT == S * C::SLOT ? 0 : take + C::SLOT;

            // ---- raise the maxima where a score exceeds them by more than the headroom
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                raise |= top[nt][0] > m[nt][0] + C::HEADROOM || top[nt][1] > m[nt][1] + C::HEADROOM;
            if (__any_sync(FULL, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[nt][e];
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
                        x = fmaxf(x, m[nt][e]);
                        const float f = x == m[nt][e] ? 1.f : exp2_fast(m[nt][e] - x);
                        m[nt][e] = x;
                        l[nt][e] *= f;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[nt][i][e] *= f;
                            o[nt][i][e + 2] *= f;
                        }
                    }
            }

            // ---- weights, and their operand layout
            uint32_t ph[TS][NT][2], pl[TS][NT][2];          // 16-bit parts
            uint32_t fh[TS][NT][2][2], fl[TS][NT][2][2];    // TF32 parts, two k-steps of 8 tokens
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float base = m[nt][e & 1] == NEG_INF ? 0.f : m[nt][e & 1] - C::BIAS;
                        const float x = exp2_fast(sc[ts][nt][e] - base);
                        l[nt][e & 1] += x;
                        if constexpr (Q8) w[e] = sc[ts][nt][e] == NEG_INF ? 0.f : x * vs[ts][e >> 1];
                        else w[e] = x;
                    }
                    if constexpr (F32) {
                        // token c (+4, +8, +12) of column g: from the lane that holds that token's row
                        const int src = c * 4 + (g >> 1);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float a = __shfl_sync(FULL, w[2 * k], src + 16 * j);
                                const float b = __shfl_sync(FULL, w[2 * k + 1], src + 16 * j);
                                split_tf32(__float_as_uint(g & 1 ? b : a), fh[ts][nt][k][j], fl[ts][nt][k][j]);
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t hi = pack2<BF16>(w[2 * k], w[2 * k + 1]);
                            const float2 back = unpack2<BF16>(hi);
                            const uint32_t lo = pack2<BF16>(w[2 * k] - back.x, w[2 * k + 1] - back.y);
                            ph[ts][nt][k] = transpose8x8(hi);
                            pl[ts][nt][k] = transpose8x8(lo);
                        }
                    }
                }

            // ---- O^T += V^T P^T
            copy_wait<S - 1>();
            const uint32_t vsm = ring0 + take + lane * C::CHV;
            constexpr int VW = C::CHV / 4;  // words of a value piece
            // `only`: -1, or the single query row to add, with values that it does not see left out
            auto add_values = [&](int only) {
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                    for (int ts = 0; ts < TS; ++ts) {
                        uint32_t v[4][VW];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            lds<VW>(v[k], vsm + ((ts * 4 + k) * VB + vb) * 32 * C::CHV);
                            if (only >= 0) {
                                const int t = tile_t + ts * 16 + (F32 ? c + 4 * k : 2 * c + (k & 1) + 8 * (k >> 1));
                                if (!seen(only, t)) {
#pragma unroll
                                    for (int j = 0; j < VW; ++j) v[k][j] = 0u;
                                }
                            }
                        }
                        auto mine = [&](uint32_t x, int nt) { return only < 0 || only == nt * 8 + g ? x : 0u; };
                        if constexpr (F32) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int j = 0; j < VW; j += 2) {
                                    const uint32_t a[4] = {v[2 * k][j], v[2 * k][j + 1], v[2 * k + 1][j], v[2 * k + 1][j + 1]};
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        const uint32_t bh[2] = {mine(fh[ts][nt][k][0], nt), mine(fh[ts][nt][k][1], nt)};
                                        const uint32_t bl[2] = {mine(fl[ts][nt][k][0], nt), mine(fl[ts][nt][k][1], nt)};
                                        mma_f32(o[nt][vb * MPV + j / 2], a, bh, bl);
                                    }
                                }
                        } else {
                            uint32_t a[MPV][4];
#pragma unroll
                            for (int j = 0; j < VW; ++j) {
                                if constexpr (Q8) {
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        const uint32_t lo = __byte_perm(v[2 * k][j], v[2 * k + 1][j], 0x5140);
                                        const uint32_t hi = __byte_perm(v[2 * k][j], v[2 * k + 1][j], 0x7362);
                                        widen<CT>(lo, a[2 * j][2 * k], a[2 * j][2 * k + 1]);
                                        widen<CT>(hi, a[2 * j + 1][2 * k], a[2 * j + 1][2 * k + 1]);
                                    }
                                } else {
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        a[j][2 * k] = __byte_perm(v[2 * k][j], v[2 * k + 1][j], 0x5410);
                                        a[j][2 * k + 1] = __byte_perm(v[2 * k][j], v[2 * k + 1][j], 0x7632);
                                    }
                                }
                            }
#pragma unroll
                            for (int j = 0; j < MPV; ++j)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma16<BF16>(o[nt][vb * MPV + j], a[j][0], a[j][1], a[j][2], a[j][3],
                                                mine(pl[ts][nt][0], nt), mine(pl[ts][nt][1], nt));
                                    mma16<BF16>(o[nt][vb * MPV + j], a[j][0], a[j][1], a[j][2], a[j][3],
                                                mine(ph[ts][nt][0], nt), mine(ph[ts][nt][1], nt));
                                }
                        }
                    }
            };
            // A value that some rows of the tile see and others do not would reach the others as
            // 0 * inf if it is not finite: such a tile is added row by row.
            bool rough = false;
            if (CT != GDN_INT8 && edge && use.s.n > 1) {
                uint32_t x[VW];
                for (int i = 0; i < 4 * TS * VB; ++i) {
                    lds<VW>(x, vsm + i * 32 * C::CHV);
#pragma unroll
                    for (int j = 0; j < VW; ++j) rough |= non_finite<CT>(x[j]);
                }
                rough = __any_sync(FULL, rough);
            }
            if (rough) {
                for (int r = 0; r < rows; ++r) add_values(r);
            } else {
                add_values(-1);
            }
            refill<S>(issue_k, issue_v, false);
            take = take + C::SLOT == S * C::SLOT ? 0 : take + C::SLOT;
        }

        // ---- join the warps
        float2 *mlp = ml + parity * (W + 1) * ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(FULL, x, 4);
                x += __shfl_xor_sync(FULL, x, 8);
                x += __shfl_xor_sync(FULL, x, 16);
                if (g == 0) mlp[warp * ROWS + nt * 8 + 2 * c + e] = make_float2(m[nt][e], x);
            }
        __syncthreads();
        // a part without a maximum has zeros (or the NaN that its scores are)
        auto part_factor = [&](float part, float all) { return part == NEG_INF ? 1.f : exp2_fast(part - all); };
        if (tid < ROWS) {
            float mm = NEG_INF, ll = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) mm = fmaxf(mm, mlp[w * ROWS + tid].x);
#pragma unroll
            for (int w = 0; w < W; ++w) ll += mlp[w * ROWS + tid].y * part_factor(mlp[w * ROWS + tid].x, mm);
            mlp[W * ROWS + tid] = make_float2(mm, ll);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mm = NEG_INF;
#pragma unroll
                for (int w = 0; w < W; ++w) mm = fmaxf(mm, mlp[w * ROWS + nt * 8 + 2 * c + e].x);
                const float f = part_factor(m[nt][e], mm);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[nt][i][e] *= f;
                    o[nt][i][e + 2] *= f;
                }
            }
        const bool whole = use.seg_chunks == use.s.chunks;
        // owner(x): the CTA whose share holds chunk x
        const long long unit0 = start + (total * (blockIdx.x + 1) / ctas - start - use.left) - use.chunk;  // the unit's first chunk
        const int c0 = (int)(((unit0 + 1) * ctas - 1) / total);
        const int c1 = (int)(((unit0 + use.s.chunks) * ctas - 1) / total);
        auto store_row = [&](int r, int ch, float4 x, float2 st) {  // joined, unnormalised
            const int i = (row0 + r) / p.G, hq = (row0 + r) - i * p.G;
            const long long token = use.s.cu0 + i;
            const bool any = pos0 + i >= 0;  // a query at a position before the cache sees nothing
            const float inv = any ? 1.f / st.y : 0.f;
            const long long at = (token * p.Hq + (long long)head * p.G + hq);
            const float y[4] = {any ? x.x * inv : 0.f, any ? x.y * inv : 0.f, any ? x.z * inv : 0.f, any ? x.w * inv : 0.f};
            if constexpr (F32) {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * D + ch) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
                const bool bf = BF16 || (Q8 && p.io_bf16);
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at * D + ch) =
                    bf ? make_uint2(pack2<true>(y[0], y[1]), pack2<true>(y[2], y[3]))
                       : make_uint2(pack2<false>(y[0], y[1]), pack2<false>(y[2], y[3]));
            }
            if (p.lse && ch == 0) p.lse[at] = any ? (st.x - C::BIAS + log2f(st.y)) * 0.6931471805599453f : NEG_INF;
        };
        const long long my_slot = 2LL * blockIdx.x + (blockIdx.x == c0 ? 1 : 0);
        float2 *part_ml = reinterpret_cast<float2 *>(p.partials);
        float *part_o = p.partials + 4LL * gridDim.x * ROWS;
#pragma unroll
        for (int ph_ = 0; ph_ < D / ITEMS; ++ph_) {
            if (ph_ > 0) __syncthreads();
            // four output tiles: 8 values a lane and row
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4 *dst = reinterpret_cast<float4 *>(buf + (warp * ROWS + nt * 8 + 2 * c + e) * BUF_ROW + g * 8);
                    const int i = ph_ * 4;
                    dst[0] = make_float4(o[nt][i][e], o[nt][i][e + 2], o[nt][i + 1][e], o[nt][i + 1][e + 2]);
                    dst[1] = make_float4(o[nt][i + 2][e], o[nt][i + 2][e + 2], o[nt][i + 3][e], o[nt][i + 3][e + 2]);
                }
            __syncthreads();
            for (int i = tid; i < rows * (ITEMS / 4); i += C::THREADS) {
                const int r = i / (ITEMS / 4), x4 = i % (ITEMS / 4);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(buf + (w * ROWS + r) * BUF_ROW + x4 * 4);
                    sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
                }
                // value 4 x4 of the phase: lane group x4 / 2, output tiles ph_ * 4 + (x4 & 1) * 2 and the next
                const int mt = ph_ * 4 + (x4 & 1) * 2;
                const int ch = (mt / MPV * 8 + x4 / 2) * C::CPL + 2 * (mt % MPV);
                if (whole) {
                    store_row(r, ch, sum, mlp[W * ROWS + r]);
                } else {
                    *reinterpret_cast<float4 *>(part_o + (my_slot * ROWS + r) * D + ch) = sum;
                    if (ch == 0) part_ml[my_slot * ROWS + r] = mlp[W * ROWS + r];
                }
            }
        }
        // ---- join the CTAs: the last one to arrive adds all parts, in CTA order
        if (!whole) {
            __threadfence();
            __syncthreads();
            const int parts = c1 - c0 + 1;
            if (tid == 0) *found = atomicAdd(&p.counters[c0], 1) == parts - 1;
            __syncthreads();
            if (*found) {
                __threadfence();
                float *fac = buf;  // [parts][ROWS]
                for (int r = warp; r < rows; r += W) {
                    float mm = NEG_INF, ll = 0.f;
                    for (int i = lane; i < parts; i += 32)
                        mm = fmaxf(mm, __ldcg(&part_ml[(2LL * (c0 + i) + (i == 0)) * ROWS + r]).x);
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(FULL, mm, s));
                    for (int i = lane; i < parts; i += 32) {
                        const float2 x = __ldcg(&part_ml[(2LL * (c0 + i) + (i == 0)) * ROWS + r]);
                        const float f = part_factor(x.x, mm);
                        fac[i * ROWS + r] = f;
                        ll += x.y * f;
                    }
                    ll = warp_sum(ll);
                    if (lane == 0) mlp[W * ROWS + r] = make_float2(mm, ll);
                }
                __syncthreads();
                for (int i = tid; i < rows * (D / 4); i += C::THREADS) {
                    const int r = i / (D / 4), ch = i % (D / 4) * 4;
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < parts; ++k) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(
                            part_o + ((2LL * (c0 + k) + (k == 0)) * ROWS + r) * D + ch));
                        const float f = fac[k * ROWS + r];
                        sum.x += f * x.x, sum.y += f * x.y, sum.z += f * x.z, sum.w += f * x.w;
                    }
                    store_row(r, ch, sum, mlp[W * ROWS + r]);
                }
                if (tid == 0) p.counters[c0] = 0;
                __syncthreads();
            }
        }
        parity ^= 1;
        next_segment<C>(use, p, warp);
        if (use.left <= 0) break;
    }
    copy_wait<0>();
}

template <int CT, int D, int NT>
cudaError_t launch_sized(const PagedAttnParams &p, cudaStream_t stream) {
    using C = Cfg<CT, D, NT>;
    auto kernel = paged_attention_kernel<CT, C>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3((unsigned)attention_ctas()), dim3(C::THREADS), C::SMEM, stream, p);
}

// Query rows a pass: as few groups of 8 as hold the rows of one key head
// (fewer idle columns), at most what the registers hold.
template <int CT, int D>
cudaError_t launch_dim(const PagedAttnParams &p, cudaStream_t stream) {
    constexpr int MAX = max_row_tiles(CT == GDN_F32, D);
    const int nt = row_tiles(CT == GDN_F32, D, p.rows_hint);
    if constexpr (MAX >= 4)
        if (nt == 4) return launch_sized<CT, D, 4>(p, stream);
    if constexpr (MAX >= 2)
        if (nt == 2) return launch_sized<CT, D, 2>(p, stream);
    return launch_sized<CT, D, 1>(p, stream);
}

}  // namespace attn

template <int CT>
cudaError_t launch_paged_attention(const PagedAttnParams &p, cudaStream_t stream) {
    switch (p.c.d) {
        case 64: return attn::launch_dim<CT, 64>(p, stream);
        case 128: return attn::launch_dim<CT, 128>(p, stream);
        default: return attn::launch_dim<CT, 256>(p, stream);
    }
}

}  // namespace gdn
