// Attention of new tokens over a paged key-value cache.
//
//   o = sum_t softmax_t(scale q k_t) v_t
//
// Every cached row is read once and used for the few query rows of its head
// (G = query heads per key head, times the new tokens), 2 G flops a byte at 16
// bits, so the kernel is bound by HBM and everything below serves to keep the
// memory pipe full: the products run on warp-level tensor instructions, whose
// rate is several times what the stream needs at 8 query rows a key head.  With
// more rows the consumers' instructions bound it (below).  tcgen05 tiles in the
// orientation used here, 128 cached tokens by 16 to 64 query rows, would have no
// padding and hold the outputs outside the registers; they are not built.
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
// rows of four (eight).  Tensor copies swizzle the rows so that these reads
// meet no bank twice.
//
// Roles.  A CTA per SM: W consumer warps multiply tiles of 16 or 32 tokens,
// each from its own ring of slots; producer warps keep the rings full, a slot
// at a time and ahead across the ends of sequences; joiner warps fetch the next
// segment's queries and add the consumers' parts of a finished one while these
// go on.  Consumers share nothing while they stream.  (When the consumers copied
// for themselves, each copy's ~700 cycles of issue stood between two tiles: draft
// verification ran 58.7 us instead of 52.5 us, many int8 requests 49 us instead of 42 us.)
//
// Work split.  The lengths are on the device, so the split is made there: all
// (sequence, key head, group of query rows) units are cut into chunks of W
// tiles, laid end to end, and dealt to the CTAs in equal runs.  A unit that
// spans several CTAs leaves unnormalised parts with their maxima and sums in
// the workspace, and a second kernel, a row to a CTA, joins them in order.
//
// Numerics.  Scores, maxima, sums and outputs are FP32.  The weights P of 16-bit
// values go to the tensor cores as two 16-bit parts (hi + lo, about 22 bits for
// FP16 values and 16 for BF16), which leaves the rounding of the result as the
// only one that matters; over 8-bit values they are single FP16 numbers.  FP32
// caches use three TF32 products for each (hi hi, hi lo, lo hi).  The running
// maximum is only raised when a score exceeds it by more than 2^8 (the exponent
// headroom of the weights), so most tiles need no reduction across lanes and no
// rescaling.  8-bit rows: key scales multiply scores and value scales multiply
// weights, so the maximum is taken over score + log2(value scale) (2^-80 for a row
// of zeros, whose scale says nothing); BF16 query
// rows are scaled to [1, 2) by a power of two as they are fetched, because 8-bit
// caches use FP16 products whatever the I/O type.
//
// Measured (one key head serves 4 query heads, heads of 128, FP16): 64 x 4096
// tokens 158-163 us, 6.6-6.8 TB/s (0.97 to 1.0 of a copy's rate); one context of 131071
// 82-84 us, 6.4-6.5 TB/s; a decode step of 64 x 128 to 2048, writes included, 54-55 us
// (5.3 TB/s); 64 e4m3 contexts of up to 16384, two heads of 256, 91 us (6.0 TB/s).
// Long streams are bound by HBM.  Short units are bound by the fixed work of a
// segment (about 1 us a CTA: queries, statistics, parts) and of a call (2.6 us to
// the first copy, 2.4 us for the join): 16 x 512 tokens 9.6 us.  16 query rows are
// bound by the consumers' instructions: draft verification (16 x 4 tokens of 8
// heads a key head, up to 8191) reads the cache twice and takes 45 us.  Prompts work, but
// each unit of 16 rows walks its sequence's whole cache: 4 x 512 tokens over 4096 cached, 32
// heads over 8, BF16, take 1.04 ms, 140 TFLOP/s (0.07 of the library's matrix rate).
#pragma once

#include "attn_internal.cuh"
#include "ptx.cuh"

namespace gdn {
namespace attn {

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// 4 bytes of a line that stays in L2 for its other readers.
__device__ __forceinline__ void copy_async4_kept(uint32_t dst, const void *src, int src_bytes, uint64_t policy) {
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 4, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ uint64_t keep_policy() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int N>  // N 32-bit words (2 or 4) of shared memory
__device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    }
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
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (BF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// x = hi + lo with hi rounded to TF32 (to nearest in magnitude, so that lo and
// the dropped lo lo products have no sign in common; in integers: with
// the convert instruction 8 x 4096 tokens of heads of 128 took 58.6 us instead of 49.1 us).  The tensor cores drop lo's bits
// past TF32, which leaves 21 bits.  From 0x7f7ff000 on (the largest numbers, infinities, NaN) hi is
// cut instead, since rounding would carry into the exponent or the sign; lo is then NaN for an x
// that is not finite, whatever the cut leaves of its bits.  (An infinity kept in hi alone would cost a compare and a
// select more, 60.6 us instead of 49.8 us, and meet the other operand's lo, whose sign is any, in its product.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
    const float f = __uint_as_float(x);
    hi = (fabsf(f) < __uint_as_float(0x7f7ff000u) ? x + 0x1000u : x) & 0xffffe000u;
    lo = __float_as_uint(f - __uint_as_float(hi));
}
// D += A B for FP32 operands.  The tensor cores cut what they add off at the bits of the largest
// addend, always towards zero, so a D should hold a few products only and be added to
// longer sums in FP32: 8 x 4099 tokens of heads of 64 had an error (by norm, against 64 bits) of 1.2e-6
// that way, and have 5.2e-7, where one product of 32 bits each has 3.6e-7.
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

// The same for keys, where int8 may stay biased: a byte x + 128 as the low half of an FP16
// number is the subnormal (x + 128) 2^-24, exactly.  The scores' bias of -128 2^-24 sum(q)
// and scale of 2^24 belong to it.  (1152 + x, as above, would lose four more bits of a score to its bias.)
template <int CT>
__device__ __forceinline__ void widen_keys(uint32_t w, uint32_t &p01, uint32_t &p23) {
    if constexpr (CT == GDN_INT8) {
        const uint32_t u = w ^ 0x80808080u;
        p01 = __byte_perm(u, 0u, 0x4140);
        p23 = __byte_perm(u, 0u, 0x4342);
    } else {
        widen<CT>(w, p01, p23);
    }
}

struct Yes { __device__ constexpr bool operator()() const { return true; } };
struct No { __device__ constexpr bool operator()() const { return false; } };

// Whether a 32-bit word of 16- or 32-bit cache elements holds an infinity or NaN.
template <int CT>
__device__ __forceinline__ bool non_finite(uint32_t w) {
    if constexpr (CT == GDN_F32) return (w & 0x7f800000u) == 0x7f800000u;
    if constexpr (CT == GDN_F16) return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
    if constexpr (CT == GDN_BF16) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    return false;
}
// A word of e4m3 values with zeros for its NaN (0x7f and 0xff).
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if ((w >> i & 0x7fu) == 0x7fu) w &= ~(0xffu << i);
    return w;
}

// ---------------------------------------------------------------- configuration

// One sequence as the kernel sees it.
struct Seq {
    int b, len, n, cu0;
    int first;  // first cache position any query sees
    int t0;     // `first` rounded down to a tile
    int tiles, chunks, row_groups, units;
};

// A walk over a CTA's chunks, one segment (part of one unit) at a time.
struct Walk {
    Seq s;
    int unit, pos;           // the current segment's unit and where in its share of the work it starts
    int chunk, seg_chunks;   // the segment's chunks
    int head, row0;          // the unit's key head and first query row
    int seg_work, left;      // the work of the segment, and of this CTA from there on
    int tile, tile_end;  // the segment's tiles
};

constexpr int SMEM_LIMIT = 232448;

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
    static constexpr int HALF = TT * RB;                // a tile's keys; its values
    static constexpr int SPAN = RB < 128 ? RB : 128;    // row bytes a tensor copy takes
    static constexpr int BOXES = RB / SPAN;             // spans a row; each half is [BOXES][TT][SPAN]
    // A ring slot holds a tile's keys and values or a consumer's part of a finished segment ([ROWS][D] floats); an
    // extra beside it the scales of 8-bit rows (keys, values), or the part's statistics.
    static constexpr int TILE = 2 * HALF, PART = ROWS * D * 4;
    static constexpr int SLOT = ((TILE > PART ? TILE : PART) + 1023) / 1024 * 1024;
    static constexpr int EXTRA = Q8 && TT > ROWS ? TT * 8 : ROWS * 8;
    // Row r's 16-byte piece x of a part is at x ^ part_swizzle(r): the lanes that store together (rows 2 c, pieces
    // CPL / 4 apart) then meet no bank twice.
    static __device__ __forceinline__ int part_swizzle(int r) {
        const int c = r >> 1 & 3;
        return CPL == 4 ? 2 * c : CPL == 8 ? (c & 1) | (c & 2) << 1 : c;
    }
    // Bytes a staged query row; the padding keeps the lanes' reads of 8 rows free of bank conflicts.
    static constexpr int QROW = D * (F32 ? 4 : 2) + (Q8 ? 16 : 64);
    static constexpr int QUERIES = 2 * ROWS * (QROW + 8);  // and each row's (scale, bias)
    static constexpr int HEAD = 2048;                    // scan, flags, barriers and segments
    // Warps: W consumers, NP producers and NJ joiners.  16 warps have 128 registers a thread, which they divide by
    // role (a consumer's outputs take HELD); where the outputs take more than 64, or the ring has no room for more, 8 have 255.
    static constexpr int HELD = NT * D / 4;
    static constexpr int FACTORS = 8 * ROWS * 4 + ROWS * 8;
    static constexpr int ROOM = (SMEM_LIMIT - 1024 - HEAD - QUERIES - FACTORS) / (SLOT + EXTRA);  // slots that fit
    static constexpr int W = HELD <= 64 && ROOM >= 16 ? 8 : ROOM >= 8 ? 4 : 3;
    static constexpr int NP = W == 8 ? 4 : W == 4 ? 2 : 1, NJ = W == 8 ? 4 : 2;
    static constexpr int PER = W / NP;  // consumers a producer feeds
    static constexpr int LAUNCH_REGS = 128, CONSUMER_REGS = 168, PRODUCER_REGS = 88, JOINER_REGS = 88;
    static_assert(8 * CONSUMER_REGS + 4 * PRODUCER_REGS + 4 * JOINER_REGS <= 16 * LAUNCH_REGS, "registers of the block");
    // What a unit costs besides its chunks (fetching queries, statistics, joining), in chunks; those of FP32 take
    // longer.  With 0 the CTAs with many short units are late: draft verification 49.1 us against 45.0 us, many int8
    // requests 44.7 us against 41.4 us; with 1 46.1 and 41.4 us; FP32 heads 22.8 us with 1 and 24.6 us with 2.
    static constexpr int UNIT_WORK = F32 ? 1 : 2;
    static constexpr int THREADS = 32 * (W + NP + NJ);
    static constexpr int S = ROOM / W < 8 ? ROOM / W : 8;  // ring slots a consumer
    static constexpr int SMEM = 1024 + HEAD + QUERIES + FACTORS + W * S * (SLOT + EXTRA);  // (1024: the ring's alignment)
    // Weights of 8-bit values are single FP16 numbers: next to values of 8 bits, 11 are plenty.  With the second part
    // 256 short int8 requests run 43.5 us instead of 41.7 us and e4m3 drafts 40.0 us instead of 36.4 us (long contexts
    // the same); without it the error of those requests is 2.4e-4, where the output's rounding alone is 2.1e-4.
    static constexpr bool SPLIT_P = !Q8;
    static constexpr float BIAS = CT == GDN_F16 || Q8 ? 6.f : -8.f;  // weights are 2^(s - m + BIAS)
    // A tile's scores before the output of the tile before: 82.5 us instead of 87.6 us for a context of 131071 tokens,
    // 161 us instead of 170 us for 64 x 4096 (FP16, 8 heads of 128).  Where a consumer holds more (two groups of rows)
    // or converts (8 and 32 bits) it runs longer instead: draft verification 52.2 us against 49.4 us, many int8
    // requests 45.2 us against 42.1 us, FP32 50.6 us against 48.9 us.
    static constexpr bool AHEAD = !Q8 && !F32 && NT == 1;
    static constexpr float HEADROOM = 8.f;  // a score may exceed the maximum by this: FP16 weights stay below 2^14
    static_assert(S >= 2 && W % NP == 0 && 512 + 2 * W * S * 8 + 64 <= 1600 && 1600 + 2 * (int)sizeof(Walk) <= HEAD && HALF % 1024 == 0,
                  "ring and barriers");
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
    // (tokens past the last sequence's are an error of the packing, not of that sequence)
    if (flag && (bad_cu || (b == p.B - 1 && cu1 != p.T))) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    if (flag && bad_len) flag_error(p.status, GDN_DEVERR_KV_LEN);
    if (bad_cu || bad_len) s.n = 0;
    const int upto = s.len - s.n + 1;  // (compared, not subtracted: a window may be as large as an int)
    s.first = p.window > 0 && upto > p.window ? upto - p.window : 0;
    s.t0 = s.first / C::TT * C::TT;
    s.tiles = s.len > s.t0 ? (s.len - s.t0 - 1) / C::TT + 1 : 0;
    s.chunks = s.tiles > 0 ? (s.tiles - 1) / C::W + 1 : 1;
    s.row_groups = (int)(((long long)s.n * p.G + C::ROWS - 1) / C::ROWS);
    s.units = p.c.H * s.row_groups;
    return s;
}

template <class C>
__device__ __forceinline__ void open_segment(Walk &w) {
    w.head = w.s.row_groups == 1 ? w.unit : (int)((uint32_t)w.unit / (uint32_t)w.s.row_groups);
    w.row0 = (w.unit - w.head * w.s.row_groups) * C::ROWS;
    w.seg_work = min(w.s.chunks + C::UNIT_WORK - w.pos, w.left);
    w.chunk = max(0, w.pos - C::UNIT_WORK);
    w.seg_chunks = max(0, w.pos + w.seg_work - C::UNIT_WORK) - w.chunk;
    if (w.seg_chunks == 0) w.left = 0;  // only a unit's fixed work is left: the next CTA, which has its chunks, does it
    w.tile = w.chunk * C::W;
    w.tile_end = min((w.chunk + w.seg_chunks) * C::W, w.s.tiles);
}

template <class C>
__device__ __forceinline__ void next_segment(Walk &w, const PagedAttnParams &p) {
    w.left -= w.seg_work;
    if (w.left <= 0) return;
    w.pos = 0;
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
    open_segment<C>(w);
}

__device__ __forceinline__ long long divide(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The first `rem` CTAs take one unit of work more than the others.
struct Shares {
    long long each, rem;
    __device__ __forceinline__ long long begin(int cta) const { return cta * each + min((long long)cta, rem); }
    __device__ __forceinline__ int owner(long long x) const {
        const long long big = rem * (each + 1);
        return (int)(x < big ? divide(x, each + 1) : rem + divide(x - big, each));
    }
};

// The warp waits for a barrier's phase.  A wait that runs out (WAIT_LIMIT cycles;
// it never does while the other roles run) marks the CTA dead: all waits of it
// return false, its warps leave, and it writes no results.
constexpr long long WAIT_LIMIT = 4000000000LL;
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, volatile int *dead) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, ptx::mbar_try_wait_for(bar, parity, 20000))) {
        if (clock64() - t0 > WAIT_LIMIT) *dead = 1;
        if (__any_sync(0xffffffffu, *dead != 0)) return false;
    }
    return true;
}

// The barrier receives this lane's arrival when all its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
// The same, and whether x is set in any of the threads.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
    int any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(threads), "r"((int)x)
        : "memory");
    return any != 0;
}

// What a CTA leaves for the join: the unit whose head it holds but not its end.
struct Split {
    int parts;  // CTAs that hold parts of it, from this one on; 0: there is none
    int rows, row0, head, cu0, pos0;
    int pad[2];  // 32 bytes, so that what follows the records is aligned
};

// The maximum before any score: as low as a finite number can be, so that any score raises it and 2^(-inf - NONE) is 0.
constexpr float NONE = -3.402823466e38f;

// What a part's sums count for when its maximum is `part` and that of all parts `all`.
__device__ __forceinline__ float part_factor(float part, float all) { return exp2_fast(part - all); }

// Four channels of joined row r of a unit, x unnormalised, st = (maximum, sum).
template <int CT, class C>
__device__ __forceinline__ void store_row(const PagedAttnParams &p, int row, int head, int cu0, int pos0, int ch, float4 x,
                                          float2 st) {
    const int i = (int)((uint32_t)row / (uint32_t)p.G), hq = row - i * p.G;
    const bool any = pos0 + i >= 0;  // a query at a position before the cache sees nothing
    const float inv = any ? 1.f / st.y : 0.f;
    const long long at = (long long)(cu0 + i) * p.Hq + (long long)head * p.G + hq;
    const float4 y = any ? make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (C::F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * C::D + ch) = y;
    } else {
        const bool bf = C::BF16 || (C::Q8 && p.io_bf16);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at * C::D + ch) =
            bf ? make_uint2(pack2<true>(y.x, y.y), pack2<true>(y.z, y.w)) : make_uint2(pack2<false>(y.x, y.y), pack2<false>(y.z, y.w));
    }
    if (p.lse && ch == 0)
        p.lse[at] = any ? (st.x - C::BIAS + log2f(st.y)) * 0.6931471805599453f : __int_as_float(0xff800000);
}

// The workspace: a Split per CTA, then two parts a CTA (0: the end or middle of
// a unit that another CTA began, 1: the head of one): (maximum, sum) of each
// row, and the rows.
template <class C>
struct Parts {
    Split *split;
    float2 *ml;
    float *o;
    __device__ __forceinline__ Parts(float *base, int ctas) {
        split = reinterpret_cast<Split *>(base);
        ml = reinterpret_cast<float2 *>(base + (size_t)ctas * (sizeof(Split) / 4));
        o = base + (size_t)ctas * (sizeof(Split) / 4 + 4 * C::ROWS);
    }
};

// ---------------------------------------------------------------- the kernel

// The registers that a role's warps (whole groups of four) go on with.
template <int N>
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// BY_ROWS: pages are not a multiple of 8 tokens, rows are copied one by one (see launch_sized).
template <int CT, class C, bool BY_ROWS>
__global__ void __launch_bounds__(C::THREADS, 1) paged_attention_kernel(const __grid_constant__ PagedAttnParams p,
                                                                        const __grid_constant__ CUtensorMap k_map,
                                                                        const __grid_constant__ CUtensorMap v_map, int box_shift) {
    constexpr int NT = C::NT, ROWS = C::ROWS, D = C::D, TS = C::TS, TT = C::TT, W = C::W, S = C::S;
    constexpr int KB = C::KB, VB = C::VB, MT = C::MT, MPV = C::MPV;
    constexpr bool Q8 = C::Q8, F32 = C::F32, BF16 = C::BF16;
    constexpr uint32_t FULL = 0xffffffffu;
    const float NEG_INF = __int_as_float(0xff800000);

    extern __shared__ __align__(1024) uint8_t smem[];
    long long *scan = reinterpret_cast<long long *>(smem);               // [warps] sums
    Walk *first = reinterpret_cast<Walk *>(smem + 128);                  // where this CTA's share begins
    volatile int *dead = reinterpret_cast<volatile int *>(smem + 272);   // a wait ran out
    int *part_slot = reinterpret_cast<int *>(smem + 288);                // [W] where a consumer left its part
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + 512);           // [W][S] a slot's tile has landed, or it is free for a part
    uint64_t *empty = full + W * S;                                      // [W][S] its tile or part has been used
    uint64_t *q_full = empty + W * S, *q_empty = q_full + 2;             // [2] a segment and its queries
    uint64_t *j_full = q_empty + 2, *j_empty = j_full + 1;               // the consumers' parts of a segment
    Walk *segments = reinterpret_cast<Walk *>(smem + 1600);              // [2] for the consumers; none left: the end
    uint8_t *queries = smem + C::HEAD;                                   // [2][ROWS][QROW]
    float2 *q_stat = reinterpret_cast<float2 *>(queries + 2 * ROWS * C::QROW);  // [2][ROWS] scores' (scale, bias)
    float2 *joined = reinterpret_cast<float2 *>(queries + C::QUERIES);   // [ROWS] maxima and sums
    float *factor = reinterpret_cast<float *>(joined + ROWS);            // [W][ROWS]
    uint8_t *extras = reinterpret_cast<uint8_t *>(factor + 8 * ROWS);    // [W][S][EXTRA]
    uint8_t *ring = smem + (C::SMEM - W * S * C::SLOT - 1024);           // [W][S][SLOT], on a 1024-byte boundary
    ring += (1024 - (ptx::smem_u32(ring) & 1023)) & 1023;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    if (tid < W * S) {
        ptx::mbar_init(full + tid, Q8 || BY_ROWS ? 33 : 1);  // tensor copies, and each lane's other copies
        ptx::mbar_init(empty + tid, 1);
    }
    if (tid < 2) {
        ptx::mbar_init(q_full + tid, 32 * C::NJ);
        ptx::mbar_init(q_empty + tid, W);
    }
    if (tid == 0) {
        ptx::mbar_init(j_full, W);
        ptx::mbar_init(j_empty, 1);
        *dead = 0;
    }
    if (!BY_ROWS && tid == 32) {
        ptx::prefetch_tensor_map(&k_map);
        ptx::prefetch_tensor_map(&v_map);
    }
    ptx::fence_mbar_init();
    dependent_prologue();

    // ---- this CTA's share of the work
    Shares shares;
    long long total, start;
    {
        const int per = (p.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = load_seq<C>(p, b, blockIdx.x == 0);
            sum += (long long)s.units * (s.chunks + C::UNIT_WORK);
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
        for (int i = 0; i < C::THREADS / 32; ++i) {
            if (i < warp) before += scan[i];
            total += scan[i];
        }
        const int ctas = (int)min((long long)gridDim.x, total);  // those with work
        if (blockIdx.x >= ctas) {
            if (tid == 0) Parts<C>(p.partials, gridDim.x).split[blockIdx.x].parts = 0;
            return;
        }
        shares.each = divide(total, ctas);
        shares.rem = total - shares.each * ctas;
        start = shares.begin(blockIdx.x);
        long long excl = before + incl - sum;
        if (start >= excl && start < excl + sum) {
            for (int b = b0;; ++b) {
                const Seq s = load_seq<C>(p, b, false);
                const long long here = (long long)s.units * (s.chunks + C::UNIT_WORK);
                if (start < excl + here) {
                    Walk w;
                    w.s = s;
                    w.unit = (int)divide(start - excl, s.chunks + C::UNIT_WORK);
                    w.pos = (int)(start - excl - (long long)w.unit * (s.chunks + C::UNIT_WORK));
                    w.left = (int)(shares.begin(blockIdx.x + 1) - start);
                    *first = w;
                    break;
                }
                excl += here;
            }
        }
        __syncthreads();
    }
    Walk use = *first;  // what the warp is at

    // ---- joiners: fetch the queries of the segments and add the consumers' parts of them
    if (warp >= W + C::NP) {
        if constexpr (W == 8) give_registers<C::JOINER_REGS>();
        constexpr int THREADS = 32 * C::NJ;
        const int j = tid - 32 * (W + C::NP);
        const Parts<C> parts(p.partials, gridDim.x);
        int split_parts = 0;
        open_segment<C>(use);
        // The queries of a segment into shared memory, ROWS / NJ rows a warp with all loads in flight at once (the
        // consumers' copies queue up in front of a later one: it took 5 us).  Scores are (K q + bias) scale:
        // queries over 8-bit rows go as FP16, BF16 ones scaled by a power of two that brings the row's largest
        // magnitude to [1, 2), and int8 keys are multiplied as (128 + k) 2^-24 (see widen_keys).
        auto fetch = [&](const Walk &w, int segment) {
            const int b = segment & 1;
            if (w.left <= 0) {  // the end
                if (!ring_wait(q_empty + b, ((segment >> 1) + 1) & 1, dead)) return;
                if (j == 0) segments[b].left = 0;
                ptx::mbar_arrive(q_full + b);
                return;
            }
            const int rows = min(ROWS, w.s.n * p.G - w.row0);
            constexpr int EB = F32 ? 4 : 2, LANE = D * EB / 32;  // bytes a lane takes of a row: 4 to 32
            constexpr int WORDS = LANE / 4, BATCH = ROWS / C::NJ;
            const int r0 = BATCH * (warp - W - C::NP);
            const int group = w.row0 + min(lane, rows - 1);  // lane r: where row r is
            const int token = w.s.n == 1 ? 0 : (int)((uint32_t)group / (uint32_t)p.G);
            const long long head = (long long)w.head * p.G + group - token * p.G;
            const long long row = ((long long)(w.s.cu0 + token) * p.q_stride + head * D) * EB;
            uint32_t x[BATCH][WORDS];
#pragma unroll
            for (int r = 0; r < BATCH; ++r) {
                const uint8_t *src = static_cast<const uint8_t *>(p.q) + __shfl_sync(FULL, row, r0 + r) + lane * LANE;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) x[r][i] = 0u;
                if (r0 + r < rows) {
                    if constexpr (WORDS == 1) x[r][0] = *reinterpret_cast<const uint32_t *>(src);
                    if constexpr (WORDS == 2) lds<2>(x[r], src);
                    if constexpr (WORDS == 4) lds<4>(x[r], src);
                    if constexpr (WORDS == 8) {
                        lds<4>(reinterpret_cast<uint32_t(&)[4]>(x[r][0]), src);
                        lds<4>(reinterpret_cast<uint32_t(&)[4]>(x[r][4]), src + 16);
                    }
                }
            }
            if (!ring_wait(q_empty + b, ((segment >> 1) + 1) & 1, dead)) return;
            if (j == 0) segments[b] = w;
#pragma unroll
            for (int r = 0; r < BATCH; ++r) {
                float scale = p.scale_log2, sum = 0.f;
                if constexpr (Q8) {
                    if (p.io_bf16) {
                        float top = 0.f;
#pragma unroll
                        for (int i = 0; i < WORDS; ++i) {
                            const float2 f = unpack2<true>(x[r][i]);
                            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
                        // the exponent of top, kept where both powers of two are normal
                        int e = (int)(__float_as_uint(top) >> 23 & 255) - 127;
                        e = top > 0.f && top <= 3.402823466e38f ? min(max(e, -100), 126) : 0;
                        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                        scale *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                        for (int i = 0; i < WORDS; ++i) {
                            const float2 f = unpack2<true>(x[r][i]);
                            x[r][i] = pack2<false>(f.x * down, f.y * down);
                        }
                    }
                    if constexpr (CT == GDN_INT8) {
#pragma unroll
                        for (int i = 0; i < WORDS; ++i) {
                            const float2 f = unpack2<false>(x[r][i]);
                            sum += f.x + f.y;
                        }
                        sum = warp_sum(sum);
                        scale *= 16777216.f;
                    }
                }
                uint32_t *dst = reinterpret_cast<uint32_t *>(queries + (b * ROWS + r0 + r) * C::QROW + lane * LANE);
                if constexpr (WORDS == 1) dst[0] = x[r][0];
                if constexpr (WORDS == 2) *reinterpret_cast<uint2 *>(dst) = make_uint2(x[r][0], x[r][1]);
                if constexpr (WORDS >= 4) {
#pragma unroll
                    for (int i = 0; i < WORDS; i += 4)
                        *reinterpret_cast<uint4 *>(dst + i) = make_uint4(x[r][i], x[r][i + 1], x[r][i + 2], x[r][i + 3]);
                }
                if (lane == 0) q_stat[b * ROWS + r0 + r] = make_float2(scale, -128.f / 16777216.f * sum);
            }
            ptx::mbar_arrive(q_full + b);
        };
        fetch(use, 0);
        for (int segment = 0; use.left > 0; ++segment) {
            Walk next = use;
            next_segment<C>(next, p);
            fetch(next, segment + 1);
            const int head = use.head, row0 = use.row0, rows = min(ROWS, use.s.n * p.G - row0);
            const int pos0 = use.s.len - use.s.n;
            const bool whole = use.seg_chunks == use.s.chunks;
            if (named_any(1, THREADS, !ring_wait(j_full, segment & 1, dead))) break;  // (all of them, or none)
            const float4 *part[W];
            const float2 *part_stat[W];  // (maximum, sum)
            int at[W];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                at[w] = w * S + part_slot[w];
                part[w] = reinterpret_cast<const float4 *>(ring + at[w] * C::SLOT);
                part_stat[w] = reinterpret_cast<const float2 *>(extras + at[w] * C::EXTRA);
            }
            for (int r = j; r < ROWS; r += THREADS) {
                float2 st[W];
                float mm = NONE, ll = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    st[w] = part_stat[w][r];
                    mm = fmaxf(mm, st[w].x);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float f = part_factor(st[w].x, mm);
                    factor[w * ROWS + r] = f;
                    ll += st[w].y * f;
                }
                joined[r] = make_float2(mm, ll);
            }
            named_sync(1, THREADS);
            const long long slot = 2LL * blockIdx.x + (use.chunk == 0 ? 1 : 0);
            for (int i = j; i < rows * (D / 4); i += THREADS) {
                const int r = i / (D / 4), ch = i % (D / 4) * 4;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float4 x = part[w][r * (D / 4) + (ch / 4 ^ C::part_swizzle(r))];
                    const float f = factor[w * ROWS + r];
                    sum.x += f * x.x, sum.y += f * x.y, sum.z += f * x.z, sum.w += f * x.w;
                }
                if (whole) {
                    store_row<CT, C>(p, row0 + r, head, use.s.cu0, pos0, ch, sum, joined[r]);
                } else {
                    *reinterpret_cast<float4 *>(parts.o + (slot * ROWS + r) * D + ch) = sum;
                    if (ch == 0) parts.ml[slot * ROWS + r] = joined[r];
                }
            }
            ptx::fence_proxy_async_smem();  // tensor copies will overwrite what the consumers stored
            named_sync(1, THREADS);
            if (j == 0) {
#pragma unroll
                for (int w = 0; w < W; ++w) ptx::mbar_arrive(empty + at[w]);
                ptx::mbar_arrive(j_empty);
                if (!whole && use.chunk == 0) {  // the head of a unit that goes on: this CTA's last segment
                    split_parts = shares.owner(shares.begin(blockIdx.x + 1) - use.left - use.pos + C::UNIT_WORK + use.s.chunks - 1) - (int)blockIdx.x + 1;
                    parts.split[blockIdx.x] = {split_parts, rows, row0, head, use.s.cu0, pos0, {0, 0}};
                }
            }
            use = next;
        }
        if (j == 0) {
            if (split_parts == 0) parts.split[blockIdx.x].parts = 0;
            if (*dead) flag_error(p.status, GDN_DEVERR_TIMEOUT);
        }
        return;
    }

    // ---- producers: warp W + i copies the tiles of consumers i PER, ... ahead of them
    if (warp >= W) {
        if constexpr (W == 8) give_registers<C::PRODUCER_REGS>();
        constexpr int PER = C::PER;
        const int base = (warp - W) * PER;  // the first consumer
        // A tile's keys (values) are `subs` boxes of box_tokens tokens, each within a page.  For each of its consumers'
        // tiles, lane i looks up box i % subs of the i / subs-th next.
        constexpr int TT_SHIFT = TS == 2 ? 5 : 4;
        const int box_tokens = 1 << box_shift, sub_shift = TT_SHIFT - box_shift, subs = 1 << sub_shift, batch = 32 >> sub_shift;
        // (The loop over the consumers is not unrolled: the roles' code together has to stay in the instruction cache.)
        uint32_t puts = 0;     // byte q: consumer q's slot that is filled next
        uint32_t wrapped = 0;  // bit q: the parity of its rounds through the ring
        auto put = [&](int q) { return (int)(puts >> 8 * q & 255); };
        auto step = [&](int q) {
            puts += 1u << 8 * q;
            if (put(q) == S) puts -= (uint32_t)S << 8 * q, wrapped ^= 1u << q;
        };
        const uint64_t keep = Q8 ? keep_policy() : 0;
        auto feed = [&]() {  // returns early in a dead CTA
            open_segment<C>(use);
            while (use.left > 0) {
                const int head = use.head;
                for (int k0 = 0; k0 < use.seg_chunks; k0 += batch) {
                    const int tile = use.tile + k0 * W + base;
                    int page[PER], in_page[PER];  // where the lane's boxes are
                    uint32_t boxes[PER];          // the lanes with boxes that are read
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        const int my_tile = tile + (lane >> sub_shift) * W + q;
                        const int t = use.s.t0 + my_tile * TT + ((lane & (subs - 1)) << box_shift);
                        const bool wanted = my_tile < use.tile_end && t < use.s.len && t + box_tokens > use.s.first;
                        page[q] = in_page[q] = 0;
                        if (wanted) {
                            const int i = p.page_shift >= 0 ? t >> p.page_shift : (int)((uint32_t)t / (uint32_t)p.c.page_size);
                            in_page[q] = t - i * p.c.page_size;
                            page[q] = p.block_table[use.s.b * p.bt_stride + i];
                        }
                        boxes[q] = __ballot_sync(FULL, wanted);
                    }
#pragma unroll
                    for (int q = 0; q < PER; ++q)  // a page outside the pool reads as zeros, like num_pages
                        if ((uint32_t)page[q] >= (uint32_t)p.c.num_pages) {
                            flag_error(p.status, GDN_DEVERR_PAGE);
                            page[q] = p.c.num_pages;
                        }
                    const int end = (min(k0 + batch, use.seg_chunks) - k0) * PER;
#pragma unroll 1
                    for (int n = 0; n < end; ++n) {
                        const int q = n % PER, box0 = n / PER * subs;
                        if (tile + n / PER * W + q >= use.tile_end) continue;
                        int at_page = page[0], at_off = in_page[0];
                        uint32_t mine = boxes[0];
#pragma unroll
                        for (int i = 1; i < PER; ++i)
                            if (q == i) at_page = page[i], at_off = in_page[i], mine = boxes[i];
                        const bool my_box = mine >> lane & 1;
                        mine = mine >> box0 & (FULL >> (32 - subs));
                        const int slot = (base + q) * S + put(q);
                        uint8_t *dst = ring + slot * C::SLOT;
                        uint64_t *bar = full + slot;
                        if (!ring_wait(empty + slot, (wrapped >> q & 1) ^ 1, dead)) return;
                        if constexpr (BY_ROWS) {
                            if (lane == 0) ptx::mbar_arrive(bar);
                            // lane box0 + i looked up token i: its row's byte offset, -1 if it is not read
                            long long row = -1;
                            if (my_box && at_page < p.c.num_pages)
                                row = (at_page * p.c.page_stride + at_off * p.c.token_stride + head * p.c.head_stride) * C::ESZ;
                            constexpr int PIECES = C::RB / 16, PER_SPAN = C::SPAN / 16;
                            const uint32_t to = ptx::smem_u32(dst);
#pragma unroll 4
                            for (int k = lane; k < TT * PIECES; k += 32) {
                                const int token = k / PIECES, x = k % PIECES, y = x % PER_SPAN;
                                const long long o = __shfl_sync(FULL, row, box0 + token);
                                const uint32_t at = to + (x / PER_SPAN) * TT * C::SPAN + token * C::SPAN +
                                                    ((y ^ (C::SPAN == 64 ? token >> 1 & 3 : token & 7)) << 4);
                                const long long src = o < 0 ? 0 : o + x * 16;
                                copy_async16(at, static_cast<const uint8_t *>(p.c.k) + src, o < 0 ? 0 : 16);
                                copy_async16(at + C::HALF, static_cast<const uint8_t *>(p.c.v) + src, o < 0 ? 0 : 16);
                            }
                        } else {
                            constexpr int MOST = TT / 8;  // boxes of 8 tokens or more
                            int pg[MOST], off[MOST];
#pragma unroll
                            for (int b = 0; b < MOST; ++b) {
                                if (b > 0 && b >= subs) break;
                                pg[b] = __shfl_sync(FULL, at_page, box0 + b);
                                off[b] = __shfl_sync(FULL, at_off, box0 + b);
                            }
                            if (ptx::elect_one()) {
                                ptx::mbar_arrive_expect_tx(bar, __popc(mine) * (2 * C::RB) << box_shift);
                                if (subs == 1) {  // all spans at once
                                    ptx::tma_load_5d(dst, &k_map, 0, off[0], 0, head, pg[0], bar);
                                    ptx::tma_load_5d(dst + C::HALF, &v_map, 0, off[0], 0, head, pg[0], bar);
                                } else {
#pragma unroll
                                    for (int b = 0; b < MOST; ++b) {
                                        if (!(mine >> b & 1)) continue;
                                        uint8_t *to = dst + (b << box_shift) * C::SPAN;
#pragma unroll 1
                                        for (int x = 0; x < C::BOXES; ++x) {
                                            ptx::tma_load_5d(to + x * TT * C::SPAN, &k_map, 0, off[b], x, head, pg[b], bar);
                                            ptx::tma_load_5d(to + C::HALF + x * TT * C::SPAN, &v_map, 0, off[b], x, head, pg[b], bar);
                                        }
                                    }
                                }
                            }
                            __syncwarp();
                        }
                        if constexpr (Q8) {
                            // TS == 2: a token a lane; 16 tokens: the upper lanes fetch the value scales.  (Those of tokens
                            // past the end are of the same page, and masked like their scores.)
                            const int token = lane & (TT - 1), sub = token >> box_shift;
                            const int pg = __shfl_sync(FULL, at_page, box0 + sub);
                            const int off = __shfl_sync(FULL, at_off, box0 + sub) + (token & (box_tokens - 1));
                            const int ok = (mine >> sub & 1) && pg < p.c.num_pages ? 4 : 0;
                            const long long at = ok ? (long long)pg * p.s_page_stride32 + (long long)off * p.s_token_stride32 +
                                                          (long long)head * p.s_head_stride32
                                                    : 0;
                            const uint32_t to = ptx::smem_u32(extras + slot * C::EXTRA + 4 * lane);
                            copy_async4_kept(to, (TS == 2 || lane < 16 ? p.c.k_scale : p.c.v_scale) + at, ok, keep);
                            if (TS == 2) copy_async4_kept(to + 4 * TT, p.c.v_scale + at, ok, keep);
                        }
                        if (Q8 || BY_ROWS) copy_arrive(bar);
                        step(q);
                    }
                }
#pragma unroll
                for (int q = 0; q < PER; ++q) {  // a slot for each consumer's part of the segment
                    const int slot = (base + q) * S + put(q);
                    if (!ring_wait(empty + slot, (wrapped >> q & 1) ^ 1, dead)) return;
                    if (Q8 || BY_ROWS || lane == 0) ptx::mbar_arrive(full + slot);
                    if ((Q8 || BY_ROWS) && lane == 0) ptx::mbar_arrive(full + slot);
                    step(q);
                }
                next_segment<C>(use, p);
            }
        };
        feed();
        copy_wait_all();
        if (*dead)  // nobody waits for the tensor copies in flight: a millisecond for them to land
            for (int i = 0; i < 1000; ++i) __nanosleep(1000);
        return;
    }

    // ---- consumers: warp w multiplies tiles w, w + W, ... of each segment
    if constexpr (W == 8) take_registers<C::CONSUMER_REGS>();
    uint8_t *slots = ring + warp * (S * C::SLOT);  // this warp's
    uint64_t *landed = full + warp * S, *used = empty + warp * S;
    int at = 0;          // the slot that is used next
    uint32_t phase = 0;  // bit i: the parity of slot i's next landing

    // Where the lane's pieces are in a slot: key row g (and g + 8), piece c (odd steps: + 4); value rows
    // 2 c, 2 c + 1 (and + 8), its piece g.  Swizzled as the tensor copies leave them.
    constexpr bool HALF_LINE = C::SPAN == 64;
    const int k_at = g * C::SPAN + ((c ^ (HALF_LINE ? g >> 1 : g)) << 4);
    const int v_at0 = 2 * c * C::SPAN + (HALF_LINE ? ((g >> 1 ^ c) << 4) + (g & 1) * 8 : (g ^ 2 * c) << 4);
    const int v_at1 = (2 * c + 1) * C::SPAN + (HALF_LINE ? ((g >> 1 ^ c) << 4) + (g & 1) * 8 : (g ^ (2 * c + 1)) << 4);

    float2 col[NT][2];  // the scores' (scale, bias) of the lane's two columns
    float o[NT][MT][4], m[NT][2], l[NT][2];
    int rows = 0;                // query rows of the unit
    int at_pos[NT][2];           // the positions of the queries of the lane's two columns
    int all_lo = 0, all_hi = 0;  // positions that every query row of the unit sees: [all_lo, all_hi)
    auto sees = [&](int pos, int t) { return t <= pos && (p.window == 0 || pos - t < p.window); };
    for (int segment = 0;; ++segment) {
        const Walk &at_use = segments[segment & 1];
        int use_tile, use_end, use_t0;
        {
            if (!ring_wait(q_full + (segment & 1), segment >> 1 & 1, dead) || at_use.left <= 0) return;
            use_tile = at_use.tile + warp, use_end = at_use.tile_end, use_t0 = at_use.s.t0;
            rows = min(ROWS, at_use.s.n * p.G - at_use.row0);
            const int pos0 = at_use.s.len - at_use.s.n;  // the first query's position
            auto position = [&](int r) {           // of row r's query (rows past the last repeat it)
                return at_use.s.n == 1 ? pos0 : pos0 + (int)((uint32_t)(at_use.row0 + min(r, rows - 1)) / (uint32_t)p.G);
            };
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                at_pos[nt][0] = position(nt * 8 + 2 * c);
                at_pos[nt][1] = position(nt * 8 + 2 * c + 1);
            }
            all_hi = position(0) + 1;
            const int upto = position(rows - 1) + 1;
            all_lo = p.window > 0 && upto > p.window ? upto - p.window : 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                col[nt][0] = q_stat[(segment & 1) * ROWS + nt * 8 + 2 * c];
                col[nt][1] = q_stat[(segment & 1) * ROWS + nt * 8 + 2 * c + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = NONE;
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
            }
        }
        // ---- scores of the tile in a slot: S^T = K Q^T
        float sc[TS][NT][4];
        auto scores = [&](int slot) {
            float sc2[TS][NT][4];
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[ts][nt][e] = sc2[ts][nt][e] = 0.f;
            const uint8_t *ks = slots + slot * C::SLOT;
            // lane (g, c) holds, of query row 8 nt + g, the channels that its key pieces have
            const uint8_t *qs = queries + ((segment & 1) * ROWS + g) * C::QROW + c * (Q8 ? 32 : 16);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint32_t q[NT][Q8 ? 8 : 4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint8_t *src = qs + nt * 8 * C::QROW + kb * (Q8 ? 128 : 64);
                    lds<4>(reinterpret_cast<uint32_t(&)[4]>(q[nt][0]), src);
                    if constexpr (Q8) lds<4>(reinterpret_cast<uint32_t(&)[4]>(q[nt][4]), src + 16);
                }
#pragma unroll
                for (int ts = 0; ts < TS; ++ts) {
                    uint32_t x[4], y[4];
                    const uint8_t *piece = ks + (kb / 2) * TT * C::SPAN + ts * 16 * C::SPAN + (kb % 2 ? k_at ^ 64 : k_at);
                    lds<4>(x, piece);
                    lds<4>(y, piece + 8 * C::SPAN);
                    if constexpr (Q8) {
                        uint32_t u[8], v[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            widen_keys<CT>(x[j], u[2 * j], u[2 * j + 1]);
                            widen_keys<CT>(y[j], v[2 * j], v[2 * j + 1]);
                        }
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16<false>((j & 2) ? sc2[ts][nt] : sc[ts][nt], u[j], v[j], u[j + 1], v[j + 1], q[nt][j],
                                             q[nt][j + 1]);
                    } else if constexpr (F32) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float t[4] = {0.f, 0.f, 0.f, 0.f};  // (see mma_f32)
#pragma unroll
                            for (int j = 0; j < 4; j += 2) {
                                const uint32_t a[4] = {x[j], y[j], x[j + 1], y[j + 1]};
                                uint32_t bh[2], bl[2];
                                split_tf32(q[nt][j], bh[0], bl[0]);
                                split_tf32(q[nt][j + 1], bh[1], bl[1]);
                                mma_f32(t, a, bh, bl);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) (kb % 2 ? sc2 : sc)[ts][nt][e] += t[e];
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j += 2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16<BF16>(j ? sc2[ts][nt] : sc[ts][nt], x[j], y[j], x[j + 1], y[j + 1], q[nt][j], q[nt][j + 1]);
                    }
                }
            }
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[ts][nt][e] += sc2[ts][nt][e];
        };
        auto arrived = [&](int slot) {
            const bool ok = ring_wait(landed + slot, phase >> slot & 1, dead);
            phase ^= 1u << slot;
            return ok;
        };
        if (C::AHEAD && use_tile < use_end) {
            if (!arrived(at)) return;
            scores(at);
        }
        for (; use_tile < use_end; use_tile += W) {
            const int tile_t = use_t0 + use_tile * TT;
            const bool edge = tile_t < all_lo || tile_t + TT > all_hi;
            if (!C::AHEAD) {
                if (!arrived(at)) return;
                scores(at);
            }

            // the lane's tokens are rows g and g + 8 of each subtile
            float vs[TS][2], lv[TS][2];
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = NEG_INF;
            const float *scales = reinterpret_cast<const float *>(extras + (warp * S + at) * C::EXTRA);
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float ksc = 1.f;
                    if constexpr (Q8) {
                        const int i = ts * 16 + g + 8 * h;
                        ksc = scales[i];
                        vs[ts][h] = scales[TT + i];
                        lv[ts][h] = log2_fast(fmaxf(fabsf(vs[ts][h]), 1e-30f));  // (rows of zeros may have scale 0)
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &x = sc[ts][nt][2 * h + e];
                            if constexpr (CT == GDN_INT8) x += col[nt][e].y;
                            x *= Q8 ? col[nt][e].x * ksc : col[nt][e].x;
                        }
                }
            if (__builtin_expect(edge, 0)) {
#pragma unroll
                for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!sees(at_pos[nt][e & 1], tile_t + ts * 16 + g + 8 * (e >> 1))) sc[ts][nt][e] = NEG_INF;
            }
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top[nt][e & 1] = fmaxf(top[nt][e & 1], Q8 ? sc[ts][nt][e] + lv[ts][e >> 1] : sc[ts][nt][e]);

            // ---- raise the maxima where a score exceeds them by more than the headroom
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                raise |= top[nt][0] > m[nt][0] + C::HEADROOM || top[nt][1] > m[nt][1] + C::HEADROOM;
            if (__any_sync(FULL, raise)) {
                if constexpr (Q8) {
                    // A row of zeros has scale 1, whatever the scales of the others: it must not raise the maximum, which
                    // would leave the weights of rows with small scales too few bits.  So it goes with a scale of 0, and
                    // counts as 2^-80 in the maximum: low enough that weights beside it stay normal FP16 numbers down to
                    // scales of 2^-100, high enough that its own term of the sum stays far inside FP32.
                    // (Looked for only where a score would raise the maximum beside a scale of 1: 64 x 4096 tokens 91 us either way.)
                    bool ones = false;
#pragma unroll
                    for (int ts = 0; ts < TS; ++ts) ones |= vs[ts][0] == 1.f || vs[ts][1] == 1.f;
                    if (__any_sync(FULL, ones)) {
                        const uint8_t *vrow = slots + at * C::SLOT + C::HALF;
#pragma unroll
                        for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t any = 0;  // of the row's pieces c, c + 4, ... of each span (in whatever order they lie)
#pragma unroll
                                for (int x = 0; x < C::BOXES; ++x)
#pragma unroll
                                    for (int k = c; k < C::SPAN / 16; k += 4) {
                                        uint32_t w[4];
                                        lds<4>(w, vrow + x * TT * C::SPAN + (ts * 16 + g + 8 * h) * C::SPAN + k * 16);
                                        any |= w[0] | w[1] | w[2] | w[3];
                                    }
                                if constexpr (CT == GDN_FP8_E4M3) any &= 0x7f7f7f7fu;  // zeros of either sign
                                any |= __shfl_xor_sync(FULL, any, 1);
                                any |= __shfl_xor_sync(FULL, any, 2);
                                if (any == 0 && vs[ts][h] == 1.f) vs[ts][h] = 0.f, lv[ts][h] = -80.f;
                            }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = NEG_INF;
#pragma unroll
                        for (int ts = 0; ts < TS; ++ts)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    top[nt][e & 1] = fmaxf(top[nt][e & 1], sc[ts][nt][e] + lv[ts][e >> 1]);
                    }
                }
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
                        const float x = exp2_fast(sc[ts][nt][e] - (m[nt][e & 1] - C::BIAS));
                        l[nt][e & 1] += x;
                        w[e] = Q8 ? x * vs[ts][e >> 1] : x;
                    }
                    if (Q8 && __builtin_expect(edge, 0)) {  // (the scale of a masked row may be anything)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sc[ts][nt][e] == NEG_INF) w[e] = 0.f;
                    }
                    if constexpr (F32) {
                        // k-slots c and c + 4 are tokens 2 c and 2 c + 1 (+ 8): from the lanes that hold their rows, column g
                        const int src = c * 8 + (g >> 1);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float a = __shfl_sync(FULL, w[2 * k], src + 4 * j);
                                const float b = __shfl_sync(FULL, w[2 * k + 1], src + 4 * j);
                                split_tf32(__float_as_uint(g & 1 ? b : a), fh[ts][nt][k][j], fl[ts][nt][k][j]);
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t hi = pack2<BF16>(w[2 * k], w[2 * k + 1]);
                            ph[ts][nt][k] = transpose8x8(hi);
                            if constexpr (C::SPLIT_P) {
                                const float2 back = unpack2<BF16>(hi);
                                pl[ts][nt][k] = transpose8x8(pack2<BF16>(w[2 * k] - back.x, w[2 * k + 1] - back.y));
                            }
                        }
                    }
                }

            // ---- O^T += V^T P^T
            const uint8_t *vsm = slots + at * C::SLOT + C::HALF;
            constexpr int VW = C::CHV / 4;  // words of a value piece
            // `only` (careful): the single query row to add to, with values that it does not see left out
            auto add_values = [&](int only, int only_pos, auto careful) {
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                    for (int ts = 0; ts < TS; ++ts) {
                        uint32_t v[4][VW];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            lds<VW>(v[k], vsm + vb * TT * C::SPAN + (ts * 16 + 8 * (k >> 1)) * C::SPAN + ((k & 1) ? v_at1 : v_at0));
                            if constexpr (careful()) {
                                const int t = tile_t + ts * 16 + 2 * c + (k & 1) + 8 * (k >> 1);
                                if (!sees(only_pos, t)) {
#pragma unroll
                                    for (int j = 0; j < VW; ++j) v[k][j] = 0u;
                                }
                            }
                        }
                        // acc += a product, in the lane's columns that are meant (the others may have seen 0 * inf)
                        auto into = [&](float(&acc)[4], int nt, auto product) {
                            if constexpr (careful()) {
                                float t[4] = {acc[0], acc[1], acc[2], acc[3]};
                                product(t);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (only == nt * 8 + 2 * c + (e & 1)) acc[e] = t[e];
                            } else {
                                product(acc);
                            }
                        };
                        if constexpr (F32) {
#pragma unroll
                            for (int j = 0; j < VW; j += 2)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    into(o[nt][vb * MPV + j / 2], nt, [&](float(&acc)[4]) {
                                        float t[4] = {0.f, 0.f, 0.f, 0.f};  // (see mma_f32)
#pragma unroll
                                        for (int k = 0; k < 2; ++k) {
                                            const uint32_t a[4] = {v[2 * k][j], v[2 * k][j + 1], v[2 * k + 1][j], v[2 * k + 1][j + 1]};
                                            mma_f32(t, a, fh[ts][nt][k], fl[ts][nt][k]);
                                        }
#pragma unroll
                                        for (int e = 0; e < 4; ++e) acc[e] += t[e];
                                    });
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
                                for (int nt = 0; nt < NT; ++nt)
                                    into(o[nt][vb * MPV + j], nt, [&](float(&acc)[4]) {
                                        if constexpr (C::SPLIT_P)
                                            mma16<BF16>(acc, a[j][0], a[j][1], a[j][2], a[j][3], pl[ts][nt][0], pl[ts][nt][1]);
                                        mma16<BF16>(acc, a[j][0], a[j][1], a[j][2], a[j][3], ph[ts][nt][0], ph[ts][nt][1]);
                                    });
                        }
                    }
            };
            // A tile at an end of what is cached holds other rows too (of other tokens, or never written): their
            // values are zeroed.  A value that some query rows see and others do not would reach the others as 0 *
            // inf if it is not finite: such a tile is added row by row.  (A row of 8-bit values that is not finite
            // has a NaN scale, which masks with its weight; its NaN bytes are zeroed.)
            bool rough = false;
            if (__builtin_expect(edge, 0)) {
                const int first = at_use.s.first, len = at_use.s.len;
                const bool several = at_use.s.n > 1;
#pragma unroll 1
                for (int i = lane * 16; i < C::HALF; i += 512) {  // [BOXES][TT][SPAN] bytes
                    const int t = tile_t + i / C::SPAN % TT;
                    uint4 *x = reinterpret_cast<uint4 *>(slots + at * C::SLOT + C::HALF + i);
                    if (t < first || t >= len)
                        *x = make_uint4(0, 0, 0, 0);
                    else if (!Q8 && several)
                        rough |= non_finite<CT>(x->x) || non_finite<CT>(x->y) || non_finite<CT>(x->z) || non_finite<CT>(x->w);
                    else if (CT == GDN_FP8_E4M3 && several)
                        *x = make_uint4(without_nan(x->x), without_nan(x->y), without_nan(x->z), without_nan(x->w));
                }
                ptx::fence_proxy_async_smem();  // (a later tensor copy overwrites what was stored here)
                if (!Q8) rough = __any_sync(FULL, rough);
                __syncwarp();
            }
            // The next tile's scores before this one's output, so that neither waits for the other.
            const int next = at + 1 == S ? 0 : at + 1;
            if (C::AHEAD && use_tile + W < use_end) {
                if (!arrived(next)) return;
                scores(next);
            }
            if (!Q8 && __builtin_expect(rough, 0)) {
#pragma unroll 1
                for (int r = 0; r < rows; ++r) add_values(r, at_use.s.len - at_use.s.n + (at_use.row0 + r) / p.G, Yes());
            } else {
                add_values(0, 0, No());
            }
            __syncwarp();  // all of its readers are behind
            if (lane == 0) ptx::mbar_arrive(used + at);
            at = next;
        }
        {
            // ---- this warp's part of the segment, for the joiners
            if (!arrived(at)) return;
            if (segment > 0 && !ring_wait(j_empty, (segment - 1) & 1, dead)) return;  // the joiners take one segment at a time
            float4 *part = reinterpret_cast<float4 *>(slots + at * C::SLOT);
            float2 *part_stat = reinterpret_cast<float2 *>(extras + (warp * S + at) * C::EXTRA);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
                    x += __shfl_xor_sync(FULL, x, 4);
                    x += __shfl_xor_sync(FULL, x, 8);
                    x += __shfl_xor_sync(FULL, x, 16);
                    const int r = nt * 8 + 2 * c + e;
                    if (g == 0) part_stat[r] = make_float2(m[nt][e], x);
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                        for (int i = 0; i < MPV; i += 2) {
                            const float(&a)[4] = o[nt][vb * MPV + i], (&b)[4] = o[nt][vb * MPV + i + 1];
                            const int x = ((vb * 8 + g) * C::CPL + 2 * i) / 4;
                            part[r * (D / 4) + (x ^ C::part_swizzle(r))] = make_float4(a[e], a[e + 2], b[e], b[e + 2]);
                        }
                }
            if (lane == 0) part_slot[warp] = at;
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(j_full);
                ptx::mbar_arrive(q_empty + (segment & 1));
            }
            at = at + 1 == S ? 0 : at + 1;
        }
    }
}

// ---------------------------------------------------------------- joining split units

constexpr int JOIN_GROUPS = 8, JOIN_BATCH = 4;

// CTA (i, r): row r of the unit whose head CTA i of the attention kernel holds.
// Each of its `groups` groups of D / 4 threads takes every groups-th part, JOIN_BATCH loads in flight.
template <int CT, class C>
__global__ void __launch_bounds__(JOIN_GROUPS * C::D / 4) join_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int D = C::D, ROWS = C::ROWS, LANES = D / 4, BATCH = JOIN_BATCH;
    __shared__ float4 sums[JOIN_GROUPS][LANES];
    __shared__ float2 stats[JOIN_GROUPS];
    const int groups = blockDim.x / LANES;
    dependent_prologue();
    const Parts<C> parts(p.partials, gridDim.x);
    const int i = blockIdx.x, r = blockIdx.y;
    const Split s = parts.split[i];
    if (r >= s.rows || s.parts == 0) return;
    const int x = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 all = make_float2(NONE, 0.f);
    auto add = [&](const float2 (&st)[BATCH], const float4 (&v)[BATCH]) {
        float mm = all.x;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) mm = fmaxf(mm, st[k].x);
        const float f0 = part_factor(all.x, mm);
        sum.x *= f0, sum.y *= f0, sum.z *= f0, sum.w *= f0;
        all = make_float2(mm, all.y * f0);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const float f = part_factor(st[k].x, mm);
            sum.x += f * v[k].x, sum.y += f * v[k].y, sum.z += f * v[k].z, sum.w += f * v[k].w;
            all.y += f * st[k].y;
        }
    };
    for (int k0 = grp; k0 < s.parts; k0 += BATCH * groups) {
        float2 st[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int part = k0 + k * groups;
            st[k] = make_float2(NONE, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (part < s.parts) {
                const long long slot = 2LL * (i + part) + (part == 0);
                st[k] = parts.ml[slot * ROWS + r];
                v[k] = *reinterpret_cast<const float4 *>(parts.o + (slot * ROWS + r) * D + x * 4);
            }
        }
        add(st, v);
    }
    sums[grp][x] = sum;
    if (x == 0) stats[grp] = all;
    __syncthreads();
    if (grp != 0) return;
    for (int k0 = 1; k0 < groups; k0 += BATCH) {
        float2 st[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            st[k] = k0 + k < groups ? stats[k0 + k] : make_float2(NONE, 0.f);
            v[k] = k0 + k < groups ? sums[k0 + k][x] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        add(st, v);
    }
    store_row<CT, C>(p, s.row0 + r, s.head, s.cu0, s.pos0, x * 4, sum, all);
}

template <int CT, int D, int NT>
cudaError_t launch_sized(const PagedAttnParams &p, cudaStream_t stream) {
    using C = Cfg<CT, D, NT>;
    // Tensor copies of the largest power of two of tokens, up to a tile, that never crosses a page; below 8
    // tokens they are so many (a lane issues them one by one) that 16-byte copies of single rows by all lanes
    // are faster: pages of 7 tokens, 8 x 4099 x 8 heads of 64, FP32, took half the time (28 us then, 23 us now).
    int box_tokens = C::TT, box_shift = C::TS == 2 ? 5 : 4;
    while (p.c.page_size % box_tokens) box_tokens >>= 1, --box_shift;
    const bool by_rows = box_tokens < 8;
    if (by_rows) box_tokens = 1, box_shift = 0;
    if constexpr (C::W == 8) {
        // the roles divide what the block is launched with, which has to be all of it
        static int whole = 0;  // 1: it is, -1: not
        if (__atomic_load_n(&whole, __ATOMIC_RELAXED) == 0) {
            cudaFuncAttributes tensor{}, rows{};
            cudaError_t e = cudaFuncGetAttributes(&tensor, paged_attention_kernel<CT, C, false>);
            if (e == cudaSuccess) e = cudaFuncGetAttributes(&rows, paged_attention_kernel<CT, C, true>);
            if (e != cudaSuccess) return e;
            const bool ok = tensor.numRegs == C::LAUNCH_REGS && rows.numRegs == C::LAUNCH_REGS;
            __atomic_store_n(&whole, ok ? 1 : -1, __ATOMIC_RELAXED);
        }
        if (__atomic_load_n(&whole, __ATOMIC_RELAXED) < 0) return cudaErrorInvalidConfiguration;
    }
    auto kernel = by_rows ? paged_attention_kernel<CT, C, true> : paged_attention_kernel<CT, C, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int spans = box_tokens == C::TT ? C::BOXES : 1;  // whole tiles land in one copy
    CUtensorMap k_map{}, v_map{};
    if (!by_rows &&
        (!encode_cache_rows(&k_map, p.c.k, C::ESZ, D, p.c.H, p.c.page_size, p.c.num_pages, p.c.head_stride, p.c.token_stride,
                            p.c.page_stride, box_tokens, spans) ||
         !encode_cache_rows(&v_map, p.c.v, C::ESZ, D, p.c.H, p.c.page_size, p.c.num_pages, p.c.head_stride, p.c.token_stride,
                            p.c.page_stride, box_tokens, spans)))
        return cudaErrorInvalidValue;
    const unsigned ctas = (unsigned)attention_ctas();
    const cudaError_t e2 =
        launch_dependent(kernel, dim3(ctas), dim3(C::THREADS), C::SMEM, stream, p, k_map, v_map, box_shift);
    // a unit of one chunk is never split
    if (e2 != cudaSuccess || (long long)p.pages_per_seq * p.c.page_size <= C::W * C::TT) return e2;
    // As many groups a row as one batch of theirs needs for the parts of a unit (CTAs with small shares of the work
    // join little): with 8 always, whose CTAs do not all fit at once, draft verification took 49.5 us instead of
    // 45.8 us and 16 x 512 tokens 10.9 us instead of 9.6 us; with 2 always one key head of 131071 tokens 31 us instead of 22 us.
    const long long units = (long long)p.B * p.c.H * ((p.rows_hint + C::ROWS - 1) / C::ROWS), most = ctas / units + 2;
    int groups = D == 64 ? 2 : 1;
    while (groups < JOIN_GROUPS && groups * JOIN_BATCH < most) groups *= 2;
    return launch_dependent(join_kernel<CT, C>, dim3(ctas, C::ROWS), dim3(groups * D / 4), 0, stream, p);
}

// Query rows a pass: 8 where one key head has no more, else 16 (fewer idle columns
// against fewer passes over the cache).
template <int CT, int D>
cudaError_t launch_dim(const PagedAttnParams &p, cudaStream_t stream) {
    constexpr int MAX = max_row_tiles(CT == GDN_F32, D);
    const int nt = row_tiles(CT == GDN_F32, D, p.rows_hint);
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
