// What the forward and the backward kernel of the gated linear recurrence share: tiles of
// tokens and channels, the packing's effect on a tile, and the scan over a cluster's tiles.
//
// Per channel h_t = g_t h_(t-1) + u_t maps the state in front of a run of tokens affinely
// to the one behind it, h -> A h + B.  A cluster of CTAs takes a slab of channels through
// all packed tokens, a tile of TILE tokens a CTA at a time; a half-warp takes TT tokens of
// its CTA's tile, a lane VC channels.  Each half-warp works out its own (A, B) and every
// state with nothing in front; the CTA folds its half-warps' maps in order and gives the
// result to all CTAs of the cluster, which fold those in order behind the carry of the
// tiles before.  Every input is read once and every output written once, nothing passes
// through global memory between CTAs, and the order of all sums is fixed.
//
// Sequences only matter at their ends.  A token that begins one (or belongs to none)
// resets the state: what stands in front of it is not multiplied by 0 but left out, so
// infinities and NaN of one sequence do not reach the next.
#pragma once

#include <type_traits>

#include "layer_internal.cuh"
#include "ptx.cuh"

namespace gdn {
namespace recur {

constexpr int CHECK = GDN_RECURRENCE_CHECKPOINT;
constexpr int LANES = 16;  // lanes beside one another along the channels
constexpr int MAX_CLUSTER = 16;  // (8 is what every device takes)
enum { RESET = 1, LOAD = 2, LAST = 4, VALID = 8 };  // LOAD: a sequence begins here; RESET: so, or no sequence's token

// The largest b in [0, hi] with cu[b] <= t (0 if there is none).
__device__ __forceinline__ int last_start(const int32_t *cu, int hi, int t) {
    int lo = 0;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The packing, in shared memory if it is short: every tile looks its tokens up in it.  (Room for 512 sequences took the
// L1 cache down a step, and rows that are copied 4 bytes at a time from 33 to 44 us.)
constexpr int STAGED = 64;
struct Packing {
    int cu[STAGED + 1], slots[STAGED];
};
struct Lookup {
    const int32_t *cu, *slots;
};
// (the caller synchronises the CTA after it)
__device__ __forceinline__ Lookup stage_packing(const RecurrenceParams &p, Packing &k) {
    Lookup l = {p.cu, p.slots};
    if (!p.cu || p.B > STAGED) return l;
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) {
        k.cu[b] = p.cu[b];
        if (p.slots && b < p.B) k.slots[b] = p.slots[b];
    }
    l.cu = k.cu;
    if (p.slots) l.slots = k.slots;
    return l;
}

// What token t is, its sequence's slot, and the tokens from it to its sequence's end.
__device__ __forceinline__ int token_of(const RecurrenceParams &p, const Lookup &l, int t, bool flag, int &slot, int &rest) {
    slot = rest = 0;
    if (t >= p.T || p.B == 0) return RESET;
    int b, begin, end;
    if (l.cu) {
        b = last_start(l.cu, p.B - 1, t);
        begin = l.cu[b];
        end = l.cu[b + 1];
    } else {
        b = t / p.S;
        begin = b * p.S;
        end = begin + p.S;
    }
    if (t < begin || t >= end || end > p.T) return RESET;  // (the last: a packing out of order)
    slot = l.slots ? l.slots[b] : b;
    if (slot < 0 || slot >= p.num_slots) {
        if (flag) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
        slot = 0;
        return RESET;
    }
    rest = end - t;
    return VALID | (t == begin ? RESET | LOAD : 0) | (t == end - 1 ? LAST : 0);
}

// Which of a tile's tokens are what, a bit a token, and their slots.
template <int TILE>
struct Tokens {
    int plain;  // the tile lies inside a sequence, without its first and last token: the rest is not set
    unsigned reset[TILE / 32], load[TILE / 32], last[TILE / 32], valid[TILE / 32];
    int slot[TILE];
};

// Fills them for the tile at t0 (TILE / 32 warps, w: which of them).
template <int TILE>
__device__ __forceinline__ void tokens_of(Tokens<TILE> &k, const RecurrenceParams &p, const Lookup &l, int t0, bool flag, int w) {
    if (w < 0) return;
    const int lane = threadIdx.x % 32;
    int slot, rest;
    int what = token_of(p, l, t0, flag, slot, rest);
    const bool plain = what == VALID && rest > TILE;
    if (w == 0 && lane == 0) k.plain = plain;
    if (plain) return;
    what = token_of(p, l, t0 + 32 * w + lane, flag, slot, rest);
    k.slot[32 * w + lane] = slot;
    const unsigned reset = __ballot_sync(0xffffffffu, what & RESET), load = __ballot_sync(0xffffffffu, what & LOAD);
    const unsigned last = __ballot_sync(0xffffffffu, what & LAST), valid = __ballot_sync(0xffffffffu, what & VALID);
    if (lane == 0) {
        k.reset[w] = reset;
        k.load[w] = load;
        k.last[w] = last;
        k.valid[w] = valid;
    }
}

// The bits of run `sub` of TT tokens.
template <int TT>
__device__ __forceinline__ unsigned bits_of(const unsigned *words, int sub) {
    return words[sub * TT / 32] >> (sub * TT % 32) & ((1u << TT) - 1);
}

// The packing's own checks, by one CTA of a call.
__device__ __forceinline__ void check_packing(const RecurrenceParams &p) {
    if (!p.cu) return;
    bool bad = threadIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.B] != p.T);
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) bad |= p.cu[b] > p.cu[b + 1];
    if (bad) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
}

// ---------------------------------------------------------------- copies into shared memory

template <int BYTES>
__device__ __forceinline__ void copy(void *dst, const void *src, bool in) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(in ? 8 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A thread copies one column of its pieces, every ROWS-th row.
template <typename E, int SLAB, int TILE, int NT, int BYTES>
__device__ __forceinline__ void copy_tile(E *dst, const E *base, long long stride, int t0, int T, int c0, int C) {
    constexpr int N = BYTES / (int)sizeof(E), ROW = SLAB / N, ROWS = NT / ROW;
    static_assert(NT % ROW == 0 && TILE % ROWS == 0, "whole rows, the same number for every thread");
    const int r = threadIdx.x / ROW, c = threadIdx.x % ROW * N;
    const bool column = c0 + c < C;
    int left = T - t0 - r;
    const E *src = base + (long long)(t0 + r) * stride + (c0 + c);
    dst += r * SLAB + c;
    stride *= ROWS;
#pragma unroll
    for (int k = 0; k < TILE / ROWS; ++k) {
        const bool in = column && left > 0;
        copy<BYTES>(dst, in ? src : base, in);
        src += stride;
        dst += ROWS * SLAB;
        left -= ROWS;
    }
}

// A tile of E's, [TILE][SLAB], from rows `stride` apart; zeros past T and C.  bytes: what base, stride and C are whole
// multiples of: 8, 4, or less (what 16 divides comes by tensor copies, or 8 bytes at a time).
template <typename E, int SLAB, int TILE, int NT>
__device__ __forceinline__ void load_tile(E *dst, const void *base, long long stride, int t0, int T, int c0, int C, int bytes) {
    const E *src = static_cast<const E *>(base);
    if (bytes == 8) {
        copy_tile<E, SLAB, TILE, NT, 8>(dst, src, stride, t0, T, c0, C);
    } else if (bytes == 4) {
        copy_tile<E, SLAB, TILE, NT, 4>(dst, src, stride, t0, T, c0, C);
    } else {
        src += (long long)t0 * stride + c0;
#pragma unroll 16
        for (int i = threadIdx.x; i < TILE * SLAB; i += NT) {
            const int r = i / SLAB, c = i % SLAB;
            dst[i] = t0 + r < T && c0 + c < C ? src[r * stride + c] : from_f32<E>(0.f);
        }
    }
}

// Brings such a tile's rows to L2 (the first and the last channel's line of each) for plain loads, which wait for what they load
// (65,536 BF16 tokens of 1001 channels backwards: 1080 -> 932 us).
template <typename E, int SLAB, int TILE, int NT>
__device__ __forceinline__ void prefetch_tile(const void *base, long long stride, int t0, int T, int c0, int C) {
    const int last = min(SLAB, C - c0) - 1;
    for (int i = threadIdx.x; i < 2 * TILE; i += NT) {
        if (t0 + i / 2 >= T) break;
        const E *p = static_cast<const E *>(base) + (long long)(t0 + i / 2) * stride + c0 + (i % 2 ? last : 0);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
}

// Tensor map of such rows for boxes of a tile; false if the driver does not take it.
template <typename E, int SLAB, int TILE>
bool tile_map(CUtensorMap *map, const void *base, long long stride, int T, long long C) {
    if constexpr (sizeof(E) == 2) return encode_rows_f16(map, base, C, stride, T, SLAB, TILE, false);
    else return encode_rows_f32_strided(map, static_cast<const float *>(base), C, stride, T, SLAB, TILE);
}

// 16, 8 or 4 if address and rows are whole multiples of it, else 2; for rows of C elements `stride` apart.
inline int whole_bytes(const void *ptr, long long stride, long long C, size_t elem) {
    const unsigned long long all = reinterpret_cast<uintptr_t>(ptr) | (unsigned long long)stride * elem | (unsigned long long)C * elem;
    return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}
// Whether rows of C elements without gaps can be accessed `bytes` at a time.
inline bool whole_rows(const void *ptr, long long C, size_t elem, size_t bytes) {
    return (reinterpret_cast<uintptr_t>(ptr) | (unsigned long long)C * elem) % bytes == 0;
}

// ---------------------------------------------------------------- accesses of VC neighbouring elements

template <typename E, int VC>
union Pack {
    E e[VC];
    uint4 u4;
    uint2 u2;
    uint32_t u1, words[4];
    __device__ __forceinline__ Pack() {}
};

// In one access.
template <typename E, int VC>
__device__ __forceinline__ void read(const E *src, float (&f)[VC]) {
    Pack<E, VC> v;
    if constexpr (sizeof(E) * VC == 16) v.u4 = *reinterpret_cast<const uint4 *>(src);
    else if constexpr (sizeof(E) * VC == 8) v.u2 = *reinterpret_cast<const uint2 *>(src);
    else if constexpr (sizeof(E) * VC == 4) v.u1 = *reinterpret_cast<const uint32_t *>(src);
    else v.e[0] = *src;
    if constexpr (std::is_same<E, __nv_bfloat16>::value && VC % 2 == 0) {
        // (an instruction a number: BF16 is the upper half of FP32)
#pragma unroll
        for (int i = 0; i < VC; i += 2) {
            f[i] = __uint_as_float(v.words[i / 2] << 16);
            f[i + 1] = __uint_as_float(v.words[i / 2] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VC; ++i) f[i] = to_f32(v.e[i]);
    }
}

template <typename E, int PAIRS>
__device__ __forceinline__ void pairs_of(const E *src, F2 (&f)[PAIRS]) {
    float g[2 * PAIRS];
    read<E, 2 * PAIRS>(src, g);
#pragma unroll
    for (int v = 0; v < PAIRS; ++v) f[v] = F2(g[2 * v], g[2 * v + 1]);
}

template <int VC>
__device__ __forceinline__ void put_pack(float *dst, const Pack<float, VC> &v) {
    if constexpr (VC == 4) *reinterpret_cast<uint4 *>(dst) = v.u4;
    else *reinterpret_cast<uint2 *>(dst) = v.u2;
}

template <typename E, int VC>
__device__ __forceinline__ void pack(Pack<E, VC> &v, const float (&f)[VC]) {
    if constexpr (sizeof(E) == 2 && VC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VC; i += 2) {
            uint32_t two;
            if constexpr (std::is_same<E, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(two) : "f"(f[i + 1]), "f"(f[i]));
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(two) : "f"(f[i + 1]), "f"(f[i]));
            v.words[i / 2] = two;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VC; ++i) v.e[i] = from_f32<E>(f[i]);
    }
}

// `inside` of them at most; vec: they are aligned, and all inside or none.
template <typename E, int VC>
__device__ __forceinline__ void store(E *dst, const float (&f)[VC], int inside, bool vec) {
    Pack<E, VC> v;
    pack(v, f);
    if (vec) {
        if (inside <= 0) return;
        if constexpr (sizeof(E) * VC == 16) *reinterpret_cast<uint4 *>(dst) = v.u4;
        else if constexpr (sizeof(E) * VC == 8) *reinterpret_cast<uint2 *>(dst) = v.u2;
        else if constexpr (sizeof(E) * VC == 4) *reinterpret_cast<uint32_t *>(dst) = v.u1;
        else dst[0] = v.e[0];
    } else {
#pragma unroll
        for (int i = 0; i < VC; ++i)
            if (i < inside) dst[i] = v.e[i];
    }
}

template <int VC>
__device__ __forceinline__ void load(const float *src, float (&f)[VC], int inside, bool vec) {
    if (vec && inside > 0) {
        read<float, VC>(src, f);
    } else {
#pragma unroll
        for (int i = 0; i < VC; ++i) f[i] = i < inside ? src[i] : 0.f;
    }
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p`, in this CTA's shared memory, in that of CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void store_cluster(uint32_t a, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
// 8 bytes to another CTA's shared memory, counted by the barrier there.
__device__ __forceinline__ void store_async(uint32_t a, uint32_t bar, float x, float y) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(a), "f"(x), "f"(y), "r"(bar)
                 : "memory");
}

// What the CTAs of a cluster tell one another about their tiles: each channel's map (A, B), or A = NaN if a reset
// closes the tile, so that nothing from in front of it comes through (where an A is NaN by itself, B is too).  Twice, for a round and the next.
template <int SLAB>
struct Exchange {
    alignas(16) float2 map[2][MAX_CLUSTER][SLAB];
    alignas(8) uint64_t full[2];
};

// Waits for a phase of `bar`; after about a second without it the caller goes on and the status word says so.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, int32_t *status) {
    if (!ptx::mbar_wait_bounded(bar, parity, 2000000000ll)) flag_error(status, GDN_DEVERR_TIMEOUT);
}

// The same for a barrier that other CTAs' stores complete.
__device__ __forceinline__ void wait_cluster(uint64_t *bar, uint32_t parity, int32_t *status) {
    const long long t0 = clock64();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(ptx::smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return;
        if (clock64() - t0 > 2000000000ll) break;
    }
    flag_error(status, GDN_DEVERR_TIMEOUT);
}

// Thread c of SLAB: channel c's map of this CTA's tile to every CTA; returns what stands in front of the tile, given what
// stands in front of the cluster's (`run`, which becomes what stands behind them).  FORWARD: tiles in the order of the ranks.
template <bool FORWARD, int SLAB>
__device__ __forceinline__ float exchange(Exchange<SLAB> &x, int n, int cluster, int rank, int c, float A, float B, bool closed,
                                          float &run, int32_t *status) {
    const int buf = n & 1;
    uint64_t *bar = &x.full[buf];
    if (c == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)cluster * SLAB * 8);
    if (closed) A = __int_as_float(0x7fc00000);
#pragma unroll 1
    for (int r = 0; r < cluster; ++r) store_async(in_cta(&x.map[buf][rank][c], r), in_cta(bar, r), A, B);
    wait_cluster(bar, n >> 1 & 1, status);
    float front = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < cluster; k0 += 4) {  // four loads at once: their latency is what a round waits for
        float2 m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = min(k0 + k, cluster - 1);
            m[k] = x.map[buf][FORWARD ? r : cluster - 1 - r][c];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k0 + k >= cluster) break;
            if ((FORWARD ? k0 + k : cluster - 1 - k0 - k) == rank) front = run;
            run = isnan(m[k].x) ? m[k].y : fmaf(m[k].x, run, m[k].y);
        }
    }
    return front;
}

// A cluster's launch as a programmatic dependent (launch_dependent with clusters).
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned clusters, unsigned size, unsigned threads, size_t smem,
                            cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

// Clusters of each size (1 to MAX_CLUSTER) of a kernel that are resident at once on the current device.
struct Resident {
    int most[MAX_CLUSTER + 1];
};
template <typename Kernel>
cudaError_t resident_clusters(Kernel kernel, unsigned threads, size_t smem, Resident &out) {
    for (int size = 1; size <= MAX_CLUSTER; ++size) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = size;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&out.most[size], kernel, &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// CTAs a cluster: the largest size at which all clusters are resident at once and has no more CTAs than tiles, or the least
// of as few rounds.  (A size at which some clusters wait for others: 1.4 times as long.)
inline int cluster_size(const Resident &r, long long slabs, long long tiles) {
    int size = 1;
    for (int s = 2; s <= MAX_CLUSTER && s <= tiles; ++s)
        if (slabs <= r.most[s]) size = s;
    const long long rounds = (tiles + size - 1) / size;
    return tiles ? (int)((tiles + rounds - 1) / rounds) : 1;
}

// Two channels a lane instead of four where slabs of four are few: up to 1600 channels.  BF16, raw, us forwards / backwards
// with two and with four:
//   16,384 tokens   512: 32 / 70 and 37 / 77, 1024: 42 / 93 and 46 / 96, 1536: 55 / 126 and 56 / 118,
//                   2048: 72 / 163 and 66 / 141, 2560: 83 / 192 and 85 / 180, 4096: 128 / 302 and 118 / 256
//   2048 tokens     1024: 9.7 / 17.9 and 11.7 / 18.2, 1536: 10.9 / 21.3 and 12.2 / 21.7, 2048: 14.1 / 27.7 and 12.5 / 23.1
// The rule looks at the channels alone and takes the slower form in places: backwards at 1536 from 4000 tokens on (39.0 instead
// of 35.6 at 4131), forwards with unit input past 1600 (4131 tokens: 2048 28.3 instead of 26.0, 4096 45.6 instead of 42.9).
inline bool narrow_slabs(long long C) {
    constexpr int SLAB = 4 * LANES;
    return (C + SLAB - 1) / SLAB * 6 <= current_device_sms();
}

// A kernel's shared memory set and its residency looked up, once a device (as current_device_sms); a template of
// what tells the kernels apart, since they share a type.
template <typename T, int MODE, int VC, typename Kernel>
cudaError_t prepare_clusters(Kernel kernel, unsigned threads, size_t smem, const Resident **out) {
    constexpr int kMaxDevices = 128;
    static Resident known[kMaxDevices];
    static int ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        Resident r;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        if ((e = resident_clusters(kernel, threads, smem, r)) != cudaSuccess) return e;
        known[dev] = r;  // (two threads that come here at once write the same)
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    *out = &known[dev];
    return cudaSuccess;
}

}  // namespace recur
}  // namespace gdn
