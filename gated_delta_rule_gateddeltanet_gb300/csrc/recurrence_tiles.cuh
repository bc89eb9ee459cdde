// What the forward and the backward kernel of the gated linear recurrence share: tiles of
// tokens and channels, the packing's effect on a tile, and the scan over tiles.
//
// Per channel h_t = g_t h_(t-1) + u_t maps the state in front of a run of tokens affinely
// to the one behind it, h -> A h + B.  A tile is TILE packed tokens of a slab of 32 VC
// channels; its warps take TT tokens each, a lane VC channels.  Each warp works out its own
// (A, B) and every state with nothing in front, the tile folds its warps' maps in order,
// and the carry into the tile comes from the tiles before it: a tile publishes its (A, B)
// as soon as it has them and the state behind it once it knows the one in front, and looks
// back over the former to the nearest of the latter.  The maps are applied one after
// another in order, wherever that begins, so the results do not depend on which tiles were
// ready.  Every input is read once and every output written once.
//
// Sequences only matter at their ends.  A token that begins one (or belongs to none)
// resets the state: what stands in front of it is not multiplied by 0 but left out, so
// infinities and NaN of one sequence do not reach the next.  A tile that holds a reset
// knows the state behind it at once, which cuts the chain.
//
// Tiles are handed out in order by a counter, so that a tile only ever waits for tiles
// that a running CTA already has; the waits are bounded all the same.
#pragma once

#include "layer_internal.cuh"

namespace gdn {
namespace recur {

constexpr int TILE = GDN_RECURRENCE_CHECKPOINT;
enum { RESET = 1, LOAD = 2, LAST = 4, VALID = 8 };  // LOAD: a sequence begins here; RESET: so, or no sequence's token

// Workspace: counter, flags, first sequences, maps and states of the tiles (floats).
struct Layout {
    long long tiles, time_tiles, slabs;
    size_t flags, first, maps, states, sums, bytes;
};

inline Layout layout(int T, int C, int slab, bool sums) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout l;
    l.time_tiles = ((long long)T + TILE - 1) / TILE;
    l.slabs = ((long long)C + slab - 1) / slab;
    l.tiles = l.time_tiles * l.slabs;
    l.flags = 256;
    l.first = l.flags + up(4 * (size_t)l.tiles);
    l.maps = l.first + up(4 * (size_t)(l.time_tiles + 1));
    l.states = l.maps + (l.time_tiles > 1 ? 8 * (size_t)l.tiles * slab : 0);
    l.sums = l.states + (l.time_tiles > 1 ? 4 * (size_t)l.tiles * slab : 0);
    l.bytes = l.sums + (sums ? 8 * (size_t)l.time_tiles * l.slabs * slab : 0);
    return l;
}

// Device view of it.
struct Work {
    int32_t *counter, *flags, *first;
    float *maps, *states, *sums;
    int time_tiles, slabs, tiles;
};

inline Work work_of(void *workspace, const Layout &l) {
    char *w = static_cast<char *>(workspace);
    Work k;
    k.counter = reinterpret_cast<int32_t *>(w);
    k.flags = reinterpret_cast<int32_t *>(w + l.flags);
    k.first = reinterpret_cast<int32_t *>(w + l.first);
    k.maps = reinterpret_cast<float *>(w + l.maps);
    k.states = reinterpret_cast<float *>(w + l.states);
    k.sums = reinterpret_cast<float *>(w + l.sums);
    k.time_tiles = (int)l.time_tiles;
    k.slabs = (int)l.slabs;
    k.tiles = (int)l.tiles;
    return k;
}

// The largest b in [lo, hi] with cu[b] <= t (lo if there is none).
__device__ __forceinline__ int last_start(const int32_t *cu, int lo, int hi, int t) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The sequence of every tile's first token, cleared flags and counter, and the packing's checks.
constexpr int PLAN_THREADS = 256;
__global__ void plan_kernel(const RecurrenceParams p, const Work k);

// What each token of tile j is (threads 0 .. TILE - 1).
__device__ __forceinline__ void token_of(const RecurrenceParams &p, const Work &k, int j, bool flag, int &what, int &slot) {
    const int i = threadIdx.x, t = j * TILE + i;
    what = RESET;
    slot = 0;
    if (t >= p.T) return;
    int b, begin, end;
    if (p.cu) {
        const int lo = k.time_tiles > 1 ? k.first[j] : 0, hi = k.time_tiles > 1 ? k.first[j + 1] : p.B - 1;
        b = last_start(p.cu, lo, hi, t);
        begin = p.cu[b];
        end = p.cu[b + 1];
    } else {
        b = t / p.S;
        begin = b * p.S;
        end = begin + p.S;
    }
    if (t < begin || t >= end) return;
    slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.num_slots) {
        if (flag) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
        slot = 0;
        return;
    }
    what = VALID | (t == begin ? RESET | LOAD : 0) | (t == end - 1 ? LAST : 0);
}

// ---------------------------------------------------------------- copies into shared memory

__device__ __forceinline__ void copy16(void *dst, const void *src, bool in) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src, bool in) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A tile of E's, [TILE][SLAB], from rows `stride` apart; zeros past T and C.  vec: base, stride and C are
// whole 16 bytes.  Threads tid of `threads`.
template <typename E, int SLAB>
__device__ __forceinline__ void load_tile(E *dst, const void *base, long long stride, int t0, int T, int c0, int C, bool vec,
                                          int tid, int threads) {
    const E *src = static_cast<const E *>(base) + (long long)t0 * stride + c0;
    if (vec) {
        constexpr int N = 16 / (int)sizeof(E), ROW = SLAB / N;
#pragma unroll 4
        for (int i = tid; i < TILE * ROW; i += threads) {
            const int r = i / ROW, c = i % ROW * N;
            const bool in = t0 + r < T && c0 + c < C;
            copy16(dst + r * SLAB + c, in ? src + r * stride + c : base, in);
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < TILE * SLAB; i += threads) {
            const int r = i / SLAB, c = i % SLAB;
            dst[i] = t0 + r < T && c0 + c < C ? src[r * stride + c] : from_f32<E>(0.f);
        }
    }
}

// SLAB floats, zeros past C.
template <int SLAB>
__device__ __forceinline__ void load_row(float *dst, const float *src, int c0, int C, int tid, int threads) {
    for (int i = tid; i < SLAB; i += threads) copy4(dst + i, c0 + i < C ? src + c0 + i : src, c0 + i < C);
}

// VC neighbouring elements as floats, in one access.
template <typename E, int VC>
__device__ __forceinline__ void read(const E *src, float (&f)[VC]) {
    union {
        E e[VC];
        uint4 u4;
        uint2 u2;
        uint32_t u1;
    } v;
    if constexpr (sizeof(E) * VC == 16) v.u4 = *reinterpret_cast<const uint4 *>(src);
    else if constexpr (sizeof(E) * VC == 8) v.u2 = *reinterpret_cast<const uint2 *>(src);
    else if constexpr (sizeof(E) * VC == 4) v.u1 = *reinterpret_cast<const uint32_t *>(src);
    else v.e[0] = *src;
#pragma unroll
    for (int i = 0; i < VC; ++i) f[i] = to_f32(v.e[i]);
}

// VC neighbouring elements of a row to memory; vec: they are aligned and all inside.
template <typename E, int VC>
__device__ __forceinline__ void store(E *dst, const float (&f)[VC], int inside, bool vec) {
    union {
        E e[VC];
        uint4 u4;
        uint2 u2;
        uint32_t u1;
    } v;
#pragma unroll
    for (int i = 0; i < VC; ++i) v.e[i] = from_f32<E>(f[i]);
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

// ---------------------------------------------------------------- the scan over tiles

__device__ __forceinline__ int load_acquire(const int32_t *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int32_t *p, int v) {
    asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <int VC>
__device__ __forceinline__ void put(float *dst, const float (&f)[VC]) {
    if constexpr (VC == 4) __stcg(reinterpret_cast<float4 *>(dst), make_float4(f[0], f[1], f[2], f[3]));
    else __stcg(reinterpret_cast<float2 *>(dst), make_float2(f[0], f[1]));
}
template <int VC>
__device__ __forceinline__ void get(const float *src, float (&f)[VC]) {
    if constexpr (VC == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
        f[0] = v.x, f[1] = v.y;
    }
}

enum { NOT_YET = 0, MAP = 1, STATE = 2 };
// Polls (about a second) after which a wait gives up.
constexpr int WAIT_LIMIT = 1 << 20;

// One warp: the tile in place `seq` of its slab's chain has the map (A, B); `closed`: its result does not depend on what
// stands in front (it holds a reset); `open`: it needs the state in front; `follow`: a tile comes after it.
// Returns the state in front in `carry` (0 if it does not need one).
template <int VC>
__device__ __forceinline__ void chain(const Work &k, int seq, int slab, const float (&A)[VC], const float (&B)[VC], bool closed,
                                      bool open, bool follow, int32_t *status, float (&carry)[VC]) {
    const int lane = threadIdx.x % 32;
    const long long me = (long long)seq * k.slabs + slab;
    constexpr int SLAB = 32 * VC;
    auto state = [&](long long tile) { return k.states + tile * SLAB + lane * VC; };
    auto map = [&](long long tile) { return k.maps + tile * 2 * SLAB + lane * VC; };
    auto publish = [&](int what) {
        __syncwarp();
        if (lane == 0) store_release(k.flags + me, what);
    };
    if (follow) {
        if (closed || !open) {
            put<VC>(state(me), B);
            publish(STATE);
        } else {
            put<VC>(map(me), A);
            put<VC>(map(me) + SLAB, B);
            publish(MAP);
        }
    }
#pragma unroll
    for (int i = 0; i < VC; ++i) carry[i] = 0.f;
    if (!open) return;
    int at = -1;
    for (int n = 0;; ++n) {
        const int before = seq - 1 - lane;
        const int f = before >= 0 ? load_acquire(k.flags + (long long)before * k.slabs + slab) : NOT_YET;
        const unsigned states = __ballot_sync(0xffffffffu, f == STATE), some = __ballot_sync(0xffffffffu, f != NOT_YET);
        if (states) {
            const int nearest = __ffs(states) - 1;
            if ((~some & ((1u << nearest) - 1)) == 0) {
                at = nearest;
                break;
            }
        }
        if (n >= WAIT_LIMIT) break;
    }
    __syncwarp();
    if (at < 0) {
        if (lane == 0) flag_error(status, GDN_DEVERR_TIMEOUT);
#pragma unroll
        for (int i = 0; i < VC; ++i) carry[i] = __int_as_float(0x7fc00000);
    } else {
        get<VC>(state(me - (long long)(at + 1) * k.slabs), carry);
#pragma unroll 4
        for (; at > 0; --at) {
            float a[VC], b[VC];
            get<VC>(map(me - (long long)at * k.slabs), a);
            get<VC>(map(me - (long long)at * k.slabs) + SLAB, b);
#pragma unroll
            for (int i = 0; i < VC; ++i) carry[i] = fmaf(a[i], carry[i], b[i]);
        }
    }
    if (follow && !closed) {
        float s[VC];
#pragma unroll
        for (int i = 0; i < VC; ++i) s[i] = fmaf(A[i], carry[i], B[i]);
        put<VC>(state(me), s);
        publish(STATE);
    }
}

}  // namespace recur
}  // namespace gdn
