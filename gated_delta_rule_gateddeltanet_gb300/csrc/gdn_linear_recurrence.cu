// The gated linear recurrence, forward: h_t = g_t h_(t-1) + w_t x_t a channel.
#include "recurrence_tiles.cuh"

namespace gdn {
namespace recur {

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const RecurrenceParams p, const Work k) {
    dependent_prologue();
    const int i = blockIdx.x * PLAN_THREADS + threadIdx.x;
    if (i == 0) {
        *k.counter = 0;
        if (p.cu && (p.cu[0] != 0 || p.cu[p.B] != p.T)) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    }
    if (i < k.tiles) k.flags[i] = NOT_YET;
    if (!p.cu) return;
    if (i <= k.time_tiles) k.first[i] = last_start(p.cu, 0, p.B - 1, min(i * (long long)TILE, (long long)p.T - 1));
    if (i < p.B && p.cu[i] > p.cu[i + 1]) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
}

}  // namespace recur

namespace {

using namespace recur;

// ---------------------------------------------------------------- long sequences

constexpr int TT = 8, W = TILE / TT, NT = 32 * W;

enum { VEC_X = 1, VEC_A = 2, VEC_B = 4, VEC_Y = 8, VEC_STATE = 16 };

template <typename T, int MODE>
struct Shape {
    using G = typename GateType<T, MODE>::type;
    static constexpr int VC = sizeof(G) == 4 ? 2 : 4, SLAB = 32 * VC;
    struct Shared {
        T x[TILE * SLAB];
        G a[TILE * SLAB], b[TILE * SLAB];
        float A_log[SLAB], dt_bias[SLAB];
        float A[W][SLAB], B[W][SLAB];  // the warps' maps, then those of what stands in front of each in the tile
        float carry[SLAB];
        int what[2][TILE], slot[2][TILE];
        int resets[W + 1];  // whether a warp's tokens hold a reset; whether one stands before a warp's in the tile
        int next;
    };
};

template <typename T, int MODE>
__global__ void __launch_bounds__(NT, 2) recurrence_tile_kernel(const RecurrenceParams p, const Work k, int vec) {
    dependent_prologue();
    using S = Shape<T, MODE>;
    using G = typename S::G;
    constexpr int VC = S::VC, SLAB = S::SLAB;
    extern __shared__ __align__(16) unsigned char raw[];
    typename S::Shared &sm = *reinterpret_cast<typename S::Shared *>(raw);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool chained = k.time_tiles > 1, has_b = p.b != nullptr;

    auto fetch = [&](int tile, int buf, int tid, int threads) {
        const int j = tile / k.slabs, c0 = (tile - j * k.slabs) * SLAB, t0 = j * TILE;
        load_tile<T, SLAB>(sm.x, p.x, p.x_stride, t0, p.T, c0, p.C, vec & VEC_X, tid, threads);
        load_tile<G, SLAB>(sm.a, p.a, p.a_stride, t0, p.T, c0, p.C, vec & VEC_A, tid, threads);
        if (has_b) load_tile<G, SLAB>(sm.b, p.b, p.b_stride, t0, p.T, c0, p.C, vec & VEC_B, tid, threads);
        if (MODE != RECUR_PRECOMPUTED) {
            load_row<SLAB>(sm.A_log, p.A_log, c0, p.C, tid, threads);
            load_row<SLAB>(sm.dt_bias, p.dt_bias, c0, p.C, tid, threads);
        }
    };
    auto tokens = [&](int tile, int buf) {
        if (threadIdx.x >= TILE) return;
        int what, slot;
        token_of(p, k, tile / k.slabs, tile % k.slabs == 0, what, slot);
        sm.what[buf][threadIdx.x] = what;
        sm.slot[buf][threadIdx.x] = slot;
    };

    int cur = blockIdx.x, nxt = k.tiles;
    if (chained) {
        if (threadIdx.x == 0) {
            cur = atomicAdd(k.counter, 1);
            nxt = atomicAdd(k.counter, 1);
            sm.resets[0] = cur;
            sm.next = nxt;
        }
        __syncthreads();
        cur = sm.resets[0];
        nxt = sm.next;
        __syncthreads();
    }
    if (cur < k.tiles) {
        fetch(cur, 0, threadIdx.x, NT);
        tokens(cur, 0);
    }
    for (int buf = 0; cur < k.tiles; buf ^= 1) {
        const int j = cur / k.slabs, slab = cur - j * k.slabs, c0 = slab * SLAB + lane * VC, inside = p.C - c0;
        copies_done();
        __syncthreads();

        // every token's state and decay with nothing in front of the warp's tokens
        float h[TT][VC], P[TT][VC];
        unsigned after = 0;  // tokens at or behind a reset among the warp's
        {
            float rate[VC], dt[VC];
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                rate[v] = MODE ? expf(sm.A_log[lane * VC + v]) : 0.f;
                dt[v] = MODE ? sm.dt_bias[lane * VC + v] : 0.f;
            }
            bool reset = false;
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const int r = warp * TT + i, what = sm.what[buf][r];
                float x[VC], a[VC], b[VC] = {};
                read<T, VC>(sm.x + r * SLAB + lane * VC, x);
                read<G, VC>(sm.a + r * SLAB + lane * VC, a);
                if (has_b) read<G, VC>(sm.b + r * SLAB + lane * VC, b);
                float g[VC], u[VC];
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const Gate q = gate_of<MODE>(a[v], b[v], rate[v], dt[v], has_b);
                    g[v] = q.g;
                    u[v] = q.w * x[v];
                }
                if (what & RESET) {
                    float h0[VC] = {};
                    if ((what & LOAD) && p.init)
                        load<VC>(p.init + (long long)sm.slot[buf][r] * p.C + c0, h0, inside, vec & VEC_STATE);
                    reset = true;
#pragma unroll
                    for (int v = 0; v < VC; ++v) {
                        h[i][v] = what & VALID ? fmaf(g[v], h0[v], u[v]) : 0.f;
                        P[i][v] = 0.f;
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < VC; ++v) {
                        h[i][v] = i ? fmaf(g[v], h[i - 1][v], u[v]) : u[v];
                        P[i][v] = i ? g[v] * P[i - 1][v] : g[v];
                    }
                }
                if (reset) after |= 1u << i;
            }
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                sm.A[warp][lane * VC + v] = P[TT - 1][v];
                sm.B[warp][lane * VC + v] = h[TT - 1][v];
            }
            if (lane == 0) sm.resets[warp] = after != 0;
        }
        __syncthreads();

        if (warp == 0) {
            // the map of the tile, and on the way that of what stands in front of each warp's tokens
            float A[VC], B[VC], carry[VC];
#pragma unroll
            for (int v = 0; v < VC; ++v) A[v] = 1.f, B[v] = 0.f;
            bool closed = false;
            int front = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const bool r = sm.resets[w];
                front |= (int)closed << w;
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const float a = sm.A[w][lane * VC + v], b = sm.B[w][lane * VC + v];
                    sm.A[w][lane * VC + v] = A[v];
                    sm.B[w][lane * VC + v] = B[v];
                    B[v] = r ? b : fmaf(a, B[v], b);
                    A[v] = r ? 0.f : a * A[v];
                }
                closed |= r;
            }
            const bool open = chained && j > 0 && !(sm.what[buf][0] & RESET);
            chain<VC>(k, j, slab, A, B, closed, open, j + 1 < k.time_tiles, p.status, carry);
#pragma unroll
            for (int v = 0; v < VC; ++v) sm.carry[lane * VC + v] = carry[v];
            if (lane == 0) sm.resets[W] = front;
            if (p.checkpoints) store<float, VC>(p.checkpoints + (long long)j * p.C + c0, carry, inside, vec & VEC_STATE);
        } else {
            // meanwhile the other warps ask for the next tile
            if (threadIdx.x == 32) sm.next = chained ? atomicAdd(k.counter, 1) : k.tiles;
            if (nxt < k.tiles) fetch(nxt, buf ^ 1, threadIdx.x - 32, NT - 32);
        }
        if (nxt < k.tiles) tokens(nxt, buf ^ 1);
        __syncthreads();

        float front[VC];
        const bool cut = sm.resets[W] >> warp & 1;
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float a = sm.A[warp][lane * VC + v], b = sm.B[warp][lane * VC + v];
            front[v] = cut ? b : fmaf(a, sm.carry[lane * VC + v], b);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int r = warp * TT + i, what = sm.what[buf][r];
            if (!(what & VALID)) continue;
            if (!(after >> i & 1))
#pragma unroll
                for (int v = 0; v < VC; ++v) h[i][v] = fmaf(P[i][v], front[v], h[i][v]);
            store<T, VC>(static_cast<T *>(p.y) + (long long)(j * TILE + r) * p.C + c0, h[i], inside, vec & VEC_Y);
            if ((what & LAST) && p.final_state)
                store<float, VC>(p.final_state + (long long)sm.slot[buf][r] * p.C + c0, h[i], inside, vec & VEC_STATE);
        }
        if (j == 0) {
            // sequences without tokens keep their state; checks that the plan makes where there is one
            if (slab == 0 && !chained && p.cu) {
                if (threadIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.B] != p.T)) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
                for (int b = threadIdx.x; b < p.B; b += NT)
                    if (p.cu[b] > p.cu[b + 1]) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
            }
            if (p.cu && p.final_state) {
                for (int b0 = warp * 32; b0 < p.B; b0 += NT) {
                    const int mine = b0 + lane;
                    unsigned empty = __ballot_sync(0xffffffffu, mine < p.B && p.cu[mine] == p.cu[mine + 1]);
                    for (; empty; empty &= empty - 1) {
                        const int b = b0 + __ffs(empty) - 1, slot = p.slots ? p.slots[b] : b;
                        if (slot < 0 || slot >= p.num_slots) {
                            if (lane == 0 && slab == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
                            continue;
                        }
                        float h0[VC] = {};
                        if (p.init) load<VC>(p.init + (long long)slot * p.C + c0, h0, inside, vec & VEC_STATE);
                        store<float, VC>(p.final_state + (long long)slot * p.C + c0, h0, inside, vec & VEC_STATE);
                    }
                }
            }
        }
        cur = nxt;
        nxt = sm.next;
    }
}

// ---------------------------------------------------------------- short sequences

// A thread carries VC channels through a sequence's tokens.
constexpr int SHORT_NT = 128, SHORT_LEN = 16, AHEAD = 4;

template <typename T, int MODE, int VC>
__global__ void __launch_bounds__(SHORT_NT) recurrence_short_kernel(const RecurrenceParams p) {
    dependent_prologue();
    using G = typename GateType<T, MODE>::type;
    const int c = (blockIdx.x * SHORT_NT + threadIdx.x) * VC, b = blockIdx.y;
    if (c == 0 && b == 0 && p.cu && (p.cu[0] != 0 || p.cu[p.B] != p.T)) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
    if (c >= p.C) return;
    const int begin = recurrence_start(p, b), end = recurrence_start(p, b + 1);
    const int slot = p.slots ? p.slots[b] : b;
    float rate[VC], dt[VC], h[VC] = {};
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        rate[v] = MODE ? expf(p.A_log[c + v]) : 0.f;
        dt[v] = MODE ? p.dt_bias[c + v] : 0.f;
    }
    if (begin < 0 || end < begin || end > p.T) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_CU_SEQLENS);
        return;
    }
    if (slot < 0 || slot >= p.num_slots) {
        if (c == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
        return;
    }
    if (p.init) load<VC>(p.init + (long long)slot * p.C + c, h, VC, VC > 1);
    for (int t0 = begin; t0 < end; t0 += AHEAD) {
        float x[AHEAD][VC] = {}, a[AHEAD][VC] = {}, bv[AHEAD][VC] = {};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const long long t = t0 + i;
            if (t >= end) break;
            read<T, VC>(static_cast<const T *>(p.x) + t * p.x_stride + c, x[i]);
            read<G, VC>(static_cast<const G *>(p.a) + t * p.a_stride + c, a[i]);
            if (p.b) read<G, VC>(static_cast<const G *>(p.b) + t * p.b_stride + c, bv[i]);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const long long t = t0 + i;
            if (t >= end) break;
            if (p.checkpoints && t % TILE == 0) {
                float s[VC];
#pragma unroll
                for (int v = 0; v < VC; ++v) s[v] = t == begin ? 0.f : h[v];
                store<float, VC>(p.checkpoints + t / TILE * p.C + c, s, VC, VC > 1);
            }
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const Gate q = gate_of<MODE>(a[i][v], bv[i][v], rate[v], dt[v], p.b != nullptr);
                h[v] = fmaf(q.g, h[v], q.w * x[i][v]);
            }
            store<T, VC>(static_cast<T *>(p.y) + t * p.C + c, h, VC, VC > 1);
        }
    }
    if (p.final_state) store<float, VC>(p.final_state + (long long)slot * p.C + c, h, VC, VC > 1);
}

// ---------------------------------------------------------------- launches

bool whole(const void *ptr, long long stride, int C, size_t elem, size_t bytes) {
    return reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && stride * elem % bytes == 0 && C * elem % bytes == 0;
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, int longest, cudaStream_t stream) {
    using S = Shape<T, MODE>;
    using G = typename S::G;
    if (longest <= SHORT_LEN) {
        constexpr int VC = 4;
        const bool vec = whole(p.x, p.x_stride, p.C, sizeof(T), VC * sizeof(T)) && whole(p.a, p.a_stride, p.C, sizeof(G), VC * sizeof(G)) &&
                         whole(p.b, p.b_stride, p.C, sizeof(G), VC * sizeof(G)) && whole(p.y, p.C, p.C, sizeof(T), VC * sizeof(T)) &&
                         whole(p.init, p.C, p.C, 4, 16) && whole(p.final_state, p.C, p.C, 4, 16) && whole(p.checkpoints, p.C, p.C, 4, 16);
        const int step = SHORT_NT * (vec ? VC : 1);
        const dim3 grid((unsigned)((p.C + step - 1) / step), (unsigned)p.B);
        if (vec) return launch_dependent(recurrence_short_kernel<T, MODE, VC>, grid, dim3(SHORT_NT), 0, stream, p);
        return launch_dependent(recurrence_short_kernel<T, MODE, 1>, grid, dim3(SHORT_NT), 0, stream, p);
    }
    const Layout l = layout(p.T, p.C, S::SLAB, false);
    const Work k = work_of(p.workspace, l);
    constexpr int VC = S::VC;
    const int vec = (whole(p.x, p.x_stride, p.C, sizeof(T), 16) ? VEC_X : 0) | (whole(p.a, p.a_stride, p.C, sizeof(G), 16) ? VEC_A : 0) |
                    (whole(p.b, p.b_stride, p.C, sizeof(G), 16) ? VEC_B : 0) |
                    (whole(p.y, p.C, p.C, sizeof(T), VC * sizeof(T)) ? VEC_Y : 0) |
                    (whole(p.init, p.C, p.C, 4, VC * 4) && whole(p.final_state, p.C, p.C, 4, VC * 4) &&
                             whole(p.checkpoints, p.C, p.C, 4, VC * 4) ? VEC_STATE : 0);
    constexpr int smem = (int)sizeof(typename S::Shared);
    auto kernel = recurrence_tile_kernel<T, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    long long ctas = l.tiles;
    if (l.time_tiles > 1) {
        const long long items = std::max<long long>(l.tiles, p.B), most = 3LL * current_device_sms();
        e = launch_dependent(plan_kernel, dim3((unsigned)((items + PLAN_THREADS) / PLAN_THREADS)), dim3(PLAN_THREADS), 0, stream, p, k);
        if (e != cudaSuccess) return e;
        ctas = std::min(ctas, most);
    }
    return launch_dependent(kernel, dim3((unsigned)ctas), dim3(NT), smem, stream, p, k, vec);
}

template <typename T>
cudaError_t launch_mode(const RecurrenceParams &p, int mode, int longest, cudaStream_t stream) {
    switch (mode) {
        case RECUR_PRECOMPUTED: return launch_typed<T, RECUR_PRECOMPUTED>(p, longest, stream);
        case RECUR_RAW: return launch_typed<T, RECUR_RAW>(p, longest, stream);
        default: return launch_typed<T, RECUR_RAW_UNIT>(p, longest, stream);
    }
}

}  // namespace

// (a slab of 64 channels takes no less than one of 128)
size_t recurrence_workspace_bytes(int T, int C, int longest) {
    if (longest <= SHORT_LEN || T <= TILE) return 0;
    return std::max(layout(T, C, 64, false).bytes, layout(T, C, 128, false).bytes);
}

cudaError_t launch_recurrence(const RecurrenceParams &p, int io_dtype, int mode, int longest, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return launch_mode<__half>(p, mode, longest, stream);
        case GDN_BF16: return launch_mode<__nv_bfloat16>(p, mode, longest, stream);
        default: return launch_mode<float>(p, mode, longest, stream);
    }
}

}  // namespace gdn
