// The gated linear recurrence, forward: h_t = g_t h_(t-1) + w_t x_t a channel.
//
// An HBM stream where the gates come ready (x, a, b read and y written once), and where
// they are worked out here a matter of instructions: 30 a channel of a token, of which an
// SM has 44 to spend at 8 bytes a channel.  Over 16,384 tokens of 4096 channels: FP32
// gates 163 us at FP32 (6.6 TB/s, 0.97 of a copy's rate) and 124 us at BF16 (6.5 TB/s); raw
// gates 166 us at FP32 (6.5 TB/s) and 118 us at BF16 (4.5 TB/s), with unit_input 144 us.
// The latter are bound by latency: the issue slots are 45% busy, and the largest stalls are the
// chains of dependent instructions and the barrier at which most warps stand while a thread a channel
// folds the half-warps' maps and waits for the cluster's; the 8 x 4 states and decays of a lane's tokens are 64 registers, so that only
// two CTAs share an SM to cover for one another.  One token of 64 sequences of 2560 channels: 1.9 us, a launch.
#include "recurrence_tiles.cuh"

namespace gdn {
namespace {

using namespace recur;

// ---------------------------------------------------------------- long sequences

// (Packed BF16 prompts, 9078 tokens of 4096 channels, raw: 74 us.  When it was 77, 512 threads of 4 tokens a half-warp
// took 99 us, 256 of 4 and three CTAs an SM 81 us, 128 of 8 and four 82 us: as many elements on an SM, with more to exchange for each.)
constexpr int NT = 256, SUBS = NT / LANES;
constexpr int TT = 8, TILE = TT * SUBS;  // tokens of a half-warp, and of a CTA
constexpr int COPIER = 96;  // a thread that has nothing else to do between the two halves of a round

// What the host found to be aligned.
struct Access {
    int x, a, b;   // bytes of a copy
    bool y, state;  // VC elements at once
};
struct Maps {
    CUtensorMap x, a, b;  // of what is copied 16 bytes at a time
};

template <typename T, int MODE, int VC_>
struct Shape {
    using G = typename GateType<T, MODE>::type;
    static constexpr int VC = VC_, SLAB = LANES * VC;
    struct Shared {
        alignas(128) T x[TILE * SLAB];
        alignas(128) G a[TILE * SLAB], b[TILE * SLAB];
        alignas(16) float A[SUBS][SLAB], B[SUBS][SLAB];  // the half-warps' maps, then those of what stands in front of each
        Exchange<SLAB> exchange;
        alignas(16) float carry[SLAB];
        Tokens<TILE> tokens[2];
        Packing packing;
        alignas(8) uint64_t full;
    };
};

template <typename T, int MODE, int VC>
__global__ void __launch_bounds__(NT, VC == 2 ? 3 : 2) recurrence_kernel(const RecurrenceParams p, const Access access,
                                                           const __grid_constant__ Maps maps, int cluster) {
    dependent_prologue();
    using S = Shape<T, MODE, VC>;
    using G = typename S::G;
    constexpr int SLAB = S::SLAB, PAIRS = VC / 2;
    extern __shared__ __align__(128) unsigned char raw[];
    typename S::Shared &sm = *reinterpret_cast<typename S::Shared *>(raw);
    const int tid = threadIdx.x, lane = tid % LANES, sub = tid / LANES;
    const int rank = cluster > 1 ? cluster_rank() : 0, slab = blockIdx.x / cluster;
    const int s0 = slab * SLAB, c0 = s0 + lane * VC, inside = p.C - c0;
    const bool has_b = p.b != nullptr;

    F2 rate[PAIRS], dt[PAIRS];
#pragma unroll
    for (int v = 0; v < PAIRS; ++v) {
        float r[2] = {}, d[2] = {};
        if (MODE != RECUR_PRECOMPUTED)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (2 * v + k < inside) r[k] = -LOG2E * expf(p.A_log[c0 + 2 * v + k]), d[k] = p.dt_bias[c0 + 2 * v + k];
        rate[v] = F2(r[0], r[1]);
        dt[v] = F2(d[0], d[1]);
    }
    if (tid == 0) {
        ptx::mbar_init(&sm.full, 1);
        ptx::mbar_init(&sm.exchange.full[0], 1);
        ptx::mbar_init(&sm.exchange.full[1], 1);
        ptx::fence_mbar_init();
    }
    const Lookup lookup = stage_packing(p, sm.packing);
    __syncthreads();

    const bool bulk = access.x == 16 || access.a == 16 || (has_b && access.b == 16);
    const bool own = access.x != 16 || access.a != 16 || (has_b && access.b != 16);  // copies of the threads' own
    auto fetch = [&](int t0) {
        if (bulk && tid == COPIER && t0 < p.T) {
            constexpr uint32_t XB = sizeof(T) * TILE * SLAB, GB = sizeof(G) * TILE * SLAB;
            ptx::mbar_arrive_expect_tx(&sm.full, (access.x == 16 ? XB : 0) + (access.a == 16 ? GB : 0) +
                                                     (has_b && access.b == 16 ? GB : 0));
            if (access.x == 16) ptx::tma_load_2d(sm.x, &maps.x, s0, t0, &sm.full);
            if (access.a == 16) ptx::tma_load_2d(sm.a, &maps.a, s0, t0, &sm.full);
            if (has_b && access.b == 16) ptx::tma_load_2d(sm.b, &maps.b, s0, t0, &sm.full);
        }
        if (access.x != 16) load_tile<T, SLAB, TILE, NT>(sm.x, p.x, p.x_stride, t0, p.T, s0, p.C, access.x);
        if (access.a != 16) load_tile<G, SLAB, TILE, NT>(sm.a, p.a, p.a_stride, t0, p.T, s0, p.C, access.a);
        if (has_b && access.b != 16) load_tile<G, SLAB, TILE, NT>(sm.b, p.b, p.b_stride, t0, p.T, s0, p.C, access.b);
    };

    const int step = cluster * TILE, rounds = (p.T + step - 1) / step;
    fetch(rank * TILE);
    tokens_of(sm.tokens[0], p, lookup, rank * TILE, slab == 0, tid / 32 - (NT - TILE) / 32);
    if (blockIdx.x == 0) check_packing(p);
    if (cluster > 1) cluster_sync();  // every CTA has its barriers before another writes to its shared memory
    else __syncthreads();
    float run = 0.f;  // the state in front of the cluster's tiles, channel tid of the slab
    for (int n = 0, buf = 0; n < rounds; ++n, buf ^= 1) {
        const int t0 = n * step + rank * TILE;
        const Tokens<TILE> &tokens = sm.tokens[buf];
        if (bulk && t0 < p.T) wait(&sm.full, n & 1, p.status);
        if (own) {
            copies_done();
            __syncthreads();
            if (access.x == 2) prefetch_tile<T, SLAB, TILE, NT>(p.x, p.x_stride, t0 + step, p.T, s0, p.C);
            if (access.a == 2) prefetch_tile<G, SLAB, TILE, NT>(p.a, p.a_stride, t0 + step, p.T, s0, p.C);
            if (has_b && access.b == 2) prefetch_tile<G, SLAB, TILE, NT>(p.b, p.b_stride, t0 + step, p.T, s0, p.C);
        }

        // every token's state and decay with nothing in front of the half-warp's tokens
        const bool plain = tokens.plain;  // as most are
        const unsigned reset = plain ? 0 : bits_of<TT>(tokens.reset, sub), loads = plain ? 0 : bits_of<TT>(tokens.load, sub);
        const unsigned valid = plain ? (1u << TT) - 1 : bits_of<TT>(tokens.valid, sub);
        const unsigned lasts = plain ? 0 : bits_of<TT>(tokens.last, sub);
        const bool quick = plain || __all_sync(0xffffffffu, (reset | lasts) == 0 && valid == (1u << TT) - 1);  // the warp's tokens
        F2 h[TT][PAIRS], P[TT][PAIRS];
        auto scan = [&](auto inside_a_sequence) {
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const int r = sub * TT + i;
                float x[VC], a[VC], b[VC] = {};
                read<T, VC>(sm.x + r * SLAB + lane * VC, x);
                read<G, VC>(sm.a + r * SLAB + lane * VC, a);
                if (has_b) read<G, VC>(sm.b + r * SLAB + lane * VC, b);
                F2 front[PAIRS];
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    front[v] = F2(0.f);
                    if (i > 0 && (inside_a_sequence || !(reset >> i & 1))) front[v] = h[i - 1][v];
                }
                if (!inside_a_sequence && (loads >> i & 1) && p.init) {
                    float h0[VC];
                    load<VC>(p.init + (long long)tokens.slot[r] * p.C + c0, h0, inside, false);
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) front[v] = F2(h0[2 * v], h0[2 * v + 1]);
                }
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    const GatePair q =
                        gate_pair<MODE>(F2(a[2 * v], a[2 * v + 1]), F2(b[2 * v], b[2 * v + 1]), rate[v], dt[v], has_b);
                    const F2 u = mul2(weight_of<MODE>(q, has_b), F2(x[2 * v], x[2 * v + 1]));
                    h[i][v] = i == 0 && inside_a_sequence ? u : fma2(q.g, front[v], u);
                    P[i][v] = i == 0 ? q.g : mul2(q.g, P[i - 1][v]);
                }
            }
        };
        if (quick) scan(std::true_type());
        else scan(std::false_type());
        {
            Pack<float, VC> A, B;
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) {
                P[TT - 1][v].get(A.e[2 * v], A.e[2 * v + 1]);
                h[TT - 1][v].get(B.e[2 * v], B.e[2 * v + 1]);
            }
            put_pack(&sm.A[sub][lane * VC], A);
            put_pack(&sm.B[sub][lane * VC], B);
        }
        __syncthreads();

        const bool more = n + 1 < rounds;
        if (more) fetch(t0 + step);
        if (tid < SLAB) {
            // the map of the tile, and on the way that of what stands in front of each half-warp's tokens
            // (in short loops: the kernel's code has to stay in the instruction cache)
            float A = 1.f, B = 0.f;
            bool closed = false;
#pragma unroll 1
            for (int s0 = 0; s0 < SUBS; s0 += 8) {
                float a[8], b[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) a[s] = sm.A[s0 + s][tid], b[s] = sm.B[s0 + s][tid];
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    sm.A[s0 + s][tid] = A;
                    sm.B[s0 + s][tid] = B;
                    B = fmaf(a[s], B, b[s]);
                    A *= a[s];
                    if (!plain && bits_of<TT>(tokens.reset, s0 + s)) {
                        B = b[s];
                        A = 0.f;
                        closed = true;
                    }
                }
            }
            if (cluster > 1) {
                sm.carry[tid] = exchange<true>(sm.exchange, n, cluster, rank, tid, A, B, closed, run, p.status);
            } else {
                sm.carry[tid] = run;
                run = closed ? B : fmaf(A, run, B);
            }
        }
        if (more) tokens_of(sm.tokens[buf ^ 1], p, lookup, t0 + step, slab == 0, tid / 32 - (NT - TILE) / 32);  // (not by the threads above)
        __syncthreads();

        unsigned before = 0;  // whether a reset stands before the half-warp's tokens in the tile
        if (!plain) {
            before = tokens.reset[sub * TT / 32] & ((1u << (sub * TT % 32)) - 1);
#pragma unroll
            for (int w = 0; w < TILE / 32 - 1; ++w) before |= w < sub * TT / 32 ? tokens.reset[w] : 0;
        }
        float front[VC], A[VC], B[VC], carry[VC];
        read<float, VC>(&sm.A[sub][lane * VC], A);
        read<float, VC>(&sm.B[sub][lane * VC], B);
        read<float, VC>(&sm.carry[lane * VC], carry);
#pragma unroll
        for (int v = 0; v < VC; ++v) front[v] = before ? B[v] : fmaf(A[v], carry[v], B[v]);
        const int first = t0 + sub * TT;
        if (p.checkpoints && first % CHECK == 0 && first < p.T)
            store<float, VC>(p.checkpoints + (long long)(first / CHECK) * p.C + c0, front, inside, access.state);
        F2 front2[PAIRS];
#pragma unroll
        for (int v = 0; v < PAIRS; ++v) front2[v] = F2(front[2 * v], front[2 * v + 1]);
        T *y = static_cast<T *>(p.y) + (long long)first * p.C + c0;
        if (quick && access.y) {
#pragma unroll
            for (int i = 0; i < TT; ++i, y += p.C) {
                float out[VC];
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) fma2(P[i][v], front2[v], h[i][v]).get(out[2 * v], out[2 * v + 1]);
                if (inside > 0) store<T, VC>(y, out, VC, true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TT; ++i, y += p.C) {
                float out[VC];
                const bool open = !(reset & ((2u << i) - 1));
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    if (open) h[i][v] = fma2(P[i][v], front2[v], h[i][v]);
                    h[i][v].get(out[2 * v], out[2 * v + 1]);
                }
                if (valid >> i & 1) store<T, VC>(y, out, inside, access.y);
                if ((lasts >> i & 1) && p.final_state)
                    store<float, VC>(p.final_state + (long long)tokens.slot[sub * TT + i] * p.C + c0, out, inside, false);
            }
        }
    }

    // sequences without tokens keep their state
    if (rank != 0 || !p.cu || !p.final_state) return;
    for (int b = sub; b < p.B; b += SUBS) {
        if (p.cu[b] != p.cu[b + 1]) continue;
        const int slot = p.slots ? p.slots[b] : b;
        if (slot < 0 || slot >= p.num_slots) {
            if (lane == 0 && slab == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
            continue;
        }
        float h0[VC] = {};
        if (p.init) load<VC>(p.init + (long long)slot * p.C + c0, h0, inside, access.state);
        store<float, VC>(p.final_state + (long long)slot * p.C + c0, h0, inside, access.state);
    }
}

// ---------------------------------------------------------------- short sequences

// A thread carries VC channels through a sequence's tokens.  (Up to SHORT_LEN of them: a tile's hand-overs cost about as
// much as 16 tokens' loads, AHEAD of them at once.)
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
    if (p.init) load<VC>(p.init + (long long)slot * p.C + c, h, VC, true);
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
            if (p.checkpoints && t % CHECK == 0) store<float, VC>(p.checkpoints + t / CHECK * p.C + c, h, VC, true);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const Gate q = gate_of<MODE>(a[i][v], bv[i][v], rate[v], dt[v], p.b != nullptr);
                h[v] = fmaf(q.g, h[v], q.w() * x[i][v]);
            }
            store<T, VC>(static_cast<T *>(p.y) + t * p.C + c, h, VC, true);
        }
    }
    if (p.final_state) store<float, VC>(p.final_state + (long long)slot * p.C + c, h, VC, true);
}

// ---------------------------------------------------------------- launches

template <typename T, int MODE>
cudaError_t launch_short(const RecurrenceParams &p, cudaStream_t stream) {
    using G = typename GateType<T, MODE>::type;
    constexpr int VC = 4;
    auto whole = [&](const void *ptr, long long stride, size_t elem) {
        return (reinterpret_cast<uintptr_t>(ptr) | (unsigned long long)stride * elem) % (VC * elem) == 0;
    };
    const bool vec = p.C % VC == 0 && whole(p.x, p.x_stride, sizeof(T)) && whole(p.a, p.a_stride, sizeof(G)) &&
                     whole(p.b, p.b_stride, sizeof(G)) && whole(p.y, p.C, sizeof(T)) && whole(p.init, p.C, 4) &&
                     whole(p.final_state, p.C, 4) && whole(p.checkpoints, p.C, 4);
    const int step = SHORT_NT * (vec ? VC : 1);
    const dim3 grid((unsigned)((p.C + step - 1) / step), (unsigned)p.B);
    if (vec) return launch_dependent(recurrence_short_kernel<T, MODE, VC>, grid, dim3(SHORT_NT), 0, stream, p);
    return launch_dependent(recurrence_short_kernel<T, MODE, 1>, grid, dim3(SHORT_NT), 0, stream, p);
}

template <typename T, int MODE, int VC>
cudaError_t launch_tiles(const RecurrenceParams &p, cudaStream_t stream) {
    using S = Shape<T, MODE, VC>;
    using G = typename S::G;
    Access access;
    access.x = whole_bytes(p.x, p.x_stride, p.C, sizeof(T));
    access.a = whole_bytes(p.a, p.a_stride, p.C, sizeof(G));
    access.b = whole_bytes(p.b, p.b_stride, p.C, sizeof(G));
    Maps maps{};
    if (access.x == 16 && !tile_map<T, S::SLAB, TILE>(&maps.x, p.x, p.x_stride, p.T, p.C)) access.x = 8;
    if (access.a == 16 && !tile_map<G, S::SLAB, TILE>(&maps.a, p.a, p.a_stride, p.T, p.C)) access.a = 8;
    if (p.b && access.b == 16 && !tile_map<G, S::SLAB, TILE>(&maps.b, p.b, p.b_stride, p.T, p.C)) access.b = 8;
    access.y = whole_rows(p.y, p.C, sizeof(T), VC * sizeof(T));
    access.state = whole_rows(p.init, p.C, 4, VC * 4) && whole_rows(p.final_state, p.C, 4, VC * 4) &&
                   whole_rows(p.checkpoints, p.C, 4, VC * 4);
    constexpr size_t smem = sizeof(typename S::Shared);
    auto kernel = recurrence_kernel<T, MODE, VC>;
    const Resident *resident;
    const cudaError_t e = prepare_clusters<T, MODE, VC>(kernel, NT, smem, &resident);
    if (e != cudaSuccess) return e;
    const long long slabs = ((long long)p.C + S::SLAB - 1) / S::SLAB, tiles = ((long long)p.T + TILE - 1) / TILE;
    const int size = cluster_size(*resident, slabs, tiles);
    return launch_clusters(kernel, (unsigned)slabs, (unsigned)size, NT, smem, stream, p, access, maps, size);
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, int longest, cudaStream_t stream) {
    if (longest <= SHORT_LEN) return launch_short<T, MODE>(p, stream);
    if constexpr (sizeof(typename GateType<T, MODE>::type) == 4) return launch_tiles<T, MODE, 2>(p, stream);
    else return narrow_slabs(p.C) ? launch_tiles<T, MODE, 2>(p, stream) : launch_tiles<T, MODE, 4>(p, stream);
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

cudaError_t launch_recurrence(const RecurrenceParams &p, int io_dtype, int mode, int longest, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return launch_mode<__half>(p, mode, longest, stream);
        case GDN_BF16: return launch_mode<__nv_bfloat16>(p, mode, longest, stream);
        default: return launch_mode<float>(p, mode, longest, stream);
    }
}

}  // namespace gdn
