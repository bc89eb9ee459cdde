// The gated linear recurrence, backward: l_t = dy_t + g_(t+1) l_(t+1) a channel, and the
// gradients of the inputs from it.
#include "recurrence_tiles.cuh"

namespace gdn {
namespace {

using namespace recur;

constexpr int NT = 256, SUBS = NT / LANES;
constexpr int TT = 4, TILE = TT * SUBS;  // tokens of a half-warp, and of a CTA
constexpr int COPIER = 160;  // a thread that has nothing else to do between the two halves of a round
static_assert(TILE == CHECK, "a tile begins at a checkpoint");

struct Access {
    int x, a, b, dy;            // bytes of a copy
    bool dx, da, db, state;  // VC elements at once
};
struct Maps {
    CUtensorMap x, a, b, dy;  // of what is copied 16 bytes at a time
};

template <typename T, int MODE>
struct Shape {
    using G = typename GateType<T, MODE>::type;
    static constexpr int VC = sizeof(G) == 4 ? 2 : 4, SLAB = LANES * VC;
    struct Tile {
        alignas(128) T x[TILE * SLAB];
        alignas(128) T dy[TILE * SLAB];
        alignas(128) G a[TILE * SLAB];
        alignas(128) G b[TILE * SLAB];
    };
    struct Shared {
        Tile tile[2];
        // The half-warps' maps forwards (F) and backwards (R), then the state in front of each (FB) and the map of
        // what stands behind each in the tile (RA, RB)
        alignas(16) float FA[SUBS][SLAB], FB[SUBS][SLAB], RA[SUBS][SLAB], RB[SUBS][SLAB];
        alignas(16) float sum_A[SUBS][SLAB], sum_dt[SUBS][SLAB];
        alignas(16) float4 map[2][MAX_CLUSTER][SLAB];  // the cluster's tiles' maps backwards (A, B, whether a sequence ends in it)
        alignas(16) float carry[SLAB];
        alignas(16) float2 sums[MAX_CLUSTER][SLAB];
        Tokens<TILE> tokens[2];
        alignas(8) uint64_t full[2], maps[2];
    };
};

template <typename T, int MODE>
__global__ void __launch_bounds__(NT, 2) recurrence_backward_kernel(const RecurrenceParams p, const Access access,
                                                                    const __grid_constant__ Maps maps, int cluster) {
    dependent_prologue();
    using S = Shape<T, MODE>;
    using G = typename S::G;
    constexpr int VC = S::VC, SLAB = S::SLAB;
    constexpr bool RAW = MODE != RECUR_PRECOMPUTED;
    extern __shared__ __align__(128) unsigned char raw[];
    typename S::Shared &sm = *reinterpret_cast<typename S::Shared *>(raw);
    const int tid = threadIdx.x, lane = tid % LANES, sub = tid / LANES;
    const int rank = cluster > 1 ? cluster_rank() : 0, slab = blockIdx.x / cluster;
    const int s0 = slab * SLAB, c0 = s0 + lane * VC, inside = p.C - c0;
    const bool has_b = p.b != nullptr;

    float rate[VC], dt[VC];
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        rate[v] = RAW && v < inside ? expf(p.A_log[c0 + v]) : 0.f;
        dt[v] = RAW && v < inside ? p.dt_bias[c0 + v] : 0.f;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.full[i], 1);
            ptx::mbar_init(&sm.maps[i], 1);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();

    const bool bulk = access.x == 16 || access.dy == 16 || access.a == 16 || (has_b && access.b == 16);
    auto fetch = [&](int t0, int buf) {
        typename S::Tile &tile = sm.tile[buf];
        if (bulk && tid == COPIER && t0 < p.T) {
            constexpr uint32_t XB = sizeof(T) * TILE * SLAB, GB = sizeof(G) * TILE * SLAB;
            uint64_t *bar = &sm.full[buf];
            ptx::mbar_arrive_expect_tx(bar, (access.x == 16 ? XB : 0) + (access.dy == 16 ? XB : 0) + (access.a == 16 ? GB : 0) +
                                                (has_b && access.b == 16 ? GB : 0));
            if (access.x == 16) ptx::tma_load_2d(tile.x, &maps.x, s0, t0, bar);
            if (access.a == 16) ptx::tma_load_2d(tile.a, &maps.a, s0, t0, bar);
            if (has_b && access.b == 16) ptx::tma_load_2d(tile.b, &maps.b, s0, t0, bar);
            if (access.dy == 16) ptx::tma_load_2d(tile.dy, &maps.dy, s0, t0, bar);
        }
        if (access.x != 16) load_tile<T, SLAB, TILE, NT>(tile.x, p.x, p.x_stride, t0, p.T, s0, p.C, access.x);
        if (access.a != 16) load_tile<G, SLAB, TILE, NT>(tile.a, p.a, p.a_stride, t0, p.T, s0, p.C, access.a);
        if (has_b && access.b != 16) load_tile<G, SLAB, TILE, NT>(tile.b, p.b, p.b_stride, t0, p.T, s0, p.C, access.b);
        if (access.dy != 16) load_tile<T, SLAB, TILE, NT>(tile.dy, p.dy, p.dy_stride, t0, p.T, s0, p.C, access.dy);
    };

    // rounds run from the last tokens to the first
    const int step = cluster * TILE, rounds = (p.T + step - 1) / step;
    if (rounds > 0) {  // (a call without tokens has none)
        fetch((rounds - 1) * step + rank * TILE, 0);
        tokens_of(sm.tokens[0], p, (rounds - 1) * step + rank * TILE, slab == 0, tid / 32 - (NT - TILE) / 32);
    }
    if (blockIdx.x == 0) check_packing(p);
    if (cluster > 1) cluster_sync();  // every CTA has its barriers before another writes to its shared memory
    float run = 0.f;                     // what reaches the state behind the cluster's tiles, channel tid of the slab
    float total_A = 0.f, total_dt = 0.f;  // channel tid's sums
    const int skipped = (rounds - 1) * step + rank * TILE >= p.T;  // a tile behind the last token is not copied
    for (int n = 0, buf = 0; n < rounds; ++n, buf ^= 1) {
        const int t0 = (rounds - 1 - n) * step + rank * TILE;
        const Tokens<TILE> &tokens = sm.tokens[buf];
        const typename S::Tile &tile = sm.tile[buf];
        if (bulk && t0 < p.T) wait(&sm.full[buf], (n >> 1) - (buf ? 0 : skipped) & 1, p.status);
        copies_done();
        __syncthreads();
        const bool more = n + 1 < rounds;
        constexpr unsigned ALL = (1u << TT) - 1;
        const bool plain = tokens.plain;  // as most are
        const unsigned reset = plain ? 0 : bits_of<TT>(tokens.reset, sub), loads = plain ? 0 : bits_of<TT>(tokens.load, sub);
        const unsigned valid = plain ? ALL : bits_of<TT>(tokens.valid, sub), lasts = plain ? 0 : bits_of<TT>(tokens.last, sub);
        // Backwards a sequence's last token cuts off what stands behind it, and so does one of no sequence.
        const unsigned cuts = lasts | (~valid & ALL);
        const int place = sub * TT * SLAB + lane * VC;
        auto row = [&](int i) { return (long long)tokens.slot[sub * TT + i] * p.C + c0; };

        Gate q[TT][VC];
        {
            Pack<float, VC> A, B;  // forwards
#pragma unroll
            for (int v = 0; v < VC; ++v) A.e[v] = 1.f, B.e[v] = 0.f;
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                float x[VC], a[VC], b[VC] = {}, front[VC];
                read<T, VC>(tile.x + place + i * SLAB, x);
                read<G, VC>(tile.a + place + i * SLAB, a);
                if (has_b) read<G, VC>(tile.b + place + i * SLAB, b);
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    q[i][v] = gate_of<MODE>(a[v], b[v], rate[v], dt[v], has_b);
                    front[v] = reset >> i & 1 ? 0.f : B.e[v];
                }
                if ((loads >> i & 1) && p.init) load<VC>(p.init + row(i), front, inside, false);
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    B.e[v] = fmaf(q[i][v].g, front[v], q[i][v].w() * x[v]);
                    A.e[v] *= q[i][v].g;
                }
            }
            put_pack(&sm.FA[sub][lane * VC], A);
            put_pack(&sm.FB[sub][lane * VC], B);
#pragma unroll
            for (int v = 0; v < VC; ++v) B.e[v] = 0.f;  // backwards
#pragma unroll
            for (int i = TT - 1; i >= 0; --i) {
                float dy[VC];
                read<T, VC>(tile.dy + place + i * SLAB, dy);
                if (cuts >> i & 1) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) B.e[v] = 0.f;
                    if ((lasts >> i & 1) && p.dfinal) {
                        float d[VC];
                        load<VC>(p.dfinal + row(i), d, inside, false);
#pragma unroll
                        for (int v = 0; v < VC; ++v) B.e[v] = d[v];
                    }
                }
#pragma unroll
                for (int v = 0; v < VC; ++v) B.e[v] = valid >> i & 1 ? q[i][v].g * (dy[v] + B.e[v]) : 0.f;
            }
            put_pack(&sm.RA[sub][lane * VC], A);
            put_pack(&sm.RB[sub][lane * VC], B);
        }
        __syncthreads();

        if (more) fetch(t0 - step, buf ^ 1);
        if (tid < SLAB) {
            // the map backwards of the tile, and on the way that of what stands behind each half-warp's tokens
            float A = 1.f, B = 0.f, a[SUBS], b[SUBS];
            bool closed = false;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) a[s] = sm.RA[s][tid], b[s] = sm.RB[s][tid];
#pragma unroll
            for (int s = SUBS - 1; s >= 0; --s) {
                sm.RA[s][tid] = A;
                sm.RB[s][tid] = B;
                B = fmaf(a[s], B, b[s]);
                A *= a[s];
                if (!plain && (bits_of<TT>(tokens.last, s) | (bits_of<TT>(tokens.valid, s) ^ ALL))) {
                    B = b[s];
                    A = 0.f;
                    closed = true;
                }
            }
            if (cluster > 1) {
                uint64_t *bar = &sm.maps[buf];
                if (tid == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)cluster * SLAB * 16);
                for (int r = 0; r < cluster; ++r)
                    store_async(in_cta(&sm.map[buf][rank][tid], r), in_cta(bar, r), A, B, closed ? 1.f : 0.f);
                wait_cluster(bar, n >> 1 & 1, p.status);
                for (int r = cluster - 1; r >= 0; --r) {
                    const float4 m = sm.map[buf][r][tid];
                    if (r == rank) sm.carry[tid] = run;
                    run = m.z != 0.f ? m.y : fmaf(m.x, run, m.y);
                }
            } else {
                sm.carry[tid] = run;
                run = closed ? B : fmaf(A, run, B);
            }
        } else if (tid < 2 * SLAB) {
            // the state in front of each half-warp's tokens
            const int c = tid - SLAB;
            float h = s0 + c < p.C && t0 < p.T ? p.states[(long long)(t0 / CHECK) * p.C + s0 + c] : 0.f;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                const float a = sm.FA[s][c], b = sm.FB[s][c];
                sm.FB[s][c] = h;
                h = !plain && bits_of<TT>(tokens.reset, s) ? b : fmaf(a, h, b);
            }
        }
        if (more) tokens_of(sm.tokens[buf ^ 1], p, t0 - step, slab == 0, tid / 32 - (NT - TILE) / 32);  // (not by the threads above)
        __syncthreads();

        // the states again, each before its token
        float before[TT][VC];
        {
            float h[VC];
            read<float, VC>(&sm.FB[sub][lane * VC], h);
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                float x[VC];
                read<T, VC>(tile.x + place + i * SLAB, x);
                if (reset >> i & 1) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) h[v] = 0.f;
                    if ((loads >> i & 1) && p.init) load<VC>(p.init + row(i), h, inside, false);
                }
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    before[i][v] = h[v];
                    h[v] = fmaf(q[i][v].g, h[v], q[i][v].w() * x[v]);
                }
            }
        }
        // whether something cuts off what stands behind the half-warp's tokens within the tile
        bool cut = false;
        if (!plain) {
#pragma unroll
            for (int w = 0; w < TILE / 32; ++w) {
                const unsigned c = tokens.last[w] | ~tokens.valid[w];
                const int own = sub * TT / 32;
                cut |= w > own ? c != 0 : w == own ? (c >> (sub * TT % 32) >> TT) != 0 : false;
            }
        }
        float m[VC], sum_A[VC] = {}, sum_dt[VC] = {};
        {
            float A[VC], B[VC], carry[VC];
            read<float, VC>(&sm.RA[sub][lane * VC], A);
            read<float, VC>(&sm.RB[sub][lane * VC], B);
            read<float, VC>(&sm.carry[lane * VC], carry);
#pragma unroll
            for (int v = 0; v < VC; ++v) m[v] = cut ? B[v] : fmaf(A[v], carry[v], B[v]);
        }
        long long at = (long long)(t0 + sub * TT + TT - 1) * p.C + c0;
#pragma unroll
        for (int i = TT - 1; i >= 0; --i, at -= p.C) {
            float x[VC], a[VC], dy[VC], dx[VC], da[VC], db[VC];
            read<T, VC>(tile.x + place + i * SLAB, x);
            read<G, VC>(tile.a + place + i * SLAB, a);
            read<T, VC>(tile.dy + place + i * SLAB, dy);
            if (cuts >> i & 1) {
#pragma unroll
                for (int v = 0; v < VC; ++v) m[v] = 0.f;
                if ((lasts >> i & 1) && p.dfinal) load<VC>(p.dfinal + row(i), m, inside, false);
            }
            if (!(valid >> i & 1)) continue;
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float l = m[v] + dy[v];
                const GateGrad d = gate_grad<MODE>(q[i][v], a[v], l * before[i][v], l * x[v], rate[v], dt[v]);
                dx[v] = l * q[i][v].w();
                da[v] = d.da;
                db[v] = d.db;
                sum_A[v] += d.dA;
                sum_dt[v] += d.da;
                m[v] = q[i][v].g * l;
            }
            store<T, VC>(static_cast<T *>(p.dx) + at, dx, inside, access.dx);
            store<G, VC>(static_cast<G *>(p.da) + at, da, inside, access.da);
            if (has_b) store<G, VC>(static_cast<G *>(p.db) + at, db, inside, access.db);
            if ((loads >> i & 1) && p.dinit) store<float, VC>(p.dinit + row(i), m, inside, false);
        }
        if constexpr (RAW) {
            Pack<float, VC> A, B;
#pragma unroll
            for (int v = 0; v < VC; ++v) A.e[v] = sum_A[v], B.e[v] = sum_dt[v];
            put_pack(&sm.sum_A[sub][lane * VC], A);
            put_pack(&sm.sum_dt[sub][lane * VC], B);
            __syncthreads();
            if (tid < SLAB) {
                float a = 0.f, d = 0.f;
#pragma unroll
                for (int s = 0; s < SUBS; ++s) a += sm.sum_A[s][tid], d += sm.sum_dt[s][tid];
                total_A += a;
                total_dt += d;
            }
        }
    }

    if constexpr (RAW) {
        // the cluster's sums, in the order of its CTAs
        if (cluster > 1) {
            if (tid < SLAB) store_cluster(in_cta(&sm.sums[rank][tid], 0), total_A, total_dt);
            cluster_sync();
            if (rank == 0 && tid < SLAB) {
                total_A = total_dt = 0.f;
                for (int r = 0; r < cluster; ++r) {
                    const float2 s = sm.sums[r][tid];
                    total_A += s.x;
                    total_dt += s.y;
                }
            }
        }
        if (rank == 0 && tid < SLAB && s0 + tid < p.C) {
            if (p.dA_log) p.dA_log[s0 + tid] = total_A;
            if (p.ddt_bias) p.ddt_bias[s0 + tid] = total_dt;
        }
    }
    // a sequence without tokens passes its last state's gradient on
    if (rank != 0 || !p.cu || !p.dinit) return;
    for (int b = sub; b < p.B; b += SUBS) {
        if (p.cu[b] != p.cu[b + 1]) continue;
        const int slot = p.slots ? p.slots[b] : b;
        if (slot < 0 || slot >= p.num_slots) {
            if (lane == 0 && slab == 0) flag_error(p.status, GDN_DEVERR_STATE_SLOT);
            continue;
        }
        float d[VC] = {};
        if (p.dfinal) load<VC>(p.dfinal + (long long)slot * p.C + c0, d, inside, access.state);
        store<float, VC>(p.dinit + (long long)slot * p.C + c0, d, inside, access.state);
    }
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, cudaStream_t stream) {
    using S = Shape<T, MODE>;
    using G = typename S::G;
    constexpr int VC = S::VC;
    Access access;
    access.x = whole_bytes(p.x, p.x_stride, p.C, sizeof(T));
    access.dy = whole_bytes(p.dy, p.dy_stride, p.C, sizeof(T));
    access.a = whole_bytes(p.a, p.a_stride, p.C, sizeof(G));
    access.b = whole_bytes(p.b, p.b_stride, p.C, sizeof(G));
    Maps maps{};
    if (access.x == 16 && !tile_map<T, S::SLAB, TILE>(&maps.x, p.x, p.x_stride, p.T, p.C)) access.x = 4;
    if (access.dy == 16 && !tile_map<T, S::SLAB, TILE>(&maps.dy, p.dy, p.dy_stride, p.T, p.C)) access.dy = 4;
    if (access.a == 16 && !tile_map<G, S::SLAB, TILE>(&maps.a, p.a, p.a_stride, p.T, p.C)) access.a = 4;
    if (p.b && access.b == 16 && !tile_map<G, S::SLAB, TILE>(&maps.b, p.b, p.b_stride, p.T, p.C)) access.b = 4;
    access.dx = whole_rows(p.dx, p.C, sizeof(T), VC * sizeof(T));
    access.da = whole_rows(p.da, p.C, sizeof(G), VC * sizeof(G));
    access.db = whole_rows(p.db, p.C, sizeof(G), VC * sizeof(G));
    access.state = whole_rows(p.dfinal, p.C, 4, VC * 4) && whole_rows(p.dinit, p.C, 4, VC * 4);
    constexpr size_t smem = sizeof(typename S::Shared);
    auto kernel = recurrence_backward_kernel<T, MODE>;
    const Resident *resident;
    const cudaError_t e = prepare_clusters<T, MODE>(kernel, NT, smem, &resident);
    if (e != cudaSuccess) return e;
    const long long slabs = ((long long)p.C + S::SLAB - 1) / S::SLAB, tiles = ((long long)p.T + TILE - 1) / TILE;
    const int size = cluster_size(*resident, slabs, tiles);
    return launch_clusters(kernel, (unsigned)slabs, (unsigned)size, NT, smem, stream, p, access, maps, size);
}

template <typename T>
cudaError_t launch_mode(const RecurrenceParams &p, int mode, cudaStream_t stream) {
    switch (mode) {
        case RECUR_PRECOMPUTED: return launch_typed<T, RECUR_PRECOMPUTED>(p, stream);
        case RECUR_RAW: return launch_typed<T, RECUR_RAW>(p, stream);
        default: return launch_typed<T, RECUR_RAW_UNIT>(p, stream);
    }
}

}  // namespace

cudaError_t launch_recurrence_backward(const RecurrenceParams &p, int io_dtype, int mode, cudaStream_t stream) {
    switch (io_dtype) {
        case GDN_F16: return launch_mode<__half>(p, mode, stream);
        case GDN_BF16: return launch_mode<__nv_bfloat16>(p, mode, stream);
        default: return launch_mode<float>(p, mode, stream);
    }
}

}  // namespace gdn
