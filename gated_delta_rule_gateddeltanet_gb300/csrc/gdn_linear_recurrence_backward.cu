// The gated linear recurrence, backward: l_t = dy_t + g_(t+1) l_(t+1) a channel, and the
// gradients of the inputs from it.
//
// The same scan as forwards, from the last tokens to the first, with m_t = g_t l_t as its
// state; the forward states, which dg needs, are worked out again inside each tile from the
// checkpoint in front of it (a tile is GDN_RECURRENCE_CHECKPOINT tokens).  x, a, b, dy are
// read once and dx, da, db written once; the parameters' gradients are added up tile by tile
// in shared memory, a thread's in its own entries, and summed over a cluster's CTAs in order.
//
// Over 16,384 tokens of 4096 channels: FP32 gates 313 us at FP32 (6.0 TB/s, 0.89 of a copy's
// rate) and 237 us at BF16 (6.2 TB/s); raw gates 379 us at FP32 and 256 us at BF16 (3.7 TB/s),
// with unit_input 314 us.  The 16-bit raw ones are bound by latency as forwards: 67 instructions a
// channel of a token, of which an SM has time for 77 at 14 bytes, but the issue slots are 48% busy; half
// of the warps stand at a barrier while the others fold and exchange.  What counted: no spills (beside
// tiles that fill the shared memory, the L1 cache is too small for them: 394 -> 278 us), code for tokens
// inside a sequence apart from the rest, which the instruction cache then holds, and no branches in
// the unrolled gradients (274 -> 257 us).
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

template <typename T, int MODE, int VC_>
struct Shape {
    using G = typename GateType<T, MODE>::type;
    static constexpr int VC = VC_, SLAB = LANES * VC;
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
        Exchange<SLAB> exchange;
        alignas(16) float carry[SLAB];
        Tokens<TILE> tokens[2];
        Packing packing;
        alignas(8) uint64_t full[2];
    };
};

template <typename T, int MODE, int VC>
__global__ void __launch_bounds__(NT, VC == 2 ? 3 : 2) recurrence_backward_kernel(const RecurrenceParams p, const Access access,
                                                                    const __grid_constant__ Maps maps, int cluster) {
    dependent_prologue();
    using S = Shape<T, MODE, VC>;
    using G = typename S::G;
    constexpr int SLAB = S::SLAB, PAIRS = VC / 2;
    constexpr bool RAW = MODE != RECUR_PRECOMPUTED;
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
        if (RAW)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (2 * v + k < inside) r[k] = -LOG2E * expf(p.A_log[c0 + 2 * v + k]), d[k] = p.dt_bias[c0 + 2 * v + k];
        rate[v] = F2(r[0], r[1]);
        dt[v] = F2(d[0], d[1]);
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sm.full[i], 1);
            ptx::mbar_init(&sm.exchange.full[i], 1);
        }
        ptx::fence_mbar_init();
    }
    const Lookup lookup = stage_packing(p, sm.packing);
    __syncthreads();

    const bool bulk = access.x == 16 || access.dy == 16 || access.a == 16 || (has_b && access.b == 16);
    const bool own = access.x != 16 || access.dy != 16 || access.a != 16 || (has_b && access.b != 16);  // the threads' own copies
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
        tokens_of(sm.tokens[0], p, lookup, (rounds - 1) * step + rank * TILE, slab == 0, tid / 32 - (NT - TILE) / 32);
    }
    if (blockIdx.x == 0) check_packing(p);
    if (cluster > 1) cluster_sync();  // every CTA has its barriers before another writes to its shared memory
    else __syncthreads();
    float run = 0.f;                     // what reaches the state behind the cluster's tiles, channel tid of the slab
    if constexpr (RAW) {
        Pack<float, VC> zero;
#pragma unroll
        for (int v = 0; v < VC; ++v) zero.e[v] = 0.f;
        put_pack(&sm.sum_A[sub][lane * VC], zero);
        put_pack(&sm.sum_dt[sub][lane * VC], zero);
    }
    const int skipped = (rounds - 1) * step + rank * TILE >= p.T;  // a tile behind the last token is not copied
    for (int n = 0, buf = 0; n < rounds; ++n, buf ^= 1) {
        const int t0 = (rounds - 1 - n) * step + rank * TILE;
        const Tokens<TILE> &tokens = sm.tokens[buf];
        const typename S::Tile &tile = sm.tile[buf];
        if (bulk && t0 < p.T) wait(&sm.full[buf], (n >> 1) - (buf ? 0 : skipped) & 1, p.status);
        if (own) {
            copies_done();
            __syncthreads();
            if (n + 1 < rounds) {
                if (access.x == 2) prefetch_tile<T, SLAB, TILE, NT>(p.x, p.x_stride, t0 - step, p.T, s0, p.C);
                if (access.dy == 2) prefetch_tile<T, SLAB, TILE, NT>(p.dy, p.dy_stride, t0 - step, p.T, s0, p.C);
                if (access.a == 2) prefetch_tile<G, SLAB, TILE, NT>(p.a, p.a_stride, t0 - step, p.T, s0, p.C);
                if (has_b && access.b == 2) prefetch_tile<G, SLAB, TILE, NT>(p.b, p.b_stride, t0 - step, p.T, s0, p.C);
            }
        }
        const bool more = n + 1 < rounds;
        float checkpoint = 0.f;  // channel tid - SLAB's, on its way while the gates are worked out
        if (tid >= SLAB && tid < 2 * SLAB && s0 + tid - SLAB < p.C && t0 < p.T)
            checkpoint = p.states[(long long)(t0 / CHECK) * p.C + s0 + tid - SLAB];
        constexpr unsigned ALL = (1u << TT) - 1;
        const bool plain = tokens.plain;  // as most are
        const unsigned reset = plain ? 0 : bits_of<TT>(tokens.reset, sub), loads = plain ? 0 : bits_of<TT>(tokens.load, sub);
        const unsigned valid = plain ? ALL : bits_of<TT>(tokens.valid, sub), lasts = plain ? 0 : bits_of<TT>(tokens.last, sub);
        // Backwards a sequence's last token cuts off what stands behind it, and so does one of no sequence.
        const unsigned cuts = lasts | (~valid & ALL);
        const int place = sub * TT * SLAB + lane * VC;
        const bool quick = plain || __all_sync(0xffffffffu, (reset | cuts) == 0);  // the warp's tokens lie inside a sequence
        auto row = [&](int i) { return (long long)tokens.slot[sub * TT + i] * p.C + c0; };

        auto state_of = [&](const float *pool, int i, F2 (&f)[PAIRS]) {
            float g[VC];
            load<VC>(pool + row(i), g, inside, false);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) f[v] = F2(g[2 * v], g[2 * v + 1]);
        };
        auto put = [&](float *dst, const F2 (&f)[PAIRS]) {
            Pack<float, VC> v;
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) f[k].get(v.e[2 * k], v.e[2 * k + 1]);
            put_pack(dst + lane * VC, v);
        };
        GatePair q[TT][PAIRS];
        F2 u[TT][PAIRS];  // a token's w x, and later the state before it
        auto gates = [&](auto inside_a_sequence) {
            F2 A[PAIRS], B[PAIRS];  // forwards
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) A[v] = F2(1.f), B[v] = F2(0.f);
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                F2 x[PAIRS], a[PAIRS], b[PAIRS];
                pairs_of(tile.x + place + i * SLAB, x);
                pairs_of(tile.a + place + i * SLAB, a);
                if (has_b) pairs_of(tile.b + place + i * SLAB, b);
                if (!inside_a_sequence && (reset >> i & 1)) {
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) B[v] = F2(0.f);
                    if ((loads >> i & 1) && p.init) state_of(p.init, i, B);
                }
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    q[i][v] = gate_pair<MODE>(a[v], b[v], rate[v], dt[v], has_b);
                    u[i][v] = mul2(weight_of<MODE>(q[i][v]), x[v]);
                    B[v] = fma2(q[i][v].g, B[v], u[i][v]);
                    A[v] = mul2(A[v], q[i][v].g);
                }
            }
            put(sm.FA[sub], A);
            put(sm.FB[sub], B);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) B[v] = F2(0.f);  // backwards
#pragma unroll
            for (int i = TT - 1; i >= 0; --i) {
                F2 dy[PAIRS];
                pairs_of(tile.dy + place + i * SLAB, dy);
                if (!inside_a_sequence && (cuts >> i & 1)) {
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) B[v] = F2(0.f);
                    if ((lasts >> i & 1) && p.dfinal) state_of(p.dfinal, i, B);
                }
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) B[v] = mul2(q[i][v].g, add2(dy[v], B[v]));
                if (!inside_a_sequence && !(valid >> i & 1))
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) B[v] = F2(0.f);
            }
            put(sm.RA[sub], A);
            put(sm.RB[sub], B);
        };
        if (quick) gates(std::true_type());
        else gates(std::false_type());
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
                sm.carry[tid] = exchange<false>(sm.exchange, n, cluster, rank, tid, A, B, closed, run, p.status);
            } else {
                sm.carry[tid] = run;
                run = closed ? B : fmaf(A, run, B);
            }
        } else if (tid < 2 * SLAB) {
            // the state in front of each half-warp's tokens
            const int c = tid - SLAB;
            float h = checkpoint;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                const float a = sm.FA[s][c], b = sm.FB[s][c];
                sm.FB[s][c] = h;
                h = !plain && bits_of<TT>(tokens.reset, s) ? b : fmaf(a, h, b);
            }
        }
        if (more) tokens_of(sm.tokens[buf ^ 1], p, lookup, t0 - step, slab == 0, tid / 32 - (NT - TILE) / 32);  // (not by the threads above)
        __syncthreads();

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
        F2 m[PAIRS], sum_A[PAIRS], sum_dt[PAIRS];
        {
            F2 A[PAIRS], B[PAIRS], carry[PAIRS];
            pairs_of(&sm.RA[sub][lane * VC], A);
            pairs_of(&sm.RB[sub][lane * VC], B);
            pairs_of(&sm.carry[lane * VC], carry);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) {
                m[v] = B[v];
                if (!cut) m[v] = fma2(A[v], carry[v], B[v]);
                sum_A[v] = sum_dt[v] = F2(0.f);
            }
        }
        auto gradients = [&](auto inside_a_sequence) {
            // the states again
            F2 h[PAIRS];
            pairs_of(&sm.FB[sub][lane * VC], h);
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                if (!inside_a_sequence && (reset >> i & 1)) {
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) h[v] = F2(0.f);
                    if ((loads >> i & 1) && p.init) state_of(p.init, i, h);
                }
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    const F2 next = fma2(q[i][v].g, h[v], u[i][v]);
                    u[i][v] = h[v];
                    h[v] = next;
                }
            }
            long long at = (long long)(t0 + sub * TT + TT - 1) * p.C + c0;
#pragma unroll
            for (int i = TT - 1; i >= 0; --i, at -= p.C) {
                if (!inside_a_sequence && (cuts >> i & 1)) {
#pragma unroll
                    for (int v = 0; v < PAIRS; ++v) m[v] = F2(0.f);
                    if ((lasts >> i & 1) && p.dfinal) state_of(p.dfinal, i, m);
                    if (!(valid >> i & 1)) continue;
                }
                F2 x[PAIRS], a[PAIRS], dy[PAIRS];
                float dx[VC], da[VC], db[VC];
                pairs_of(tile.x + place + i * SLAB, x);
                pairs_of(tile.a + place + i * SLAB, a);
                pairs_of(tile.dy + place + i * SLAB, dy);
#pragma unroll
                for (int v = 0; v < PAIRS; ++v) {
                    const F2 l = add2(m[v], dy[v]);
                    const GradPair d = grad_pair<MODE>(q[i][v], a[v], mul2(l, u[i][v]), mul2(l, x[v]), rate[v], dt[v]);
                    mul2(l, d.w).get(dx[2 * v], dx[2 * v + 1]);
                    d.da.get(da[2 * v], da[2 * v + 1]);
                    d.db.get(db[2 * v], db[2 * v + 1]);
                    if (RAW) {
                        sum_A[v] = add2(sum_A[v], d.dA);
                        sum_dt[v] = add2(sum_dt[v], d.da);
                    }
                    m[v] = mul2(q[i][v].g, l);
                }
                if (inside_a_sequence) {
                    if (inside > 0) {
                        store<T, VC>(static_cast<T *>(p.dx) + at, dx, VC, true);
                        store<G, VC>(static_cast<G *>(p.da) + at, da, VC, true);
                        if (has_b) store<G, VC>(static_cast<G *>(p.db) + at, db, VC, true);
                    }
                } else {
                    store<T, VC>(static_cast<T *>(p.dx) + at, dx, inside, access.dx);
                    store<G, VC>(static_cast<G *>(p.da) + at, da, inside, access.da);
                    if (has_b) store<G, VC>(static_cast<G *>(p.db) + at, db, inside, access.db);
                    if ((loads >> i & 1) && p.dinit) {
                        float first[VC];
#pragma unroll
                        for (int v = 0; v < PAIRS; ++v) m[v].get(first[2 * v], first[2 * v + 1]);
                        store<float, VC>(p.dinit + row(i), first, inside, false);
                    }
                }
            }
        };
        if (quick && access.dx && access.da && access.db) gradients(std::true_type());
        else gradients(std::false_type());
        if constexpr (RAW) {
            // (in shared memory, since registers are short; a thread's entries are its own)
            F2 before[PAIRS];
            pairs_of(&sm.sum_A[sub][lane * VC], before);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) sum_A[v] = add2(before[v], sum_A[v]);
            put(sm.sum_A[sub], sum_A);
            pairs_of(&sm.sum_dt[sub][lane * VC], before);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) sum_dt[v] = add2(before[v], sum_dt[v]);
            put(sm.sum_dt[sub], sum_dt);
        }
    }

    if constexpr (RAW) {
        __syncthreads();
        float total_A = 0.f, total_dt = 0.f;  // channel tid's sums
        if (tid < SLAB)
            for (int s = 0; s < SUBS; ++s) total_A += sm.sum_A[s][tid], total_dt += sm.sum_dt[s][tid];
        // the cluster's sums, in the order of its CTAs (where the maps of the last round but one were: whoever has the
        // last round's has them from CTAs that are past that one)
        if (cluster > 1) {
            float2(*sums)[SLAB] = sm.exchange.map[rounds & 1];
            if (tid < SLAB) store_cluster(in_cta(&sums[rank][tid], 0), total_A, total_dt);
            cluster_sync();
            if (rank == 0 && tid < SLAB) {
                total_A = total_dt = 0.f;
                for (int r = 0; r < cluster; ++r) {
                    const float2 s = sums[r][tid];
                    total_A += s.x;
                    total_dt += s.y;
                }
            }
        }
        if (rank == 0 && tid < SLAB && s0 + tid < p.C) {
            if (p.dA_log) p.dA_log[s0 + tid] = LN2 * total_A;  // (from base-2 logarithms)
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

template <typename T, int MODE, int VC>
cudaError_t launch_tiles(const RecurrenceParams &p, cudaStream_t stream) {
    using S = Shape<T, MODE, VC>;
    using G = typename S::G;
    Access access;
    access.x = whole_bytes(p.x, p.x_stride, p.C, sizeof(T));
    access.dy = whole_bytes(p.dy, p.dy_stride, p.C, sizeof(T));
    access.a = whole_bytes(p.a, p.a_stride, p.C, sizeof(G));
    access.b = whole_bytes(p.b, p.b_stride, p.C, sizeof(G));
    Maps maps{};
    if (access.x == 16 && !tile_map<T, S::SLAB, TILE>(&maps.x, p.x, p.x_stride, p.T, p.C)) access.x = 8;
    if (access.dy == 16 && !tile_map<T, S::SLAB, TILE>(&maps.dy, p.dy, p.dy_stride, p.T, p.C)) access.dy = 8;
    if (access.a == 16 && !tile_map<G, S::SLAB, TILE>(&maps.a, p.a, p.a_stride, p.T, p.C)) access.a = 8;
    if (p.b && access.b == 16 && !tile_map<G, S::SLAB, TILE>(&maps.b, p.b, p.b_stride, p.T, p.C)) access.b = 8;
    access.dx = whole_rows(p.dx, p.C, sizeof(T), VC * sizeof(T));
    access.da = whole_rows(p.da, p.C, sizeof(G), VC * sizeof(G));
    access.db = whole_rows(p.db, p.C, sizeof(G), VC * sizeof(G));
    access.state = whole_rows(p.dfinal, p.C, 4, VC * 4) && whole_rows(p.dinit, p.C, 4, VC * 4);
    constexpr size_t smem = sizeof(typename S::Shared);
    auto kernel = recurrence_backward_kernel<T, MODE, VC>;
    const Resident *resident;
    const cudaError_t e = prepare_clusters<T, MODE, VC>(kernel, NT, smem, &resident);
    if (e != cudaSuccess) return e;
    const long long slabs = ((long long)p.C + S::SLAB - 1) / S::SLAB, tiles = ((long long)p.T + TILE - 1) / TILE;
    const int size = cluster_size(*resident, slabs, tiles);
    return launch_clusters(kernel, (unsigned)slabs, (unsigned)size, NT, smem, stream, p, access, maps, size);
}

template <typename T, int MODE>
cudaError_t launch_typed(const RecurrenceParams &p, cudaStream_t stream) {
    if constexpr (sizeof(typename GateType<T, MODE>::type) == 4) return launch_tiles<T, MODE, 2>(p, stream);
    else return narrow_slabs(p.C) ? launch_tiles<T, MODE, 2>(p, stream) : launch_tiles<T, MODE, 4>(p, stream);
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
