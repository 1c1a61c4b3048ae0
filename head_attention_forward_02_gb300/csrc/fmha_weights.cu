// fmha_weights.cu -- the attention weight that every cached key got from a
// call's queries, added to a running score per key.
//
// Operation: sequence b has L = seqlen[b] cached keys in entry e and
// n = n_query[b] query tokens; with the LSE that the attention call returned,
//   acc_out[e, g, j] = acc_in[e, g, j] +
//     sum over query tokens t that see key j, heads h of group g:
//       exp(scale * q[b, t, h].K_cache[e, j, g] - lse[b, h, t])
// for j < L.  The sum runs over queries, so the kernel computes
// S^T = K Q^T (M = 128 keys, N = up to 128 packed query rows): a thread owns
// one key (TMEM lane) and adds its columns up in a register; nothing is
// exchanged between threads and no atomics are needed.
//
// Every cached key (128 * E bytes) takes 2 * 128 * n * G flops and n * G
// exponentials: with one query token the call is bound by reading K, with
// more than a few dozen rows by the exponentials (two for each 128 * 2 flops
// of the tensor core's 8192 a cycle).
//
// A unit is 256 keys of one kv head (two MMA tiles that share the query
// stream) and its query chunks (TB = 128 / G tokens each).  The chunks of all
// units form one sequence, cut evenly over the CTAs; a unit that is cut
// leaves partial sums (256 floats) in the workspace and a second kernel adds
// them in CTA order, so results do not depend on timing.
#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kWeightsMaxCtas = 152;     // CTAs at most (bounds the workspace)
constexpr int kUnitKeys = 2 * kRows;
constexpr int kWThreads = 320;           // 8 softmax warps, producer, MMA issuer
constexpr int kWProd = 8, kWMma = 9;

template <int ELEM>
struct WCfg : ElemCfg<ELEM> {
    using B = ElemCfg<ELEM>;
    static constexpr int NK = 4 * 32768 / B::TILE_BYTES;      // K ring stages (one 128-key tile each): 128 KB
    static constexpr int NQ = 2 * 32768 / B::TILE_BYTES;      // Q ring stages (one chunk each): 64 KB
    static constexpr int OFF_K = 0;
    static constexpr int OFF_Q = NK * B::TILE_BYTES;
    static constexpr int OFF_BARS = OFF_Q + NQ * B::TILE_BYTES;
    static constexpr int SMEM_BYTES = OFF_BARS + 4096 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

struct WMeta {                           // one partial sum in the workspace
    int64_t row;                         // its unit's first element of acc
    int keys;                            // keys of the unit below L (0: no partial here)
    int last;                            // the unit ends with this partial
};

struct WParams {
    const float *lse;                    // [B, H, Sq]
    const float *acc_in;                 // [B_cache, H_k, S_max] or NULL
    float *acc_out;
    const int *seqlen, *batch_idx, *n_query;
    WMeta *meta;                         // [2 * ncta]
    float *part;                         // [2 * ncta][256]
    int B, Sq, H, H_k, G, B_cache, S_max;
    int TB;                              // query tokens of a chunk
    int NMMA;                            // MMA N: TB * G rounded up to 16
    int causal;
    float c;                             // scale * log2(e)
};

struct WSched {
    int64_t left;                        // chunks of this CTA
    int b, g, tile, skip;                // its first unit, and chunks of that unit that are other CTAs'
};

struct WBars {
    uint64_t k_full[8], k_empty[8], q_full[4], q_empty[4];
    uint64_t s_full[2][2], s_free[2][2], drain;
    uint32_t tmem_base;
    int abort;
    WSched sched;
    float lse[2][2][kRows];              // per group and buffer: a chunk's LSE in log2 units
};
static_assert(sizeof(WBars) <= 4096, "barrier block");

__device__ __forceinline__ int w_keys(const WParams &p, int b, bool report) {
    return clamped(p.seqlen[b], 0, p.S_max, report);
}
__device__ __forceinline__ int w_queries(const WParams &p, int b, bool report) {
    return p.n_query ? clamped(p.n_query[b], 0, p.Sq, report) : p.Sq;
}

// Query t of a sequence sees key j iff j <= t + L - n (causal): the first
// chunk of unit `tile` that holds a query which sees one of its keys.
__device__ __forceinline__ int w_first_chunk(const WParams &p, int L, int n, int tile) {
    if (!p.causal) return 0;
    const int t = tile * kUnitKeys - (L - n);
    return t > 0 ? t / p.TB : 0;
}
// Chunks of a unit; a sequence without queries still copies acc: one empty chunk.
__device__ __forceinline__ int w_cost(const WParams &p, int L, int n, int tile) {
    return imax(1, (n + p.TB - 1) / p.TB - w_first_chunk(p, L, n, tile));
}
// Units [0, *uniform) of one head cost the same; the sum over all of them.
__device__ __forceinline__ int64_t w_head_cost(const WParams &p, int L, int n, int *uniform) {
    const int nt = (L + kUnitKeys - 1) / kUnitKeys;
    int u = nt;
    if (p.causal) {
        const int64_t x = (int64_t)p.TB - 1 + L - n;         // last key whose tile still starts at chunk 0
        u = x < 0 ? 0 : imin(nt, (int)(x / kUnitKeys) + 1);
    }
    *uniform = u;
    int64_t cost = u > 0 ? (int64_t)u * w_cost(p, L, n, 0) : 0;
    for (int t = u; t < nt; ++t) cost += w_cost(p, L, n, t);
    return cost;
}

// One warp: this CTA's share of the chunks and where it starts.
__device__ void w_schedule(const WParams &p, WSched *sc, int lane) {
    int64_t T = 0;
    int uni;
    for (int b = lane; b < p.B; b += 32) {
        const bool report = blockIdx.x == 0;                 // values outside their bounds, once a call
        if (report) cache_entry(p.batch_idx, b, p.B_cache, true);
        T += p.H_k * w_head_cost(p, w_keys(p, b, report), w_queries(p, b, report), &uni);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    const int64_t per = (T + gridDim.x - 1) / gridDim.x;
    const int64_t G0 = min((int64_t)blockIdx.x * per, T), G1 = min(G0 + per, T);
    WSched s;
    s.left = G1 - G0;
    s.b = p.B;
    s.g = s.tile = s.skip = 0;
    int64_t base = 0;
    for (int bb = 0; bb < p.B && G0 < G1; bb += 32) {
        const int b = bb + lane;
        int64_t head = 0;
        if (b < p.B) head = w_head_cost(p, w_keys(p, b, false), w_queries(p, b, false), &uni);
        int64_t incl = p.H_k * head;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, head > 0 && base + incl > G0);
        if (hit) {
            const int l = __ffs(hit) - 1;
            if (lane == l) {
                int64_t r = G0 - (base + incl - p.H_k * head);
                const int L = w_keys(p, b, false), n = w_queries(p, b, false);
                s.b = b;
                s.g = (int)(r / head);
                r -= s.g * head;
                const int64_t c0 = w_cost(p, L, n, 0);
                s.tile = uni > 0 ? (int)min((int64_t)uni, r / c0) : 0;
                r -= s.tile * c0;
                while (r >= w_cost(p, L, n, s.tile)) r -= w_cost(p, L, n, s.tile++);
                s.skip = (int)r;
                *sc = s;
            }
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *sc = s;
}

struct WItem {
    int b, g, tile, entry, L, n;
    int c0, c1;                          // query chunks [c0, c1) of the unit that are this CTA's
    int nkt;                             // key tiles of the unit: 2, or 1 at the end of a sequence
    bool begins, ends;                   // the unit's first / last chunk is among them
};

struct WCursor {
    int b = -1, g = 0, tile = 0, skip = 0;
    int64_t left = 0;
};

__device__ bool w_next(const WParams &p, const WSched &sc, WCursor &cur, WItem &it) {
    if (cur.b < 0) {
        cur.b = sc.b;
        cur.g = sc.g;
        cur.tile = sc.tile;
        cur.skip = sc.skip;
        cur.left = sc.left;
    }
    for (;;) {
        if (cur.b >= p.B || cur.left <= 0) return false;
        const int L = w_keys(p, cur.b, false), n = w_queries(p, cur.b, false);
        if (cur.tile * kUnitKeys < L) {
            const int cost = w_cost(p, L, n, cur.tile), fc = w_first_chunk(p, L, n, cur.tile);
            const int take = (int)min((int64_t)(cost - cur.skip), cur.left);
            it.b = cur.b;
            it.g = cur.g;
            it.tile = cur.tile;
            it.entry = cache_entry(p.batch_idx, cur.b, p.B_cache, false);
            it.L = L;
            it.n = n;
            it.nkt = L - cur.tile * kUnitKeys > kRows ? 2 : 1;
            it.begins = cur.skip == 0;
            it.ends = cur.skip + take == cost;
            it.c0 = fc + cur.skip;
            it.c1 = imin(it.c0 + take, (n + p.TB - 1) / p.TB);   // none without queries
            cur.left -= take;
            cur.skip = 0;
            ++cur.tile;
            return true;
        }
        cur.tile = 0;
        if (++cur.g == p.H_k) {
            cur.g = 0;
            ++cur.b;
        }
    }
}

template <class C>
__device__ void w_producer(const WParams &p, const WSched &sc, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                           uint8_t *smem, WBars *bars) {
    volatile int *abort_flag = &bars->abort;
    uint32_t kf = 0, qf = 0;
    bool ok = test_gate_open(abort_flag);
    WCursor cur;
    while (ok) {
        WItem it;
        if (!w_next(p, sc, cur, it)) break;
        const int e = it.entry >= 0 ? it.entry : p.B_cache;   // out of range: zero fill
        for (int x = 0; ok && x < it.nkt; ++x, ++kf) {
            const int st = kf % C::NK;
            if (kf >= C::NK && !mbar_wait(smem_u32(&bars->k_empty[st]), (kf / C::NK - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint32_t fb = smem_u32(&bars->k_full[st]);
            mbar_expect_tx(fb, C::TILE_BYTES);
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_4d(smem_u32(smem + C::OFF_K + st * C::TILE_BYTES + pn * kPanelBytes), tmK, fb, pn * C::BOX,
                            it.g, it.tile * kUnitKeys + x * kRows, e);
        }
        for (int c = it.c0; ok && c < it.c1; ++c, ++qf) {
            const int st = qf % C::NQ;
            if (qf >= C::NQ && !mbar_wait(smem_u32(&bars->q_empty[st]), (qf / C::NQ - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint32_t fb = smem_u32(&bars->q_full[st]);
            mbar_expect_tx(fb, C::PANELS * p.TB * p.G * 128);
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_3d(smem_u32(smem + C::OFF_Q + st * C::TILE_BYTES + pn * kPanelBytes), tmQ, fb, pn * C::BOX,
                            it.g * p.G, it.b * p.Sq + c * p.TB);
        }
    }
    if (ok) {
        // the last release of every stage must arrive before exit
        for (uint32_t f = kf > C::NK ? kf - C::NK : 0; f < kf; ++f)
            if (!mbar_wait(smem_u32(&bars->k_empty[f % C::NK]), (f / C::NK) & 1, abort_flag)) break;
        for (uint32_t f = qf > C::NQ ? qf - C::NQ : 0; f < qf; ++f)
            if (!mbar_wait(smem_u32(&bars->q_empty[f % C::NQ]), (f / C::NQ) & 1, abort_flag)) break;
    } else {
        // aborted: let the copies already issued land before the CTA exits
        for (uint32_t f = kf > C::NK ? kf - C::NK : 0; f < kf; ++f)
            mbar_wait_drain(smem_u32(&bars->k_full[f % C::NK]), (f / C::NK) & 1);
        for (uint32_t f = qf > C::NQ ? qf - C::NQ : 0; f < qf; ++f)
            mbar_wait_drain(smem_u32(&bars->q_full[f % C::NQ]), (f / C::NQ) & 1);
    }
}

// S^T of every (chunk, key tile) into that tile's two alternating buffers.
template <class C>
__device__ void w_mma(const WParams &p, const WSched &sc, uint8_t *smem, WBars *bars, uint32_t tmem_any) {
    volatile int *abort_flag = &bars->abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    const uint32_t idesc = mma_idesc(C::FMT, p.NMMA, false);
    uint32_t kf = 0, qf = 0, cnt[2] = {0, 0};
    bool ok = true;
    WCursor cur;
    while (ok) {
        WItem it;
        if (!w_next(p, sc, cur, it)) break;
        for (int x = 0; ok && x < it.nkt; ++x)
            ok = warp_wait(smem_u32(&bars->k_full[(kf + x) % C::NK]), ((kf + x) / C::NK) & 1, abort_flag);
        for (int c = it.c0; ok && c < it.c1; ++c, ++qf) {
            const int qst = qf % C::NQ;
            if (!warp_wait(smem_u32(&bars->q_full[qst]), (qf / C::NQ) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint64_t q = smem_desc(smem_u32(smem + C::OFF_Q + qst * C::TILE_BYTES), 16, 1024);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || x >= it.nkt) continue;
                const uint32_t i = cnt[x]++, buf = i & 1;
                if (i >= 2 && !warp_wait(smem_u32(&bars->s_free[x][buf]), ((i - 2) >> 1) & 1, abort_flag)) {
                    ok = false;
                    continue;
                }
                tc_fence_after();
                const uint64_t k =
                    smem_desc(smem_u32(smem + C::OFF_K + ((kf + x) % C::NK) * C::TILE_BYTES), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < kD / C::MMA_K; ++kk) {
                    const uint32_t off = (kk * 32 / 128) * kPanelBytes + (kk * 32) % 128;
                    mma_ss<C::FP8>(tmem + (2 * x + buf) * kRows, k + (off >> 4), q + (off >> 4), idesc, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(&bars->s_full[x][buf]));
            }
            if (ok) tc_commit(smem_u32(&bars->q_empty[qst]));
        }
        if (!ok) break;
        for (int x = 0; x < it.nkt; ++x) tc_commit(smem_u32(&bars->k_empty[(kf + x) % C::NK]));
        kf += it.nkt;
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain));
    mbar_wait_drain(smem_u32(&bars->drain), 0);
}

// Barrier 1 + x over the 128 threads of key tile x, with a vote: all go on or all give up.
__device__ __forceinline__ bool group_all(int x, bool v) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(1 + x)
                 : "memory");
    return r != 0;
}

// Weights: warps 4x .. 4x + 3 own key tile x of every unit, a key a thread.
__device__ void w_sum(const WParams &p, const WSched &sc, WBars *bars, uint32_t tmem, int warp, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 2 * x * kRows;
    const int rt = r / p.G, rh = r % p.G;                // as a chunk's column: its token and head
    uint32_t cnt = 0;
    int parts = 0;                                       // bit s: slot s of this CTA holds a partial
    WCursor cur;
    for (;;) {
        WItem it;
        if (!w_next(p, sc, cur, it)) break;
        const int key = it.tile * kUnitKeys + x * kRows + r;
        const bool whole = it.begins && it.ends;
        const int64_t at = ((int64_t)(it.entry < 0 ? 0 : it.entry) * p.H_k + it.g) * p.S_max + key;
        float old = 0.f;
        if (whole && p.acc_in && key < it.L && it.entry >= 0) old = p.acc_in[at];
        // LSE of this thread's column of chunk c, in log2 units; +inf (weight
        // 0) where the row saw no key
        auto load_lse = [&](int c) {
            const int t = c * p.TB + rt;
            if (rt >= p.TB || t >= it.n) return INFINITY;
            const float v = p.lse[((int64_t)it.b * p.H + it.g * p.G + rh) * p.Sq + t];
            return v == -INFINITY ? INFINITY : v * kLog2e;
        };
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        bool ok = true;
        if (x < it.nkt) {
            float next = it.c0 < it.c1 ? load_lse(it.c0) : 0.f;
            for (int c = it.c0; c < it.c1; ++c, ++cnt) {
                const uint32_t buf = cnt & 1;
                float *lse = bars->lse[x][buf];
                lse[r] = next;           // the threads that read it two chunks ago are past the last barrier
                if (c + 1 < it.c1) next = load_lse(c + 1);
                if (!group_all(x, warp_wait(smem_u32(&bars->s_full[x][buf]), (cnt >> 1) & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int cols = imin(p.TB, it.n - c * p.TB) * p.G;      // valid columns
                // columns below lo are queries that do not see this key
                int lo = 0;
                if (p.causal) {
                    const int t = key - (it.L - it.n) - c * p.TB;        // first token of the chunk that sees it
                    lo = t <= 0 ? 0 : t >= p.TB ? kRows : t * p.G;
                }
                const uint32_t s_tm = lane_base + buf * kRows;
#pragma unroll 1
                for (int q = 0; q < cols; q += 32) {
                    uint32_t s[32];
                    tmem_ld32(s_tm + q, s);
                    tmem_wait_ld(s);
                    if (q + 32 <= cols && __all_sync(0xffffffffu, lo <= q)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[i & 3] += ex2(fmaf(__uint_as_float(s[i]), p.c, -lse[q + i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const bool in = q + i >= lo && q + i < cols;
                            const float w = ex2(fmaf(__uint_as_float(s[i]), p.c, -lse[q + i]));
                            sum[i & 3] += in ? w : 0.f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[x][buf]));
            }
        }
        if (!ok) break;
        const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (whole) {
            if (key < it.L && it.entry >= 0) p.acc_out[at] = old + total;
        } else {
            const int slot = it.begins ? 1 : 0;
            parts |= 1 << slot;
            p.part[((int64_t)2 * blockIdx.x + slot) * kUnitKeys + x * kRows + r] = total;
            if (threadIdx.x == 0) {
                WMeta m;
                m.row = at;
                m.keys = it.entry < 0 ? 0 : imin(kUnitKeys, it.L - it.tile * kUnitKeys);
                m.last = it.ends;
                p.meta[2 * blockIdx.x + slot] = m;
            }
        }
    }
    if (threadIdx.x == 0) {
        // an empty slot; a missing continuation also ends its unit (a CTA that gave up)
        for (int s = 0; s < 2; ++s)
            if (!(parts >> s & 1)) p.meta[2 * blockIdx.x + s] = WMeta{0, 0, 1};
    }
}

template <int ELEM>
__global__ void __launch_bounds__(kWThreads, 1)
    fmha_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const WParams p) {
    using C = WCfg<ELEM>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    WBars *bars = reinterpret_cast<WBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(smem_u32(&bars->k_full[s]), 1);
            mbar_init(smem_u32(&bars->k_empty[s]), 1);
        }
        for (int s = 0; s < C::NQ; ++s) {
            mbar_init(smem_u32(&bars->q_full[s]), 1);
            mbar_init(smem_u32(&bars->q_empty[s]), 1);
        }
        for (int x = 0; x < 2; ++x)
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&bars->s_full[x][b]), 1);
                mbar_init(smem_u32(&bars->s_free[x][b]), 4);
            }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWMma) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == kWProd) {
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
        }
        w_schedule(p, &bars->sched, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const WSched sc = bars->sched;
    if (warp < 8) {
        w_sum(p, sc, bars, tmem, warp, lane);
    } else if (warp == kWProd) {
        if (lane == 0) w_producer<C>(p, sc, &tmQ, &tmK, smem, bars);
    } else {
        w_mma<C>(p, sc, smem, bars, tmem);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWMma) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// CTA c joins the unit that CTA c of the kernel above began and did not end.
__global__ void __launch_bounds__(kUnitKeys) fmha_weights_join_kernel(const WParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WMeta m = p.meta[2 * blockIdx.x + 1];
    if (m.keys == 0 || (int)threadIdx.x >= m.keys) return;
    float sum = p.part[((int64_t)2 * blockIdx.x + 1) * kUnitKeys + threadIdx.x];
    for (unsigned c = blockIdx.x + 1, last = m.last; !last && c < gridDim.x; ++c) {
        const WMeta x = p.meta[2 * c];
        sum += p.part[(int64_t)2 * c * kUnitKeys + threadIdx.x];
        last = x.last;
    }
    const int64_t at = m.row + threadIdx.x;
    p.acc_out[at] = (p.acc_in ? p.acc_in[at] : 0.f) + sum;
}

int w_tokens(int Sq, int G) { return imin(kRows / G, Sq); }

}  // namespace

int weights_set_wait_limit(unsigned long long ns) { return cache_set_wait_limit(ns); }
int weights_set_test_gate(int on) { return cache_set_test_gate(on); }
int weights_read_status(int reset) { return cache_read_status(reset); }

}  // namespace fmha

using namespace fmha;

extern "C" size_t fmha_cache_weights_workspace_size(void) {
    return (size_t)2 * kWeightsMaxCtas * (kUnitKeys * sizeof(float) + sizeof(WMeta));
}

extern "C" int fmha_cache_weights(fmha_tensor q, fmha_tensor k_cache, const float *lse, const float *acc_in,
                                  float *acc_out, int B, int Sq, int H, int H_k, int D, int B_cache, int S_max,
                                  const int *seqlen, const int *batch_idx, const int *n_query, float scale, int mask,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    // ---- host-side validation: nothing is launched on a bad argument ----
    if (B < 0 || Sq < 0 || H <= 0 || H_k <= 0 || H % H_k != 0 || H / H_k > kRows || D != kD) return FMHA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY)) return FMHA_ERR_INVALID_ARG;
    if (mask != FMHA_MASK_NONE && mask != FMHA_MASK_CAUSAL) return FMHA_ERR_INVALID_ARG;
    if (B == 0 || Sq == 0) return FMHA_OK;
    if (S_max <= 0 || B_cache <= 0 || !seqlen || !lse || !acc_out) return FMHA_ERR_INVALID_ARG;
    if (!q.data || !k_cache.data) return FMHA_ERR_INVALID_ARG;
    const int dt = q.dtype;
    if (dt != FMHA_F16 && dt != FMHA_BF16 && dt != FMHA_E4M3) return FMHA_ERR_UNSUPPORTED;
    if (k_cache.dtype != dt) return FMHA_ERR_UNSUPPORTED;
    if (misaligned(q.data, 16) || misaligned(k_cache.data, 16)) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {(const void *)lse, (const void *)acc_in, (const void *)acc_out, (const void *)seqlen,
                            (const void *)batch_idx, (const void *)n_query})
        if (misaligned(ptr, 4)) return FMHA_ERR_INVALID_ARG;
    if ((int64_t)B * Sq >= (int64_t(1) << 31) / kRows || S_max > (1 << 30)) return FMHA_ERR_INVALID_ARG;
    const size_t acc_bytes = (size_t)B_cache * H_k * S_max * sizeof(float);
    const char *ai = reinterpret_cast<const char *>(acc_in), *ao = reinterpret_cast<const char *>(acc_out);
    if (acc_in && ai != ao && ai < ao + acc_bytes && ao < ai + acc_bytes) return FMHA_ERR_INVALID_ARG;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < fmha_cache_weights_workspace_size())
        return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    const int sms = sm_count();
    if (sms <= 0) return FMHA_ERR_CUDA;

    WParams p{};
    p.lse = lse;
    p.acc_in = acc_in;
    p.acc_out = acc_out;
    p.seqlen = seqlen;
    p.batch_idx = batch_idx;
    p.n_query = n_query;
    p.B = B;
    p.Sq = Sq;
    p.H = H;
    p.H_k = H_k;
    p.G = H / H_k;
    p.B_cache = B_cache;
    p.S_max = S_max;
    p.TB = w_tokens(Sq, p.G);
    p.NMMA = (p.TB * p.G + 15) / 16 * 16;
    p.causal = mask == FMHA_MASK_CAUSAL;
    p.c = scale * kLog2e;
    const int chunks = (Sq + p.TB - 1) / p.TB;
    const int64_t work = (int64_t)B * H_k * (((int64_t)S_max + kUnitKeys - 1) / kUnitKeys) * chunks;
    const int grid = (int)(work < imin(sms, kWeightsMaxCtas) ? work : imin(sms, kWeightsMaxCtas));
    p.part = static_cast<float *>(workspace);
    p.meta = reinterpret_cast<WMeta *>(p.part + (size_t)2 * kWeightsMaxCtas * kUnitKeys);

    CUtensorMap tq, tk;
    const cuuint32_t box_d = dt == FMHA_E4M3 ? 128 : 64;
    const cuuint64_t dq[3] = {kD, (cuuint64_t)H, (cuuint64_t)B * Sq};
    const cuuint32_t bq[3] = {box_d, (cuuint32_t)p.G, (cuuint32_t)p.TB};
    const cuuint64_t dk[4] = {kD, (cuuint64_t)H_k, (cuuint64_t)S_max, (cuuint64_t)B_cache};
    const cuuint32_t bk[4] = {box_d, 1, kRows, 1};
    if (!make_map(&tq, dt, q.data, 3, dq, bq) || !make_map(&tk, dt, k_cache.data, 4, dk, bk, row_promotion(dt))) return FMHA_ERR_CUDA;

    auto kern = dt == FMHA_BF16 ? fmha_weights_kernel<FMHA_BF16>
                : dt == FMHA_F16 ? fmha_weights_kernel<FMHA_F16> : fmha_weights_kernel<FMHA_E4M3>;
    const int smem = dt == FMHA_E4M3 ? WCfg<FMHA_E4M3>::SMEM_BYTES : WCfg<FMHA_BF16>::SMEM_BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return cuda_failed();
    kern<<<grid, kWThreads, smem, stream>>>(tq, tk, p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;
    if (chunks > 1) {                    // else no unit is ever cut
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kUnitKeys);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, fmha_weights_join_kernel, p) != cudaSuccess) return cuda_failed();
    }
    return FMHA_OK;
}
