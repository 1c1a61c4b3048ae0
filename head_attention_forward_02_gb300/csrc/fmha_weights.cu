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
// A unit is 512 keys of one kv head (four MMA tiles that share the query
// stream: with two, a chunk took the 1950 cycles that the SMs together need to
// fetch theirs from L2) and its query chunks (TB = 128 / G tokens each).  The
// chunks of all units form one sequence, kv heads fastest, so that a CTA reads
// the heads' rows of the same keys one after another (they are adjacent in the
// cache).  The sequence is cut evenly over the CTAs; a unit that is cut leaves
// partial sums (a float a key) in the workspace and a second kernel adds them
// in CTA order, so results do not depend on timing.
//
// Measured: one token a sequence (B=32, H=32, H_k=8, 8192 keys, ragged) 63 us,
// 5.6 TB/s of keys; the last 33 tokens of four e4m3 prompts of 16384 (H=64,
// H_k=8) 33 us; every row of a prompt of 4096 (H=32, H_k=8, causal) 67 us,
// 1.02 PFLOP/s.  A chunk takes 3700 cycles where its MMAs and its exponentials
// need 2050 each: S has one TMEM buffer a tile, so the chain freed -> issued ->
// there -> loaded -> half of it added is serial for a tile, and four tiles in
// flight do not fill either unit (without the exponentials the prompt takes
// 62 us, without the LSE loads 64, without both and 7/8 of the MMAs 47).
#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kWeightsMaxCtas = 152;     // CTAs at most (bounds the workspace)
constexpr int kGroups = 4;               // groups of four summing warps, a key tile of the unit each
constexpr int kUnitMax = kGroups * kRows;                    // keys of the largest unit
constexpr int kWProd = 16, kWLse = 17, kWMma = 18;           // then the producer, LSE loader and two MMA issuers
constexpr int kWThreads = 640;

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
    float *part;                         // [2 * ncta][UK]
    int B, Sq, H, H_k, G, B_cache, S_max;
    int TB;                              // query tokens of a chunk
    int UK;                              // keys of a unit: 512, or 256 where those are too few
    int NMMA;                            // MMA N: TB * G rounded up to 16
    int causal;
    int whole;                           // units are not cut: a CTA takes those that begin in its share
    float c;                             // scale * log2(e)
};

struct WItem {
    int b, g, tile, entry, L, n;         // b < 0: no more items
    int c0, c1;                          // query chunks [c0, c1) of the unit that are this CTA's
    int nkt;                             // K tiles to load: UK / 128, or fewer at the end of a sequence
    bool begins, ends;                   // the unit's first / last chunk is among them
};

constexpr int kWItems = 4;               // work items published ahead
constexpr int kWStages = 14;             // ring stages at most, K's and Q's together

struct WBars {
    uint64_t full[kWStages], empty[kWStages];            // K ring, then Q ring
    uint64_t s_full[kGroups], s_free[kGroups], drain[2];
    uint64_t lse_full[2], lse_free[2];
    uint64_t item_full[kWItems], item_empty[kWItems];
    WItem item[kWItems];
    uint32_t tmem_base;
    int abort;
    alignas(16) float lse[2][kRows];     // by buffer: a chunk's -LSE in log2 units
};

// Ring stages of 128 rows, 224 KB in all.  Where a sequence's rows fill one
// chunk (ONE) the stream is K's, 160 KB of it in flight; else it is Q's, 32 KB
// a chunk (16-bit) from L2.
template <int ELEM, bool ONE>
struct WCfg : ElemCfg<ELEM> {
    using B = ElemCfg<ELEM>;
    static constexpr int NK = (ONE ? 5 : 4) * 32768 / B::TILE_BYTES;
    static constexpr int NQ = (ONE ? 2 : 3) * 32768 / B::TILE_BYTES;
    static_assert(NK + NQ <= kWStages, "ring barriers");
    static constexpr int OFF_K = 0;
    static constexpr int OFF_Q = NK * B::TILE_BYTES;
    static constexpr int OFF_BARS = OFF_Q + NQ * B::TILE_BYTES;
    static constexpr int SMEM_BYTES = OFF_BARS + sizeof(WBars) + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ int w_keys(const WParams &p, int b, bool report) {
    return clamped(p.seqlen[b], 0, p.S_max, report);
}
__device__ __forceinline__ int w_queries(const WParams &p, int b, bool report) {
    return p.n_query ? clamped(p.n_query[b], 0, p.Sq, report) : p.Sq;
}

// Chunks of a sequence's n rows.
__device__ __forceinline__ int w_chunks(const WParams &p, int n) { return (n + p.TB - 1) / p.TB; }

// Query t of a sequence sees key j iff j <= t + L - n (causal): the first
// chunk of unit `tile` that holds a query which sees one of its keys.
__device__ __forceinline__ int w_first_chunk(const WParams &p, int L, int n, int tile) {
    if (!p.causal) return 0;
    const int t = tile * p.UK - (L - n);
    return t > 0 ? t / p.TB : 0;
}
// Chunks of a unit; a sequence without queries still copies acc: one empty chunk.
__device__ __forceinline__ int w_cost(const WParams &p, int L, int n, int tile) {
    return imax(1, w_chunks(p, n) - w_first_chunk(p, L, n, tile));
}
// Units [0, *uniform) of one head cost the same; the sum over all of them.
__device__ __forceinline__ int64_t w_head_cost(const WParams &p, int L, int n, int *uniform) {
    const int nt = (L + p.UK - 1) / p.UK;
    int u = nt;
    if (p.causal) {
        const int64_t x = (int64_t)p.TB - 1 + L - n;         // last key whose unit still starts at chunk 0
        u = x < 0 ? 0 : imin(nt, (int)(x / p.UK) + 1);
    }
    *uniform = u;
    int64_t cost = u > 0 ? (int64_t)u * w_cost(p, L, n, 0) : 0;
    for (int t = u; t < nt; ++t) cost += w_cost(p, L, n, t);
    return cost;
}

// Where the producer is in this CTA's chunks.
struct WCursor {
    int64_t left;                        // chunks still to hand out
    int b, g, tile, skip;                // next unit, and chunks of it that are other CTAs'
    int L, n, entry;                     // of sequence b
};

__device__ __forceinline__ void w_load_seq(const WParams &p, WCursor &cur) {
    cur.L = w_keys(p, cur.b, false);
    cur.n = w_queries(p, cur.b, false);
    cur.entry = cache_entry(p.batch_idx, cur.b, p.B_cache, false);
}

// One warp: this CTA's share of the chunks and where it starts (the same in every lane).
__device__ void w_schedule(const WParams &p, WCursor &cur, int lane) {
    int64_t T = 0;
    int uni;
    for (int b = lane; b < p.B; b += 32) T += p.H_k * w_head_cost(p, w_keys(p, b, false), w_queries(p, b, false), &uni);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    const int64_t per = (T + gridDim.x - 1) / gridDim.x;
    const int64_t G0 = min((int64_t)blockIdx.x * per, T), G1 = min(G0 + per, T);
    if (blockIdx.x == gridDim.x - 1)     // reports values outside their bounds, once a call
        for (int b = lane; b < p.B; b += 32) {
            w_keys(p, b, true);
            w_queries(p, b, true);
            cache_entry(p.batch_idx, b, p.B_cache, true);
        }
    cur.left = G1 - G0;
    cur.b = p.B;
    cur.g = cur.tile = cur.skip = 0;
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
            cur.b = bb + l;
            w_load_seq(p, cur);
            head = __shfl_sync(0xffffffffu, head, l);
            uni = __shfl_sync(0xffffffffu, uni, l);
            int64_t r = G0 - (__shfl_sync(0xffffffffu, base + incl, l) - p.H_k * head);
            auto cost = [&](int tile) { return (int64_t)p.H_k * w_cost(p, cur.L, cur.n, tile); };
            cur.tile = uni > 0 ? (int)min((int64_t)uni, r / cost(0)) : 0;
            r -= cur.tile * cost(0);
            while (r >= cost(cur.tile)) r -= cost(cur.tile++);
            const int unit = w_cost(p, cur.L, cur.n, cur.tile);
            cur.g = (int)(r / unit);
            r -= (int64_t)cur.g * unit;
            if (!p.whole) {
                cur.skip = (int)r;
            } else if (r > 0) {          // the unit began in the share before
                cur.left -= unit - r;
                if (++cur.g == p.H_k) {
                    cur.g = 0;
                    ++cur.tile;
                }
            }
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ bool w_next(const WParams &p, WCursor &cur, WItem &it) {
    it.b = -1;
    for (;;) {
        if (cur.b >= p.B || cur.left <= 0) return false;
        if (cur.tile * p.UK < cur.L) {
            const int cost = w_cost(p, cur.L, cur.n, cur.tile), fc = w_first_chunk(p, cur.L, cur.n, cur.tile);
            const int take = p.whole ? cost : (int)min((int64_t)(cost - cur.skip), cur.left);
            it.b = cur.b;
            it.g = cur.g;
            it.tile = cur.tile;
            it.entry = cur.entry;
            it.L = cur.L;
            it.n = cur.n;
            it.nkt = imin(p.UK / kRows, (cur.L - cur.tile * p.UK + kRows - 1) / kRows);
            it.begins = cur.skip == 0;
            it.ends = cur.skip + take == cost;
            it.c0 = fc + cur.skip;
            it.c1 = imin(it.c0 + take, w_chunks(p, cur.n));          // none without queries
            cur.left -= take;
            cur.skip = 0;
            if (++cur.g == p.H_k) {
                cur.g = 0;
                ++cur.tile;
            }
            return true;
        }
        cur.tile = 0;
        if (++cur.b < p.B) w_load_seq(p, cur);
    }
}

// Items: the producer publishes them ahead of its loads; the other warps take
// a copy each and hand the slot back.
__device__ __forceinline__ bool w_publish(WBars *bars, uint32_t i, const WItem &it, volatile int *abort_flag) {
    const uint32_t st = i % kWItems;
    if (i >= kWItems && !mbar_wait(smem_u32(&bars->item_empty[st]), (i / kWItems - 1) & 1, abort_flag)) return false;
    bars->item[st] = it;
    mbar_arrive(smem_u32(&bars->item_full[st]));
    return true;
}

__device__ __forceinline__ bool w_take(WBars *bars, uint32_t i, WItem &it, volatile int *abort_flag, int lane) {
    const uint32_t st = i % kWItems;
    if (!warp_wait(smem_u32(&bars->item_full[st]), (i / kWItems) & 1, abort_flag)) return false;
    it = bars->item[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[st]));
    return it.b >= 0;
}

template <class C>
__device__ void w_producer(const WParams &p, WCursor &cur, int gate, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                           uint8_t *smem, WBars *bars) {
    volatile int *abort_flag = &bars->abort;
    uint64_t *k_full = bars->full, *k_empty = bars->empty, *q_full = k_full + C::NK, *q_empty = k_empty + C::NK;
    uint32_t kf = 0, qf = 0;
    bool ok = !gate || test_gate_open(abort_flag);
    WItem it, next;
    if (ok) {
        w_next(p, cur, it);
        ok = w_publish(bars, 0, it, abort_flag);
    }
    for (uint32_t i = 1; ok && it.b >= 0; ++i, it = next) {
        const int e = it.entry >= 0 ? it.entry : p.B_cache;   // out of range: zero fill
        auto load_q = [&](int c) {
            const int st = qf % C::NQ;
            if (qf >= C::NQ && !mbar_wait(smem_u32(&q_empty[st]), (qf / C::NQ - 1) & 1, abort_flag)) return false;
            const uint32_t fb = smem_u32(&q_full[st]);
            mbar_expect_tx(fb, C::PANELS * p.TB * p.G * 128);
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_3d(smem_u32(smem + C::OFF_Q + st * C::TILE_BYTES + pn * kPanelBytes), tmQ, fb, pn * C::BOX,
                            it.g * p.G, it.b * p.Sq + c * p.TB);
            ++qf;
            return true;
        };
        // the first chunk's Q goes ahead of K, whose stages come free later
        if (it.c0 < it.c1) ok = load_q(it.c0);
        for (int x = 0; ok && x < it.nkt; ++x) {
            const int st = kf % C::NK;
            if (kf >= C::NK && !mbar_wait(smem_u32(&k_empty[st]), (kf / C::NK - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint32_t fb = smem_u32(&k_full[st]);
            mbar_expect_tx(fb, C::TILE_BYTES);
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_4d(smem_u32(smem + C::OFF_K + st * C::TILE_BYTES + pn * kPanelBytes), tmK, fb, pn * C::BOX,
                            it.g, it.tile * p.UK + x * kRows, e);
            ++kf;
        }
        if (!ok) break;
        w_next(p, cur, next);
        ok = w_publish(bars, i, next, abort_flag);
        for (int c = it.c0 + 1; ok && c < it.c1; ++c) ok = load_q(c);
    }
    // the last release of every stage must arrive before exit; when the CTA
    // gave up, only the copies already issued
    for (uint32_t f = kf > C::NK ? kf - C::NK : 0; f < kf; ++f) {
        if (ok) ok = mbar_wait(smem_u32(&k_empty[f % C::NK]), (f / C::NK) & 1, abort_flag);
        if (!ok) mbar_wait_drain(smem_u32(&k_full[f % C::NK]), (f / C::NK) & 1);
    }
    for (uint32_t f = qf > C::NQ ? qf - C::NQ : 0; f < qf; ++f) {
        if (ok) ok = mbar_wait(smem_u32(&q_empty[f % C::NQ]), (f / C::NQ) & 1, abort_flag);
        if (!ok) mbar_wait_drain(smem_u32(&q_full[f % C::NQ]), (f / C::NQ) & 1);
    }
}

// S^T of every (chunk, key tile): tile x of a unit is group x's, and issuer x % 2
// issues it, so that one issuer's waits pass under the other's MMAs (with one,
// a tile took 900 cycles for 512 of MMAs).  Both wait for every K tile and
// give it back, so that neither misses a phase of its barrier.
template <class C>
__device__ void w_mma(const WParams &p, uint8_t *smem, WBars *bars, uint32_t tmem_any, int who, int lane) {
    volatile int *abort_flag = &bars->abort;
    uint64_t *k_full = bars->full, *k_empty = bars->empty, *q_full = k_full + C::NK, *q_empty = k_empty + C::NK;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    const uint32_t idesc = mma_idesc(C::FMT, p.NMMA, false);
    uint32_t kf = 0, qf = 0;             // K tiles and chunks so far
    uint32_t cnt[2] = {0, 0};            // of groups who and who + 2: their chunks
    bool ok = true;
    WItem it;
    for (uint32_t i = 0; ok && w_take(bars, i, it, abort_flag, lane); ++i) {
        int landed = 0;                  // K tiles of the unit that are here
        for (int c = it.c0; ok && c < it.c1; ++c, ++qf) {
            const int qst = qf % C::NQ;
            if (!warp_wait(smem_u32(&q_full[qst]), (qf / C::NQ) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint64_t q = smem_desc(smem_u32(smem + C::OFF_Q + qst * C::TILE_BYTES), 16, 1024);
#pragma unroll
            for (int y = 0; y < kGroups / 2; ++y) {
                const int x = who + 2 * y;
                if (!ok || x >= it.nkt) continue;
                for (; ok && landed <= x; ++landed)
                    ok = warp_wait(smem_u32(&k_full[(kf + landed) % C::NK]), ((kf + landed) / C::NK) & 1, abort_flag);
                if (ok && cnt[y] > 0) ok = warp_wait(smem_u32(&bars->s_free[x]), (cnt[y] - 1) & 1, abort_flag);
                if (!ok) continue;
                ++cnt[y];
                tc_fence_after();
                const int st = (kf + x) % C::NK;
                const uint64_t k = smem_desc(smem_u32(smem + C::OFF_K + st * C::TILE_BYTES), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < kD / C::MMA_K; ++kk) {
                    const uint32_t off = (kk * 32 / 128) * kPanelBytes + (kk * 32) % 128;
                    mma_ss<C::FP8>(tmem + x * kRows, k + (off >> 4), q + (off >> 4), idesc, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(&bars->s_full[x]));
                if (c == it.c1 - 1) tc_commit(smem_u32(&k_empty[st]));       // the unit's last use of it
            }
            if (ok) tc_commit(smem_u32(&q_empty[qst]));
        }
        for (; ok && landed < it.nkt; ++landed)
            ok = warp_wait(smem_u32(&k_full[(kf + landed) % C::NK]), ((kf + landed) / C::NK) & 1, abort_flag);
        if (!ok) break;
        // the other issuer's tiles, and all of them where there is no chunk
        for (int x = 0; x < it.nkt; ++x)
            if (lane == 0 && ((x & 1) != who || it.c0 >= it.c1)) mbar_arrive(smem_u32(&k_empty[(kf + x) % C::NK]));
        kf += it.nkt;
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain[who]));
    mbar_wait_drain(smem_u32(&bars->drain[who]), 0);
}

// One warp: -LSE of every chunk's columns, in log2 units (-inf, weight 0,
// where the row saw no key), into one of two buffers in shared memory.  (With
// the summing threads loading it, a chunk had two barriers of 128 threads more.)
__device__ void w_load_lse(const WParams &p, WBars *bars, int lane) {
    volatile int *abort_flag = &bars->abort;
    uint32_t n = 0;                      // chunks so far
    WItem it;
    for (uint32_t i = 0; w_take(bars, i, it, abort_flag, lane); ++i) {
        const float *lse = p.lse + ((int64_t)it.b * p.H + it.g * p.G) * p.Sq;
        float next[4];                   // a chunk's values are fetched before the buffer of the chunk before is free
        auto fetch = [&](int c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 32 * k + lane, rt = r / p.G, t = c * p.TB + rt;
                next[k] = rt < p.TB && t < it.n ? lse[(int64_t)(r - rt * p.G) * p.Sq + t] : -INFINITY;
            }
        };
        fetch(it.c0);
        for (int c = it.c0; c < it.c1; ++c, ++n) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = next[k];
            if (c + 1 < it.c1) fetch(c + 1);
            const uint32_t buf = n & 1;
            if (n >= 2 && !warp_wait(smem_u32(&bars->lse_free[buf]), ((n - 2) >> 1) & 1, abort_flag)) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) bars->lse[buf][32 * k + lane] = v[k] == -INFINITY ? -INFINITY : v[k] * -kLog2e;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->lse_full[buf]));
        }
    }
}

// Weights: warps 4 x .. 4 x + 3 own key tile x of every unit, a key a thread.
// Four warps an SM sub-partition hide one another's latencies (two, with twice
// the columns in registers, took 1500 cycles for 128 columns of a tile, of
// which they issued 350).
__device__ void w_sum(const WParams &p, WBars *bars, uint32_t tmem, int warp, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int x = warp >> 2, r = warp * 32 + lane;       // key tile, key of the unit
    const uint32_t s_tm = tmem + ((uint32_t)((warp & 3) * 32) << 16) + x * kRows;
    const uint64_t c2 = pack_f2(p.c, p.c);
    uint32_t n = 0, m = 0;                               // chunks so far, and those of this group's tiles
    int parts = 0;                                       // bit s: slot s of this CTA holds a partial
    WItem it;
    for (uint32_t i = 0; w_take(bars, i, it, abort_flag, lane); ++i) {
        const int key = it.tile * p.UK + r;
        const bool whole = it.begins && it.ends, mine = key < it.L && it.entry >= 0;
        const int64_t at = ((int64_t)(it.entry < 0 ? 0 : it.entry) * p.H_k + it.g) * p.S_max + key;
        const float old = whole && p.acc_in && mine ? p.acc_in[at] : 0.f;
        uint64_t sum[2] = {0, 0};        // two pairs of partial sums
        bool ok = true;
        for (int c = it.c0; c < it.c1; ++c, ++n) {
            const float *lse = bars->lse[n & 1];
            if (!warp_wait(smem_u32(&bars->lse_full[n & 1]), (n >> 1) & 1, abort_flag) ||
                (x < it.nkt && !warp_wait(smem_u32(&bars->s_full[x]), m++ & 1, abort_flag))) {
                ok = false;
                break;
            }
            if (x >= it.nkt) {           // no tile at the end of a sequence
                if (lane == 0) mbar_arrive(smem_u32(&bars->lse_free[n & 1]));
                continue;
            }
            tc_fence_after();
            const int cols = imin(p.TB, it.n - c * p.TB) * p.G;        // valid columns
            // columns below lo are queries that do not see this key
            int lo = 0;
            if (p.causal) {
                const int t = key - (it.L - it.n) - c * p.TB;           // first token of the chunk that sees it
                lo = t <= 0 ? 0 : t >= p.TB ? kRows : t * p.G;
            }
            // 32 columns: weights of pairs
            auto add = [&](const uint32_t (&s)[32], int q) {
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const ulonglong2 nl = *reinterpret_cast<const ulonglong2 *>(lse + q + k);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint64_t s2 = pack_f2(__uint_as_float(s[k + 2 * z]), __uint_as_float(s[k + 2 * z + 1]));
                        float a, b;
                        unpack_f2(fma_f2(s2, c2, z ? nl.y : nl.x), a, b);
                        sum[z] = add_f2(sum[z], pack_f2(ex2(a), ex2(b)));
                    }
                }
            };
            // S^T is in registers: the next chunk's may come
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[x]));
            };
            if (p.NMMA == kRows && cols == p.TB * p.G && __all_sync(0xffffffffu, lo == 0)) {
#pragma unroll 1
                for (int q = 0; q < kRows; q += 64) {
                    uint32_t s[2][32];
                    tmem_ld32(s_tm + q, s[0]);
                    tmem_ld32(s_tm + q + 32, s[1]);
                    tmem_wait_ld(s[0]);
                    tmem_wait_ld(s[1]);
                    if (q > 0) release();
                    add(s[0], q);
                    add(s[1], q + 32);
                }
            } else {
#pragma unroll 1
                for (int q = 0; q < cols; q += 32) {
                    // a bit for every column that counts; the others' scores become -inf
                    const int l = lo - q, h = cols - q;
                    const uint32_t vis = (l <= 0 ? 0xffffffffu : l >= 32 ? 0u : 0xffffffffu << l) &
                                         (h >= 32 ? 0xffffffffu : (1u << h) - 1u);
                    if (__all_sync(0xffffffffu, vis == 0u)) continue;
                    uint32_t s[32];
                    tmem_ld32(s_tm + q, s);
                    tmem_wait_ld(s);
                    if (!__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((vis >> k) & 1u)) s[k] = 0xff800000u;
                    }
                    add(s, q);
                }
                release();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->lse_free[n & 1]));
        }
        if (!ok) break;
        float t0, t1, t2, t3;
        unpack_f2(sum[0], t0, t1);
        unpack_f2(sum[1], t2, t3);
        const float total = (t0 + t1) + (t2 + t3);
        if (whole) {
            if (mine) p.acc_out[at] = old + total;
        } else {
            const int slot = it.begins ? 1 : 0;
            parts |= 1 << slot;
            p.part[((int64_t)2 * blockIdx.x + slot) * p.UK + r] = total;
            if (threadIdx.x == 0) {
                const int keys = it.entry < 0 ? 0 : imin(p.UK, it.L - it.tile * p.UK);
                p.meta[2 * blockIdx.x + slot] = WMeta{at, keys, it.ends};
            }
        }
    }
    if (threadIdx.x == 0) {
        // an empty slot; a missing continuation also ends its unit (a CTA that gave up)
        for (int s = 0; s < 2; ++s)
            if (!(parts >> s & 1)) p.meta[2 * blockIdx.x + s] = WMeta{0, 0, 1};
    }
}

template <int ELEM, bool ONE>
__global__ void __launch_bounds__(kWThreads, 1)
    fmha_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const WParams p) {
    using C = WCfg<ELEM, ONE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    WBars *bars = reinterpret_cast<WBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NK + C::NQ; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 2);         // both issuers
        }
        for (int x = 0; x < kGroups; ++x) {
            mbar_init(smem_u32(&bars->s_full[x]), 1);
            mbar_init(smem_u32(&bars->s_free[x]), 4);
        }
        const int summing = p.UK / 32;                       // warps that sum
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars->lse_full[b]), 1);
            mbar_init(smem_u32(&bars->lse_free[b]), summing);
        }
        for (int s = 0; s < kWItems; ++s) {
            mbar_init(smem_u32(&bars->item_full[s]), 1);
            mbar_init(smem_u32(&bars->item_empty[s]), summing + 3);
        }
        mbar_init(smem_u32(&bars->drain[0]), 1);
        mbar_init(smem_u32(&bars->drain[1]), 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWMma) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    // rows of a full chunk that hold no query (G = 3: two) are zero, so that
    // all 128 columns can be summed (those have an LSE that makes them 0)
    if (p.NMMA == kRows && p.TB * p.G < kRows) {
        const int pieces = (kRows - p.TB * p.G) * 8;
        for (int i = threadIdx.x; i < pieces * C::NQ * C::PANELS; i += kWThreads)
            *reinterpret_cast<uint4 *>(smem + C::OFF_Q + (i / pieces) * kPanelBytes + p.TB * p.G * 128 + i % pieces * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        proxy_fence();
    }
    WCursor cur;
    int gate = 0;
    if (warp == kWProd) {
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
        }
        gate = g_test_gate;              // read along with the lengths
        w_schedule(p, cur, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < kWProd) {
        if (warp * 32 < p.UK) w_sum(p, bars, tmem, warp, lane);
    } else if (warp == kWProd) {
        if (lane == 0) w_producer<C>(p, cur, gate, &tmQ, &tmK, smem, bars);
    } else if (warp == kWLse) {
        w_load_lse(p, bars, lane);
    } else {
        w_mma<C>(p, smem, bars, tmem, warp - kWMma, lane);
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
__global__ void __launch_bounds__(kUnitMax) fmha_weights_join_kernel(const WParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WMeta m = p.meta[2 * blockIdx.x + 1];
    if ((int)threadIdx.x >= m.keys) return;
    float sum = p.part[((int64_t)2 * blockIdx.x + 1) * p.UK + threadIdx.x];
    for (unsigned c = blockIdx.x + 1, last = m.last; !last && c < gridDim.x; ++c) {
        sum += p.part[(int64_t)2 * c * p.UK + threadIdx.x];
        last = p.meta[2 * c].last;
    }
    const int64_t at = m.row + threadIdx.x;
    p.acc_out[at] = (p.acc_in ? p.acc_in[at] : 0.f) + sum;
}

using WKernel = void (*)(CUtensorMap, CUtensorMap, WParams);
template <int ELEM>
WKernel w_kernel(bool one) {
    return one ? fmha_weights_kernel<ELEM, true> : fmha_weights_kernel<ELEM, false>;
}

int w_tokens(int Sq, int G) { return imin(kRows / G, Sq); }

}  // namespace

int weights_set_wait_limit(unsigned long long ns) { return cache_set_wait_limit(ns); }
int weights_set_test_gate(int on) { return cache_set_test_gate(on); }
int *weights_status_word() { return symbol_address(g_status); }

}  // namespace fmha

using namespace fmha;

extern "C" size_t fmha_cache_weights_workspace_size(void) {
    return (size_t)2 * kWeightsMaxCtas * (kUnitMax * sizeof(float) + sizeof(WMeta));
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
    if ((int64_t)B * Sq >= (int64_t(1) << 31) / kRows || S_max > kMaxCacheRows) return FMHA_ERR_INVALID_ARG;
    const size_t acc_bytes = (size_t)B_cache * H_k * S_max * sizeof(float);
    if (acc_in && acc_in != acc_out && overlap(acc_in, acc_bytes, acc_out, acc_bytes)) return FMHA_ERR_INVALID_ARG;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < fmha_cache_weights_workspace_size())
        return FMHA_ERR_INVALID_ARG;
    const size_t seq_bytes = (size_t)B * sizeof(int), row = kD * (dt == FMHA_E4M3 ? 1 : 2);
    const Bytes out[2] = {{acc_out, acc_bytes}, {workspace, fmha_cache_weights_workspace_size()}};
    const Bytes in[6] = {{q.data, (size_t)B * Sq * H * row}, {k_cache.data, (size_t)B_cache * S_max * H_k * row},
                         {lse, (size_t)B * H * Sq * sizeof(float)}, {seqlen, seq_bytes}, {batch_idx, seq_bytes},
                         {n_query, seq_bytes}};
    if (outputs_clash(out, in) || overlap(out[1], Bytes{acc_in, acc_bytes})) return FMHA_ERR_INVALID_ARG;
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
    p.c = log2_scale(scale);
    const int chunks = (Sq + p.TB - 1) / p.TB;
    // units of 512 keys, or of half that where they would not fill the SMs
    const bool one = chunks == 1;
    p.UK = (int64_t)B * H_k * (((int64_t)S_max + kUnitMax - 1) / kUnitMax) * chunks >= sms ? kUnitMax : kUnitMax / 2;
    const int64_t units = (int64_t)B * H_k * (((int64_t)S_max + p.UK - 1) / p.UK), work = units * chunks;
    const int most = imin(sms, kWeightsMaxCtas), grid = (int)(work < most ? work : most);
    // Units of two chunks stay whole where a CTA gets at most one: nothing has to
    // be joined, and the host saves 3 us of 17.  Cut / whole in us, 32/8 heads:
    // B=3, 44 e4m3 rows 8.9 / 8.2; B=2, 64 rows on 4000 keys 13.0 / 11.7; three
    // chunks (90 rows on 1000 keys) 10.3 / 11.6; four (128) 9.6 / 12.3.
    p.whole = chunks == 2 && units <= grid;
    p.part = static_cast<float *>(workspace);
    p.meta = reinterpret_cast<WMeta *>(p.part + (size_t)2 * kWeightsMaxCtas * kUnitMax);

    CUtensorMap tq, tk;
    const cuuint32_t box_d = dt == FMHA_E4M3 ? 128 : 64;
    const cuuint64_t dq[3] = {kD, (cuuint64_t)H, (cuuint64_t)B * Sq};
    const cuuint32_t bq[3] = {box_d, (cuuint32_t)p.G, (cuuint32_t)p.TB};
    const cuuint64_t dk[4] = {kD, (cuuint64_t)H_k, (cuuint64_t)S_max, (cuuint64_t)B_cache};
    const cuuint32_t bk[4] = {box_d, 1, kRows, 1};
    if (!make_map(&tq, dt, q.data, 3, dq, bq) || !make_map(&tk, dt, k_cache.data, 4, dk, bk, row_promotion(dt)))
        return FMHA_ERR_CUDA;

    auto kern = dt == FMHA_BF16  ? w_kernel<FMHA_BF16>(one)
                : dt == FMHA_F16 ? w_kernel<FMHA_F16>(one) : w_kernel<FMHA_E4M3>(one);
    constexpr int smem = WCfg<FMHA_BF16, true>::SMEM_BYTES;      // the same of every kernel
    static_assert(WCfg<FMHA_BF16, false>::SMEM_BYTES == smem && WCfg<FMHA_E4M3, true>::SMEM_BYTES == smem &&
                      WCfg<FMHA_E4M3, false>::SMEM_BYTES == smem, "");
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return cuda_failed();
    kern<<<grid, kWThreads, smem, stream>>>(tq, tk, p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;
    if (!one && !p.whole) {              // else no unit is ever cut
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(p.UK);
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
