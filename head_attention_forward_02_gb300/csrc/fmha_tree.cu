// fmha_tree.cu -- attention of a tree of drafted tokens over a K/V cache, and
// the commit of the accepted drafts into that cache.
//
// Operation: sequence b has L = seqlen[b] cached tokens in entry
// e = batch_idx[b] and n = n_draft[b] <= T drafted tokens.  The keys of kv
// head g are K_cache[e, 0..L-1, g] and K_new[b, 0..n-1, g] (values alike);
// draft t sees every cached key and the drafts j with tree_mask[b, t, j] != 0
// (without a mask: j <= t).  With x = scale * q.k over what it sees,
//   O[b, t, h] = out_scale * sum_j exp(x_j - LSE) v_j,  LSE = ln sum_j exp(x_j).
//
// A cached key and value (2 * 128 * E bytes) serves T * G query rows
// (G = H / H_k), 4 * 128 flops each: 16-bit types need more than about 280
// rows a kv head to be bound by the tensor cores instead of HBM.  So the
// rows of a kv head's whole group are packed together, t-major, into blocks
// of 128 MMA rows (128 / G tokens each), a work unit being one block of one
// kv head, or two blocks that share the K/V stream where there are more rows
// than one block holds.  The key tiles of all units form one sequence that is
// cut evenly over the CTAs, one per SM; a CTA streams its part through a ring
// of 128-key tiles filled by TMA, and the drafts' keys are the unit's last
// tiles, so the tree mask touches those alone.
//
// Two groups of four softmax warps work on a unit: each on a row block of its
// own, or, where there is one block (SPLIT), on every other key tile of it,
// with an O of its own that the epilogue adds up.  Per 128-key tile:
// S = Q K^T (M = 128 rows, N = 128), P = exp2(S * c - m) by one thread per row
// (TMEM lane = row, so no exchange between threads), written back to TMEM over
// S in two halves, and O += P V of a half as soon as it is there.  Each group
// has an MMA warp of its own, and one group's MMAs run under the other's
// softmax.  The reference m is kept lazily: O is rescaled only when P would
// leave a range in which the type holds it well.
// P is rounded to the inputs' type for the P V product (by up to 2^-8 / 2^-11 /
// 2^-4 of a weight for bf16 / fp16 / e4m3, where it is not subnormal there), its
// row sum and O stay in fp32.  e4m3 has 2^-9 for its last step: of many keys
// far below one (a sink before a long context) all would round to nothing, so
// there the reference also moves down again, before small weights have cost
// more than 2^-5 of their row's.
//
// A unit cut between CTAs leaves normalised fp32 partials and their LSE in the
// workspace, at most two per CTA, and a second kernel joins them; units that
// one CTA covers are written to O directly.
//
// Measured (kernel and merge, in us; S: from the start to the first S of a CTA,
// tiles: from a unit's first S to its last P V, ends: what its units' ends take, all
// of the average CTA; spread: from its end to the last one's):
//                                              all   S  tiles  ends  spread  merge
//   B=32 T=64 32/8 heads, 8192 keys, bf16      221   7    175    17       6     12
//   B=16 T=27 32/8, 4096 ragged, f16            51   5     23     6       5      6
//   B=16 T=5  64/8, 16384 ragged, e4m3       75-84   4     58     5      10      4
// (e4m3: 75 on one GPU, 84 on another.)  In the tiles' time keys and values come
// at 6.2, 7.9 (with what the ring held before) and 6.1 TB/s.  The spread of e4m3
// is not the cut's: CTAs take 680 to 940 ns a tile, the same ones pass after
// pass.  B=1, T=8, 1000 keys: 13.7 us, all latency.
#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kTreeMaxCtas = 152;            // CTAs of the attention kernel at most (bounds the workspace)
constexpr int kStagesMax = 12;
constexpr int kItems = 4;                    // work items published ahead
constexpr int kTreeProd = 8, kTreeMma = 9;   // warps: two softmax groups of four, producer, an MMA issuer a group
constexpr int kTreeThreads = 352;

template <int ELEM, bool SPLIT_>
struct TreeCfg : ElemCfg<ELEM> {
    using B = ElemCfg<ELEM>;
    static constexpr bool SPLIT = SPLIT_;                     // one row block a unit, its key tiles split between the groups
    static constexpr int NRB = SPLIT ? 1 : 2;                 // row blocks of a unit
    // K and V tiles are separate ring stages; with Q they fill 224 KB.  With
    // SPLIT each group has a ring of its own: a barrier's phases must all be
    // waited for by the same warp, since a wait that is two phases early
    // passes on the parity of the phase before the last.
    static constexpr int NS = (7 * 32768 - NRB * B::TILE_BYTES) / B::TILE_BYTES < kStagesMax
                                  ? (7 * 32768 - NRB * B::TILE_BYTES) / B::TILE_BYTES
                                  : kStagesMax;
    static constexpr int RING = SPLIT ? NS / 2 : NS;          // stages of a ring
    static constexpr int OFF_KV = NRB * B::TILE_BYTES;
    static constexpr int OFF_BARS = OFF_KV + NS * B::TILE_BYTES;
    static constexpr int OFF_STAT = OFF_BARS + 1024;          // SPLIT: (m, l) of group 1's rows
    static constexpr int SMEM_BYTES = OFF_STAT + kRows * 8 + 1024;   // 1 KB alignment
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    // log2 of the largest P right after the reference is set, and how far it may
    // grow before the reference is set again (e4m3 ends at 448, fp16 at 65504).
    // fp16's steps are 2^-24 and more: with its largest at 2^7 a weight is off by
    // 2^-32 of the row's sum at most where P is below its normal range.
    static constexpr float BIAS = B::FP8 ? 4.f : ELEM == FMHA_F16 ? 7.f : 0.f;
    static constexpr float GROWN = B::FP8 ? 8.75f : ELEM == FMHA_F16 ? 15.f : 8.f;
    // e4m3: P below 2^-6 is rounded to steps of 2^-9, so a tile's 128 weights are
    // off by 2^-3 together at most.  So that these sum to 2^-5 of the row's sum
    // at most, a row whose sum is below LOST a tile gets a lower reference from a
    // tile without a P of 2^(BIAS - 1) (a tile with one adds more than LOST).
    // By 2^DOWN at most, and not above SUM_MAX, so that nothing overflows: what a
    // tile could lose then is below 2^-33 of the sum.  (0.4% of 75 us for 16 x 5
    // drafts on 16384 keys, where it is hardly ever needed.)
    static constexpr float LOST = 4.f, DOWN = 40.f, SUM_MAX = 0x1p30f;
    // What a unit's ends cost a CTA, in tiles' time: the ring runs empty and is
    // filled again (of 16 ragged f16 sequences, 40 us, a CTA of two units' parts
    // would end 4 us after one that stays in a unit).
    static constexpr int EDGE = NS / 2;
    static_assert(EDGE >= 1, "a ring of two tiles");
    // TMEM: S of each group, P over S, then O of each group
    static constexpr int O_COL = 2 * kRows;
};

struct TreeMeta {                        // whose partial a workspace slot holds
    int b, g, u, n;                      // its unit, and the sequence's drafts (0: no partial here)
    int last;                            // the unit ends with this partial
};

struct TreeParams {
    void *o;                            // [B, T, H, D]
    float *lse;                         // [B, H, T] or NULL
    const int *seqlen, *batch_idx, *n_draft;
    const uint8_t *mask;                // [B or 1, T, T] or NULL
    int64_t mask_stride;
    float *part_o, *part_lse;           // [2 * ncta][NRB * 128][D], [2 * ncta][NRB * 128]
    TreeMeta *meta;                     // [2 * ncta]
    int B, T, H, H_k, G, B_cache, S_max;
    int TB;                             // tokens of a row block
    int NRB;
    int edge;                           // tiles that a unit's ends cost beside its own
    int whole;                          // units are not cut: a CTA takes those that begin in its part
    int ncta;
    float c;                            // scale * log2(e)
    float out_scale;
};

struct TreeItem {
    int b, g, u, entry, L, n;           // b < 0: no more items
    int t0, t1, nt, nc;                 // this CTA's tiles [t0, t1) of the unit's nt; the first nc are cached keys
};

struct TreeBars {
    uint64_t q_full, q_empty, drain[2], stat_full, epi_done;
    uint64_t s_full[2], p_full[2][2], o_full[2], turn[2];   // by group; p_full by half
    uint64_t kv_full[kStagesMax], kv_empty[kStagesMax];
    uint64_t item_full[kItems], item_empty[kItems];
    TreeItem item[kItems];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(TreeBars) <= 1024, "barrier block");

// ---------------------------------------------------------------------------
// Work: the tiles of all (sequence b, kv head g, row-block group u), u fastest
// so that the units that read the same keys run at the same time.  A unit is
// `edge` tiles of nothing, for the work at its ends, and then its own.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int tree_cached(const TreeParams &p, int b, bool report) {
    return clamped(p.seqlen[b], 0, p.S_max, report);
}
__device__ __forceinline__ int tree_drafts(const TreeParams &p, int b, bool report) {
    return p.n_draft ? clamped(p.n_draft[b], 0, p.T, report) : p.T;
}
// row-block groups of a kv head, key tiles of a unit
__device__ __forceinline__ int tree_groups(const TreeParams &p, int n) {
    return (n + p.TB * p.NRB - 1) / (p.TB * p.NRB);
}
__device__ __forceinline__ int tree_tiles(int L, int n) { return (L + kRows - 1) / kRows + (n + kRows - 1) / kRows; }

__device__ __forceinline__ int64_t tree_seq_tiles(const TreeParams &p, int b) {
    const int n = tree_drafts(p, b, false);
    return (int64_t)p.H_k * tree_groups(p, n) * (tree_tiles(tree_cached(p, b, false), n) + p.edge);
}

// Where the producer is in this CTA's tiles [G0, G1).
struct TreeCursor {
    int64_t off, G0, G1;                // off: where the unit at hand begins
    int b, g, u;
    int L, n, entry, nt, nu;            // of sequence b
};

__device__ __forceinline__ void tree_load_seq(const TreeParams &p, TreeCursor &cur) {
    cur.n = tree_drafts(p, cur.b, false);
    cur.L = tree_cached(p, cur.b, false);
    cur.entry = cache_entry(p.batch_idx, cur.b, p.B_cache, false);
    cur.nt = tree_tiles(cur.L, cur.n);
    cur.nu = tree_groups(p, cur.n);     // 0: a sequence without drafts has no unit
}

// One warp: this CTA's range and its first unit (the same in every lane).
__device__ void tree_schedule(const TreeParams &p, TreeCursor &cur, int lane) {
    const int64_t n0 = lane < p.B ? tree_seq_tiles(p, lane) : 0;     // kept: most batches are this small
    int64_t T = n0;
    for (int b = lane + 32; b < p.B; b += 32) T += tree_seq_tiles(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    const int64_t per = (T + gridDim.x - 1) / gridDim.x;
    cur.G0 = min((int64_t)blockIdx.x * per, T);
    cur.G1 = min(cur.G0 + per, T);
    cur.b = p.B;
    cur.off = T;
    if (blockIdx.x == gridDim.x - 1)    // reports values outside their bounds, once a call
        for (int b = lane; b < p.B; b += 32) {
            tree_cached(p, b, true);
            tree_drafts(p, b, true);
            cache_entry(p.batch_idx, b, p.B_cache, true);
        }
    int64_t base = 0;
    for (int bb = 0; bb < p.B && cur.G0 < cur.G1; bb += 32) {
        const int b = bb + lane;
        const int64_t n = bb == 0 ? n0 : b < p.B ? tree_seq_tiles(p, b) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && base + incl > cur.G0);
        if (hit) {
            const int l = __ffs(hit) - 1;
            cur.b = bb + l;
            cur.off = __shfl_sync(0xffffffffu, base + incl - n, l);
            tree_load_seq(p, cur);
            // units of this sequence that end at or before G0, or begin before it
            const int skip = (int)((cur.G0 - cur.off + (p.whole ? cur.nt + p.edge - 1 : 0)) / (cur.nt + p.edge));
            cur.off += (int64_t)skip * (cur.nt + p.edge);
            cur.g = skip / cur.nu;
            cur.u = skip % cur.nu;
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ bool tree_next(const TreeParams &p, TreeCursor &cur, TreeItem &it) {
    it.b = -1;
    if (cur.b >= p.B || cur.off >= cur.G1) return false;
    while (cur.nu == 0 || cur.g == p.H_k) {
        if (++cur.b >= p.B) return false;
        cur.g = cur.u = 0;
        tree_load_seq(p, cur);
    }
    it.t0 = p.whole ? 0 : imax(0, (int)(max(cur.G0, cur.off) - cur.off) - p.edge);
    it.t1 = p.whole ? cur.nt : (int)(min(cur.G1, cur.off + p.edge + cur.nt) - cur.off) - p.edge;
    if (it.t1 <= 0) return false;       // the range ends before the unit's first tile
    it.b = cur.b;
    it.g = cur.g;
    it.u = cur.u;
    it.entry = cur.entry;
    it.L = cur.L;
    it.n = cur.n;
    it.nt = cur.nt;
    it.nc = (cur.L + kRows - 1) / kRows;
    cur.off += p.edge + cur.nt;
    if (++cur.u == cur.nu) {
        cur.u = 0;
        ++cur.g;
    }
    return true;
}

__device__ __forceinline__ int tile_keys(const TreeItem &it, int t) {
    return imin(kRows, t >= it.nc ? it.n - (t - it.nc) * kRows : it.L - t * kRows);
}

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------

// Stage and parity of the n-th tile of group x's ring: K of the group's c-th
// tile is n = 2 c, V is 2 c + 1.
template <class C>
__device__ __forceinline__ uint32_t ring_stage(int x, uint32_t n) { return (C::SPLIT ? x * C::RING : 0) + n % C::RING; }
template <class C>
__device__ __forceinline__ uint32_t ring_parity(uint32_t n) { return (n / C::RING) & 1; }

// Items: the producer publishes them ahead of its loads; the other warps take
// a copy each and hand the slot back.
__device__ __forceinline__ bool publish_item(TreeBars *bars, uint32_t i, const TreeItem &it, volatile int *abort_flag) {
    const uint32_t st = i % kItems;
    if (i >= kItems && !mbar_wait(smem_u32(&bars->item_empty[st]), (i / kItems - 1) & 1, abort_flag)) return false;
    bars->item[st] = it;
    mbar_arrive(smem_u32(&bars->item_full[st]));
    return true;
}

__device__ __forceinline__ bool take_item(TreeBars *bars, uint32_t i, TreeItem &it, volatile int *abort_flag, int lane) {
    const uint32_t st = i % kItems;
    if (!warp_wait(smem_u32(&bars->item_full[st]), (i / kItems) & 1, abort_flag)) return false;
    it = bars->item[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[st]));
    return it.b >= 0;
}

// TMA producer: per item the Q blocks, then its K and V tiles into the ring.
// The next item is worked out (a few dependent loads) behind the first tile's
// loads.
template <class C>
__device__ void tree_producer(const TreeParams &p, TreeCursor &cur, int gate, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                              const CUtensorMap *tmV, const CUtensorMap *tmKn, const CUtensorMap *tmVn, uint8_t *smem,
                              TreeBars *bars) {
    volatile int *abort_flag = &bars->abort;
    uint32_t fill[2] = {0, 0}, qn = 0;  // tiles loaded by ring, Q blocks
    bool ok = !gate || test_gate_open(abort_flag);
    TreeItem it, next;
    if (ok) {
        tree_next(p, cur, it);
        ok = publish_item(bars, 0, it, abort_flag);
    }
    while (ok && it.b >= 0) {
        // the one Q slot: free once the S MMAs of the item before are done
        if (qn > 0 && !mbar_wait(smem_u32(&bars->q_empty), (qn - 1) & 1, abort_flag)) {
            ok = false;
            break;
        }
        const uint32_t qb = smem_u32(&bars->q_full);
        const int tok0 = it.u * C::NRB * p.TB;
        // a box holds TB tokens x G heads; tokens past the sequence's own
        // (another sequence's, or zero fill) give rows that are never stored
        const int nblk = !C::SPLIT && tok0 + p.TB < it.n ? 2 : 1;
        mbar_expect_tx(qb, nblk * C::PANELS * p.TB * p.G * 128);
        for (int x = 0; x < nblk; ++x)
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_3d(smem_u32(smem + x * C::TILE_BYTES + pn * kPanelBytes), tmQ, qb, pn * C::BOX, it.g * p.G,
                            it.b * p.T + tok0 + x * p.TB);
        ++qn;
        const int e = it.entry >= 0 ? it.entry : p.B_cache;   // out of range: zero fill
        for (int t = it.t0; ok && t < it.t1; ++t) {
            const bool drafts = t >= it.nc;
            const int row = (drafts ? t - it.nc : t) * kRows;
            const int x = C::SPLIT ? (t - it.t0) & 1 : 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t n = x ? fill[1] : fill[0], st = ring_stage<C>(x, n);
                if (n >= C::RING && !mbar_wait(smem_u32(&bars->kv_empty[st]), ring_parity<C>(n) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&bars->kv_full[st]);
                mbar_expect_tx(fb, C::TILE_BYTES);
                const uint32_t dst = smem_u32(smem + C::OFF_KV + st * C::TILE_BYTES);
                const CUtensorMap *tm = drafts ? (kv ? tmVn : tmKn) : (kv ? tmV : tmK);
#pragma unroll
                for (int pn = 0; pn < C::PANELS; ++pn)
                    tma_load_4d(dst + pn * kPanelBytes, tm, fb, pn * C::BOX, it.g, row, drafts ? it.b : e);
                if (x) ++fill[1];
                else ++fill[0];
            }
            if (ok && t == it.t0) {
                tree_next(p, cur, next);
                ok = publish_item(bars, qn, next, abort_flag);
            }
        }
        it = next;
    }
    // the last release of every stage and of the Q slot must arrive before
    // exit; when the CTA gave up, only the copies already issued
#pragma unroll
    for (int x = 0; x < (C::SPLIT ? 2 : 1); ++x)
        for (uint32_t n = fill[x] > C::RING ? fill[x] - C::RING : 0; n < fill[x]; ++n) {
            const uint32_t st = ring_stage<C>(x, n);
            if (ok) ok = mbar_wait(smem_u32(&bars->kv_empty[st]), ring_parity<C>(n), abort_flag);
            if (!ok) mbar_wait_drain(smem_u32(&bars->kv_full[st]), ring_parity<C>(n));
        }
    if (qn > 0) {
        if (ok) ok = mbar_wait(smem_u32(&bars->q_empty), (qn - 1) & 1, abort_flag);
        if (!ok) mbar_wait_drain(smem_u32(&bars->q_full), (qn - 1) & 1);
    }
}

// MMA issuer of group x (one warp, one elected lane).  MMAs of one warp
// execute in issue order (promised for those into one accumulator, observed for
// others), so S of the next tile may overwrite the columns of
// P once P V is issued: the chain is P V, next S, softmax.  Where both groups
// work on the same tiles their chains would settle in step, with both softmax
// passes, then both groups' MMAs, at the same time (4200 cycles a tile against
// 3650 when they happened to alternate); so there the issuers take turns, one
// step each, and one group's MMAs run under the other's softmax.
template <class C>
__device__ void tree_mma(uint8_t *smem, TreeBars *bars, uint32_t tmem_any, int x, int lane) {
    volatile int *abort_flag = &bars->abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    const uint32_t s_tm = tmem + x * kRows, o_tm = tmem + C::O_COL + x * kD;
    constexpr uint32_t kIdS = mma_idesc(C::FMT, kRows, false);
    constexpr uint32_t kIdPV = mma_idesc(C::FMT, kD, true);
    constexpr int kStep = C::SPLIT ? 2 : 1;
    const uint64_t q = smem_desc(smem_u32(smem + (C::SPLIT ? 0 : x) * C::TILE_BYTES), 16, 1024);
    const uint64_t k0 = smem_desc(smem_u32(smem + C::OFF_KV), 16, 1024);
    const uint64_t v0 = smem_desc(smem_u32(smem + C::OFF_KV), kPanelBytes, 1024);   // MN-major: LBO = panel stride
    uint32_t c = 0, turns = 0;          // tiles of this group, its turns
    bool ok = true;
    TreeItem it;
    for (uint32_t i = 0; ok && take_item(bars, i, it, abort_flag, lane); ++i) {
        if (!warp_wait(smem_u32(&bars->q_full), i & 1, abort_flag)) {
            ok = false;
            break;
        }
        const int tb = it.t0 + (C::SPLIT ? x : 0);
        bool first = true;
        for (int t = tb; ok && t < it.t1 + kStep; t += kStep) {
            // the tiles of this step first: their waits are off the chain
            const uint32_t nk = 2 * c, nv = 2 * c - 1;           // K of tile t, V of the tile before
            const uint32_t kst = ring_stage<C>(x, nk), vst = ring_stage<C>(x, nv);
            if ((t > tb && !warp_wait(smem_u32(&bars->kv_full[vst]), ring_parity<C>(nv), abort_flag)) ||
                (t < it.t1 && !warp_wait(smem_u32(&bars->kv_full[kst]), ring_parity<C>(nk), abort_flag))) {
                ok = false;
                break;
            }
            if (t > tb) {               // P V of the tile before
                const int halves = tile_keys(it, t - kStep) > kRows / 2 ? 2 : 1;
                const uint64_t v = v0 + ((vst * C::TILE_BYTES) >> 4);
                for (int h = 0; h < halves; ++h) {
                    if (!warp_wait(smem_u32(&bars->p_full[x][h]), (c - 1) & 1, abort_flag) ||
                        (!C::SPLIT && h == 0 &&
                         !warp_wait(smem_u32(&bars->turn[x]), (turns & 1) ^ (x ^ 1), abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // k-steps of MMA_K keys: columns of P, rows of V
#pragma unroll
                    for (int kk = 0; kk < kRows / 2 / C::MMA_K; ++kk)
                        mma_ts<C::FP8>(o_tm, s_tm + h * (kRows / 2 * C::E / 4) + kk * (C::MMA_K * C::E / 4),
                                       v + ((h * (kRows / 2) * 128 + kk * C::MMA_K * 128) >> 4), kIdPV,
                                       !first || h > 0 || kk > 0 ? 1u : 0u);
                }
                if (!ok) break;
                first = false;
            }
            if (!C::SPLIT && t == tb && !warp_wait(smem_u32(&bars->turn[x]), (turns & 1) ^ (x ^ 1), abort_flag)) {
                ok = false;
                break;
            }
            if (t < it.t1) {
                tc_fence_after();
                const uint64_t k = k0 + ((kst * C::TILE_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < kD / C::MMA_K; ++kk) {
                    // each k-step (16 dims of 16 bits or 32 of 8) is 32 bytes of a 128-byte panel row
                    const uint32_t off = (kk * 32 / 128) * kPanelBytes + (kk * 32) % 128;
                    mma_ss<C::FP8>(s_tm, q + (off >> 4), k + (off >> 4), kIdS, kk > 0 ? 1u : 0u);
                    // the other warp wakes up behind the MMAs still to issue
                    if (!C::SPLIT && kk == kD / C::MMA_K - 3 && lane == 0) mbar_arrive(smem_u32(&bars->turn[x ^ 1]));
                }
                tc_commit(smem_u32(&bars->s_full[x]));           // also: P V of the tile before is done
                tc_commit(smem_u32(&bars->kv_empty[kst]));
                if (t + kStep >= it.t1) tc_commit(smem_u32(&bars->q_empty));
                ++c;
            }
            if (t > tb) tc_commit(smem_u32(&bars->kv_empty[vst]));
            if (!C::SPLIT) {
                if (t >= it.t1 && lane == 0) mbar_arrive(smem_u32(&bars->turn[x ^ 1]));
                ++turns;
            }
        }
        if (!ok) break;
        if (tb < it.t1) tc_commit(smem_u32(&bars->o_full[x]));
        else tc_commit(smem_u32(&bars->q_empty));        // an item of one tile is group 0's alone
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain[x]));
    mbar_wait_drain(smem_u32(&bars->drain[x]), 0);
}

// The 128 tree-mask bits of this thread's row for drafts [j0, j0 + 128):
// bit i of w[i / 32] is set where draft token tok sees draft j0 + i.  A warp
// reads each of its tokens' mask rows once, 32 bytes at a time.
__device__ __forceinline__ void tree_bits(const TreeParams &p, const TreeItem &it, int tok, int j0, int lane,
                                          uint32_t (&w)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = 0u;
    if (!p.mask) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int cnt = imin(tok, it.n - 1) + 1 - (j0 + 32 * q);     // drafts j <= tok
            w[q] = cnt >= 32 ? 0xffffffffu : cnt > 0 ? (1u << cnt) - 1u : 0u;
        }
        return;
    }
    const uint8_t *m = p.mask + (int64_t)it.b * p.mask_stride;
    const int lo = __shfl_sync(0xffffffffu, tok, 0), hi = imin(__shfl_sync(0xffffffffu, tok, 31), it.n - 1);
    // eight tokens' loads in flight at a time
    for (int t0 = lo; t0 <= hi; t0 += 8) {
        bool see[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int jj = j0 + 32 * q + lane;
                see[i][q] = t0 + i <= hi && jj < it.n && m[(int64_t)(t0 + i) * p.T + jj] != 0;
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t bits = __ballot_sync(0xffffffffu, see[i][q]);
                if (t0 + i == tok) w[q] = bits;
            }
    }
}

// 32 bytes, a whole sector, in one store
__device__ __forceinline__ void store_sector(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Softmax and epilogue: warp w of group x owns the rows 32 (w % 4) .. + 31 of
// its block (TMEM lanes), one row a thread.
template <class C>
__device__ void tree_softmax(const TreeParams &p, uint8_t *smem, TreeBars *bars, uint32_t tmem, int warp, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int x = warp >> 2;                            // group
    const int r = (warp & 3) * 32 + lane;               // row of the block = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_tm = lane_base + C::O_COL + x * kD;
    const int rt = r / p.G, rh = r % p.G;               // token of the block, head of the group
    float2 *stat = reinterpret_cast<float2 *>(smem + C::OFF_STAT);
    uint32_t c = 0;                                     // tiles of this group
    uint32_t shared = 0;                                // SPLIT: items so far that group 1 had tiles of
    int parts = 0;                                      // bit s: slot s of this CTA holds a partial
    TreeItem it;
    for (uint32_t i = 0; take_item(bars, i, it, abort_flag, lane); ++i) {
        const int tok = (C::SPLIT ? it.u : 2 * it.u + x) * p.TB + rt;
        const bool row_ok = rt < p.TB && tok < it.n;
        const bool work = __any_sync(0xffffffffu, row_ok);   // else the warp only keeps step
        float m = -INFINITY;                            // reference (log2 units) of P and O
        float l = 0.f;                                  // row sum
        float lost = 0.f;                               // e4m3: tiles so far, each in the units P had then,
        float low = -INFINITY;                          // and the maximum below which a tile moves m down
        bool ok = true;
        constexpr int kStep = C::SPLIT ? 2 : 1;
        const int tb = it.t0 + (C::SPLIT ? x : 0);
        // the tree bits of the first draft tile are fetched before the first S is waited for
        uint32_t bits[4] = {0u, 0u, 0u, 0u};
        int bits_t = it.nc + (C::SPLIT ? (it.nc - tb) & 1 : 0);
        if (bits_t < tb) bits_t = tb;
        if (work && bits_t < it.t1) tree_bits(p, it, tok, (bits_t - it.nc) * kRows, lane, bits);
        for (int t = tb; t < it.t1; t += kStep, ++c) {
            const bool drafts = t >= it.nc;
            const int nk = tile_keys(it, t), halves = nk > kRows / 2 ? 2 : 1;
            if (work && drafts && t != bits_t) tree_bits(p, it, tok, (t - it.nc) * kRows, lane, bits);
            if (!warp_wait(smem_u32(&bars->s_full[x]), c & 1, abort_flag)) {
                ok = false;
                break;
            }
            if (nk < kRows) {
                // rows past the keys (stale cache contents, possibly not
                // finite): V is zeroed so that P = 0 contributes 0 (by both
                // groups where both use the tile: each before its own P V)
                const uint32_t nv = 2 * c + 1, vst = ring_stage<C>(x, nv);
                if (!warp_wait(smem_u32(&bars->kv_full[vst]), ring_parity<C>(nv), abort_flag)) {
                    ok = false;
                    break;
                }
                if (r >= nk) {
                    proxy_fence();
                    uint8_t *v = smem + C::OFF_KV + vst * C::TILE_BYTES + r * 128;
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4 *>(v + pn * kPanelBytes + (k << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    proxy_fence();
                }
            }
            if (!work) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&bars->p_full[x][0]));
                    mbar_arrive(smem_u32(&bars->p_full[x][1]));
                }
                continue;
            }
            tc_fence_after();
            const uint32_t s_tm = lane_base + x * kRows;
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(s_tm + 32 * q, s[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_wait_ld(s[q]);
            if (drafts || nk < kRows) {
                // a bit per key: those below nk, of drafts the tree's
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int cnt = nk - 32 * q;
                    uint32_t vis = cnt >= 32 ? 0xffffffffu : cnt > 0 ? (1u << cnt) - 1u : 0u;
                    if (drafts) vis &= bits[q];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((vis >> k) & 1u)) s[q][k] = 0xff800000u;
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 32; k += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mx[y] = max3(mx[y], __uint_as_float(s[q][k + 2 * y]), __uint_as_float(s[q][k + 2 * y + 1]));
            const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
            const bool need = tmax > m + C::GROWN || (C::FP8 && tmax < low);
            if (__any_sync(0xffffffffu, need)) {
                float alpha = 1.f;
                if (need) {
                    const float ref = fmaxf(tmax - C::BIAS, m - C::DOWN);
                    alpha = m == -INFINITY ? 0.f : ex2(m - ref);
                    m = ref;
                    l *= alpha;
                    lost *= alpha;
                }
                if (t > tb) {
                    // the P V of the tile before is in O: S, issued behind it, is there
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        uint32_t o[16];
                        tmem_ld16(o_tm + 16 * q, o);
                        tmem_wait_ld16(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tmem_st16(o_tm + 16 * q, o);
                    }
                }
            }
            lost += 1.f;
            // a row that has seen no key yet: every score is -inf, P = 0
            const float mr = m == -INFINITY ? 0.f : -m;
            const uint64_t c2 = pack_f2(p.c, p.c), m2 = pack_f2(mr, mr);
            uint64_t ls[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h < halves) {
#pragma unroll
                    for (int q = 2 * h; q < 2 * h + 2; ++q) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float a, b;
                            unpack_f2(fma_f2(pack_f2(__uint_as_float(s[q][k]), __uint_as_float(s[q][k + 1])), c2, m2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            ls[(k >> 1) & 1] = add_f2(ls[(k >> 1) & 1], pack_f2(a, b));
                            s[q][k] = __float_as_uint(a);
                            s[q][k + 1] = __float_as_uint(b);
                        }
                        auto f = [&](int k) { return __uint_as_float(s[q][k]); };
                        if constexpr (C::FP8) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = pack4_e4m3(f(4 * k), f(4 * k + 1), f(4 * k + 2), f(4 * k + 3));
                            tmem_st8(s_tm + 8 * q, w);
                        } else {
                            uint32_t w[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) w[k] = pack2<C::FMT == 1u>(f(2 * k), f(2 * k + 1));
                            tmem_st16(s_tm + 16 * q, w);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[x][h]));
            }
            float la, lb, lc, ld;
            unpack_f2(ls[0], la, lb);
            unpack_f2(ls[1], lc, ld);
            l += (la + lb) + (lc + ld);
            if constexpr (C::FP8) low = l < fminf(C::LOST * (lost + 1.f), C::SUM_MAX) ? m + (C::BIAS - 1.f) : -INFINITY;
        }
        if (!ok) break;

        // epilogue: O of a unit that this CTA covers alone, else a partial
        const bool two = C::SPLIT && it.t1 - it.t0 > 1;      // group 1 has an O of the same rows
        float f0 = 1.f, f1 = 0.f;                       // SPLIT: factors of the two groups' O
        if constexpr (C::SPLIT) {
            if (x == 1) {
                stat[r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->stat_full));
                // group 0 reads this group's O: not overwritten before it has
                if (!warp_wait(smem_u32(&bars->epi_done), i & 1, abort_flag)) break;
                continue;
            }
            if (!warp_wait(smem_u32(&bars->stat_full), i & 1, abort_flag)) break;
            if (two && !warp_wait(smem_u32(&bars->o_full[1]), shared++ & 1, abort_flag)) break;
            const float2 s1 = stat[r];
            const float mm = fmaxf(m, s1.x);
            f0 = m == -INFINITY ? 0.f : ex2(m - mm);
            f1 = s1.x == -INFINITY ? 0.f : ex2(s1.x - mm);
            l = l * f0 + s1.y * f1;
            m = mm;
        }
        if (!warp_wait(smem_u32(&bars->o_full[x]), i & 1, abort_flag)) break;
        // slot 2 * cta: a unit that an earlier CTA began; 2 * cta + 1: one that begins here
        const bool whole = it.t1 - it.t0 == it.nt;
        const int part = 2 * blockIdx.x + (it.t0 == 0 ? 1 : 0);
        if (threadIdx.x == 0 && !whole) {
            parts |= it.t0 == 0 ? 2 : 1;
            p.meta[part] = TreeMeta{it.b, it.g, it.u, it.n, it.t1 == it.nt};
        }
        if (work) {
            tc_fence_after();
            const bool empty = l == 0.f;                // the row saw no key (O may hold anything)
            const float inv = (whole ? p.out_scale : 1.f) / l;
            const float lse = empty ? -INFINITY : (m + log2f(l)) * kLn2;
            const int h = it.g * p.G + rh;
            const int64_t slot = (int64_t)part * (C::NRB * kRows) + (C::SPLIT ? 0 : x) * kRows + r;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                tmem_ld32(o_tm + 32 * q, o);
                tmem_wait_ld(o);
                if (two) {
                    uint32_t o1[32];
                    tmem_ld32(o_tm + kD + 32 * q, o1);
                    tmem_wait_ld(o1);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = empty ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
                if (row_ok && !whole) {
                    float *dst = p.part_o + slot * kD + 32 * q;
#pragma unroll
                    for (int k = 0; k < 4; ++k) store_sector(dst + 8 * k, o + 8 * k);
                } else if (row_ok) {
                    uint8_t *dst = static_cast<uint8_t *>(p.o) +
                                   ((((int64_t)it.b * p.T + tok) * p.H + h) * kD + 32 * q) * C::E;
                    uint32_t w[8 * C::E];
#pragma unroll
                    for (int k = 0; k < 8 * C::E; ++k) {
                        auto f = [&](int i) { return __uint_as_float(o[k * 4 / C::E + i]); };
                        if constexpr (C::FP8) w[k] = pack4_e4m3(f(0), f(1), f(2), f(3));
                        else w[k] = pack2<C::FMT == 1u>(f(0), f(1));
                    }
                    if ((reinterpret_cast<uintptr_t>(p.o) & 31u) == 0) {
#pragma unroll
                        for (int k = 0; k < C::E; ++k) store_sector(dst + 32 * k, w + 8 * k);
                    } else {
#pragma unroll
                        for (int k = 0; k < 2 * C::E; ++k)
                            reinterpret_cast<uint4 *>(dst)[k] =
                                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                }
            }
            if (row_ok) {
                if (!whole) p.part_lse[slot] = lse;
                else if (p.lse) p.lse[((int64_t)it.b * p.H + h) * p.T + tok] = lse;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (C::SPLIT && lane == 0) mbar_arrive(smem_u32(&bars->epi_done));
    }
    if (threadIdx.x == 0)               // empty slots; one that is missing (a CTA that gave up) also ends its unit
        for (int s = 0; s < 2; ++s)
            if (!(parts >> s & 1)) p.meta[2 * blockIdx.x + s] = TreeMeta{0, 0, 0, 0, 1};
}

template <int ELEM, bool SPLIT>
__global__ void __launch_bounds__(kTreeThreads, 1)
    fmha_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                     const __grid_constant__ CUtensorMap tmVn, const TreeParams p) {
    using C = TreeCfg<ELEM, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TreeBars *bars = reinterpret_cast<TreeBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 2);              // both MMA warps
        mbar_init(smem_u32(&bars->stat_full), 4);
        mbar_init(smem_u32(&bars->epi_done), 4);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bars->s_full[x]), 1);
            mbar_init(smem_u32(&bars->p_full[x][0]), 4);
            mbar_init(smem_u32(&bars->p_full[x][1]), 4);
            mbar_init(smem_u32(&bars->o_full[x]), 1);
            mbar_init(smem_u32(&bars->drain[x]), 1);
            mbar_init(smem_u32(&bars->turn[x]), 1);
        }
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), C::SPLIT ? 1 : 2);   // the MMA warps that use a tile
        }
        for (int s = 0; s < kItems; ++s) {
            mbar_init(smem_u32(&bars->item_full[s]), 1);
            mbar_init(smem_u32(&bars->item_empty[s]), 10);   // the softmax and MMA warps
        }
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kTreeMma) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    TreeCursor cur;
    int gate = 0;
    if (warp == kTreeProd) {
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmKn);
            prefetch_tmap(&tmVn);
        }
        gate = g_test_gate;             // read along with the lengths
        tree_schedule(p, cur, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // the merge kernel may be scheduled as CTAs of this grid exit; it waits
    // for this grid's completion before it reads the partials
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < kTreeProd) {
        tree_softmax<C>(p, smem, bars, tmem, warp, lane);
    } else if (warp == kTreeProd) {
        if (lane == 0) tree_producer<C>(p, cur, gate, &tmQ, &tmK, &tmV, &tmKn, &tmVn, smem, bars);
    } else {
        tree_mma<C>(smem, bars, tmem, warp - kTreeMma, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTreeMma) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the units that several CTAs covered:
//   O = out_scale * sum_c w_c O_c / sum_c w_c with w_c = exp(LSE_c - max LSE).
// CTA (c, y) takes eight rows, a warp each, of the unit that CTA c of the kernel
// above began and did not end; the metadata says where it goes on, so nothing
// of the schedule is worked out again.  Nearly every cut unit has two
// partials: their rows are fetched in the same round trip as the metadata and
// joined by straight code (the kernel is short enough that its instruction
// fetches count); more partials take the loop.  Bound by L2: 64 drafts of 32
// sequences leave 40 MB of partials, read in 9.6 us (four rows a warp, all
// loads first, made 16 sequences of 27 drafts 55 us instead of 51).
constexpr int kMergeWarps = 8;

template <int ELEM>
__device__ __forceinline__ void tree_store_row(const TreeParams &p, const TreeMeta &m, int q, float4 acc, float wsum,
                                               float mx, int lane) {
    const int per = p.TB * p.G, x = q / per, rr = q - x * per;       // block, row of the block
    const int tok = (m.u * p.NRB + x) * p.TB + rr / p.G, h = m.g * p.G + rr % p.G;
    if (tok >= m.n) return;
    const float inv = wsum == 0.f ? 0.f : p.out_scale / wsum;
    const int64_t out = ((int64_t)m.b * p.T + tok) * p.H + h;
    if constexpr (ELEM == FMHA_E4M3) {
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.o) + out * kD + lane * 4) =
            pack4_e4m3(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + out * kD + lane * 4) =
            make_uint2(pack2<ELEM == FMHA_BF16>(acc.x * inv, acc.y * inv), pack2<ELEM == FMHA_BF16>(acc.z * inv, acc.w * inv));
    }
    if (lane == 0 && p.lse)
        p.lse[((int64_t)m.b * p.H + h) * p.T + tok] = wsum == 0.f ? -INFINITY : mx + __logf(wsum);
}

template <int ELEM>
__global__ void __launch_bounds__(32 * kMergeWarps) fmha_tree_merge_kernel(const TreeParams p) {
    const int lane = threadIdx.x & 31, c0 = blockIdx.x;
    const int q = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);          // row of the unit, without padding
    const int per = p.TB * p.G;                                           // rows of a block that hold tokens
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (q >= p.NRB * per || c0 + 1 >= p.ncta) return;
    const int r = q / per * kRows + q % per;
    auto slot = [&](int c) { return ((int64_t)2 * (c0 + c) + (c == 0 ? 1 : 0)) * (p.NRB * kRows) + r; };
    const float4 *o_c = reinterpret_cast<const float4 *>(p.part_o) + lane;
    const TreeMeta m = p.meta[2 * c0 + 1];
    const bool two = p.meta[2 * (c0 + 1)].last;
    const float la = p.part_lse[slot(0)], lb = p.part_lse[slot(1)];
    const float4 a = o_c[slot(0) * (kD / 4)], b = o_c[slot(1) * (kD / 4)];
    if (m.n == 0) return;                                                 // CTA c0 began no unit that it did not end
    if (two) {
        float mx = fmaxf(la, lb);
        if (mx == -INFINITY || la != la || lb != lb) mx = 0.f;            // no key: weights 0; NaN in, NaN out
        const float wa = __expf(la - mx), wb = __expf(lb - mx);
        const float4 o = make_float4(wa * a.x + wb * b.x, wa * a.y + wb * b.y, wa * a.z + wb * b.z, wa * a.w + wb * b.w);
        tree_store_row<ELEM>(p, m, q, o, wa + wb, mx, lane);
        return;
    }
    // the partials of CTAs c0 .. c0 + nch - 1
    int nch = 2;
    for (;;) {
        const int c = c0 + nch + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, c >= p.ncta || p.meta[2 * c].last);
        nch += hit ? __ffs(hit) : 32;
        if (hit) break;
    }
    nch = imin(nch, p.ncta - c0);
    float mx = -INFINITY;
    bool nan = false;
    for (int c = lane; c < nch; c += 32) {
        const float v = p.part_lse[slot(c)];
        nan |= v != v;
        mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY || __any_sync(0xffffffffu, nan)) mx = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    for (int cb = 0; cb < nch; cb += 8) {
        // eight partials' rows and LSEs in flight
        float4 v[8];
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t s = slot(imin(cb + i, nch - 1));
            v[i] = o_c[s * (kD / 4)];
            w[i] = p.part_lse[s];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = cb + i < nch ? __expf(w[i] - mx) : 0.f;
            wsum += x;
            acc.x += x * v[i].x;
            acc.y += x * v[i].y;
            acc.z += x * v[i].z;
            acc.w += x * v[i].w;
        }
    }
    tree_store_row<ELEM>(p, m, q, acc, wsum, mx, lane);
}

// ---------------------------------------------------------------------------
// Commit: row path[b, i] of the drafts' K/V becomes cache row seqlen[b] + i.
// A row of all kv heads is contiguous on both sides; one CTA a (sequence,
// accepted draft), so the call is one round trip to memory whatever its size.
// ---------------------------------------------------------------------------

struct CommitParams {
    uint4 *k_cache, *v_cache;
    const uint4 *k_new, *v_new;
    const int *seqlen, *batch_idx, *path, *n_accept;
    int T, P, B_cache, S_max;
    int row16;                          // 16-byte pieces of a row: H_k * 128 * E / 16
};

__global__ void __launch_bounds__(256) fmha_tree_commit_kernel(const CommitParams p) {
    const int i = blockIdx.x, b = blockIdx.y;
    const bool report = threadIdx.x == 0 && i == 0;
    const int L = clamped(p.seqlen[b], 0, p.S_max, report);
    const int n = clamped(p.n_accept[b], 0, imin(p.P, p.S_max - L), report);
    if (i >= n) return;
    const int e = cache_entry(p.batch_idx, b, p.B_cache, report);
    const int t = p.path[(int64_t)b * p.P + i];
    if (t < 0 || t >= p.T) {
        if (threadIdx.x == 0) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
        return;
    }
    if (e < 0) return;
    const int64_t src = ((int64_t)b * p.T + t) * p.row16, dst = ((int64_t)e * p.S_max + L + i) * p.row16;
    for (int x = threadIdx.x; x < p.row16; x += blockDim.x) {
        const uint4 k = p.k_new[src + x], v = p.v_new[src + x];
        p.k_cache[dst + x] = k;
        p.v_cache[dst + x] = v;
    }
}

// Rows: TB tokens of G heads fill a 128-row block; two blocks a unit where
// one does not hold the drafts' rows.
struct TreeShape {
    int TB, NRB, groups;
};
TreeShape tree_shape(int T, int G) {
    TreeShape s;
    s.TB = imin(kRows / G, T);
    const int blocks = (T + s.TB - 1) / s.TB;
    s.NRB = blocks > 1 ? 2 : 1;
    s.groups = (blocks + s.NRB - 1) / s.NRB;
    return s;
}

int tree_ctas(int64_t tiles) { return (int)(tiles < kTreeMaxCtas ? tiles : kTreeMaxCtas); }
int64_t tree_max_tiles(const TreeShape &s, int B, int T, int H_k, int S_max) {
    return (int64_t)B * H_k * s.groups * (((int64_t)S_max + kRows - 1) / kRows + (T + kRows - 1) / kRows);
}

// Are units left whole?  Then there are no partials and no merge (the host saves
// 2.7 us of 25 as well), but a CTA may take a unit more than its share.  So they
// are where the longest CTA, by the cache's size since only the device knows the
// lengths, has few tiles: six, or ten of two blocks, whose partials are twice
// as large, if no more than six of them are above the average.  Cut / whole in
// us, H_k=8, G=4: B=1 T=8 256 keys 11.6 / 11.0, 768 13.7 / 13.7, 1000 13.7 / 15.1;
// B=4, 500 ragged 15.9 / 13.0; B=32, 256 24.0 / 20.5; B=24, 500 ragged 23.7 / 25.3;
// B=16, 1000 ragged 23.3 / 26.0; two blocks (T=64): B=1, 512 19.1 / 17.7, 1000
// 20.6 / 24.0; B=8, 500 28.7 / 19.1; B=16, 1000 42.8 / 30.0, ragged 38.6 / 36.5.
bool tree_whole(const TreeShape &s, int B, int T, int H_k, int S_max, int ncta) {
    const int64_t units = (int64_t)B * H_k * s.groups, tiles = tree_max_tiles(s, B, T, H_k, S_max) / units;
    const int64_t most = tiles * ((units + ncta - 1) / ncta);
    return most <= (s.NRB == 2 ? 10 : 6) && most * ncta - tiles * units <= (int64_t)6 * ncta;
}

bool tree_sizes_ok(int B, int T, int H, int H_k, int D, int S_max) {
    return B > 0 && T > 0 && H > 0 && H_k > 0 && H % H_k == 0 && H / H_k <= kRows && D == kD && S_max > 0 &&
           S_max <= kMaxCacheRows;
}

using TreeKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, TreeParams);
template <bool SPLIT>
TreeKernel tree_kernel_for(int dt) {
    return dt == FMHA_BF16 ? fmha_tree_kernel<FMHA_BF16, SPLIT>
           : dt == FMHA_F16 ? fmha_tree_kernel<FMHA_F16, SPLIT> : fmha_tree_kernel<FMHA_E4M3, SPLIT>;
}
template <int ELEM>
int tree_edge(int nrb) {
    return nrb == 2 ? TreeCfg<ELEM, false>::EDGE : TreeCfg<ELEM, true>::EDGE;
}
template <int ELEM>
int tree_smem(int nrb) {
    return nrb == 2 ? TreeCfg<ELEM, false>::SMEM_BYTES : TreeCfg<ELEM, true>::SMEM_BYTES;
}

}  // namespace

int tree_set_wait_limit(unsigned long long ns) { return cache_set_wait_limit(ns); }
int tree_set_test_gate(int on) { return cache_set_test_gate(on); }
int *tree_status_word() { return symbol_address(g_status); }

}  // namespace fmha

using namespace fmha;

extern "C" size_t fmha_tree_workspace_size(int B, int T, int H, int H_k, int D, int S_max) {
    if (!tree_sizes_ok(B, T, H, H_k, D, S_max)) return 0;
    const TreeShape s = tree_shape(T, H / H_k);
    // two partials a CTA: an fp32 row of O and its LSE for every row of a unit, and whose they are
    return (size_t)2 * tree_ctas(tree_max_tiles(s, B, T, H_k, S_max)) *
           (s.NRB * kRows * (kD + 1) * sizeof(float) + sizeof(TreeMeta));
}

extern "C" int fmha_tree_fwd(fmha_tensor q, fmha_tensor k_cache, fmha_tensor v_cache, fmha_tensor k_new,
                             fmha_tensor v_new, fmha_tensor o, float *lse, int B, int T, int H, int H_k, int D,
                             int B_cache, int S_max, const int *seqlen, const int *batch_idx, const int *n_draft,
                             const uint8_t *tree_mask, int64_t mask_batch_stride, float scale, float out_scale,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    // ---- host-side validation: nothing is launched on a bad argument ----
    if (B < 0 || T < 0 || H <= 0 || H_k <= 0 || H % H_k != 0 || H / H_k > kRows || D != kD) return FMHA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY) || !(out_scale == out_scale) || out_scale == INFINITY ||
        out_scale == -INFINITY)
        return FMHA_ERR_INVALID_ARG;
    if (tree_mask && mask_batch_stride != 0 && mask_batch_stride < (int64_t)T * T) return FMHA_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return FMHA_OK;
    if (S_max <= 0 || S_max > kMaxCacheRows || B_cache <= 0 || !seqlen) return FMHA_ERR_INVALID_ARG;
    if (!q.data || !k_cache.data || !v_cache.data || !k_new.data || !v_new.data || !o.data) return FMHA_ERR_INVALID_ARG;
    const int dt = q.dtype;
    if (dt != FMHA_F16 && dt != FMHA_BF16 && dt != FMHA_E4M3) return FMHA_ERR_UNSUPPORTED;
    for (const fmha_tensor *t : {&k_cache, &v_cache, &k_new, &v_new, &o})
        if (t->dtype != dt) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {q.data, k_cache.data, v_cache.data, k_new.data, v_new.data, o.data})
        if (misaligned(ptr, 16)) return FMHA_ERR_UNSUPPORTED;
    if ((int64_t)B * T >= (int64_t(1) << 31) / kRows || misaligned(lse, 4) || misaligned(seqlen, 4) ||
        misaligned(batch_idx, 4) || misaligned(n_draft, 4))
        return FMHA_ERR_INVALID_ARG;
    const TreeShape sh = tree_shape(T, H / H_k);
    if (!workspace || misaligned(workspace, 256) ||
        workspace_bytes < fmha_tree_workspace_size(B, T, H, H_k, D, S_max))
        return FMHA_ERR_INVALID_ARG;
    // a unit's inputs are read by several CTAs, at their own times
    const size_t row = kD * (dt == FMHA_E4M3 ? 1 : 2), q_bytes = (size_t)B * T * H * row;
    const size_t new_bytes = (size_t)B * T * H_k * row, cache_bytes = (size_t)B_cache * S_max * H_k * row;
    const size_t seq_bytes = (size_t)B * sizeof(int);
    const Bytes out[3] = {{o.data, q_bytes}, {lse, (size_t)B * H * T * sizeof(float)},
                          {workspace, fmha_tree_workspace_size(B, T, H, H_k, D, S_max)}};
    const Bytes in[9] = {{q.data, q_bytes}, {k_cache.data, cache_bytes}, {v_cache.data, cache_bytes},
                         {k_new.data, new_bytes}, {v_new.data, new_bytes}, {seqlen, seq_bytes}, {batch_idx, seq_bytes},
                         {n_draft, seq_bytes}, {tree_mask, (size_t)(B - 1) * mask_batch_stride + (size_t)T * T}};
    if (outputs_clash(out, in)) return FMHA_ERR_INVALID_ARG;
    int rc = check_device();
    if (rc != FMHA_OK) return rc;
    const int sms = sm_count();
    if (sms <= 0) return FMHA_ERR_CUDA;

    TreeParams p{};
    p.o = o.data;
    p.lse = lse;
    p.seqlen = seqlen;
    p.batch_idx = batch_idx;
    p.n_draft = n_draft;
    p.mask = tree_mask;
    p.mask_stride = mask_batch_stride;
    p.B = B;
    p.T = T;
    p.H = H;
    p.H_k = H_k;
    p.G = H / H_k;
    p.B_cache = B_cache;
    p.S_max = S_max;
    p.TB = sh.TB;
    p.NRB = sh.NRB;
    p.edge = dt == FMHA_E4M3 ? tree_edge<FMHA_E4M3>(sh.NRB) : tree_edge<FMHA_BF16>(sh.NRB);
    p.ncta = imin(sms, tree_ctas(tree_max_tiles(sh, B, T, H_k, S_max)));
    p.whole = tree_whole(sh, B, T, H_k, S_max, p.ncta);
    p.part_o = static_cast<float *>(workspace);
    p.part_lse = p.part_o + (size_t)2 * p.ncta * sh.NRB * kRows * kD;
    p.meta = reinterpret_cast<TreeMeta *>(p.part_lse + (size_t)2 * p.ncta * sh.NRB * kRows);
    p.c = log2_scale(scale);
    p.out_scale = out_scale;

    // ---- tensor maps: boxes of one swizzle panel of dims ----
    CUtensorMap tq, tc[2], tn[2];
    const cuuint32_t box_d = dt == FMHA_E4M3 ? 128 : 64;
    {
        // q as [B * T, H, 128]: a box of one block, TB tokens x G heads
        const cuuint64_t dims[3] = {kD, (cuuint64_t)H, (cuuint64_t)B * T};
        const cuuint32_t box[3] = {box_d, (cuuint32_t)p.G, (cuuint32_t)p.TB};
        if (!make_map(&tq, dt, q.data, 3, dims, box)) return FMHA_ERR_CUDA;
    }
    for (int kv = 0; kv < 2; ++kv) {
        // cache [B_cache, S_max, H_k, 128] and drafts [B, T, H_k, 128]: 128 tokens of one head
        const cuuint64_t dc[4] = {kD, (cuuint64_t)H_k, (cuuint64_t)S_max, (cuuint64_t)B_cache};
        const cuuint64_t dn[4] = {kD, (cuuint64_t)H_k, (cuuint64_t)T, (cuuint64_t)B};
        const cuuint32_t box[4] = {box_d, 1, kRows, 1};
        if (!make_map(&tc[kv], dt, kv ? v_cache.data : k_cache.data, 4, dc, box, row_promotion(dt)) ||
            !make_map(&tn[kv], dt, kv ? v_new.data : k_new.data, 4, dn, box, row_promotion(dt)))
            return FMHA_ERR_CUDA;
    }

    auto kern = sh.NRB == 2 ? tree_kernel_for<false>(dt) : tree_kernel_for<true>(dt);
    const int smem = dt == FMHA_E4M3 ? tree_smem<FMHA_E4M3>(sh.NRB) : tree_smem<FMHA_BF16>(sh.NRB);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return cuda_failed();
    kern<<<p.ncta, kTreeThreads, smem, stream>>>(tq, tc[0], tc[1], tn[0], tn[1], p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;
    if (p.whole) return FMHA_OK;

    const int rows = sh.NRB * p.TB * p.G;                 // of a unit
    auto merge = dt == FMHA_BF16 ? fmha_tree_merge_kernel<FMHA_BF16>
                 : dt == FMHA_F16 ? fmha_tree_merge_kernel<FMHA_F16> : fmha_tree_merge_kernel<FMHA_E4M3>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ncta, (rows + kMergeWarps - 1) / kMergeWarps);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, merge, p) != cudaSuccess) return cuda_failed();
    return FMHA_OK;
}

extern "C" int fmha_tree_commit(fmha_tensor k_cache, fmha_tensor v_cache, fmha_tensor k_new, fmha_tensor v_new, int B,
                                int T, int P, int H_k, int D, int B_cache, int S_max, const int *seqlen,
                                const int *batch_idx, const int *path, const int *n_accept, cudaStream_t stream) {
    if (B < 0 || T < 0 || P < 0 || H_k <= 0 || D != kD) return FMHA_ERR_INVALID_ARG;
    if (B == 0 || P == 0) return FMHA_OK;
    if (T == 0 || S_max <= 0 || S_max > kMaxCacheRows || B_cache <= 0 || !seqlen || !path || !n_accept)
        return FMHA_ERR_INVALID_ARG;
    if (!k_cache.data || !v_cache.data || !k_new.data || !v_new.data) return FMHA_ERR_INVALID_ARG;
    const int dt = k_cache.dtype;
    if (dt != FMHA_F16 && dt != FMHA_BF16 && dt != FMHA_E4M3) return FMHA_ERR_UNSUPPORTED;
    for (const fmha_tensor *t : {&v_cache, &k_new, &v_new})
        if (t->dtype != dt) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {k_cache.data, v_cache.data, k_new.data, v_new.data})
        if (misaligned(ptr, 16)) return FMHA_ERR_UNSUPPORTED;
    if (misaligned(seqlen, 4) || misaligned(batch_idx, 4) || misaligned(path, 4) || misaligned(n_accept, 4))
        return FMHA_ERR_INVALID_ARG;
    if (B > 65535) return FMHA_ERR_UNSUPPORTED;
    const size_t row = (size_t)H_k * kD * (dt == FMHA_E4M3 ? 1 : 2);
    const size_t new_bytes = (size_t)B * T * row, cache_bytes = (size_t)B_cache * S_max * row;
    const size_t seq_bytes = (size_t)B * sizeof(int);
    const Bytes out[2] = {{k_cache.data, cache_bytes}, {v_cache.data, cache_bytes}};
    const Bytes in[6] = {{k_new.data, new_bytes}, {v_new.data, new_bytes}, {seqlen, seq_bytes}, {batch_idx, seq_bytes},
                         {path, P * seq_bytes}, {n_accept, seq_bytes}};
    if (outputs_clash(out, in)) return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    CommitParams p{};
    p.k_cache = static_cast<uint4 *>(k_cache.data);
    p.v_cache = static_cast<uint4 *>(v_cache.data);
    p.k_new = static_cast<const uint4 *>(k_new.data);
    p.v_new = static_cast<const uint4 *>(v_new.data);
    p.seqlen = seqlen;
    p.batch_idx = batch_idx;
    p.path = path;
    p.n_accept = n_accept;
    p.T = T;
    p.P = P;
    p.B_cache = B_cache;
    p.S_max = S_max;
    p.row16 = (int)(row / 16);
    const int threads = p.row16 >= 256 ? 256 : (p.row16 + 31) / 32 * 32;
    fmha_tree_commit_kernel<<<dim3(P, B), threads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FMHA_OK : FMHA_ERR_CUDA;
}
