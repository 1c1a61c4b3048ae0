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
// kv head, or two blocks (NRB = 2) that share the K/V stream where there are
// more rows than one block holds.  The key tiles of all units form one
// sequence that is cut evenly over the CTAs, one per SM; a CTA streams its
// part through a ring of 128-key tiles filled by TMA, and the drafts' keys are
// the unit's last tiles, so the tree mask touches those alone.
//
// Per tile: S = Q K^T (M = 128 rows, N = 128 keys), P = exp2(S * c - m) by one
// thread per row (TMEM lane = row, so no exchange between threads), written
// back to TMEM over S, then O += P V.  The reference m is kept lazily:
// O is rescaled only when the row maximum has grown by more than 2^8.  With
// one block S is double-buffered; with two, each block has its own S and O
// and one block's softmax runs under the other's MMAs.
// P is rounded to the inputs' type for the P V product (relative 2^-9 / 2^-12
// / 2^-4 a weight), its row sum and O stay in fp32.
//
// A unit cut between CTAs leaves normalised fp32 partials and their LSE in the
// workspace, at most two per CTA, and a second kernel joins them; units that
// one CTA covers are written to O directly.
#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kTreeMaxCtas = 152;            // CTAs of the attention kernel at most (bounds the workspace)
constexpr float kRescaleLog2 = 8.0f;
constexpr int kStagesMax = 12;

template <int ELEM, int NRB_>
struct TreeCfg : ElemCfg<ELEM> {
    using B = ElemCfg<ELEM>;
    static constexpr int NRB = NRB_;                          // 128-row blocks of a unit
    static constexpr int SW = 4 * NRB;                        // softmax warps
    static constexpr int PROD = SW, MMA = SW + 1;
    static constexpr int THREADS = (SW + 2) * 32;
    // K and V tiles are separate ring stages; with Q they fill 224 KB
    static constexpr int NS = (7 * 32768 - NRB * B::TILE_BYTES) / B::TILE_BYTES < kStagesMax
                                  ? (7 * 32768 - NRB * B::TILE_BYTES) / B::TILE_BYTES
                                  : kStagesMax;
    static constexpr int OFF_KV = NRB * B::TILE_BYTES;
    static constexpr int OFF_BARS = OFF_KV + NS * B::TILE_BYTES;
    static constexpr int SMEM_BYTES = OFF_BARS + 1024 + 1024;   // barriers, 1 KB alignment
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    // TMEM: two S buffers, then O of each block; P over S
    static constexpr int O_COL = 256;
};

struct TreeParams {
    void *o;                            // [B, T, H, D]
    float *lse;                         // [B, H, T] or NULL
    const int *seqlen, *batch_idx, *n_draft;
    const uint8_t *mask;                // [B or 1, T, T] or NULL
    int64_t mask_stride;
    float *part_o, *part_lse;           // [2 * ncta][NRB * 128][D], [2 * ncta][NRB * 128]
    int B, T, H, H_k, G, B_cache, S_max;
    int TB;                             // tokens of a row block
    int NRB;
    int ncta;
    float c;                            // scale * log2(e)
    float out_scale;
};

struct TreeSched {
    int64_t per, G0, G1;                // this CTA's tiles [G0, G1)
    int64_t off0;                       // first tile of sequence b0
    int b0;                             // first sequence with a tile at or past G0
};

struct TreeBars {
    uint64_t q_full, q_empty, drain;
    uint64_t s_full[2], p_full[2], pv_done[2], o_full[2];
    uint64_t kv_full[kStagesMax], kv_empty[kStagesMax];
    uint32_t tmem_base;
    int abort;
    TreeSched sched;
};
static_assert(sizeof(TreeBars) <= 1024, "barrier block");

// ---------------------------------------------------------------------------
// Work: the tiles of all (sequence b, kv head g, row-block group u), u fastest
// so that the units that read the same keys run at the same time.
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
    return (int64_t)p.H_k * tree_groups(p, n) * tree_tiles(tree_cached(p, b, false), n);
}

// One warp: this CTA's range and where its first segment starts.
__device__ void tree_schedule(const TreeParams &p, TreeSched *sc, int lane) {
    int64_t T = 0;
    for (int b = lane; b < p.B; b += 32) {
        T += tree_seq_tiles(p, b);
        if (blockIdx.x == 0) {          // reports values outside their bounds, once a call
            tree_cached(p, b, true);
            tree_drafts(p, b, true);
            cache_entry(p.batch_idx, b, p.B_cache, true);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    const int64_t per = (T + gridDim.x - 1) / gridDim.x;
    const int64_t G0 = min((int64_t)blockIdx.x * per, T), G1 = min(G0 + per, T);
    int b0 = p.B;
    int64_t off0 = T, base = 0;
    for (int bb = 0; bb < p.B && G0 < G1; bb += 32) {
        const int b = bb + lane;
        const int64_t n = b < p.B ? tree_seq_tiles(p, b) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && base + incl > G0);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b0 = bb + l;
            off0 = __shfl_sync(0xffffffffu, base + incl - n, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
        sc->per = per;
        sc->G0 = G0;
        sc->G1 = G1;
        sc->b0 = b0;
        sc->off0 = off0;
    }
}

struct TreeItem {
    int b, g, u, entry, L, n;
    int t0, t1, nt, nc;                 // this CTA's tiles [t0, t1) of the unit's nt; the first nc are cached keys
};

struct TreeCursor {
    int b = -1, g = 0, u = 0;
    int64_t off = 0;
};

__device__ bool tree_next(const TreeParams &p, const TreeSched &sc, TreeCursor &cur, TreeItem &it) {
    if (cur.b < 0) {
        cur.b = sc.b0;
        cur.off = sc.off0;
        if (cur.b >= p.B) return false;
        // whole units of sequence b0 that end at or before G0
        const int n = tree_drafts(p, cur.b, false);
        const int nt = tree_tiles(tree_cached(p, cur.b, false), n), nu = tree_groups(p, n);
        const int skip = (int)((sc.G0 - cur.off) / nt);
        cur.off += (int64_t)skip * nt;
        cur.g = skip / nu;
        cur.u = skip % nu;
    }
    for (;;) {
        if (cur.b >= p.B || cur.off >= sc.G1) return false;
        const int n = tree_drafts(p, cur.b, false), L = tree_cached(p, cur.b, false);
        const int nt = tree_tiles(L, n), nu = tree_groups(p, n);
        const bool hit = nu > 0;        // a sequence without drafts has no unit
        if (hit) {
            it.t0 = (int)(max(sc.G0, cur.off) - cur.off);
            it.t1 = (int)(min(sc.G1, cur.off + nt) - cur.off);
            it.b = cur.b;
            it.g = cur.g;
            it.u = cur.u;
            it.nt = nt;
            it.nc = (L + kRows - 1) / kRows;
            it.L = L;
            it.n = n;
            it.entry = cache_entry(p.batch_idx, cur.b, p.B_cache, false);
            cur.off += nt;
            if (++cur.u == nu) {
                cur.u = 0;
                ++cur.g;
            }
        }
        if (!hit || cur.g == p.H_k) {
            cur.g = 0;
            ++cur.b;
        }
        if (hit) return true;
    }
}

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------

// TMA producer: per item the Q blocks, then its K and V tiles into the ring.
template <class C>
__device__ void tree_producer(const TreeParams &p, const TreeSched &sc, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                              const CUtensorMap *tmV, const CUtensorMap *tmKn, const CUtensorMap *tmVn, uint8_t *smem,
                              TreeBars *bars) {
    volatile int *abort_flag = &bars->abort;
    uint32_t fill = 0, qn = 0;
    bool ok = test_gate_open(abort_flag);
    TreeCursor cur;
    while (ok) {
        TreeItem it;
        if (!tree_next(p, sc, cur, it)) break;
        // the one Q slot: free once the S MMAs of the item before are done
        if (qn > 0 && !mbar_wait(smem_u32(&bars->q_empty), (qn - 1) & 1, abort_flag)) {
            ok = false;
            break;
        }
        const uint32_t qb = smem_u32(&bars->q_full);
        const int tok0 = it.u * C::NRB * p.TB;
        // a box holds TB tokens x G heads; tokens past the sequence's own
        // (another sequence's, or zero fill) give rows that are never stored
        const int nblk = C::NRB == 2 && tok0 + p.TB < it.n ? 2 : 1;
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
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int st = fill % C::NS;
                const uint32_t rnd = fill / C::NS;
                if (rnd > 0 && !mbar_wait(smem_u32(&bars->kv_empty[st]), (rnd - 1) & 1, abort_flag)) {
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
                ++fill;
            }
        }
    }
    if (ok) {
        // the last release of every stage and of the Q slot must arrive before exit
        for (int st = 0; st < C::NS; ++st) {
            const uint32_t nf = fill > (uint32_t)st ? (fill - st + C::NS - 1) / C::NS : 0;
            if (nf && !mbar_wait(smem_u32(&bars->kv_empty[st]), (nf - 1) & 1, abort_flag)) break;
        }
        if (qn > 0) mbar_wait(smem_u32(&bars->q_empty), (qn - 1) & 1, abort_flag);
    } else {
        // aborted: let the copies already issued land before the CTA exits
        const uint32_t first = fill > (uint32_t)C::NS ? fill - C::NS : 0;
        for (uint32_t f = first; f < fill; ++f) mbar_wait_drain(smem_u32(&bars->kv_full[f % C::NS]), (f / C::NS) & 1);
        if (qn > 0) mbar_wait_drain(smem_u32(&bars->q_full), (qn - 1) & 1);
    }
}

// MMA issuer (one warp, one elected lane).  MMAs of one CTA execute in issue
// order, so S_j may overwrite the columns of P_i once P_i V_i is issued.
//   NRB = 1: S_j into buffer j % 2, then P_{j-1} V_{j-1}: S_j runs under the
//            softmax of tile j - 1.
//   NRB = 2: per tile and block t: P_{j-1} V_{j-1} of block t, then its S_j:
//            block t's MMAs run under the softmax of the other block.
template <class C>
__device__ void tree_mma(const TreeParams &p, const TreeSched &sc, uint8_t *smem, TreeBars *bars, uint32_t tmem_any) {
    volatile int *abort_flag = &bars->abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    constexpr uint32_t kIdS = mma_idesc(C::FMT, kRows, false);
    constexpr uint32_t kIdPV = mma_idesc(C::FMT, kD, true);
    uint32_t j = 0, qn = 0;             // tiles and items so far
    bool ok = true;

    auto issue_s = [&](int x, uint32_t buf, uint32_t kst) {
        const uint64_t q = smem_desc(smem_u32(smem + x * C::TILE_BYTES), 16, 1024);
        const uint64_t k = smem_desc(smem_u32(smem + C::OFF_KV + kst * C::TILE_BYTES), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kD / C::MMA_K; ++kk) {
            // each k-step (16 dims of 16 bits or 32 of 8) is 32 bytes of a 128-byte panel row
            const uint32_t off = (kk * 32 / 128) * kPanelBytes + (kk * 32) % 128;
            mma_ss<C::FP8>(tmem + buf * kRows, q + (off >> 4), k + (off >> 4), kIdS, kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars->s_full[buf]));
    };
    // P V of tile i (block x, P in buffer buf); `first` starts the item's O
    auto issue_pv = [&](uint32_t i, int x, uint32_t buf, uint32_t parity, bool first) -> bool {
        const uint32_t vst = (2 * i + 1) % C::NS;
        if (!warp_wait(smem_u32(&bars->p_full[buf]), parity, abort_flag) ||
            !warp_wait(smem_u32(&bars->kv_full[vst]), ((2 * i + 1) / C::NS) & 1, abort_flag))
            return false;
        tc_fence_after();
        // B = V tile MN-major: dims over the panels (LBO = panel stride), keys MMA_K rows a step
        const uint64_t v = smem_desc(smem_u32(smem + C::OFF_KV + vst * C::TILE_BYTES), kPanelBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kRows / C::MMA_K; ++kk)
            mma_ts<C::FP8>(tmem + C::O_COL + x * kD, tmem + buf * kRows + kk * (C::MMA_K * C::E / 4),
                           v + ((kk * C::MMA_K * 128) >> 4), kIdPV, !first || kk > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->pv_done[buf]));
        if (x == C::NRB - 1) tc_commit(smem_u32(&bars->kv_empty[vst]));
        return true;
    };

    TreeCursor cur;
    while (ok) {
        TreeItem it;
        if (!tree_next(p, sc, cur, it)) break;
        if (!warp_wait(smem_u32(&bars->q_full), qn & 1, abort_flag)) break;
        ++qn;
        const int nt = it.t1 - it.t0;
        for (int t = 0; ok && t <= nt; ++t) {
            const uint32_t kst = (2 * j) % C::NS;
            if (t < nt && !warp_wait(smem_u32(&bars->kv_full[kst]), ((2 * j) / C::NS) & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if constexpr (C::NRB == 1) {
                if (t < nt) {
                    issue_s(0, j & 1, kst);
                    tc_commit(smem_u32(&bars->kv_empty[kst]));
                    if (t == nt - 1) tc_commit(smem_u32(&bars->q_empty));
                }
                if (t > 0) ok = issue_pv(j - 1, 0, (j - 1) & 1, ((j - 1) >> 1) & 1, t == 1);
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (ok && t > 0) ok = issue_pv(j - 1, x, x, (j - 1) & 1, t == 1);
                    if (ok && t < nt) issue_s(x, x, kst);
                    if (ok && t == nt) tc_commit(smem_u32(&bars->o_full[x]));
                }
                if (ok && t < nt) {
                    tc_commit(smem_u32(&bars->kv_empty[kst]));
                    if (t == nt - 1) tc_commit(smem_u32(&bars->q_empty));
                }
            }
            if (t < nt) ++j;
        }
        if (!ok) break;
        if (C::NRB == 1) tc_commit(smem_u32(&bars->o_full[0]));
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain));
    mbar_wait_drain(smem_u32(&bars->drain), 0);
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
#pragma unroll 2
    for (int t = lo; t <= hi; ++t) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int jj = j0 + 32 * q + lane;
            const uint32_t bits = __ballot_sync(0xffffffffu, jj < it.n && m[(int64_t)t * p.T + jj] != 0);
            if (t == tok) w[q] = bits;
        }
    }
}

// Softmax and epilogue: warp w of a block owns its rows 32 (w % 4) .. + 31
// (TMEM lanes), one row a thread.
template <class C>
__device__ void tree_softmax(const TreeParams &p, const TreeSched &sc, uint8_t *smem, TreeBars *bars, uint32_t tmem,
                             int warp, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int x = warp >> 2;                            // row block
    const int r = (warp & 3) * 32 + lane;               // row of the block = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_tm = lane_base + C::O_COL + x * kD;
    const int rt = r / p.G, rh = r % p.G;               // token of the block, head of the group
    uint32_t j = 0, oph = 0;
    TreeCursor cur;
    for (;;) {
        TreeItem it;
        if (!tree_next(p, sc, cur, it)) break;
        const int tok = (it.u * C::NRB + x) * p.TB + rt;
        const bool row_ok = rt < p.TB && tok < it.n;
        float m = -INFINITY;                            // reference (log2 units) of P and O
        float l = 0.f;                                  // row sum
        bool ok = true;
        for (int t = it.t0; t < it.t1; ++t, ++j) {
            const uint32_t buf = C::NRB == 1 ? j & 1 : x;
            const uint32_t par = C::NRB == 1 ? (j >> 1) & 1 : j & 1;
            const bool drafts = t >= it.nc;
            // keys of this tile; fewer than 128 or drafts: a bit per key
            const int nk = imin(kRows, drafts ? it.n - (t - it.nc) * kRows : it.L - t * kRows);
            const bool masked = drafts || nk < kRows;
            uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            if (drafts) {
                tree_bits(p, it, tok, (t - it.nc) * kRows, lane, vis);
            } else if (masked) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int cnt = nk - 32 * q;
                    vis[q] = cnt >= 32 ? 0xffffffffu : cnt > 0 ? (1u << cnt) - 1u : 0u;
                }
            }
            if (!warp_wait(smem_u32(&bars->s_full[buf]), par, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t s_tm = lane_base + buf * kRows;
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(s_tm + 32 * q, s[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_wait_ld(s[q]);
            if (masked) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((vis[q] >> i) & 1u)) s[q][i] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
                for (int i = 1; i < 32; ++i) mx[q] = fmaxf(mx[q], __uint_as_float(s[q][i]));
            }
            const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
            const bool need = tmax > m + kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {
                float alpha = 1.f;
                if (need) {
                    alpha = m == -INFINITY ? 0.f : ex2(m - tmax);
                    m = tmax;
                    l *= alpha;
                }
                if (t > it.t0) {
                    // O holds the P V of the tile before once it is done
                    if (!warp_wait(smem_u32(&bars->pv_done[C::NRB == 1 ? (j - 1) & 1 : x]),
                                   C::NRB == 1 ? ((j - 1) >> 1) & 1 : (j - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tmem_ld32(o_tm + 32 * q, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(o_tm + 32 * q, o);
                    }
                }
            }
            // a row that has seen no key yet: every score is -inf, P = 0
            const float mr = m == -INFINITY ? 0.f : m;
            float ls[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float pq[32];
                ls[q] = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    pq[i] = ex2(fmaf(__uint_as_float(s[q][i]), p.c, -mr));
                    ls[q] += pq[i];
                }
                if constexpr (C::FP8) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = pack4_e4m3(pq[4 * i], pq[4 * i + 1], pq[4 * i + 2], pq[4 * i + 3]);
                    tmem_st8(s_tm + 8 * q, w);
                } else {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack2<C::FMT == 1u>(pq[2 * i], pq[2 * i + 1]);
                    tmem_st16(s_tm + 16 * q, w);
                }
            }
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            if (nk < kRows && x == 0) {
                // rows past the keys (stale cache contents, possibly not
                // finite): V is zeroed so that P = 0 contributes 0.  Block 0
                // does it; the MMA warp waits for block 0's P before it
                // issues either block's product.
                const uint32_t vst = (2 * j + 1) % C::NS;
                if (!warp_wait(smem_u32(&bars->kv_full[vst]), ((2 * j + 1) / C::NS) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                if (r >= nk) {
                    proxy_fence();
                    uint8_t *v = smem + C::OFF_KV + vst * C::TILE_BYTES + r * 128;
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(v + pn * kPanelBytes + (i << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    proxy_fence();
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[buf]));
        }
        if (!ok) break;

        // epilogue: O of a unit that this CTA covers alone, else a partial
        if (!warp_wait(smem_u32(&bars->o_full[x]), oph, abort_flag)) break;
        oph ^= 1;
        tc_fence_after();
        const bool whole = it.t1 - it.t0 == it.nt;
        const bool empty = l == 0.f;                    // the row saw no key (O may hold anything)
        const float inv = (whole ? p.out_scale : 1.f) / l;
        const float lse = empty ? -INFINITY : (m + log2f(l)) * kLn2;
        const int h = it.g * p.G + rh;
        // slot 2 * cta: a unit that an earlier CTA began; 2 * cta + 1: one that begins here
        const int64_t slot = ((int64_t)2 * blockIdx.x + (it.t0 == 0 ? 1 : 0)) * (C::NRB * kRows) + x * kRows + r;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld32(o_tm + 32 * q, o);
            tmem_wait_ld(o);
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = empty ? 0.f : __uint_as_float(o[i]) * inv;
            if (row_ok && !whole) {
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + slot * kD + 32 * q);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            } else if (row_ok) {
                uint8_t *dst = static_cast<uint8_t *>(p.o) +
                               ((((int64_t)it.b * p.T + tok) * p.H + h) * kD + 32 * q) * C::E;
                uint32_t w[8 * C::E];
                if constexpr (C::FP8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = pack4_e4m3(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack2<C::FMT == 1u>(f[2 * i], f[2 * i + 1]);
                }
#pragma unroll
                for (int i = 0; i < 2 * C::E; ++i)
                    reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        }
        if (row_ok) {
            if (!whole) p.part_lse[slot] = lse;
            else if (p.lse) p.lse[((int64_t)it.b * p.H + h) * p.T + tok] = lse;
        }
    }
}

template <int ELEM, int NRB>
__global__ void __launch_bounds__(TreeCfg<ELEM, NRB>::THREADS, 1)
    fmha_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                     const __grid_constant__ CUtensorMap tmVn, const TreeParams p) {
    using C = TreeCfg<ELEM, NRB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TreeBars *bars = reinterpret_cast<TreeBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 1);
        mbar_init(smem_u32(&bars->drain), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->p_full[i]), 4);
            mbar_init(smem_u32(&bars->pv_done[i]), 1);
            mbar_init(smem_u32(&bars->o_full[i]), 1);
        }
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::MMA) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == C::PROD) {
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmKn);
            prefetch_tmap(&tmVn);
        }
        tree_schedule(p, &bars->sched, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // the merge kernel may be scheduled as CTAs of this grid exit; it waits
    // for this grid's completion before it reads the partials
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const TreeSched sc = bars->sched;
    if (warp < C::SW) {
        tree_softmax<C>(p, sc, smem, bars, tmem, warp, lane);
    } else if (warp == C::PROD) {
        if (lane == 0) tree_producer<C>(p, sc, &tmQ, &tmK, &tmV, &tmKn, &tmVn, smem, bars);
    } else {
        tree_mma<C>(p, sc, smem, bars, tmem);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::MMA) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the units that several CTAs covered, one warp a row:
// O = out_scale * sum_c w_c O_c / sum_c w_c with w_c = exp(LSE_c - max LSE).
template <int ELEM>
__global__ void __launch_bounds__(256) fmha_tree_merge_kernel(const TreeParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);     // (b, t, h)
    if (row >= (int64_t)p.B * p.T * p.H) return;
    const int h = (int)(row % p.H), tok = (int)(row / p.H % p.T), b = (int)(row / ((int64_t)p.H * p.T));
    const int n = tree_drafts(p, b, false);
    // where the unit's tiles lie in the attention kernel's sequence of tiles
    int64_t tot = 0, pre = 0;
    for (int bb = lane; bb < p.B; bb += 32) {
        const int64_t x = tree_seq_tiles(p, bb);
        tot += x;
        if (bb < b) pre += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        tot += __shfl_xor_sync(0xffffffffu, tot, o);
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
    }
    const int nt = tree_tiles(tree_cached(p, b, false), n), g = h / p.G;
    const int blk = tok / p.TB, u = blk / p.NRB;
    const int64_t per = (tot + p.ncta - 1) / p.ncta;
    const int64_t off = pre + ((int64_t)g * tree_groups(p, n) + u) * nt;
    const int c0 = tok < n ? (int)(off / per) : 0, nch = tok < n ? (int)((off + nt - 1) / per) - c0 + 1 : 0;
    const int r = (blk % p.NRB) * kRows + (tok - blk * p.TB) * p.G + (h - g * p.G);
    auto slot = [&](int c) { return ((int64_t)2 * (c0 + c) + (c == 0 ? 1 : 0)) * (p.NRB * kRows) + r; };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nch <= 1) return;               // not a draft, or written by the attention kernel
    float mx = -INFINITY;
    bool nan = false;
    for (int c = lane; c < nch; c += 32) {
        const float x = p.part_lse[slot(c)];
        nan |= x != x;
        mx = fmaxf(mx, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (__any_sync(0xffffffffu, nan)) mx = 0.f;      // NaN in, NaN out
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    if (mx != -INFINITY) {
        for (int cb = 0; cb < nch; cb += 4) {
            float4 v[4];
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = cb + i < nch;
                const int64_t s = slot(in ? cb + i : 0);
                w[i] = in ? __expf(p.part_lse[s] - mx) : 0.f;
                v[i] = *reinterpret_cast<const float4 *>(p.part_o + s * kD + lane * 4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wsum += w[i];
                acc.x += w[i] * v[i].x;
                acc.y += w[i] * v[i].y;
                acc.z += w[i] * v[i].z;
                acc.w += w[i] * v[i].w;
            }
        }
    }
    const float inv = wsum == 0.f ? 0.f : p.out_scale / wsum;
    if constexpr (ELEM == FMHA_E4M3) {
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.o) + row * kD + lane * 4) =
            pack4_e4m3(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + row * kD + lane * 4) =
            make_uint2(pack2<ELEM == FMHA_BF16>(acc.x * inv, acc.y * inv), pack2<ELEM == FMHA_BF16>(acc.z * inv, acc.w * inv));
    }
    if (lane == 0 && p.lse) p.lse[((int64_t)b * p.H + h) * p.T + tok] = wsum == 0.f ? -INFINITY : mx + __logf(wsum);
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

bool tree_sizes_ok(int B, int T, int H, int H_k, int D, int S_max) {
    return B > 0 && T > 0 && H > 0 && H_k > 0 && H % H_k == 0 && H / H_k <= kRows && D == kD && S_max > 0;
}

using TreeKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, TreeParams);
template <int NRB>
TreeKernel tree_kernel_nrb(int dt) {
    return dt == FMHA_BF16 ? fmha_tree_kernel<FMHA_BF16, NRB>
           : dt == FMHA_F16 ? fmha_tree_kernel<FMHA_F16, NRB> : fmha_tree_kernel<FMHA_E4M3, NRB>;
}
template <int ELEM>
int tree_smem(int nrb) {
    return nrb == 2 ? TreeCfg<ELEM, 2>::SMEM_BYTES : TreeCfg<ELEM, 1>::SMEM_BYTES;
}

}  // namespace

int tree_set_wait_limit(unsigned long long ns) { return cache_set_wait_limit(ns); }
int tree_set_test_gate(int on) { return cache_set_test_gate(on); }
int tree_read_status(int reset) { return cache_read_status(reset); }

}  // namespace fmha

using namespace fmha;

extern "C" size_t fmha_tree_workspace_size(int B, int T, int H, int H_k, int D, int S_max) {
    if (!tree_sizes_ok(B, T, H, H_k, D, S_max)) return 0;
    const TreeShape s = tree_shape(T, H / H_k);
    // two partials a CTA: an fp32 row of O and its LSE for every row of a unit
    return (size_t)2 * tree_ctas(tree_max_tiles(s, B, T, H_k, S_max)) * s.NRB * kRows * (kD + 1) * sizeof(float);
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
    if (S_max <= 0 || B_cache <= 0 || !seqlen) return FMHA_ERR_INVALID_ARG;
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
    p.ncta = imin(sms, tree_ctas(tree_max_tiles(sh, B, T, H_k, S_max)));
    p.part_o = static_cast<float *>(workspace);
    p.part_lse = p.part_o + (size_t)2 * p.ncta * sh.NRB * kRows * kD;
    p.c = scale * kLog2e;
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
        if (!make_map(&tc[kv], dt, kv ? v_cache.data : k_cache.data, 4, dc, box) ||
            !make_map(&tn[kv], dt, kv ? v_new.data : k_new.data, 4, dn, box))
            return FMHA_ERR_CUDA;
    }

    auto kern = sh.NRB == 2 ? tree_kernel_nrb<2>(dt) : tree_kernel_nrb<1>(dt);
    const int smem = dt == FMHA_E4M3 ? tree_smem<FMHA_E4M3>(sh.NRB) : tree_smem<FMHA_BF16>(sh.NRB);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return cuda_failed();
    const int threads = sh.NRB == 2 ? TreeCfg<FMHA_BF16, 2>::THREADS : TreeCfg<FMHA_BF16, 1>::THREADS;
    kern<<<p.ncta, threads, smem, stream>>>(tq, tc[0], tc[1], tn[0], tn[1], p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;

    auto merge = dt == FMHA_BF16 ? fmha_tree_merge_kernel<FMHA_BF16>
                 : dt == FMHA_F16 ? fmha_tree_merge_kernel<FMHA_F16> : fmha_tree_merge_kernel<FMHA_E4M3>;
    const int64_t rows = (int64_t)B * T * H;
    const int warps = rows < 8 * 4 * sms ? 2 : 8;         // small calls spread their rows over the SMs
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + warps - 1) / warps));
    cfg.blockDim = dim3(32 * warps);
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
    if (T == 0 || S_max <= 0 || B_cache <= 0 || !seqlen || !path || !n_accept) return FMHA_ERR_INVALID_ARG;
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
    p.row16 = H_k * kD * (dt == FMHA_E4M3 ? 1 : 2) / 16;
    const int threads = p.row16 >= 256 ? 256 : (p.row16 + 31) / 32 * 32;
    fmha_tree_commit_kernel<<<dim3(P, B), threads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FMHA_OK : FMHA_ERR_CUDA;
}
