// fmha_paged.cu -- attention over a paged K/V cache held in e4m3 with a scale
// for each page and kv head.
//
// Operation: sequence b has L = seqlen[b] cached tokens, its last n among them
// the call's own (packed rows cu_q[b] .. cu_q[b + 1] - 1 of q); token j lies in
// row j % P of page p_j = table[e, j / P].  With c_j, d_j the codes of its key
// and value of kv head g, x_j = scale * k_scale[p_j, g] * q . c_j and, for
// query t, the keys j <= L - n + t (all without a mask),
//   O = out_scale * sum_j exp(x_j - LSE) v_scale[p_j, g] d_j,  LSE = ln sum_j exp(x_j).
//
// The codes go from the pages to the tensor cores as they are (TMA into
// swizzled shared memory, kind::f8f6f4), so q and the weights P have to be
// e4m3 there too.  One e4m3 number holds four bits, which is not enough of
// either; but as a sum of several the product stays exact, and with the roles
// swapped, S^T = K Q^T (M = 128 keys) and O^T = V^T P^T (M = 128 dims), each
// further term costs columns of N, not another pass over K or V:
//   q  = 2^k (q_0 + q_1 / 16), each 4 bits: all 8 bits of a bf16 row's
//        elements down to 2^-13 of its largest (2^k: a power of two per row); f16
//        has a third term, in units of the second: in columns of its own where a unit has
//        up to 8 rows, else added to the second's by an MMA of the first's shape, which
//        keeps their order;
//   P' = p_0 + p_1 / 16 + p_2 / 256, off by 2^-11 of a weight (two terms: 2^-8, and
//        small weights next to a large one lost from 2^-14 of the terms' unit on).
// A group of 16 query rows is thus 32 columns, [16 first terms | 16 second], and a
// unit one or two such groups of one kv head: single tokens, drafts, the ends of
// prompts.  More rows have a kernel of their own, further down.
//
// e4m3 ends at 448 and 2^-9, so P' = exp2(y_j - m) with y_j = x_j log2(e) +
// log2(v_scale) is relative to a reference m per row, that a group of at most
// eight key tiles has: the next group sets its own, up or down, from the maximum
// of its first tile, and O^T in TMEM and the row sums are brought to it.  A
// score that outgrows the reference opens a new group early (a reference up to
// 2^2 higher, if one was that high before, makes these fewer).
// So a long context of small weights behind a large one is not rounded to
// nothing: of a group's weight, what e4m3's smallest steps lose is 2^-10 at most
// (1024 weights of 2^-18 where the largest is 2^2 or more), or 2^-46 a key of the
// largest weight of all (a reference is not more than 2^24 below the highest so
// far, which keeps fp32 in its range).
// Row sums are of the unrounded weights, in fp32.
//
// Work: the key tiles of all units form one sequence cut evenly over the CTAs,
// one an SM; units that a cut goes through leave normalised fp32 partials,
// which a second kernel joins.  A CTA's producer warps (page ids, TMA, the scales
// by cp.async) fill rings of 128-key tiles, a q warp splits the next unit's rows
// into terms, and two pipelines, each an MMA issuer and four softmax warps with
// S^T, P^T and O^T of their own, go through the tiles: in units of up to 16 rows
// each takes every other tile with all rows, from a ring of its own, and their O
// are added up at the end; of two groups each takes one, of every tile.  A softmax
// thread is a key, and for O^T a dim.
//
// Bound by HBM where there are few rows.  64 sequences of 2100 to 8192 keys, 32/8
// heads, bf16: 108 us, 6.3 TB/s, 92% of the copy rate (one pipeline, and scales
// loaded by the softmax threads: 149); 8 of 8200 to 32768 in pages of 16, 64/8 heads,
// f16: 74 us, 72%; one sequence of 1000: 10.7 us, all latency: 2.5 to the first
// item, 5 to the first S, 7.5 to the last O, the rest the join.  16 sequences of 1500
// to 6000 with 7 tokens: 48 us where the bytes take 19 (weights as two terms: 45): a tile's chain of S, vote,
// weights and P V takes 1.1 us where its bytes take 0.73.
#include "fmha_cache.cuh"

namespace fmha {
namespace {

constexpr int kPagedMaxCtas = 152;       // bounds the workspace
constexpr int kPagedItems = 4;           // work items published ahead
constexpr int kGroupTiles = 8;           // key tiles with one reference
constexpr float kBias = 4.f;             // log2 of a group's largest P' where its reference is set
constexpr float kGrown = 8.75f;          // and how far it may grow: e4m3 ends at 2^8.8
constexpr float kAbove = 2.f;            // how far it may be set higher, to an earlier one
constexpr float kBelow = 24.f;           // how far a reference may be below the highest before it
constexpr int kStagesPaged = 6;
constexpr int kPagedBars = 4096;         // barrier block
constexpr float kNone = 1e30f;           // -m of a row that has seen no key in its group
constexpr float kLeastScale = 0x1p-60f, kMostScale = 0x1p60f;   // of values

template <bool BF_, int NG_, int NR_>
struct PagedCfg {
    static constexpr bool BF = BF_;
    static constexpr int NG = NG_;                            // groups of 16 query rows a unit holds, one or two,
    static constexpr int NR = NR_;                            // of whose rows so many are computed
    static constexpr int R = 16 * NG;                         // its rows
    static constexpr bool SPLIT = NG == 1;                    // the pipelines share out the tiles, else the groups
    static constexpr int SW = 8;                              // softmax warps
    // Producer warps: issuing a TMA load takes one warp 80 ns, and a tile of 16-token
    // pages is 16 of them (98 us instead of 67 for eight sequences of 32768); the
    // wider softmax needs the registers (above 12 warps, 128 a thread).
    static constexpr int NP = NR <= 8 ? 4 : 1;
    static constexpr int QW = SW, PROD = SW + 1, MMA = PROD + NP;   // q warp, producers, two MMA issuers
    static constexpr int THREADS = 32 * (MMA + 2);
    static constexpr int COLS = 32;                           // of a pipeline's S^T and O^T: a group's
    static constexpr bool INLINE3 = NR <= 8;                  // third terms in columns 8 .. 15 of the group, else in a tile of their own
    static constexpr int PIPE_COLS = 4 * COLS;                // TMEM: two S^T, O^T, and O^T of third terms that are apart
    static constexpr int TMEM_COLS = 2 * PIPE_COLS;
    static constexpr int P_ROW = COLS;                        // bytes of a key's P^T row
    static constexpr int P_TILE = kRows * P_ROW;
    static constexpr int P_BYTES = P_TILE * (INLINE3 ? 1 : 2);
    static constexpr uint64_t P_SWZ = 6;                      // 32-byte swizzle
    static constexpr bool QPASS = !BF && !INLINE3;            // q's third terms have an MMA of their own
    static constexpr int Q_ROWS = INLINE3 ? 8 : 16;           // rows of a group that have terms
    static constexpr int Q_BYTES = (QPASS ? 64 : 32) * NG * 128;   // by group 32 rows, and for that MMA 32 more: 16 of zeros, third terms
    static constexpr int STAGE = 2 * kPanelBytes;             // K and V of 128 keys
    static constexpr int OFF_P = 2 * Q_BYTES;                 // two buffers a pipeline
    static constexpr int OFF_KV = OFF_P + 4 * P_BYTES;
    static constexpr int NS_FIT = (226 * 1024 - kPagedBars - OFF_KV) / STAGE;
    static constexpr int NS = NS_FIT >= kStagesPaged ? kStagesPaged : SPLIT ? NS_FIT & ~1 : NS_FIT;
    static constexpr int RING = SPLIT ? NS / 2 : NS;          // stages of a ring
    static constexpr int OFF_BARS = OFF_KV + NS * STAGE;
    static constexpr int SMEM_BYTES = OFF_BARS + kPagedBars + 1024;   // 1 KB alignment
    static_assert(SMEM_BYTES <= 227 * 1024 && OFF_KV % 1024 == 0 && OFF_P % 1024 == 0, "shared memory");
    static_assert(!SPLIT || NS % 2 == 0, "a ring a pipeline");
    static_assert(!SPLIT || 2 * P_BYTES >= R * kD * 4, "pipeline 1 hands its O over in its P^T buffers");
};

struct PagedMeta {                       // whose partial a workspace slot holds
    int row0, h0, rows;                  // first q row and head of its unit; rows (0: no partial here)
    int last;                            // the unit ends with this partial
};

struct PagedParams {
    const uint8_t *q;                    // [N, H, 128]
    void *o;
    float *lse;                          // [N, H] or NULL
    const float *k_scale, *v_scale;      // [n_pages, H_k]
    const int *table, *seqlen, *batch_idx, *cu_q;
    float *part_o, *part_lse;            // [2 * ncta][R][D], [2 * ncta][R]
    PagedMeta *meta;                     // [2 * ncta]
    int B, N, max_q, H, H_k, G, B_table, width, n_pages, shift;
    int tau, tau_log;                    // tokens of a unit, a power of two
    int causal, edge, ncta;
    float c, out_scale;                  // c: scale * log2(e)
};

struct PagedItem {
    int g, L, base, entry;               // base: token t of the sequence sees keys up to base + t
    int row0, tok0, h0, rows;            // first q row, token and head; rows (0: no more items)
    int t0, t1, nt;                      // this CTA's tiles [t0, t1) of the unit's nt
};

struct PagedBars {
    uint64_t q_full[2], q_empty[2], drain[2], stat_full, epi_done;
    uint64_t s_full[2][2], s_free[2][2], p_full[2][2], pv_done[2][2];   // by pipeline and buffer
    uint64_t kv_full[kStagesPaged], kv_empty[kStagesPaged];
    uint64_t item_full[kPagedItems], item_empty[kPagedItems];
    PagedItem item[kPagedItems];
    uint32_t tmem_base;
    int abort;
    alignas(16) float zero[16];
    alignas(16) float scale[kStagesPaged][2][8];   // k_scale, v_scale of a stage's pages
    alignas(16) float qscale[2][32];     // of a q slot's rows: 2^k,
    alignas(16) int lim[2][32], at[2][32];   // the last key they see, and q row * H + head (-1: none)
    alignas(16) float nm[2][32];         // by pipeline and row: -m,
    alignas(16) float am[2][32];         // 2^(m before - m),
    float top[2][32];                    // the largest m so far, then (epilogue) the factor of O
    float red[8][16];                    // by warp: maxima or sums of its rows
    float stat_m[16], stat_l[16];        // pipeline 1's references and sums
    float other[16];                     // factor of pipeline 1's O
};
static_assert(sizeof(PagedBars) <= kPagedBars, "barrier block");

// ---------------------------------------------------------------------------
// PTX wrappers that this kernel adds
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t desc_sw(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint64_t swz) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (swz << 61);
}
// e4m3 operands, fp32 accumulator, M = 128; A and B K-major or MN-major
__device__ constexpr uint32_t paged_idesc(int n, bool mn) {
    return (1u << 4) | ((mn ? 3u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// Four k-steps of 16 with A in TMEM (16 elements: eight columns)
template <int BS>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n.reg .pred p, e;\n.reg .b32 a1, a2, a3;\n.reg .b64 b1, b2, b3;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
                 "add.u32 a1, %1, 8;\nadd.u64 b1, %2, %5;\nadd.u32 a2, %1, 16;\nadd.u64 b2, b1, %5;\nadd.u32 a3, %1, 24;\nadd.u64 b3, b2, %5;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc), "n"(BS >> 4)
                 : "memory");
}

// Four k-steps of e4m3, whose descriptors lie AS and BS bytes apart, under one election
template <int AS, int BS>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n.reg .pred p, e;\n.reg .b64 a1, a2, a3, b1, b2, b3;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
                 "add.u64 a1, %1, %5;\nadd.u64 b1, %2, %6;\nadd.u64 a2, a1, %5;\nadd.u64 b2, b1, %6;\n"
                 "add.u64 a3, a2, %5;\nadd.u64 b3, b2, %6;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(AS >> 4), "n"(BS >> 4)
                 : "memory");
}

__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Both terms' columns of NR rows of a group: first[NR], second[NR]; and the wait
// for them (which holds back other loads: hoisted above it they took too many registers).
template <int NR>
__device__ __forceinline__ void ld_terms(uint32_t taddr, uint32_t (&r)[2 * NR]) {
    if constexpr (NR == 16) {
        tmem_ld32(taddr, r);
    } else if constexpr (NR == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr + 16));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr + 16));
    }
}
template <int NR>
__device__ __forceinline__ void st_terms(uint32_t taddr, const uint32_t (&r)[2 * NR]) {
    if constexpr (NR == 16) {
        tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(r));
        tmem_st16(taddr + 16, *reinterpret_cast<const uint32_t(*)[16]>(r + 16));
    } else if constexpr (NR == 8) {
        tmem_st8(taddr, *reinterpret_cast<const uint32_t(*)[8]>(r));
        tmem_st8(taddr + 16, *reinterpret_cast<const uint32_t(*)[8]>(r + 8));
    } else {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr + 16), "r"(r[4]), "r"(r[5]),
                     "r"(r[6]), "r"(r[7])
                     : "memory");
    }
}
template <int NR>
__device__ __forceinline__ void wait_terms(uint32_t (&r)[2 * NR]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
    if constexpr (NR >= 8)
        asm volatile("" : "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
    if constexpr (NR >= 16) {
        asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]));
        asm volatile("" : "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
    }
}

// Bounded waits as in fmha_cache.cuh, but with a hint that lets the hardware
// suspend the warp for up to 20 us: most of a CTA's warps wait most of the time,
// and polling took as many issue slots as the softmax.
__device__ __forceinline__ bool hinted_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool hinted_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (hinted_try(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > g_wait_ns) {
            *abort_flag = 1;
            atomicExch(&g_status, FMHA_ERR_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    const bool r = hinted_try(bar, parity) || hinted_slow(bar, parity, abort_flag);
    return __all_sync(0xffffffffu, r);
}

// N consecutive columns, waited for; and stored.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 16) {
        tmem_ld16(taddr, r);
        tmem_wait_ld16(r);
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\ntcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr)
                     : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\ntcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr)
                     : "memory");
    }
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 16) tmem_st16(taddr, r);
    else if constexpr (N == 8) tmem_st8(taddr, r);
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
}

// Four weights as three terms each (first weight in the low byte), by way of f16,
// whose 11 bits hold a rest exactly: p = hi + mid / 16 + low / 256 in e4m3.  In one piece of
// PTX, since a 16-bit code that passes through C++ costs an instruction to widen it.
__device__ __forceinline__ void split4(const float (&e)[4], uint32_t &hi, uint32_t &mid, uint32_t &low) {
    const uint32_t p = pack2<false>(e[0], e[1]), q = pack2<false>(e[2], e[3]);
    asm("{\n.reg .b16 a, b;\n.reg .b32 x, y, u, v;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, %3;\ncvt.rn.satfinite.e4m3x2.f16x2 b, %4;\nmov.b32 %0, {a, b};\n"
        "cvt.rn.f16x2.e4m3x2 x, a;\ncvt.rn.f16x2.e4m3x2 y, b;\nsub.rn.f16x2 x, %3, x;\nsub.rn.f16x2 y, %4, y;\n"
        "mul.rn.f16x2 x, x, %5;\nmul.rn.f16x2 y, y, %5;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\ncvt.rn.satfinite.e4m3x2.f16x2 b, y;\nmov.b32 %1, {a, b};\n"
        "cvt.rn.f16x2.e4m3x2 u, a;\ncvt.rn.f16x2.e4m3x2 v, b;\nsub.rn.f16x2 x, x, u;\nsub.rn.f16x2 y, y, v;\n"
        "mul.rn.f16x2 x, x, %5;\nmul.rn.f16x2 y, y, %5;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\ncvt.rn.satfinite.e4m3x2.f16x2 b, y;\nmov.b32 %2, {a, b};\n}\n"
        : "=&r"(hi), "=&r"(mid), "=&r"(low)
        : "r"(p), "r"(q), "r"(0x4c004c00u));                 // 16, 16
}

// ---------------------------------------------------------------------------
// Work: of every sequence b, kv head g: blocks v of tau tokens, a unit each, whose
// rows are the group's heads of these tokens.  Block v's tiles reach to the last key that one of its tokens sees.
// A unit is `edge` tiles of nothing, for the work at its ends, and then its own.
// ---------------------------------------------------------------------------

struct PagedSeq {
    int L, n, row0, entry;
    int base, nv, full, all;             // blocks; the first `full` end within L, the others have `all` tiles
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int b, bool report) {
    PagedSeq s;
    s.L = clamped(p.seqlen[b], 0, p.width << p.shift, report);
    s.row0 = p.cu_q ? clamped(p.cu_q[b], 0, p.N, report) : b;
    s.n = p.cu_q ? clamped(clamped(p.cu_q[b + 1], s.row0, p.N, report) - s.row0, 0, p.max_q, report) : 1;
    s.entry = cache_entry(p.batch_idx, b, p.B_table, report);
    s.base = s.L - s.n;
    s.nv = (s.n + p.tau - 1) >> p.tau_log;
    s.full = p.causal ? imin(s.n, s.L) >> p.tau_log : 0;
    s.all = imax(1, (s.L + kRows - 1) / kRows);
    return s;
}
__device__ __forceinline__ int paged_tiles(const PagedParams &p, const PagedSeq &s, int v) {
    return v < s.full ? (imax(s.base, 0) + ((v + 1) << p.tau_log) + kRows - 1) / kRows : s.all;
}
// sum over k = 0 .. x of floor(k / 2^s), x >= -1
__device__ __forceinline__ int64_t floor_sum(int64_t x, int s) {
    const int64_t q = (x + 1) >> s, r = (x + 1) - (q << s);
    return ((q * (q - 1) / 2) << s) + q * r;
}
// tiles and edges of a head's blocks before block v
__device__ __forceinline__ int64_t paged_before(const PagedParams &p, const PagedSeq &s, int v) {
    const int f = imin(v, s.full), sh = 7 - p.tau_log;
    const int64_t d = (int64_t)(imax(s.base, 0) - 1) >> p.tau_log;     // tiles of block i: floor((i + 1 + d) / 2^sh) + 1
    const int64_t tiles = floor_sum(d + f, sh) - floor_sum(d, sh) + f + (int64_t)(v - f) * s.all;
    return tiles + (int64_t)v * p.edge;
}

struct PagedCursor {
    PagedSeq s;
    int64_t off, G0, G1;                 // off: where the unit at hand begins; this CTA's range
    int b, g, v;
};

// One warp: this CTA's range and its first unit (the same in every lane).
__device__ void paged_schedule(const PagedParams &p, PagedCursor &cur, int lane) {
    auto size = [&](int b) {
        const PagedSeq s = paged_seq(p, b, false);
        return p.H_k * paged_before(p, s, s.nv);
    };
    const int64_t n0 = lane < p.B ? size(lane) : 0;          // kept: most batches are this small
    int64_t T = n0;
    for (int b = lane + 32; b < p.B; b += 32) T += size(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    const int64_t per = (T + gridDim.x - 1) / gridDim.x;
    cur.G0 = min((int64_t)blockIdx.x * per, T);
    cur.G1 = min(cur.G0 + per, T);
    cur.b = p.B;
    cur.off = T;
    cur.g = cur.v = 0;
    if (blockIdx.x == gridDim.x - 1)     // reports values outside their bounds, once a call
        for (int b = lane; b < p.B; b += 32) paged_seq(p, b, true);
    int64_t base = 0;
    for (int bb = 0; bb < p.B && cur.G0 < cur.G1; bb += 32) {
        const int b = bb + lane;
        const int64_t n = bb == 0 ? n0 : b < p.B ? size(b) : 0;
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
            cur.s = paged_seq(p, cur.b, false);
            const int64_t head = paged_before(p, cur.s, cur.s.nv);
            int64_t x = cur.G0 - cur.off;
            cur.g = (int)(x / head);
            x -= cur.g * head;
            int lo = 0, hi = cur.s.nv;                        // the block that x lies in
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (paged_before(p, cur.s, mid) <= x) lo = mid;
                else hi = mid;
            }
            cur.v = lo;
            cur.off += cur.g * head + paged_before(p, cur.s, lo);
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ bool paged_next(const PagedParams &p, PagedCursor &cur, PagedItem &it) {
    it.rows = 0;
    if (cur.b >= p.B || cur.off >= cur.G1) return false;
    while (cur.s.nv == 0 || cur.g == p.H_k) {                // the next sequence that has tokens
        if (++cur.b >= p.B) return false;
        cur.g = cur.v = 0;
        cur.s = paged_seq(p, cur.b, false);
    }
    const int nt = paged_tiles(p, cur.s, cur.v);
    it.t0 = imax(0, (int)(max(cur.G0, cur.off) - cur.off) - p.edge);
    it.t1 = (int)(min(cur.G1, cur.off + p.edge + nt) - cur.off) - p.edge;
    if (it.t1 <= 0) return false;        // the range ends before the unit's first tile
    it.nt = nt;
    it.g = cur.g;
    it.L = cur.s.L;
    it.base = p.causal ? cur.s.base : cur.s.L;
    it.entry = cur.s.entry;
    it.tok0 = cur.v << p.tau_log;
    it.row0 = cur.s.row0 + it.tok0;
    it.h0 = cur.g * p.G;
    it.rows = imin(p.tau, cur.s.n - it.tok0) * p.G;
    cur.off += p.edge + nt;
    if (++cur.v == cur.s.nv) {
        cur.v = 0;
        ++cur.g;
    }
    return true;
}

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool paged_take(PagedBars *bars, uint32_t i, PagedItem &it, volatile int *abort_flag, int lane) {
    const uint32_t st = i % kPagedItems;
    if (!wait_all(smem_u32(&bars->item_full[st]), (i / kPagedItems) & 1, abort_flag)) return false;
    it = bars->item[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[st]));
    return it.rows > 0;
}

// Page of a sequence's token, or -1 (no such entry, or a page outside the cache).
__device__ __forceinline__ int page_id(const PagedParams &p, int entry, int i, bool report) {
    const int id = entry >= 0 ? p.table[(int64_t)entry * p.width + i] : -1;
    if (id >= 0 && id < p.n_pages) return id;
    if (report && entry >= 0) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
    return -1;
}

// Stage and parity of the n-th tile of ring x.
template <class C>
__device__ __forceinline__ uint32_t ring_stage(int x, uint32_t n) { return (C::SPLIT ? x * C::RING : 0) + n % C::RING; }
template <class C>
__device__ __forceinline__ uint32_t ring_parity(uint32_t n) { return (n / C::RING) & 1; }

__device__ const float g_one = 1.f;

// Producer warp x: loads its share of the K and V tiles, a lane a page's K or V
// with its scale.  Ids are fetched a tile ahead.  Warp 0 also publishes the items.
template <class C>
__device__ void paged_producer(const PagedParams &p, PagedCursor &cur, int gate, const CUtensorMap *tmK,
                               const CUtensorMap *tmV, uint8_t *smem, PagedBars *bars, int x, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int job = lane * C::NP + x, kv = job & 1;           // of a tile: page job / 2, its K or V
    bool ok = true;
    if (gate) ok = __all_sync(0xffffffffu, lane > 0 || test_gate_open(abort_flag));
    uint32_t fill[2] = {0, 0}, qn = 0;
    const int P = 1 << p.shift, per = kRows >> p.shift;       // pages of a tile
    auto publish = [&](uint32_t i, const PagedItem &it) -> bool {
        if (x > 0) return true;
        const uint32_t st = i % kPagedItems;
        if (i >= kPagedItems && !wait_all(smem_u32(&bars->item_empty[st]), (i / kPagedItems - 1) & 1, abort_flag)) return false;
        if (lane == 0) {
            bars->item[st] = it;
            mbar_arrive(smem_u32(&bars->item_full[st]));
        }
        __syncwarp();
        return true;
    };
    PagedItem it, next;
    if (ok) {
        paged_next(p, cur, it);
        ok = publish(0, it);
    }
    while (ok && it.rows > 0) {
        ++qn;
        const int pages = (it.L + P - 1) >> p.shift;
        auto id_of = [&](int t) {
            const int i = t * per + (job >> 1);
            return job < 2 * per && i < pages && t < it.t1 ? page_id(p, it.entry, i, true) : -1;
        };
        int id = id_of(it.t0);
        for (int t = it.t0; t < it.t1; ++t) {
            const int ahead = id_of(t + 1);
            const int ring = C::SPLIT ? (t - it.t0) & 1 : 0;
            const uint32_t n = ring ? fill[1] : fill[0], st = ring_stage<C>(ring, n);
            if (n >= C::RING && !wait_all(smem_u32(&bars->kv_empty[st]), ring_parity<C>(n) ^ 1, abort_flag)) {
                ok = false;
                break;
            }
            const int here = imax(0, imin(per, pages - t * per));
            const uint32_t fb = smem_u32(&bars->kv_full[st]);
            const int jobs = (2 * here - x + C::NP - 1) / C::NP;     // of this warp
            if (lane == 0) mbar_expect_tx(fb, imax(0, jobs) * (P << 7));
            __syncwarp();
            if (job < 2 * here) {
                const uint32_t dst = smem_u32(smem + C::OFF_KV + st * C::STAGE) + kv * kPanelBytes + (job >> 1) * (P << 7);
                // a page outside the cache: a coordinate outside it, which reads zeros
                const int head = id >= 0 ? id * p.H_k + it.g : p.n_pages * p.H_k;
                tma_load_3d(dst, kv ? tmV : tmK, fb, 0, 0, head);
                const float *src = id >= 0 ? (kv ? p.v_scale : p.k_scale) + head : &g_one;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&bars->scale[st][kv][job >> 1])), "l"(src)
                             : "memory");
            }
            // every lane's arrival, when its copies are there
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
            if (ring) ++fill[1];
            else ++fill[0];
            id = ahead;
            if (t == it.t0) {            // the next item is worked out behind the first tile's loads
                paged_next(p, cur, next);
                ok = publish(qn, next);
                if (!ok) break;
            }
        }
        it = next;
    }
    // the last release of every stage must arrive before exit; when the CTA
    // gave up, only the copies already issued
#pragma unroll
    for (int ring = 0; ring < (C::SPLIT ? 2 : 1); ++ring)
        for (uint32_t n = fill[ring] > C::RING ? fill[ring] - C::RING : 0; n < fill[ring]; ++n) {
            const uint32_t st = ring_stage<C>(ring, n);
            if (ok) ok = wait_all(smem_u32(&bars->kv_empty[st]), ring_parity<C>(n), abort_flag);
            if (!ok) mbar_wait_drain(smem_u32(&bars->kv_full[st]), ring_parity<C>(n));
        }
    for (uint32_t i = qn > 2 ? qn - 2 : 0; x == 0 && ok && i < qn; ++i)
        ok = wait_all(smem_u32(&bars->q_empty[i & 1]), (i >> 1) & 1, abort_flag);
}

// Four elements of a row of q times a power of two that brings the row's largest
// to [2^7, 2^8); g: what takes it back.  A row with an infinity or a NaN becomes
// one of NaN.  By a warp, four elements a lane.
template <bool BF>
__device__ __forceinline__ void row_scaled(uint2 v, float (&y)[4], float &g) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (BF) {
            y[2 * j] = __uint_as_float(w[j] << 16);
            y[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
            y[2 * j] = f.x;
            y[2 * j + 1] = f.y;
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = max((int)(top >> 23) - 127, -100);
    const float up = top < 0x7f800000u ? __uint_as_float((uint32_t)(127 + 7 - e) << 23) : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] *= up;
    g = __uint_as_float((uint32_t)(127 + e - 7) << 23);
}

// The next term of four elements: its codes; and `rest` without it.  In f16, which
// holds a row's scaled elements exactly where the terms do.
__device__ __forceinline__ uint32_t take_term(uint32_t (&rest)[2]) {
    uint32_t code;
    asm("{\n.reg .b16 a, b;\n.reg .b32 x, y;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\ncvt.rn.satfinite.e4m3x2.f16x2 b, %2;\nmov.b32 %0, {a, b};\n"
        "cvt.rn.f16x2.e4m3x2 x, a;\ncvt.rn.f16x2.e4m3x2 y, b;\nsub.rn.f16x2 %1, %1, x;\nsub.rn.f16x2 %2, %2, y;\n}\n"
        : "=&r"(code), "+r"(rest[0]), "+r"(rest[1]));
    return code;
}

// What is left of them, in e5m2.
__device__ __forceinline__ uint32_t last_term(const uint32_t (&rest)[2]) {
    uint32_t code;
    asm("{\n.reg .b16 a, b;\ncvt.rn.satfinite.e5m2x2.f16x2 a, %1;\ncvt.rn.satfinite.e5m2x2.f16x2 b, %2;\nmov.b32 %0, {a, b};\n}\n"
        : "=r"(code)
        : "r"(rest[0]), "r"(rest[1]));
    return code;
}

// Rows r0 .. r0 + N - 1 of an item's q as e4m3 terms in shared memory, and what
// the softmax needs to know of each row; by a warp.
template <class C, int N>
__device__ __forceinline__ void paged_terms(const PagedParams &p, uint8_t *smem, PagedBars *bars, const PagedItem &it, int slot,
                                            int r0, int lane) {
    uint8_t *qs = smem + slot * C::Q_BYTES;
    uint2 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int r = r0 + k, t = r / p.G;
        const int at = r < it.rows ? (it.row0 + t) * p.H + it.h0 + r - t * p.G : -1;
        v[k] = at >= 0 ? *reinterpret_cast<const uint2 *>(p.q + ((int64_t)at * kD + lane * 4) * 2) : make_uint2(0u, 0u);
        if (lane == k) {
            bars->at[slot][r] = at;
            bars->lim[slot][r] = it.base + it.tok0 + t;
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float y[4], g;
        row_scaled<C::BF>(v[k], y, g);
        const int r = r0 + k, row = 32 * (r >> 4) + (r & 15);
        uint32_t rest[2] = {pack2<false>(y[0], y[1]), pack2<false>(y[2], y[3])};
        // 16-byte chunk lane / 4 of a 128-byte row, swizzled
        auto term = [&](int row_) {
            *reinterpret_cast<uint32_t *>(qs + row_ * 128 + ((((lane >> 2) ^ (row_ & 7)) << 4) | ((lane & 3) << 2))) = take_term(rest);
        };
        term(row);
#pragma unroll
        for (int j = 0; j < 2; ++j) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(rest[j]) : "r"(0x4c004c00u));   // by 16
        term(row + 16);
        if constexpr (!C::BF) term(C::INLINE3 ? row + 8 : 32 * C::NG + row + 16);   // in units of the second
        if (lane == 0) bars->qscale[slot][r] = g;
    }
}

// One warp: the rows of every item but the first, an item ahead of the softmax.
// The first's are shared out among the softmax warps, which have nothing to do
// then (one warp took 6 us for 32 rows from a cold cache).
template <class C>
__device__ void paged_queries(const PagedParams &p, uint8_t *smem, PagedBars *bars, int lane) {
    volatile int *abort_flag = &bars->abort;
    PagedItem it;
    for (uint32_t i = 0; paged_take(bars, i, it, abort_flag, lane); ++i) {
        const int slot = i & 1;
        if (i == 0) continue;
        if (i >= 2 && !wait_all(smem_u32(&bars->q_empty[slot]), ((i >> 1) - 1) & 1, abort_flag)) break;
        const int rows = imin((it.rows + 15) & ~15, C::NG * C::Q_ROWS);
        for (int r0 = 0; r0 < rows; r0 += 8) paged_terms<C, 8>(p, smem, bars, it, slot, r0, lane);
        proxy_fence();
        __syncwarp();
        if (lane < C::SW) mbar_arrive(smem_u32(&bars->q_full[slot]));
    }
}

// MMA issuer of pipeline w (one warp, one elected lane).  S^T and P^T are
// double-buffered: S^T of the pipeline's next tile is issued before the P V of
// this one, so the softmax of one runs under the MMAs of the other.
template <class C>
__device__ void paged_mma(uint8_t *smem, PagedBars *bars, uint32_t tmem_any, int w, int lane) {
    volatile int *abort_flag = &bars->abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0) + w * C::PIPE_COLS;
    const uint64_t q0 = desc_sw(smem_u32(smem), 16, 1024, 2);
    const uint64_t p0 = desc_sw(smem_u32(smem + C::OFF_P + w * 2 * C::P_BYTES), C::P_TILE, 8 * C::P_ROW, C::P_SWZ);
    const uint64_t k0 = desc_sw(smem_u32(smem + C::OFF_KV), 16, 1024, 2);
    const uint64_t v0 = desc_sw(smem_u32(smem + C::OFF_KV + kPanelBytes), kPanelBytes, 1024, 2);   // MN-major
    constexpr int kStep = C::SPLIT ? 2 : 1;
    uint32_t c = 0, m = 0;               // tiles of the ring so far, tiles of MMAs so far
    bool ok = true;
    PagedItem it;
    auto issue_pv = [&](uint32_t mm, uint32_t st, bool begins) -> bool {
        const uint32_t b = mm & 1;
        if (!wait_all(smem_u32(&bars->p_full[w][b]), (mm >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint64_t v = v0 + ((st * C::STAGE) >> 4), pt = p0 + ((b * C::P_BYTES) >> 4);
        const uint32_t o_tm = tmem + 2 * C::COLS;
        // 32 keys a step
        mma4<32 * 128, 32 * C::P_ROW>(o_tm, v, pt, paged_idesc(32, true), begins ? 0u : 1u);
        if constexpr (!C::INLINE3)
            mma4<32 * 128, 32 * C::P_ROW>(o_tm + C::COLS, v, pt + (C::P_TILE >> 4), paged_idesc(16, true), begins ? 0u : 1u);
        tc_commit(smem_u32(&bars->pv_done[w][b]));
        tc_commit(smem_u32(&bars->kv_empty[st]));
        return true;
    };
    for (uint32_t i = 0; ok && paged_take(bars, i, it, abort_flag, lane); ++i) {
        const int slot = i & 1;
        const bool on = C::SPLIT || 16 * w < it.rows;
        if (!wait_all(smem_u32(&bars->q_full[slot]), (i >> 1) & 1, abort_flag)) {
            ok = false;
            break;
        }
        // this pipeline's group in q's tile
        const int grp = C::SPLIT ? 0 : w;
        const uint64_t q = q0 + ((slot * C::Q_BYTES + grp * 32 * 128) >> 4);
        const uint64_t q3 = q + ((32 * C::NG * 128) >> 4);
        const int tb = it.t0 + (C::SPLIT ? w : 0);
        uint32_t st_before = 0;
        for (int t = tb; t < it.t1; t += kStep, ++c) {
            const uint32_t st = ring_stage<C>(w, c), b = m & 1;
            if (!wait_all(smem_u32(&bars->kv_full[st]), ring_parity<C>(c), abort_flag)) {
                ok = false;
                break;
            }
            if (!on) {                   // nothing to do with this tile
                if (lane == 0) mbar_arrive(smem_u32(&bars->kv_empty[st]));
                continue;
            }
            if (m >= 2 && !wait_all(smem_u32(&bars->s_free[w][b]), ((m >> 1) - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t k = k0 + ((st * C::STAGE) >> 4);
            const uint32_t s_tm = tmem + b * C::COLS;
            mma4<32, 32>(s_tm, k, q, paged_idesc(32, false), 0u);      // 32 dims a step: 32 bytes of a row
            if constexpr (C::QPASS) mma4<32, 32>(s_tm, k, q3, paged_idesc(32, false), 1u);
            tc_commit(smem_u32(&bars->s_full[w][b]));
            if (t + kStep >= it.t1) tc_commit(smem_u32(&bars->q_empty[slot]));
            if (t > tb && !issue_pv(m - 1, st_before, t - kStep == tb)) {
                ok = false;
                break;
            }
            st_before = st;
            ++m;
        }
        if (!ok) break;
        if (tb >= it.t1 || !on) tc_commit(smem_u32(&bars->q_empty[slot]));
        else ok = issue_pv(m - 1, st_before, tb + kStep >= it.t1);   // the item's last P V: its epilogue does not wait for the next item's loads
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain[w]));
    mbar_wait_drain(smem_u32(&bars->drain[w]), 0);
}

// Named barrier of a pipeline's softmax threads, and votes over them.
__device__ __forceinline__ void soft_sync(int w) { asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory"); }
__device__ __forceinline__ bool soft_any(int w, bool v) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(1 + w)
                 : "memory");
    return r != 0;
}

// Softmax and epilogue of pipeline w.  Thread r is key r of its tiles (TMEM lane
// of S^T), and dim r of O^T.
template <class C, int NR>
__device__ void paged_softmax(const PagedParams &p, uint8_t *smem, PagedBars *bars, uint32_t tmem_all, int warp, int lane) {
    constexpr int kStep = C::SPLIT ? 2 : 1;
    volatile int *abort_flag = &bars->abort;
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tmem = tmem_all + w * C::PIPE_COLS + ((uint32_t)((warp & 3) * 32) << 16);
    uint8_t *pbuf = smem + C::OFF_P + w * 2 * C::P_BYTES;
    float *scratch = reinterpret_cast<float *>(smem + C::OFF_P + 2 * C::P_BYTES);   // pipeline 1's O at a unit's end
    const uint64_t sixteenth = pack_f2(0.0625f, 0.0625f);
    uint32_t c = 0, n = 0;               // tiles so far, and of its ring
    int parts = 0;                       // bit s: slot s of this CTA holds a partial
    PagedItem it;
    for (uint32_t i = 0;; ++i) {
        // a false return is either the end or an abort: all warps leave together
        const bool more = paged_take(bars, i, it, abort_flag, lane);
        if (soft_any(w, !more)) break;
        const int slot = i & 1, row0 = C::SPLIT ? 0 : 16 * w;     // this pipeline's rows
        const bool on = row0 < it.rows;
        const int tb = it.t0 + (C::SPLIT ? w : 0);
        if (i == 0) {
            constexpr int N = C::R / C::SW;
            if (warp * N < ((it.rows + 15) & ~15) && (warp * N & 15) < C::Q_ROWS) paged_terms<C, N>(p, smem, bars, it, slot, warp * N, lane);
            proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[slot]));
        }
        bool ok = wait_all(smem_u32(&bars->q_full[slot]), (i >> 1) & 1, abort_flag);
        uint64_t l[NR / 2];         // this key's part of the row sums, relative to m
#pragma unroll
            for (int k = 0; k < NR / 2; ++k) l[k] = 0;
        if (r < C::R) {
            bars->top[w][r] = -INFINITY;
            bars->nm[w][r] = kNone;
        }
        int since = kGroupTiles;         // tiles of the group so far
        bool first = true;
        if (!on) n += it.t1 - it.t0;     // a pipeline without rows has no tiles
        for (int t = tb; on && t < it.t1; t += kStep, ++c, ++n) {
            const uint32_t b = c & 1, st = ring_stage<C>(w, n);
            const int key = t * kRows + r, nk = it.L - t * kRows;
            ok = wait_all(smem_u32(&bars->s_full[w][b]), (c >> 1) & 1, abort_flag) && ok;
            ok = wait_all(smem_u32(&bars->kv_full[st]), ring_parity<C>(n), abort_flag) && ok;   // the scales, and V
            if (nk < kRows) {
                // rows past the keys (of an earlier tile, or of nothing): V is zeroed so that P = 0 contributes
                // 0 (by both pipelines where both use the tile: each before its own P V)
                if (ok && r >= nk) {
                    proxy_fence();
                    uint4 *v = reinterpret_cast<uint4 *>(smem + C::OFF_KV + st * C::STAGE + kPanelBytes + r * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            tc_fence_after();
            const float sv = fminf(fmaxf(bars->scale[st][1][r >> p.shift], kLeastScale), kMostScale);
            const float a = p.c * bars->scale[st][0][r >> p.shift], lsv = __log2f(sv);
            const uint64_t a2 = pack_f2(a, a), lsv2 = pack_f2(lsv, lsv);
            const bool masked = nk < kRows || t * kRows + kRows - 1 > it.base + it.tok0;
            bool fresh = since == kGroupTiles;
            uint64_t e[NR / 2];     // scores in log2 units, with the value's scale, over the reference
            for (;;) {
                float top = -INFINITY;
                uint32_t s[2 * NR];
                ld_terms<NR>(tmem + b * C::COLS, s);
                uint32_t z[NR];
                if constexpr (!C::BF && C::INLINE3) ld_cols<NR>(tmem + b * C::COLS + 8, z);
                wait_terms<NR>(s);
                if constexpr (!C::BF && C::INLINE3) {
#pragma unroll
                    for (int k = 0; k < NR; ++k) s[NR + k] = __float_as_uint(__uint_as_float(s[NR + k]) + __uint_as_float(z[k]));
                }
                const float4 *g4 = reinterpret_cast<const float4 *>(&bars->qscale[slot][row0]);
                const float4 *n4 = reinterpret_cast<const float4 *>(fresh ? bars->zero : &bars->nm[w][row0]);
#pragma unroll
                for (int k = 0; k < NR; k += 4) {
                    const float4 gg = g4[k / 4], nm = n4[k / 4];
                    const uint64_t t0 = fma_f2(pack_f2(__uint_as_float(s[NR + k]), __uint_as_float(s[NR + k + 1])), sixteenth,
                                               pack_f2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])));
                    const uint64_t t1 = fma_f2(pack_f2(__uint_as_float(s[NR + k + 2]), __uint_as_float(s[NR + k + 3])),
                                               sixteenth, pack_f2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])));
                    e[k / 2] = fma_f2(t0, mul_f2(pack_f2(gg.x, gg.y), a2), add_f2(pack_f2(nm.x, nm.y), lsv2));
                    e[k / 2 + 1] = fma_f2(t1, mul_f2(pack_f2(gg.z, gg.w), a2), add_f2(pack_f2(nm.z, nm.w), lsv2));
                }
                if (masked) {
                    const int4 *lim = reinterpret_cast<const int4 *>(&bars->lim[slot][row0]);
#pragma unroll
                    for (int k = 0; k < NR; k += 4) {
                        const int4 m = lim[k / 4];
                        float u, v;
                        unpack_f2(e[k / 2], u, v);
                        e[k / 2] = pack_f2(r < nk && key <= m.x ? u : -INFINITY, r < nk && key <= m.y ? v : -INFINITY);
                        unpack_f2(e[k / 2 + 1], u, v);
                        e[k / 2 + 1] = pack_f2(r < nk && key <= m.z ? u : -INFINITY, r < nk && key <= m.w ? v : -INFINITY);
                    }
                }
#pragma unroll
                for (int k = 0; k < NR; k += 2) {
                    float u, v;
                    unpack_f2(e[k / 2], u, v);
                    top = max3(top, u, v);
                }
                // does a score outgrow the group's reference?  Then it begins anew here.
                if (!soft_any(w, !ok || (!fresh && top > kGrown))) break;
                if (soft_any(w, !ok)) {
                    ok = false;
                    break;
                }
                fresh = true;
            }
            if (!ok) break;              // voted: the same in every warp
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[w][b]));
            if (fresh) {
                // the group's reference: the tile's maximum of every row
#pragma unroll
                for (int k = 0; k < NR; k += 2) {
                    float u, v;
                    unpack_f2(e[k / 2], u, v);
                    u = redux_max(u);
                    v = redux_max(v);
                    if (lane == 0) {
                        bars->red[warp][k] = u;
                        bars->red[warp][k + 1] = v;
                    }
                }
                soft_sync(w);
                if (r < NR) {
                    const int row = row0 + r;
                    const float top = fmaxf(fmaxf(bars->red[4 * w][r], bars->red[4 * w + 1][r]),
                                            fmaxf(bars->red[4 * w + 2][r], bars->red[4 * w + 3][r]));
                    const float M = bars->top[w][row], own = top - kBias, nm = bars->nm[w][row];
                    const float m = fmaxf(fmaxf(own, fminf(M, own + kAbove)), M - kBelow);
                    bars->top[w][row] = fmaxf(M, m);
                    // without a key so far: nothing to keep, and the next key is above the reference
                    bars->am[w][row] = nm == kNone ? 0.f : ex2(-nm - m);
                    bars->nm[w][row] = m == -INFINITY ? kNone : -m;
                }
                ok = first || wait_all(smem_u32(&bars->pv_done[w][b ^ 1]), ((c - 1) >> 1) & 1, abort_flag);
                if (soft_any(w, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!first) {        // O^T, whose last P V is that of this pipeline's tile before
                    uint32_t s[2 * NR];
                    ld_terms<NR>(tmem + 2 * C::COLS, s);
                    wait_terms<NR>(s);
#pragma unroll
                    for (int k = 0; k < NR; k += 4) {
                        const float4 am = *reinterpret_cast<const float4 *>(&bars->am[w][row0 + k]);
                        const float f[4] = {am.x, am.y, am.z, am.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            s[k + q] = __float_as_uint(__uint_as_float(s[k + q]) * f[q]);
                            s[NR + k + q] = __float_as_uint(__uint_as_float(s[NR + k + q]) * f[q]);
                        }
                    }
                    st_terms<NR>(tmem + 2 * C::COLS, s);
                    uint32_t z[NR];
                    ld_cols<NR>(tmem + (C::INLINE3 ? 2 * C::COLS + 8 : 3 * C::COLS), z);
#pragma unroll
                    for (int k = 0; k < NR; ++k)
                        z[k] = __float_as_uint(__uint_as_float(z[k]) * bars->am[w][row0 + k]);
                    st_cols<NR>(tmem + (C::INLINE3 ? 2 * C::COLS + 8 : 3 * C::COLS), z);
                }
#pragma unroll
                for (int k = 0; k < NR; k += 4) {
                    const float4 nm = *reinterpret_cast<const float4 *>(&bars->nm[w][row0 + k]);
                    const float4 am = *reinterpret_cast<const float4 *>(&bars->am[w][row0 + k]);
                    l[k / 2] = mul_f2(l[k / 2], pack_f2(am.x, am.y));
                    l[k / 2 + 1] = mul_f2(l[k / 2 + 1], pack_f2(am.z, am.w));
                    e[k / 2] = add_f2(e[k / 2], pack_f2(nm.x, nm.y));
                    e[k / 2 + 1] = add_f2(e[k / 2 + 1], pack_f2(nm.z, nm.w));
                }
                tmem_wait_st();
                tc_fence_before();
                since = 0;
            }
            ++since;
            // weights, their sums, and both terms into P^T
            const float isv = ex2(-lsv);     // of the same rounded logarithm
            const uint64_t isv2 = pack_f2(isv, isv);
            uint8_t *prow = pbuf + b * C::P_BYTES + r * C::P_ROW;
            const uint32_t swz = (r >> 2) & 1;
            uint32_t hi[NR / 4], mid[NR / 4], low[NR / 4];
#pragma unroll
            for (int k = 0; k < NR; k += 4) {
                float v[4];
                unpack_f2(e[k / 2], v[0], v[1]);
                unpack_f2(e[k / 2 + 1], v[2], v[3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = ex2(v[q]);
                l[k / 2] = fma_f2(pack_f2(v[0], v[1]), isv2, l[k / 2]);
                l[k / 2 + 1] = fma_f2(pack_f2(v[2], v[3]), isv2, l[k / 2 + 1]);
                split4(v, hi[k / 4], mid[k / 4], low[k / 4]);
            }
            uint8_t *ph = prow + (swz << 4), *pm = prow + ((1 ^ swz) << 4);
            if constexpr (NR == 16) {
                *reinterpret_cast<uint4 *>(ph) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(pm) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                *reinterpret_cast<uint4 *>(ph + C::P_TILE) = make_uint4(low[0], low[1], low[2], low[3]);
            } else if constexpr (NR == 8) {
                *reinterpret_cast<uint2 *>(ph) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(pm) = make_uint2(mid[0], mid[1]);
                *reinterpret_cast<uint2 *>(ph + 8) = make_uint2(low[0], low[1]);
            } else {
                *reinterpret_cast<uint32_t *>(ph) = hi[0];
                *reinterpret_cast<uint32_t *>(pm) = mid[0];
                *reinterpret_cast<uint32_t *>(ph + 8) = low[0];
            }
            proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[w][b]));
            first = false;
        }
        if (soft_any(w, !ok)) break;

        // epilogue: O, a dim a thread, and the row sums
        float o[NR];
        if (!first) {
            ok = wait_all(smem_u32(&bars->pv_done[w][(c - 1) & 1]), ((c - 1) >> 1) & 1, abort_flag);
            if (soft_any(w, !ok)) break;
            tc_fence_after();
            uint32_t s[2 * NR];
            ld_terms<NR>(tmem + 2 * C::COLS, s);
            wait_terms<NR>(s);
#pragma unroll
            for (int k = 0; k < NR; ++k) o[k] = fmaf(__uint_as_float(s[NR + k]), 0.0625f, __uint_as_float(s[k]));
            uint32_t z[NR];
            ld_cols<NR>(tmem + (C::INLINE3 ? 2 * C::COLS + 8 : 3 * C::COLS), z);
#pragma unroll
            for (int k = 0; k < NR; ++k) o[k] = fmaf(__uint_as_float(z[k]), 0x1p-8f, o[k]);
        } else {
#pragma unroll
            for (int k = 0; k < NR; ++k) o[k] = 0.f;
        }
        tc_fence_before();
#pragma unroll
            for (int k = 0; k < NR; k += 2) {
                float u, v;
                unpack_f2(l[k / 2], u, v);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    u += __shfl_xor_sync(0xffffffffu, u, d);
                    v += __shfl_xor_sync(0xffffffffu, v, d);
                }
                if (lane == 0) {
                    bars->red[warp][k] = u;
                    bars->red[warp][k + 1] = v;
                }
            }
        soft_sync(w);
        // this pipeline's rows: a thread each
        const int row = row0 + r;
        const bool mine = r < NR && row < it.rows;
        float sum = 0.f, m = -INFINITY;
        if (mine) {
            sum = (bars->red[4 * w][r] + bars->red[4 * w + 1][r]) + (bars->red[4 * w + 2][r] + bars->red[4 * w + 3][r]);
            const float nm = bars->nm[w][row];
            m = nm == kNone ? -INFINITY : -nm;
        }
        const bool two = C::SPLIT && it.t1 - it.t0 > 1;      // pipeline 1 has an O of the same rows
        if (C::SPLIT && w == 1) {
            if (mine) {
                bars->stat_m[row] = m;
                bars->stat_l[row] = sum;
            }
            if (two) {
#pragma unroll
                    for (int k = 0; k < NR; ++k) scratch[k * kD + r] = o[k];
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&bars->stat_full));
                mbar_arrive(smem_u32(&bars->q_empty[slot]));
            }
            // pipeline 0 reads this one's O: not overwritten before it has
            ok = wait_all(smem_u32(&bars->epi_done), i & 1, abort_flag);
            if (soft_any(w, !ok)) break;
            continue;
        }
        if (C::SPLIT) {
            ok = wait_all(smem_u32(&bars->stat_full), i & 1, abort_flag);
            if (soft_any(w, !ok)) break;
        }
        // slot 2 * cta: a unit that an earlier CTA began; 2 * cta + 1: one that begins here
        const bool whole = it.t1 - it.t0 == it.nt;
        const int part = 2 * blockIdx.x + (it.t0 == 0 ? 1 : 0);
        if (w == 0 && r == 0 && !whole) {
            parts |= it.t0 == 0 ? 2 : 1;
            p.meta[part] = PagedMeta{it.row0, it.h0, it.rows, it.t1 == it.nt};
        }
        if (mine) {
            float f0 = 1.f, f1 = 0.f;
            if (two) {
                const float m1 = bars->stat_m[row], mm = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : ex2(m - mm);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
                sum = sum * f0 + bars->stat_l[row] * f1;
                m = mm;
            }
            const bool empty = sum == 0.f;                    // the row saw no key
            const float lse = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
            const float inv = empty ? 0.f : (whole ? p.out_scale : 1.f) / sum;
            bars->top[w][row] = f0 * inv;
            if (C::SPLIT) bars->other[row] = f1 * inv;
            if (!whole) p.part_lse[(int64_t)part * C::R + row] = lse;
            else if (p.lse) p.lse[bars->at[slot][row]] = lse;
        }
        soft_sync(w);
#pragma unroll
            for (int k = 0; k < NR; ++k) {
                const int rr = row0 + k;
                if (rr >= it.rows) continue;
                const float f0 = bars->top[w][rr];
                float v = f0 == 0.f ? 0.f : o[k] * f0;
                if (two) v = fmaf(scratch[rr * kD + r], bars->other[rr], v);
                if (!whole) {
                    p.part_o[((int64_t)part * C::R + rr) * kD + r] = v;
                } else {
                    uint16_t *dst = static_cast<uint16_t *>(p.o) + (int64_t)bars->at[slot][rr] * kD + r;
                    *dst = (uint16_t)pack2<C::BF>(v, 0.f);
                }
            }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&bars->q_empty[slot]));
            if (C::SPLIT) mbar_arrive(smem_u32(&bars->epi_done));
        }
        soft_sync(w);                    // the scratch rows may be rewritten after this
    }
    if (threadIdx.x == 0)                // empty slots; one that is missing (a CTA that gave up) also ends its unit
        for (int s = 0; s < 2; ++s)
            if (!(parts >> s & 1)) p.meta[2 * blockIdx.x + s] = PagedMeta{0, 0, 0, 1};
}

template <bool BF, int NG, int NR>
__global__ void __launch_bounds__((PagedCfg<BF, NG, NR>::THREADS), 1)
    fmha_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = PagedCfg<BF, NG, NR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    PagedBars *bars = reinterpret_cast<PagedBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->q_full[s]), C::SW);        // the softmax warps, or the q warp for them
            mbar_init(smem_u32(&bars->q_empty[s]), 2 + C::SW);   // the MMA warps' commits and the softmax warps
            mbar_init(smem_u32(&bars->drain[s]), 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&bars->s_full[s][b]), 1);
                mbar_init(smem_u32(&bars->s_free[s][b]), 4);
                mbar_init(smem_u32(&bars->p_full[s][b]), 4);
                mbar_init(smem_u32(&bars->pv_done[s][b]), 1);
            }
        }
        mbar_init(smem_u32(&bars->stat_full), 4);
        mbar_init(smem_u32(&bars->epi_done), 4);
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 33 * C::NP);  // a producer's bytes, and its lanes' scales
            mbar_init(smem_u32(&bars->kv_empty[s]), C::SPLIT ? 1 : 2);   // the MMA warps that use a tile
        }
        for (int s = 0; s < kPagedItems; ++s) {
            mbar_init(smem_u32(&bars->item_full[s]), 1);
            mbar_init(smem_u32(&bars->item_empty[s]), C::SW + 3);   // the softmax, q and MMA warps
        }
        for (int k = 0; k < 16; ++k) bars->zero[k] = 0.f;
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if constexpr (C::QPASS) {            // the zeros beside q's third terms: 2 KB a group and slot
        for (int i = threadIdx.x; i < 2 * C::NG * 128; i += C::THREADS) {
            const int slot = i / (C::NG * 128), grp = i / 128 % C::NG;
            reinterpret_cast<uint4 *>(smem + slot * C::Q_BYTES + (32 * C::NG + 32 * grp) * 128)[i % 128] = make_uint4(0u, 0u, 0u, 0u);
        }
        proxy_fence();
    }
    if (warp == C::MMA) {                // pipeline 0's issuer
        tmem_alloc(smem_u32(&bars->tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    PagedCursor cur;
    int gate = 0;
    if (warp >= C::PROD && warp < C::MMA) {
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        gate = g_test_gate;              // read along with the lengths
        paged_schedule(p, cur, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // the merge kernel may be scheduled as CTAs of this grid exit; it waits
    // for this grid's completion before it reads the partials
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < C::SW) {
        paged_softmax<C, NR>(p, smem, bars, tmem, warp, lane);
    } else {
        if (warp == C::QW) paged_queries<C>(p, smem, bars, lane);
        else if (warp < C::MMA) paged_producer<C>(p, cur, gate, &tmK, &tmV, smem, bars, warp - C::PROD, lane);
        else paged_mma<C>(smem, bars, tmem, warp - C::MMA, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::MMA) {
        __syncwarp();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Chunks of prompts: units of up to 128 rows, and the roles not swapped.
//
// With more rows the kernel above is bound by what its softmax does across threads
// (a key each): the scores of 32 rows a thread, their references and votes took
// 3400 cycles a tile of 64 rows where the MMAs need 800.  Here S = Q K^T has the
// rows as M: a thread is a row (TMEM lane), its reference, sum and limit are in
// registers, nothing is exchanged, and a page's scale is one factor for its
// columns.  Two groups, each an MMA issuer and four softmax warps with K, V, S
// and O of their own, take every other tile, and their O are added up at the end.
//   S  = Q_0 K^T + Q_1 K^T + Q_2 K^T, the terms passes of their own into the same
//        accumulator, without factors; the third in e5m2, whose steps go on where e4m3's end, so that
//        as above elements of q below 2^-13 (f16 2^-10) of their row's largest are off by 2^-21 of it
//        (bf16 with two terms, f16 with three of e4m3: 2^-17; bf16's pass more takes 4%,
//        206 -> 215 us for 4 chunks of 512 on 8192 keys);
//   O += P V with both in f16, which holds every e4m3 number: a weight is off by 2^-11
//        of itself, or by 2^-25 where the group's largest is 2^7 or more (a reference
//        serves 16 tiles, so that this is 2^-21 of their weight at most).
// 128 rows share a tile's V, so that four warps that convert it cost less than
// splitting every weight into e4m3 terms did (12 instructions for four weights
// instead of two), and less shared memory traffic, which two terms of P read.
//
// A tile's scores, and its weights, are halves of 64 keys, each a link of a chain:
// S of a half, softmax, P over that S in TMEM, P V, and S of the half two tiles on,
// while the softmax is at the other half.
//
// What bounds it is that chain: of 4 chunks of 512 tokens on 8192 keys (220 us, 847
// TFLOP/s; flops 97 at the bf16 rate) a half takes a group 2700 cycles, of
// which its softmax computes 1600 and waits 900 for S; the tensor pipe is busy 50%,
// the ALU 40%, issue slots 51%.  Without one of S's passes it takes 4% less, without the
// wait for P V 2%.  With two passes and no such wait (206): without P V 3% less, without
// the conversion 7%; weights as e4m3 terms in shared memory took 229 (f16: three,
// 291), f16 ones there 232; S and P V a whole tile at a time 232; V converted a tile ahead
// 213; 16 softmax warps, two threads a row, 231; units of 256 rows, a block a
// group, 3% more.
// ---------------------------------------------------------------------------

constexpr int kRowsBars = 4096;          // barrier block
constexpr int kRowsTerms = 3;            // of q
constexpr int kRowsVs = 2;               // tiles of V as codes, for both groups
constexpr int kRowsTiles = 16;           // tiles that a reference serves at most
constexpr float kRowsGrown = 15.f;       // as kGrown: f16 ends at 2^16
constexpr float kRowsBias = 7.f;         // as kBias
constexpr int kRowsConv = 8, kRowsK = 12, kRowsMma = 13, kRowsV = 15;   // first warps of the roles behind the softmax's
constexpr int kRowsThreads = 512;        // two softmax groups and the converters, of four warps; K's and V's producers, an MMA issuer a group

template <bool BF_>
struct RowsCfg {
    static constexpr bool BF = BF_;
    static constexpr int OFF_VF = kRowsTerms * kPanelBytes;   // after q's terms, by group: V in f16,
    static constexpr int OFF_K = OFF_VF + 4 * kPanelBytes;    // and K (one tile, free once its S is there)
    static constexpr int OFF_V = OFF_K + 2 * kPanelBytes;     // V as it comes, for both
    static constexpr int OFF_BARS = OFF_V + kRowsVs * kPanelBytes;
    static constexpr int SMEM_BYTES = OFF_BARS + kRowsBars + 1024;   // 1 KB alignment
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct RowsBars {
    uint64_t q_full[2], q_empty, drain[2];                    // by group,
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // and half of a tile
    uint64_t stat_full, epi_done;
    uint64_t k_full[2], k_empty[2], v_full[kRowsVs], v_empty[kRowsVs], vf_full[2], scale_full[2][2];
    uint64_t item_full[kPagedItems], item_empty[kPagedItems];
    PagedItem item[kPagedItems];
    uint32_t tmem_base;
    int abort;
    float scale[2][2][2][8];             // by group and tile mod 2: k_scale, v_scale of its pages
    float2 stat[kRows];                  // reference and sum of group 1's rows
    float qscale[kRows];                 // of the rows of q
};
static_assert(sizeof(RowsBars) <= kRowsBars, "barrier block");

__device__ __forceinline__ bool rows_take(RowsBars *bars, uint32_t i, PagedItem &it, volatile int *abort_flag, int lane) {
    const uint32_t st = i % kPagedItems;
    if (!wait_all(smem_u32(&bars->item_full[st]), (i / kPagedItems) & 1, abort_flag)) return false;
    it = bars->item[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[st]));
    return it.rows > 0;
}

// A producer warp: the groups' tiles of K, with the pages' scales, or (V) of V.  One
// warp for both held a group's K back behind the other's V (230 us for 4 chunks of
// 512, f16 400, with one slot of either).
template <class C, bool V>
__device__ void rows_producer(const PagedParams &p, PagedCursor &cur, int gate, const CUtensorMap *tm, uint8_t *smem, RowsBars *bars,
                              int lane) {
    volatile int *abort_flag = &bars->abort;
    bool ok = true;
    if (gate) ok = __all_sync(0xffffffffu, lane > 0 || test_gate_open(abort_flag));
    uint32_t fill[2] = {0, 0}, qn = 0;
    const int P = 1 << p.shift, per = kRows >> p.shift;
    auto publish = [&](uint32_t i, const PagedItem &it) -> bool {
        const uint32_t st = i % kPagedItems;
        if (i >= kPagedItems && !wait_all(smem_u32(&bars->item_empty[st]), (i / kPagedItems - 1) & 1, abort_flag)) return false;
        if (lane == 0) {
            bars->item[st] = it;
            mbar_arrive(smem_u32(&bars->item_full[st]));
        }
        __syncwarp();
        return true;
    };
    PagedItem it, next;
    if (ok) {
        if constexpr (V) ok = rows_take(bars, 0, it, abort_flag, lane);
        else {
            paged_next(p, cur, it);
            ok = publish(0, it);
        }
    }
    while (ok && it.rows > 0) {
        ++qn;
        const int pages = (it.L + P - 1) >> p.shift;
        auto id_of = [&](int t) {
            const int i = t * per + lane;
            return lane < per && i < pages && t < it.t1 ? page_id(p, it.entry, i, !V) : -1;
        };
        int id = id_of(it.t0);
        for (int t = it.t0; t < it.t1; ++t) {
            const int ahead = id_of(t + 1), here = imax(0, imin(per, pages - t * per));
            // a page outside the cache: a coordinate outside it, which reads zeros
            const int head = id >= 0 ? id * p.H_k + it.g : p.n_pages * p.H_k;
            const int x = (t - it.t0) & 1;
            // V's tiles share a ring; K's have a slot a group
            const uint32_t n = V || x == 0 ? fill[0] : fill[1], st = V ? n % kRowsVs : 0, lap = V ? n / kRowsVs : n;
            const uint32_t full = smem_u32(V ? &bars->v_full[st] : &bars->k_full[x]);
            if (lap > 0 && !wait_all(smem_u32(V ? &bars->v_empty[st] : &bars->k_empty[x]), lap & 1 ^ 1, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_expect_tx(full, here * (P << 7));
            __syncwarp();
            if (lane < here) {
                tma_load_3d(smem_u32(smem + (V ? C::OFF_V + st * kPanelBytes : C::OFF_K + x * kPanelBytes)) + lane * (P << 7), tm, full, 0, 0, head);
                if constexpr (!V) {
                    // into the place of the tile two before in this group, which was read
                    // before S of the one before, and so before this slot was free
                    const float *ks = id >= 0 ? p.k_scale + head : &g_one, *vs = id >= 0 ? p.v_scale + head : &g_one;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&bars->scale[x][n & 1][0][lane])), "l"(ks)
                                 : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&bars->scale[x][n & 1][1][lane])), "l"(vs)
                                 : "memory");
                }
            }
            if constexpr (!V)
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars->scale_full[x][n & 1])) : "memory");
            if (V || x == 0) ++fill[0];
            else ++fill[1];
            id = ahead;
            if constexpr (!V)
                if (t == it.t0) {
                    paged_next(p, cur, next);
                    if (!publish(qn, next)) {
                        ok = false;
                        break;
                    }
                }
        }
        if constexpr (V) ok = ok && rows_take(bars, qn, it, abort_flag, lane);
        else it = next;
    }
    // no copy may be in flight when the block ends, nor a product that reads one
    ok = *abort_flag == 0;
    constexpr uint32_t kSlots = V ? kRowsVs : 1;
#pragma unroll
    for (int x = 0; x < (V ? 1 : 2); ++x)
        for (uint32_t n = fill[x] > kSlots ? fill[x] - kSlots : 0; n < fill[x]; ++n) {
            const uint32_t st = n % kSlots, lap = n / kSlots;
            if (ok) ok = wait_all(smem_u32(V ? &bars->v_empty[st] : &bars->k_empty[x]), lap & 1, abort_flag);
            if (!ok) mbar_wait_drain(smem_u32(V ? &bars->v_full[st] : &bars->k_full[x]), lap & 1);
            if (!V) mbar_wait_drain(smem_u32(&bars->scale_full[x][n & 1]), n >> 1 & 1);
        }
    if (!V && ok && qn > 0) wait_all(smem_u32(&bars->q_empty), (qn - 1) & 1, abort_flag);
}

// Converter warp w: V's codes to f16, a quarter of each tile, from rows of 128
// bytes to two panels of 64 dims; in a sequence's last tile the rows past the keys
// are zeros, so that P = 0 contributes 0.
template <class C>
__device__ void rows_convert(uint8_t *smem, RowsBars *bars, int w, int lane) {
    volatile int *abort_flag = &bars->abort;
    uint32_t n = 0, done[2] = {0, 0};    // tiles, and those of either group
    PagedItem it;
    for (uint32_t i = 0; rows_take(bars, i, it, abort_flag, lane); ++i) {
        bool ok = true;
        for (int t = it.t0; t < it.t1; ++t, ++n) {
            const int x = (t - it.t0) & 1, nk = it.L - t * kRows;
            const uint32_t st = n % kRowsVs, c = x ? done[1]++ : done[0]++;
            // the codes, and room: P V of the group's tile before is done
            ok = wait_all(smem_u32(&bars->v_full[st]), (n / kRowsVs) & 1, abort_flag) &&
                 (c == 0 || wait_all(smem_u32(&bars->pv_done[x][1]), (c - 1) & 1, abort_flag));
            if (!ok) break;
            const int ch = lane & 7, up = ch >> 2;       // 16 dims of a row; of which panel
            const uint8_t *src = smem + C::OFF_V + st * kPanelBytes;
            uint8_t *dst = smem + C::OFF_VF + (2 * x + up) * kPanelBytes;
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = 32 * w + 4 * k + (lane >> 3);
                v[k] = *reinterpret_cast<const uint4 *>(src + j * 128 + ((ch ^ (j & 7)) << 4));
                if (j >= nk) v[k] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = 32 * w + 4 * k + (lane >> 3), f = 2 * (ch & 3);
                // eight dims at a time; the panels' lanes begin with different ones, so that their banks differ
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const bool high = (o ^ up) != 0;
                    const uint32_t a = high ? v[k].z : v[k].x, b = high ? v[k].w : v[k].y;
                    uint4 y;
                    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
                        : "=r"(y.x), "=r"(y.y) : "r"(a));
                    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
                        : "=r"(y.z), "=r"(y.w) : "r"(b));
                    *reinterpret_cast<uint4 *>(dst + j * 128 + (((f + high) ^ (j & 7)) << 4)) = y;
                }
            }
            proxy_fence();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&bars->v_empty[st]));
                mbar_arrive(smem_u32(&bars->vf_full[x]));
            }
        }
        if (!ok) break;
    }
}

// MMA issuer of group x.  The code of both is the same: a copy for each, with constant
// operands, took 299 us for 4 chunks of 512.
template <class C>
__device__ void rows_mma(uint8_t *smem, RowsBars *bars, uint32_t tmem_any, int x, int lane) {
    volatile int *abort_flag = &bars->abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    const uint32_t s_tm = tmem + x * kRows, o_tm = tmem + 2 * kRows + x * kD;
    constexpr uint32_t kIdS = mma_idesc(0u, kRows / 2, false), kIdP = mma_idesc(0u, kD, true);
    constexpr uint32_t kIdLast = kIdS | (1u << 7);           // A in e5m2
    const uint64_t q = smem_desc(smem_u32(smem), 16, 1024);
    const uint64_t k = smem_desc(smem_u32(smem + C::OFF_K + x * kPanelBytes), 16, 1024);
    const uint64_t v = smem_desc(smem_u32(smem + C::OFF_VF + 2 * x * kPanelBytes), kPanelBytes, 1024);   // MN-major: LBO = panel stride
    uint32_t m = 0;                      // tiles of this group
    bool ok = true;
    PagedItem it;
    for (uint32_t i = 0; ok && rows_take(bars, i, it, abort_flag, lane); ++i) {
        if (!wait_all(smem_u32(&bars->q_full[x]), i & 1, abort_flag)) {
            ok = false;
            break;
        }
        const int tb = it.t0 + x;
        if (tb >= it.t1) tc_commit(smem_u32(&bars->q_empty));   // an item of one tile is group 0's alone
        // S of half h of tile m, over P of that of tile m - 1, so once that P V is done: MMAs into one
        // accumulator keep their order, of others nothing is promised (without the wait 215 us for 4
        // chunks of 512, with it 220); P V of tile m - 1
        auto scores = [&](int h) -> bool {
            if ((h == 0 && !wait_all(smem_u32(&bars->k_full[x]), m & 1, abort_flag)) ||
                (m > 0 && !wait_all(smem_u32(&bars->pv_done[x][h]), (m - 1) & 1, abort_flag)))
                return false;
            tc_fence_after();
#pragma unroll
            for (int term = 0; term < kRowsTerms; ++term)    // 32 dims a step: 32 bytes of a row
                mma4<32, 32>(s_tm + 64 * h, q + ((term * kPanelBytes) >> 4), k + ((h * 64 * 128) >> 4),
                             term + 1 < kRowsTerms ? kIdS : kIdLast, term > 0 ? 1u : 0u);
            tc_commit(smem_u32(&bars->s_full[x][h]));
            return true;
        };
        auto values = [&](int h, bool first) -> bool {
            if ((h == 0 && !wait_all(smem_u32(&bars->vf_full[x]), (m - 1) & 1, abort_flag)) ||
                !wait_all(smem_u32(&bars->p_full[x][h]), (m - 1) & 1, abort_flag))
                return false;
            tc_fence_after();
            // 16 keys a step: 8 columns of P's, 16 rows of V
            mma4_ts<16 * 128>(o_tm, s_tm + 64 * h, v + ((h * 64 * 128) >> 4), kIdP, first ? 0u : 1u);
            tc_commit(smem_u32(&bars->pv_done[x][h]));
            return true;
        };
        for (int t = tb; ok && t < it.t1 + 2 && tb < it.t1; t += 2) {
            const bool more = t < it.t1, before = t > tb;    // a tile here; one before it
            for (int h = 0; ok && h < 2; ++h) {
                ok = !before || values(h, h == 0 && t == tb + 2);
                ok = ok && (!more || scores(h));
            }
            if (!ok) break;
            if (more) {
                tc_commit(smem_u32(&bars->k_empty[x]));
                if (t + 2 >= it.t1) tc_commit(smem_u32(&bars->q_empty));
                ++m;
            }
        }
    }
    // no tensor-core operation may be in flight when TMEM is released
    tc_commit(smem_u32(&bars->drain[x]));
    mbar_wait_drain(smem_u32(&bars->drain[x]), 0);
}

// 16 rows of the unit's q by a warp, from r0 on, as terms in its tiles; at: of lane
// k's row r0 + k, q row * H + head (-1: none).  All loads go out first (eight at a
// time, with a division a row, took 9 us for 32).  Returns the scale of lane k's row.
template <class C>
__device__ __forceinline__ float rows_terms(const PagedParams &p, uint8_t *tile, int at, int r0, int lane) {
    uint2 v[16];
    float g = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int a = __shfl_sync(0xffffffffu, at, k);
        v[k] = a >= 0 ? *reinterpret_cast<const uint2 *>(p.q + ((int64_t)a * kD + lane * 4) * 2) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float y[4], gk;
        row_scaled<C::BF>(v[k], y, gk);
        if (lane == k) g = gk;
        uint32_t rest[2] = {pack2<false>(y[0], y[1]), pack2<false>(y[2], y[3])};
        const int row = r0 + k;
#pragma unroll
        for (int term = 0; term < kRowsTerms; ++term)
            *reinterpret_cast<uint32_t *>(tile + term * kPanelBytes + row * 128 +
                                          ((((lane >> 2) ^ (row & 7)) << 4) | ((lane & 3) << 2))) =
                term + 1 < kRowsTerms ? take_term(rest) : last_term(rest);
    }
    return g;
}

// Softmax and epilogue of group x, a row a thread.
template <class C>
__device__ void rows_softmax(const PagedParams &p, uint8_t *smem, RowsBars *bars, uint32_t tmem, int warp, int lane) {
    volatile int *abort_flag = &bars->abort;
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;   // group, row of the unit
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_tm = lane_base + x * kRows, o_tm = lane_base + 2 * kRows + x * kD;
    uint32_t c = 0;                                     // tiles of this group
    int parts = 0;                                      // bit s: slot s of this CTA holds a partial
    for (uint32_t i = 0;; ++i) {
        // read where it lies, and given back at its end: registers are scarce
        const PagedItem &it = bars->item[i % kPagedItems];
        if (!wait_all(smem_u32(&bars->item_full[i % kPagedItems]), (i / kPagedItems) & 1, abort_flag) || it.rows == 0) break;
        const bool row_ok = r < it.rows;
        // the unit's rows of q, 16 a warp, for both groups; the S MMAs of the item before are done
        if (i > 0 && !wait_all(smem_u32(&bars->q_empty), (i - 1) & 1, abort_flag)) break;
        const int k = warp * 16 + (lane & 15), tk = k / p.G;
        const float gk = rows_terms<C>(p, smem, k < it.rows ? (it.row0 + tk) * p.H + it.h0 + k - tk * p.G : -1, warp * 16, lane);
        if (lane < 16) bars->qscale[k] = gk;
        proxy_fence();
        __syncwarp();
        if (lane < 2) mbar_arrive(smem_u32(&bars->q_full[lane]));
        if (!wait_all(smem_u32(&bars->q_full[x]), i & 1, abort_flag)) break;
        const bool work = __any_sync(0xffffffffu, row_ok);   // else the warp only keeps step
        const int lim = it.base + it.tok0 + r / p.G;    // last key it sees
        const int t1 = it.t1, L = it.L;
        const float fq = p.c * bars->qscale[r];
        float m = -INFINITY, M = -INFINITY;             // reference (log2 units) of P and O, and the highest so far
        float l = 0.f;                                  // row sum
        int since = kRowsTiles;
        bool ok = true;
        const int tb = it.t0 + x;
        // a warp without rows keeps step with those that have some
        for (int t = tb; !work && ok && t < t1; t += 2, ++c)
            for (int h = 0; ok && h < 2; ++h) {
                ok = wait_all(smem_u32(&bars->s_full[x][h]), c & 1, abort_flag) &&
                     (c == 0 || wait_all(smem_u32(&bars->pv_done[x][h]), (c - 1) & 1, abort_flag));
                if (ok && lane == 0) mbar_arrive(smem_u32(&bars->p_full[x][h]));
            }
        for (int t = tb; work && t < t1; t += 2, ++c) {
            const int cnt = imin(L, lim + 1) - t * kRows;   // visible keys
            if (!wait_all(smem_u32(&bars->scale_full[x][c & 1]), c >> 1 & 1, abort_flag)) {
                ok = false;
                break;
            }
            // k_scale and log2 of v_scale of 16 columns, a page or a part of one: in lane u those of columns 16 u ...
            const float lane_ks = bars->scale[x][c & 1][0][(16 * (lane & 7)) >> p.shift];
            const float lane_vs = __log2f(fminf(fmaxf(bars->scale[x][c & 1][1][(16 * (lane & 7)) >> p.shift], kLeastScale), kMostScale));
            auto factor = [&](int u) { return fmaxf(fq * __shfl_sync(0xffffffffu, lane_ks, u), FLT_MIN); };   // not 0: -inf stays -inf
            auto summand = [&](int u) { return __shfl_sync(0xffffffffu, lane_vs, u); };
            if (since == kRowsTiles) since = 0;
            ++since;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                // P V of the half's tile before, done before S, is waited for as well, so that
                // no phase of its barrier goes unseen
                if (!wait_all(smem_u32(&bars->s_full[x][h]), c & 1, abort_flag) ||
                    (c > 0 && !wait_all(smem_u32(&bars->pv_done[x][h]), (c - 1) & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                uint32_t s[2][32];
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) tmem_ld32(s_tm + 64 * h + 32 * q, s[q]);
#pragma unroll
                for (int q = 0; q < 2; ++q) tmem_wait_ld(s[q]);
                if (__any_sync(0xffffffffu, cnt < 64 * h + 64)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * q + k >= cnt - 64 * h) s[q][k] = 0xff800000u;
                }
                float tmax = -INFINITY;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t *su = s[u >> 1] + 16 * (u & 1);
                    float a = -INFINITY, b = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        a = max3(a, __uint_as_float(su[k]), __uint_as_float(su[k + 1]));
                        b = max3(b, __uint_as_float(su[k + 2]), __uint_as_float(su[k + 3]));
                    }
                    tmax = fmaxf(tmax, fmaf(fmaxf(a, b), factor(4 * h + u), summand(4 * h + u)));
                }
                const bool need = tmax > m + kRowsGrown || (since == 1 && h == 0);
                if (__any_sync(0xffffffffu, need)) {
                    float alpha = 1.f;
                    if (need) {
                        const float own = tmax - kRowsBias, ref = fmaxf(fmaxf(own, fminf(M, own + kAbove)), M - kBelow);
                        alpha = m == -INFINITY ? 0.f : ex2(m - ref);
                        m = ref;
                        M = fmaxf(M, ref);
                        l *= alpha;
                    }
                    if (t > tb || h > 0) {   // O: once the P V of the half before is done
                        if (!wait_all(smem_u32(&bars->pv_done[x][h ^ 1]), (h ? c : c - 1) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
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
                // a row that has seen no key yet: every score is -inf, P = 0
                const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float fu = factor(4 * h + u), du = summand(4 * h + u);
                    const uint64_t f2 = pack_f2(fu, fu), d2 = pack_f2(du - mr, du - mr);
                    const uint32_t *su = s[u >> 1] + 16 * (u & 1);
                    uint64_t sum[2] = {0, 0};
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float a, b;
                        unpack_f2(fma_f2(pack_f2(__uint_as_float(su[2 * k]), __uint_as_float(su[2 * k + 1])), f2, d2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[k & 1] = add_f2(sum[k & 1], pack_f2(a, b));
                        w[k] = pack2<false>(a, b);
                    }
                    float a, b;
                    unpack_f2(add_f2(sum[0], sum[1]), a, b);
                    l = fmaf(a + b, ex2(-du), l);
                    tmem_st8(s_tm + 64 * h + 8 * u, w);      // over the scores: 16 keys, eight columns
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[x][h]));
            }
            if (!ok) break;
        }
        if (!ok) break;

        // epilogue: O of a unit that this CTA covers alone, else a partial
        if (tb < t1 && !wait_all(smem_u32(&bars->pv_done[x][1]), (c - 1) & 1, abort_flag)) break;
        const int t0 = it.t0;
        const bool two = t1 - t0 > 1;                   // group 1 has an O of the same rows
        if (x == 1) {
            bars->stat[r] = make_float2(m, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&bars->stat_full));
                mbar_arrive(smem_u32(&bars->item_empty[i % kPagedItems]));
            }
            // group 0 reads this group's O: not overwritten before it has
            if (!wait_all(smem_u32(&bars->epi_done), i & 1, abort_flag)) break;
            continue;
        }
        if (!wait_all(smem_u32(&bars->stat_full), i & 1, abort_flag)) break;
        const float2 other = bars->stat[r];
        const float mm = fmaxf(m, other.x);
        const float f0 = m == -INFINITY && l == 0.f ? 0.f : ex2(m - mm);              // factors of the groups' O; NaN stays NaN
        const float f1 = other.x == -INFINITY && other.y == 0.f ? 0.f : ex2(other.x - mm);
        l = l * f0 + other.y * f1;
        m = mm;
        const bool whole = t1 - t0 == it.nt;
        const int part = 2 * blockIdx.x + (t0 == 0 ? 1 : 0), tok = r / p.G;
        const int at = (it.row0 + tok) * p.H + it.h0 + r - tok * p.G;
        if (threadIdx.x == 0 && !whole) {
            parts |= t0 == 0 ? 2 : 1;
            p.meta[part] = PagedMeta{it.row0, it.h0, it.rows, t1 == it.nt};
        }
        if (work) {
            tc_fence_after();
            const bool empty = l == 0.f;                // the row saw no key
            const float inv = (whole ? p.out_scale : 1.f) / l;
            const float lse = empty ? -INFINITY : (m + log2f(l)) * kLn2;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                tmem_ld32(o_tm + 32 * q, o);
                tmem_wait_ld(o);
                uint32_t o1[32];
                if (two) {
                    tmem_ld32(o_tm + kD + 32 * q, o1);
                    tmem_wait_ld(o1);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float both = __uint_as_float(o[k]) * f0 + (two ? __uint_as_float(o1[k]) * f1 : 0.f);
                    o[k] = empty ? 0u : __float_as_uint(both * inv);
                }
                if (row_ok && !whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + ((int64_t)part * kRows + r) * kD + 32 * q);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else if (row_ok) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + (int64_t)at * kD + 32 * q);
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = pack2<C::BF>(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                }
            }
            if (row_ok) {
                if (!whole) p.part_lse[(int64_t)part * kRows + r] = lse;
                else if (p.lse) p.lse[at] = lse;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&bars->epi_done));
            mbar_arrive(smem_u32(&bars->item_empty[i % kPagedItems]));
        }
    }
    if (threadIdx.x == 0)               // empty slots; one that is missing (a CTA that gave up) also ends its unit
        for (int s = 0; s < 2; ++s)
            if (!(parts >> s & 1)) p.meta[2 * blockIdx.x + s] = PagedMeta{0, 0, 0, 1};
}

template <bool BF>
__global__ void __launch_bounds__(kRowsThreads, 1)
    fmha_paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using C = RowsCfg<BF>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    RowsBars *bars = reinterpret_cast<RowsBars *>(smem + C::OFF_BARS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bars->q_full[x]), 8);          // the warps that write its rows
            for (int h = 0; h < 2; ++h) {
                mbar_init(smem_u32(&bars->s_full[x][h]), 1);
                mbar_init(smem_u32(&bars->p_full[x][h]), 4);
                mbar_init(smem_u32(&bars->pv_done[x][h]), 1);
            }
            mbar_init(smem_u32(&bars->scale_full[x][0]), 32);  // the producer's lanes
            mbar_init(smem_u32(&bars->scale_full[x][1]), 32);
            mbar_init(smem_u32(&bars->drain[x]), 1);
            mbar_init(smem_u32(&bars->k_full[x]), 1);
            mbar_init(smem_u32(&bars->k_empty[x]), 1);
            mbar_init(smem_u32(&bars->vf_full[x]), 4);         // the converters
        }
        for (int s = 0; s < kRowsVs; ++s) {
            mbar_init(smem_u32(&bars->v_full[s]), 1);
            mbar_init(smem_u32(&bars->v_empty[s]), 4);
        }
        for (int s = 0; s < kPagedItems; ++s) {
            mbar_init(smem_u32(&bars->item_full[s]), 1);
            mbar_init(smem_u32(&bars->item_empty[s]), 15);       // all warps but K's
        }
        mbar_init(smem_u32(&bars->q_empty), 2);
        mbar_init(smem_u32(&bars->stat_full), 4);
        mbar_init(smem_u32(&bars->epi_done), 4);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kRowsMma) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    PagedCursor cur;
    int gate = 0;
    if (warp == kRowsK) {
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        gate = g_test_gate;
        paged_schedule(p, cur, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < kRowsConv) rows_softmax<C>(p, smem, bars, tmem, warp, lane);
    else if (warp < kRowsK) rows_convert<C>(smem, bars, warp - kRowsConv, lane);
    else if (warp == kRowsK) rows_producer<C, false>(p, cur, gate, &tmK, smem, bars, lane);
    else if (warp == kRowsV) rows_producer<C, true>(p, cur, 0, &tmV, smem, bars, lane);
    else rows_mma<C>(smem, bars, tmem, warp - kRowsMma, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kRowsMma) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the units that several CTAs covered:
//   O = out_scale * sum_c w_c O_c / sum_c w_c with w_c = exp(LSE_c - max LSE).
// CTA (c, y) takes rows, a warp each, of the unit that CTA c of the kernel above
// began and did not end; the metadata says how far it goes on.  Nearly every cut
// unit has two partials: their rows are fetched in the same round trip as the
// metadata and joined by straight code; more take the loop.
constexpr int kPagedMergeWarps = 4;

template <bool BF>
__device__ __forceinline__ void paged_store_row(const PagedParams &p, const PagedMeta &m, int r, float4 acc, float sum, float mx,
                                                int lane) {
    const float inv = sum == 0.f ? 0.f : p.out_scale / sum;
    const int t = r / p.G;
    const int64_t at = (int64_t)(m.row0 + t) * p.H + m.h0 + r - t * p.G;
    reinterpret_cast<uint2 *>(p.o)[at * (kD / 4) + lane] =
        make_uint2(pack2<BF>(acc.x * inv, acc.y * inv), pack2<BF>(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

template <bool BF>
__global__ void __launch_bounds__(32 * kPagedMergeWarps) fmha_paged_merge_kernel(const PagedParams p, int R) {
    const int lane = threadIdx.x & 31, c0 = blockIdx.x;
    const int r = blockIdx.y * kPagedMergeWarps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 + 1 >= p.ncta || r >= R) return;
    auto slot = [&](int c) { return ((int64_t)2 * (c0 + c) + (c == 0 ? 1 : 0)) * R + r; };
    const float4 *o_c = reinterpret_cast<const float4 *>(p.part_o) + lane;
    const PagedMeta m = p.meta[2 * c0 + 1];
    const bool two = p.meta[2 * (c0 + 1)].last;
    const float la = p.part_lse[slot(0)], lb = p.part_lse[slot(1)];
    const float4 a = o_c[slot(0) * (kD / 4)], b = o_c[slot(1) * (kD / 4)];
    if (r >= m.rows) return;                                 // also: CTA c0 began no unit that it did not end
    if (two) {
        float mx = fmaxf(la, lb);
        if (mx == -INFINITY || la != la || lb != lb) mx = 0.f;   // no key: weights 0; NaN in, NaN out
        const float wa = __expf(la - mx), wb = __expf(lb - mx);
        const float4 o = make_float4(wa * a.x + wb * b.x, wa * a.y + wb * b.y, wa * a.z + wb * b.z, wa * a.w + wb * b.w);
        paged_store_row<BF>(p, m, r, o, wa + wb, mx, lane);
        return;
    }
    // the partials of CTAs c0 .. c0 + n - 1
    int n = 2;
    for (;;) {
        const int c = c0 + n + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, c >= p.ncta || p.meta[2 * c].last);
        n += hit ? __ffs(hit) : 32;
        if (hit) break;
    }
    n = imin(n, p.ncta - c0);
    float mx = -INFINITY;
    bool nan = false;
    for (int c = lane; c < n; c += 32) {
        const float v = p.part_lse[slot(c)];
        nan |= v != v;
        mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY || __any_sync(0xffffffffu, nan)) mx = 0.f;   // no key: weights 0; NaN in, NaN out
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int cb = 0; cb < n; cb += 8) {
        float4 v[8];                                         // eight partials in flight
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t s = slot(imin(cb + k, n - 1));
            v[k] = reinterpret_cast<const float4 *>(p.part_o)[s * (kD / 4) + lane];
            w[k] = p.part_lse[s];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = cb + k < n ? __expf(w[k] - mx) : 0.f;
            sum += x;
            acc.x += x * v[k].x;
            acc.y += x * v[k].y;
            acc.z += x * v[k].z;
            acc.w += x * v[k].w;
        }
    }
    paged_store_row<BF>(p, m, r, acc, sum, mx, lane);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Query rows of a unit: 16 or 32 where a sequence's rows of a kv head fit them,
// else 128.  (16 sequences of 28 rows on 1500 to 6000 keys: 46 us in units of 32, 55 of
// 128; 4 sequences of 8192 keys and 64 / 80 / 128 rows: 35 / 48 / 56 in units of 64,
// two groups a pipeline, 35 / 36 / 40 of 128.)
int paged_rows(int64_t max_q, int G) { return max_q * G <= 16 ? 16 : max_q * G <= 32 ? 32 : kRows; }

using PagedKernel = void (*)(CUtensorMap, CUtensorMap, PagedParams);
struct PagedLaunch {
    PagedKernel kernel;
    int smem, threads;
};
template <bool BF, int NG, int NR>
PagedLaunch paged_launch() {
    return {fmha_paged_kernel<BF, NG, NR>, PagedCfg<BF, NG, NR>::SMEM_BYTES, PagedCfg<BF, NG, NR>::THREADS};
}
template <bool BF>
PagedLaunch paged_kernel(int rows, int per_unit) {
    if (rows == kRows) return {fmha_paged_rows_kernel<BF>, RowsCfg<BF>::SMEM_BYTES, kRowsThreads};
    if (rows == 32) return paged_launch<BF, 2, 16>();
    return per_unit <= 4 ? paged_launch<BF, 1, 4>() : per_unit <= 8 ? paged_launch<BF, 1, 8>() : paged_launch<BF, 1, 16>();
}

}  // namespace

int paged_set_wait_limit(unsigned long long ns) { return cache_set_wait_limit(ns); }
int paged_set_test_gate(int on) { return cache_set_test_gate(on); }
int *paged_status_word() { return symbol_address(g_status); }

}  // namespace fmha

using namespace fmha;

extern "C" size_t fmha_page_workspace_size(int max_q, int H, int H_k) {
    if (max_q <= 0 || H <= 0 || H_k <= 0 || H % H_k != 0 || H / H_k > kRows) return 0;
    // two partials a CTA: an fp32 row of O and its LSE for every row of a unit, and whose they are
    return (size_t)2 * kPagedMaxCtas * (paged_rows(max_q, H / H_k) * (kD + 1) * sizeof(float) + sizeof(PagedMeta));
}

extern "C" int fmha_page_fwd(fmha_tensor q, const void *k_pages, const void *v_pages, const float *k_scale,
                             const float *v_scale, fmha_tensor o, float *lse, int B, int N, int max_q, int H, int H_k,
                             int D, int n_pages, int page_size, int B_table, int max_pages, const int *table,
                             const int *seqlen, const int *batch_idx, const int *cu_q, float scale, float out_scale,
                             int mask, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    int shift = 4;
    while (shift < 7 && page_size != 1 << shift) ++shift;
    if (B < 0 || N < 0 || H <= 0 || H_k <= 0 || H % H_k != 0 || H / H_k > kRows || D != kD || page_size != 1 << shift)
        return FMHA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY) || !(out_scale == out_scale) || out_scale == INFINITY || out_scale == -INFINITY)
        return FMHA_ERR_INVALID_ARG;
    if (mask != FMHA_MASK_NONE && mask != FMHA_MASK_CAUSAL) return FMHA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return FMHA_OK;
    if (max_q <= 0 || n_pages <= 0 || B_table <= 0 || max_pages <= 0 || max_pages > kMaxCacheRows >> shift ||
        (int64_t)n_pages * H_k > 0x7ffffffe || n_pages > 0x7fffffff >> shift || (int64_t)N * H > 0x7fffffff ||
        (!cu_q && N != B))
        return FMHA_ERR_INVALID_ARG;
    if (!q.data || !k_pages || !v_pages || !o.data || !k_scale || !v_scale || !table || !seqlen)
        return FMHA_ERR_INVALID_ARG;
    const int dt = q.dtype;
    if ((dt != FMHA_F16 && dt != FMHA_BF16) || o.dtype != dt)
        return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {(const void *)q.data, k_pages, v_pages, (const void *)o.data})
        if (misaligned(ptr, 16)) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {(const void *)k_scale, (const void *)v_scale, (const void *)lse, (const void *)table,
                            (const void *)seqlen, (const void *)batch_idx, (const void *)cu_q})
        if (misaligned(ptr, 4)) return FMHA_ERR_INVALID_ARG;
    const size_t need = fmha_page_workspace_size(max_q, H, H_k);
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < need) return FMHA_ERR_INVALID_ARG;
    // a unit's inputs are read by several CTAs, at their own times
    const size_t rows_bytes = (size_t)N * H * kD * 2, pages = ((size_t)n_pages * H_k << shift) * kD;
    const size_t scales = (size_t)n_pages * H_k * sizeof(float), seqs = (size_t)B * sizeof(int);
    const Bytes out[3] = {{o.data, rows_bytes}, {lse, (size_t)N * H * sizeof(float)}, {workspace, need}};
    const Bytes in[9] = {{q.data, rows_bytes}, {k_pages, pages}, {v_pages, pages}, {k_scale, scales},
                         {v_scale, scales}, {table, (size_t)B_table * max_pages * sizeof(int)}, {seqlen, seqs},
                         {batch_idx, seqs}, {cu_q, seqs + sizeof(int)}};
    if (outputs_clash(out, in)) return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    const int sms = sm_count();
    if (sms <= 0) return FMHA_ERR_CUDA;

    const int G = H / H_k, R = paged_rows(max_q, G);
    PagedParams p{};
    p.q = static_cast<const uint8_t *>(q.data);
    p.o = o.data;
    p.lse = lse;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.seqlen = seqlen;
    p.batch_idx = batch_idx;
    p.cu_q = cu_q;
    p.B = B;
    p.N = N;
    p.max_q = max_q;
    p.H = H;
    p.H_k = H_k;
    p.G = G;
    p.B_table = B_table;
    p.width = max_pages;
    p.n_pages = n_pages;
    p.shift = shift;
    while ((2 << p.tau_log) * G <= R) ++p.tau_log;
    p.tau = 1 << p.tau_log;
    p.causal = mask == FMHA_MASK_CAUSAL;
    p.edge = 2;
    // a CTA a tile at most, of the tiles that there can be
    const int64_t units = (int64_t)H_k * ((int64_t)B + (N >> p.tau_log));
    const int64_t tiles = (((int64_t)max_pages << shift) + kRows - 1) / kRows;
    p.ncta = (int)(units >= kPagedMaxCtas || units * tiles >= kPagedMaxCtas ? kPagedMaxCtas : units * tiles);
    p.ncta = imin(p.ncta, sms);
    p.part_o = static_cast<float *>(workspace);
    p.part_lse = p.part_o + (size_t)2 * p.ncta * R * kD;
    p.meta = reinterpret_cast<PagedMeta *>(p.part_lse + (size_t)2 * p.ncta * R);
    p.c = log2_scale(scale);
    p.out_scale = out_scale;

    CUtensorMap tm[2];
    for (int kv = 0; kv < 2; ++kv) {
        // [n_pages * H_k, P, 128]: the rows of one page and head
        const cuuint64_t dims[3] = {kD, (cuuint64_t)page_size, (cuuint64_t)n_pages * H_k};
        const cuuint32_t box[3] = {kD, (cuuint32_t)page_size, 1};
        if (!make_map(&tm[kv], FMHA_E4M3, kv ? v_pages : k_pages, 3, dims, box)) return FMHA_ERR_CUDA;
    }
    const bool bf = dt == FMHA_BF16;
    const int per_unit = imin(R, G * imin(p.tau, max_q));
    const PagedLaunch k = bf ? paged_kernel<true>(R, per_unit) : paged_kernel<false>(R, per_unit);
    if (cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess) return cuda_failed();
    k.kernel<<<p.ncta, k.threads, k.smem, stream>>>(tm[0], tm[1], p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ncta, (R + kPagedMergeWarps - 1) / kPagedMergeWarps);
    cfg.blockDim = dim3(32 * kPagedMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto merge = bf ? fmha_paged_merge_kernel<true> : fmha_paged_merge_kernel<false>;
    if (cudaLaunchKernelEx(&cfg, merge, p, R) != cudaSuccess) return cuda_failed();
    return FMHA_OK;
}
