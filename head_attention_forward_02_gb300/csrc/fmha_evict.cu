// fmha_evict.cu -- eviction from a K/V cache by a score per key: the rows that
// stay are chosen per kv head and moved, in order, to the front of an entry.
//
// Operation: sequence b has L = seqlen[b] rows in entry e, and acc[e, g, j] is
// the score of row j for kv head g.  With L <= budget every row stays.  Else
// the newest `recent` rows stay, and of the L - recent before them the
// budget - recent with the largest scores (equal scores: the lowest row
// first; NaN: below every number).  kept[b, g, :] lists them in ascending
// order, -1 past the end, and row i of the output entry is row kept[b, g, i]
// of the input entry for K, V and acc; acc past the new length is zeroed.
//
// Selection (a cluster of 1, 2, 4 or 8 CTAs a kv head): the scores are mapped
// to 32-bit keys of the same order and the threshold, the need-th largest key,
// is found digit by digit (11, 11 and 10 bits) from histograms in shared
// memory; the CTAs of a cluster add the bins that hold keys to the sums that
// each of them keeps (two fp8 sequences of 65536 rows, 8 heads, to 2047: 17.1
// us for the call; reading one another's histograms whole, 20.5).
// Then every warp counts the keys above the threshold and equal to it in its
// own run of consecutive rows, and, with the counts of the runs before, writes
// its kept rows in order, the first few equal ones among them.  Whole numbers
// only, so the result does not depend on the order of the atomics.  One CTA of
// 512 threads a head took 125 us for 65536 rows of 16 heads, whose 4 MB take
// 0.6; clusters take 15 (from a cold cache), bound by latency: the launch, five
// barriers of the cluster and three rounds of atomics in shared memory.
//
// The move is bound by memory: 4 * 128 * E bytes a kept row and head (32 ragged
// bf16 sequences of 8192 rows, 8 heads, to 2048: 80 us, 6.2 TB/s from and to
// DRAM).  In place, the rows of a head move down one after another: row i comes
// from a row at or after it, so a CTA walks them in blocks, reads a whole block
// into registers, and writes it only after all of it was read.
#include <type_traits>

#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kSelKeys = 16;             // keys a thread holds
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;

struct EvictParams {
    const uint8_t *k, *v;                // [B_cache, S_max, H_k, D]
    const float *acc;                    // [B_cache, H_k, S_max]
    uint8_t *k_out, *v_out;              // [B_out, S_out, H_k, D]
    float *acc_out;                      // [B_out, H_k, S_out]
    const int *seqlen, *batch_idx, *out_idx;
    int *kept;                           // [B, H_k, budget]
    int *new_seqlen;                     // [B]
    int B, H_k, B_cache, S_max, B_out, S_out, budget, recent;
    int in_place;
};

// Order-preserving key of a score: larger score, larger key; NaN below all.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);                // -0 becomes +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const EvictParams &p, int b, bool report) {
    return clamped(p.seqlen[b], 0, p.S_max, report);
}

// Shared memory of CTA `rank` of the cluster, at the address that `p` has in
// this one: add to a word there, store one.
__device__ __forceinline__ uint32_t cluster_addr(const uint32_t *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_add(const uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_store(const uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// grid (CS * H_k, B), clusters of CS CTAs of TH threads along x
template <int CS, int TH>
__global__ void __launch_bounds__(TH) fmha_evict_select_kernel(const EvictParams p) {
    constexpr int kSelWarps = TH / 32;
    __shared__ alignas(16) uint32_t hist[kBins];                     // of this CTA's keys
    __shared__ alignas(16) uint32_t sum[CS > 1 ? 3 : 1][CS > 1 ? kBins : 4];   // the cluster's, by pass: every CTA adds to all
    __shared__ uint32_t warp_sum[kSelWarps], warp_eq[kSelWarps];
    __shared__ uint32_t s_digit, s_above, cta_gt[CS], cta_eq[CS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int g = blockIdx.x / CS, rank = blockIdx.x % CS, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool first = blockIdx.x == 0 && tid == 0;
    const int L = evict_len(p, b, first);
    const int e = cache_entry(p.batch_idx, b, p.B_cache, first);
    if (first) {
        cache_entry(p.out_idx, b, p.B_out, true);
        p.new_seqlen[b] = imin(L, p.budget);
    }
    int *kept = p.kept + ((int64_t)b * p.H_k + g) * p.budget;
    if (L <= p.budget || e < 0) {                // the same in every CTA of the cluster
        for (int i = rank * TH + tid; i < p.budget; i += CS * TH) kept[i] = i < L ? i : -1;
        return;
    }
    const int cand = L - p.recent, need = p.budget - p.recent;   // cand > need >= 0
    const float *acc = p.acc + ((int64_t)e * p.H_k + g) * p.S_max;
    for (int i = rank * TH + tid; i < p.recent; i += CS * TH) kept[need + i] = cand + i;
    if (need == 0) return;

    // this warp's run of rows [lo, hi), in blocks of kSelKeys a lane; a run of
    // one block is read once and stays in registers
    const int run = ((cand + CS * kSelWarps - 1) / (CS * kSelWarps) + 31) / 32 * 32;
    const int lo = imin(cand, (rank * kSelWarps + warp) * run), hi = imin(cand, lo + run);
    constexpr int kBlock = 32 * kSelKeys;
    const bool once = run <= kBlock;
    uint32_t key[kSelKeys];
    float x[kSelKeys];
    auto fetch = [&](int base) {
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k) {
            const int i = base + 32 * k + lane;
            x[k] = i < hi ? acc[i] : 0.f;
        }
    };
    auto to_keys = [&]() {
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k) key[k] = score_key(x[k]);
    };
    auto load = [&](int base) {
        fetch(base);
        to_keys();
    };
    if (once) fetch(lo);
    for (int i = tid; i < kBins; i += TH) hist[i] = 0;
    if (CS > 1) {
        for (int i = tid; i < 3 * kBins; i += TH) sum[0][i] = 0;
        cluster_arrive();                        // met below: nobody adds to a sum before it is zeroed
    }
    if (once) to_keys();
    if (CS > 1) cluster_wait();
    __syncthreads();

    // the need-th largest key: its digits, and how many keys equal to it stay
    uint32_t prefix = 0, want = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int base = lo; base < hi; base += kBlock) {
            if (!once) load(base);
#pragma unroll
            for (int k = 0; k < kSelKeys; ++k)
                if (base + 32 * k + lane < hi && (pass == 0 || (key[k] >> (shift + bits)) == prefix))
                    atomicAdd(&hist[(key[k] >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        if (CS > 1) {
            // few of the bins hold a key: those go to every CTA
            for (int i = tid; i < kBins; i += TH) {
                const uint32_t c = hist[i];
                if (c == 0) continue;
                hist[i] = 0;
#pragma unroll
                for (int r = 0; r < CS; ++r) cluster_add(&sum[pass][i], r, c);
            }
            cluster_arrive();
            cluster_wait();
        }
        // bins from the top, PER a thread: the one in which the count passes `want`
        constexpr int PER = kBins / TH;
        using Bins = std::conditional_t<PER == 4, uint4, uint2>;
        static_assert(PER == 4 || PER == 2, "bins of a thread");
        Bins *own = reinterpret_cast<Bins *>(CS > 1 ? sum[CS > 1 ? pass : 0] : hist) + (TH - 1 - tid);
        const Bins v = *own;
        if (CS == 1) *own = Bins{};
        uint32_t n[PER], mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            n[i] = reinterpret_cast<const uint32_t *>(&v)[PER - 1 - i];
            mine += n[i];
        }
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        const uint32_t ws = lane < kSelWarps ? warp_sum[lane] : 0u;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u);
        uint32_t above = before + incl - mine;
        if (above < want && above + mine >= want) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (above < want && above + n[i] >= want) {
                    s_digit = kBins - 1 - (tid * PER + i);
                    s_above = above;
                }
                above += n[i];
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | s_digit;
        want -= s_above;
    }

    // rows above the threshold, and those equal to it, of every warp's run
    uint32_t gt = 0, eq = 0;
    for (int base = lo; base < hi; base += kBlock) {
        if (!once) load(base);
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k) {
            const bool in = base + 32 * k + lane < hi;
            gt += in && key[k] > prefix;
            eq += in && key[k] == prefix;
        }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) {
        warp_sum[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    const uint32_t wg = lane < kSelWarps ? warp_sum[lane] : 0u, we = lane < kSelWarps ? warp_eq[lane] : 0u;
    uint32_t at_gt = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0u);
    uint32_t at_eq = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0u);
    if (CS > 1) {
        // the CTAs before this one
        const uint32_t tg = __reduce_add_sync(0xffffffffu, wg), te = __reduce_add_sync(0xffffffffu, we);
        if (tid < CS) {
            cluster_store(&cta_gt[rank], tid, tg);
            cluster_store(&cta_eq[rank], tid, te);
        }
        cluster_arrive();
        cluster_wait();                          // no CTA reaches into another's shared memory after this
#pragma unroll
        for (int c = 0; c < CS; ++c) {
            at_gt += c < rank ? cta_gt[c] : 0u;
            at_eq += c < rank ? cta_eq[c] : 0u;
        }
    }
    const uint32_t lt = (1u << lane) - 1u;
    for (int base = lo; base < hi; base += kBlock) {
        if (!once) load(base);
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k) {
            if (base + 32 * k >= hi) break;
            const int i = base + 32 * k + lane;
            const bool is_gt = i < hi && key[k] > prefix, is_eq = i < hi && key[k] == prefix;
            const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
            const uint32_t re = at_eq + __popc(me & lt);
            if (is_gt || (is_eq && re < want)) kept[at_gt + __popc(mg & lt) + min(re, want)] = i;
            at_gt += __popc(mg);
            at_eq += __popc(me);
        }
    }
}

// A CTA moves slices of SL bytes of a head's rows in 16-byte pieces, four rows'
// of a block a thread; eight where a head is walked by few CTAs, each block a
// round trip to memory (2048 of 4096 rows in place: 24.6 -> 20.5 us).
template <int SL>
struct MoveCfg {
    static constexpr int PIECES = SL / 16;
    static constexpr int ROWS_AT_ONCE = kMoveThreads / PIECES;
    static constexpr int PER = SL == 64 ? 8 : 4;
    static constexpr int BLOCK = ROWS_AT_ONCE * PER;
};

// K or V of one head: grid (H_k, B, chunks * 2 * ROW / SL).  Apart from the
// input, a chunk is every `chunks`-th block of whole rows.  In place there is
// one chunk, walked in order, and for few heads the rows are cut into slices
// of 64 bytes, which move down independently: four times the CTAs, and four
// times the rows in a block.
template <int ROW, int SL>
__global__ void __launch_bounds__(kMoveThreads) fmha_evict_move_kernel(const EvictParams p) {
    using M = MoveCfg<SL>;
    constexpr int kSlices = ROW / SL;
    const int g = blockIdx.x, b = blockIdx.y;
    const int slice = blockIdx.z % kSlices, kv = blockIdx.z / kSlices % 2;
    const int chunk = blockIdx.z / (2 * kSlices), chunks = gridDim.z / (2 * kSlices);
    const int tid = threadIdx.x, piece = tid % M::PIECES, r0 = tid / M::PIECES;
    const int L = evict_len(p, b, false), n = imin(L, p.budget);
    const int e = cache_entry(p.batch_idx, b, p.B_cache, false), d = cache_entry(p.out_idx, b, p.B_out, false);
    const int *kept = p.kept + ((int64_t)b * p.H_k + g) * p.budget;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (e < 0 || d < 0) return;
    const int64_t pitch = (int64_t)p.H_k * ROW;
    const int64_t col = (int64_t)g * ROW + slice * SL + piece * 16;
    const uint8_t *src = (kv ? p.v : p.k) + (int64_t)e * p.S_max * pitch + col;
    uint8_t *dst = (kv ? p.v_out : p.k_out) + (int64_t)d * p.S_out * pitch + col;
    const bool moves = !p.in_place || L > p.budget;
    if (moves) {
        // the rows' numbers of a block are fetched while the block before moves
        int from[M::PER];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < M::PER; ++k) {
                const int i = i0 + k * M::ROWS_AT_ONCE + r0;
                from[k] = i < n ? kept[i] : 0;
            }
        };
        const int step = chunks * M::BLOCK;
        fetch(chunk * M::BLOCK);
        for (int i0 = chunk * M::BLOCK; i0 < n; i0 += step) {
            uint4 x[M::PER];
#pragma unroll
            for (int k = 0; k < M::PER; ++k)
                if (i0 + k * M::ROWS_AT_ONCE + r0 < n) x[k] = *reinterpret_cast<const uint4 *>(src + from[k] * pitch);
            fetch(i0 + step);
            if (p.in_place) __syncthreads();                    // the block is read: it may be overwritten
#pragma unroll
            for (int k = 0; k < M::PER; ++k) {
                const int i = i0 + k * M::ROWS_AT_ONCE + r0;
                if (i < n) *reinterpret_cast<uint4 *>(dst + i * pitch) = x[k];
            }
        }
    }
    if (kv != 0 || slice != 0) return;
    // the scores of the head, and zeros behind them, by the same chunks
    const float *a = p.acc + ((int64_t)e * p.H_k + g) * p.S_max;
    float *o = p.acc_out + ((int64_t)d * p.H_k + g) * p.S_out;
    constexpr int kScores = 4;                                  // a thread
    if (moves)
        for (int i0 = chunk * kScores * kMoveThreads; i0 < n; i0 += chunks * kScores * kMoveThreads) {
            float x[kScores];
#pragma unroll
            for (int k = 0; k < kScores; ++k) {
                const int i = i0 + k * kMoveThreads + tid;
                x[k] = i < n ? a[kept[i]] : 0.f;
            }
            if (p.in_place) __syncthreads();
#pragma unroll
            for (int k = 0; k < kScores; ++k) {
                const int i = i0 + k * kMoveThreads + tid;
                if (i < n) o[i] = x[k];
            }
        }
    __syncthreads();
    float *z = o + n;
    const int rest = p.S_out - n, lead = imin(rest, (int)(-reinterpret_cast<uintptr_t>(z) & 15) / 4);
    const int quads = (rest - lead) / 4;
    for (int i = chunk * kMoveThreads + tid; i < quads; i += chunks * kMoveThreads)
        reinterpret_cast<float4 *>(z + lead)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (chunk == 0 && tid < rest - 4 * quads) z[tid < lead ? tid : tid + 4 * quads] = 0.f;
}

}  // namespace

int *evict_status_word() { return symbol_address(g_status); }

}  // namespace fmha

using namespace fmha;

extern "C" int fmha_cache_evict(fmha_tensor k_cache, fmha_tensor v_cache, const float *acc, fmha_tensor k_out,
                                fmha_tensor v_out, float *acc_out, int B, int H_k, int D, int B_cache, int S_max,
                                int B_out, int S_out, const int *seqlen, const int *batch_idx, const int *out_idx,
                                int budget, int recent, int *kept, int *new_seqlen, cudaStream_t stream) {
    // ---- host-side validation: nothing is launched on a bad argument ----
    if (B < 0 || H_k <= 0 || D != kD || budget <= 0 || recent < 0 || recent > budget) return FMHA_ERR_INVALID_ARG;
    if (B == 0) return FMHA_OK;
    if (S_max <= 0 || B_cache <= 0 || S_out <= 0 || B_out <= 0 || budget > S_out) return FMHA_ERR_INVALID_ARG;
    if (S_max > kMaxCacheRows || S_out > kMaxCacheRows) return FMHA_ERR_INVALID_ARG;
    if (!seqlen || !kept || !new_seqlen || !acc || !acc_out) return FMHA_ERR_INVALID_ARG;
    if (!k_cache.data || !v_cache.data || !k_out.data || !v_out.data) return FMHA_ERR_INVALID_ARG;
    const int dt = k_cache.dtype;
    if (dt != FMHA_F16 && dt != FMHA_BF16 && dt != FMHA_E4M3) return FMHA_ERR_UNSUPPORTED;
    for (const fmha_tensor *t : {&v_cache, &k_out, &v_out})
        if (t->dtype != dt) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {k_cache.data, v_cache.data, k_out.data, v_out.data})
        if (misaligned(ptr, 16)) return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {(const void *)acc, (const void *)acc_out, (const void *)seqlen, (const void *)batch_idx,
                            (const void *)out_idx, (const void *)kept, (const void *)new_seqlen})
        if (misaligned(ptr, 4)) return FMHA_ERR_INVALID_ARG;
    if (B > 65535) return FMHA_ERR_UNSUPPORTED;
    const int row = kD * (dt == FMHA_E4M3 ? 1 : 2);
    // the output is the input (all three, same sizes and entries), or apart from
    // it; either way K, V, the scores and the lists are arrays of their own
    const bool in_place = k_out.data == k_cache.data;
    if (in_place &&
        (v_out.data != v_cache.data || acc_out != acc || B_out != B_cache || S_out != S_max || out_idx != batch_idx))
        return FMHA_ERR_INVALID_ARG;
    const size_t in_b = (size_t)B_cache * S_max * H_k, out_b = (size_t)B_out * S_out * H_k, seq_b = (size_t)B * sizeof(int);
    const Bytes out[5] = {{k_out.data, out_b * row}, {v_out.data, out_b * row}, {acc_out, out_b * sizeof(float)},
                          {kept, (size_t)H_k * budget * seq_b}, {new_seqlen, seq_b}};
    const Bytes in[3] = {{k_cache.data, in_b * row}, {v_cache.data, in_b * row}, {acc, in_b * sizeof(float)}};
    const Bytes seq[3] = {{seqlen, seq_b}, {batch_idx, seq_b}, {out_idx, seq_b}};
    if (outputs_clash(out, seq) || (!in_place && outputs_clash(out, in))) return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    const int sms = sm_count();
    if (sms <= 0) return FMHA_ERR_CUDA;

    EvictParams p{};
    p.k = static_cast<const uint8_t *>(k_cache.data);
    p.v = static_cast<const uint8_t *>(v_cache.data);
    p.acc = acc;
    p.k_out = static_cast<uint8_t *>(k_out.data);
    p.v_out = static_cast<uint8_t *>(v_out.data);
    p.acc_out = acc_out;
    p.seqlen = seqlen;
    p.batch_idx = batch_idx;
    p.out_idx = out_idx;
    p.kept = kept;
    p.new_seqlen = new_seqlen;
    p.B = B;
    p.H_k = H_k;
    p.B_cache = B_cache;
    p.S_max = S_max;
    p.B_out = B_out;
    p.S_out = S_out;
    p.budget = budget;
    p.recent = recent;
    p.in_place = in_place ? 1 : 0;
    // CTAs of a head's selection: while all fit the SMs at once (clusters of
    // eight do not pack: half; 16 heads of 65536 rows take 17.1 us by four and
    // 18.5 by eight) and each has 2048 rows; 1024 threads where 512 would not
    // hold a CTA's keys in registers
    int cs = 8;
    while (cs > 1 && ((int64_t)B * H_k * cs > (cs == 8 ? sms / 2 : sms) || S_max / cs < 2048)) cs /= 2;
    const bool wide = S_max / cs > 512 * kSelKeys;
    {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cs * H_k, B);
        cfg.blockDim = dim3(wide ? 1024 : 512);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cs;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cs > 1 ? 1 : 0;
        auto select = wide ? (cs == 8 ? fmha_evict_select_kernel<8, 1024> : cs == 4 ? fmha_evict_select_kernel<4, 1024>
                              : cs == 2 ? fmha_evict_select_kernel<2, 1024> : fmha_evict_select_kernel<1, 1024>)
                           : (cs == 8 ? fmha_evict_select_kernel<8, 512> : cs == 4 ? fmha_evict_select_kernel<4, 512>
                              : cs == 2 ? fmha_evict_select_kernel<2, 512> : fmha_evict_select_kernel<1, 512>);
        if (cudaLaunchKernelEx(&cfg, select, p) != cudaSuccess) return cuda_failed();
    }

    // apart from the input, the blocks of a head are spread over CTAs until
    // the SMs hold eight each; in place, few heads are cut into slices
    const int64_t heads = (int64_t)2 * B * H_k;
    const bool sliced = in_place && heads < 2 * sms;
    const int block = dt == FMHA_E4M3 ? MoveCfg<128>::BLOCK : MoveCfg<256>::BLOCK;
    const int blocks = (budget + block - 1) / block;
    int chunks = (int)((8 * (int64_t)sms + heads - 1) / heads);
    if (chunks > blocks) chunks = blocks;
    if (in_place) chunks = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(H_k, B, 2 * chunks * (sliced ? row / 64 : 1));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto move = dt == FMHA_E4M3 ? (sliced ? fmha_evict_move_kernel<128, 64> : fmha_evict_move_kernel<128, 128>)
                                : (sliced ? fmha_evict_move_kernel<256, 64> : fmha_evict_move_kernel<256, 256>);
    if (cudaLaunchKernelEx(&cfg, move, p) != cudaSuccess) return cuda_failed();
    return FMHA_OK;
}
