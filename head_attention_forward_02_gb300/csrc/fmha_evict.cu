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
// Selection (one CTA a kv head): the scores are mapped to 32-bit keys of the
// same order and the threshold, the need-th largest key, is found digit by
// digit (11, 11 and 10 bits) from histograms in shared memory; a last pass
// over the scores writes the rows above it, and the first few equal to it, in
// order by a block-wide prefix sum.  Whole numbers only, so the result does not
// depend on the order of the atomics.
//
// The move is bound by memory: 4 * 128 * E bytes a kept row and head.  In
// place, the rows of a head move down one after another: row i comes from a
// row at or after it, so a CTA walks them in blocks, reads a whole block into
// registers, and writes it only after all of it was read.
#include "fmha_cache.cuh"

namespace fmha {

namespace {

constexpr int kSelThreads = 512;
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
    int row;                             // bytes of one head's row
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

__global__ void __launch_bounds__(kSelThreads) fmha_evict_select_kernel(const EvictParams p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t warp_sum[kSelThreads / 32][2];
    __shared__ uint32_t s_digit, s_above;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool first = g == 0 && tid == 0;
    const int L = evict_len(p, b, first);
    const int e = cache_entry(p.batch_idx, b, p.B_cache, first);
    if (first) {
        cache_entry(p.out_idx, b, p.B_out, true);
        p.new_seqlen[b] = imin(L, p.budget);
    }
    int *kept = p.kept + ((int64_t)b * p.H_k + g) * p.budget;
    if (L <= p.budget || e < 0) {
        for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = i < L ? i : -1;
        return;
    }
    const int cand = L - p.recent, need = p.budget - p.recent;   // cand > need >= 0
    const float *acc = p.acc + ((int64_t)e * p.H_k + g) * p.S_max;
    for (int i = tid; i < p.recent; i += kSelThreads) kept[need + i] = cand + i;
    if (need == 0) return;

    // the need-th largest key: its digits, and how many keys equal to it stay
    uint32_t prefix = 0, want = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < cand; i += kSelThreads) {
            const uint32_t k = score_key(acc[i]);
            if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        // bins from the top: the one in which the count passes `want`
        constexpr int PER = kBins / kSelThreads;
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine += hist[kBins - 1 - (tid * PER + i)];
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp][0] = incl;
        __syncthreads();
        uint32_t above = incl - mine;
        for (int w = 0; w < warp; ++w) above += warp_sum[w][0];
        if (above < want && above + mine >= want) {
            for (int i = 0; i < PER; ++i) {
                const int bin = kBins - 1 - (tid * PER + i);
                if (above + hist[bin] >= want) {
                    s_digit = bin;
                    s_above = above;
                    break;
                }
                above += hist[bin];
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | s_digit;
        want -= s_above;
        __syncthreads();
    }

    // rows above the threshold, and the first `want` equal to it, in order
    uint32_t base_gt = 0, base_eq = 0;
    for (int i0 = 0; i0 < cand; i0 += kSelThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < cand ? score_key(acc[i]) : 0u;
        const bool gt = i < cand && k > prefix, eq = i < cand && k == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_sum[warp][0] = __popc(mg);
            warp_sum[warp][1] = __popc(me);
        }
        __syncthreads();
        uint32_t rg = base_gt, re = base_eq;
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) {
            const uint32_t a = warp_sum[w][0], c = warp_sum[w][1];
            if (w < warp) {
                rg += a;
                re += c;
            }
            base_gt += a;
            base_eq += c;
        }
        const uint32_t lt = (1u << lane) - 1u;
        rg += __popc(mg & lt);
        re += __popc(me & lt);
        if (gt || (eq && re < want)) kept[rg + min(re, want)] = i;
        __syncthreads();
    }
}

// 16-byte pieces of a row, and the rows of a block: a block is 16 KB
template <int ROW>
struct MoveCfg {
    static constexpr int PIECES = ROW / 16;
    static constexpr int ROWS_AT_ONCE = kMoveThreads / PIECES;
    static constexpr int PER = 4;                               // rows a thread holds
    static constexpr int BLOCK = ROWS_AT_ONCE * PER;
};

// K or V of one head: grid (H_k, B, 2 * chunks); a chunk is every `chunks`-th
// block of rows.  In place there is one chunk, walked in order.
template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) fmha_evict_move_kernel(const EvictParams p) {
    using M = MoveCfg<ROW>;
    const int g = blockIdx.x, b = blockIdx.y, kv = blockIdx.z & 1, chunk = blockIdx.z >> 1, chunks = gridDim.z >> 1;
    const int tid = threadIdx.x, piece = tid % M::PIECES, r0 = tid / M::PIECES;
    const int L = evict_len(p, b, false), n = imin(L, p.budget);
    const int e = cache_entry(p.batch_idx, b, p.B_cache, false), d = cache_entry(p.out_idx, b, p.B_out, false);
    const int *kept = p.kept + ((int64_t)b * p.H_k + g) * p.budget;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (e < 0 || d < 0) return;
    const int64_t pitch = (int64_t)p.H_k * ROW;
    const uint8_t *src = (kv ? p.v : p.k) + (int64_t)e * p.S_max * pitch + (int64_t)g * ROW + piece * 16;
    uint8_t *dst = (kv ? p.v_out : p.k_out) + (int64_t)d * p.S_out * pitch + (int64_t)g * ROW + piece * 16;
    if (!p.in_place || L > p.budget) {
        for (int i0 = chunk * M::BLOCK; i0 < n; i0 += chunks * M::BLOCK) {
            uint4 x[M::PER];
#pragma unroll
            for (int k = 0; k < M::PER; ++k) {
                const int i = i0 + k * M::ROWS_AT_ONCE + r0;
                if (i < n) x[k] = *reinterpret_cast<const uint4 *>(src + kept[i] * pitch);
            }
            if (p.in_place) __syncthreads();                    // the block is read: it may be overwritten
#pragma unroll
            for (int k = 0; k < M::PER; ++k) {
                const int i = i0 + k * M::ROWS_AT_ONCE + r0;
                if (i < n) *reinterpret_cast<uint4 *>(dst + i * pitch) = x[k];
            }
        }
    }
    if (kv != 0 || chunk != 0) return;
    // the scores of the head, and zeros behind them
    const float *a = p.acc + ((int64_t)e * p.H_k + g) * p.S_max;
    float *o = p.acc_out + ((int64_t)d * p.H_k + g) * p.S_out;
    if (!p.in_place || L > p.budget)
        for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
            const int i = i0 + tid;
            const float x = i < n ? a[kept[i]] : 0.f;
            if (p.in_place) __syncthreads();
            if (i < n) o[i] = x;
        }
    __syncthreads();
    for (int i = n + tid; i < p.S_out; i += kMoveThreads) o[i] = 0.f;
}

}  // namespace

int evict_read_status(int reset) { return cache_read_status(reset); }

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
    // the output is the input (all three, same sizes and entries), or apart from it
    const bool in_place = k_out.data == k_cache.data;
    if (in_place) {
        if (v_out.data != v_cache.data || acc_out != acc || B_out != B_cache || S_out != S_max || out_idx != batch_idx)
            return FMHA_ERR_INVALID_ARG;
    } else {
        const size_t in_b = (size_t)B_cache * S_max * H_k, out_b = (size_t)B_out * S_out * H_k;
        struct Range { const char *p; size_t n; };
        const Range in[3] = {{(const char *)k_cache.data, in_b * row}, {(const char *)v_cache.data, in_b * row},
                             {(const char *)acc, in_b * sizeof(float)}};
        const Range out[3] = {{(const char *)k_out.data, out_b * row}, {(const char *)v_out.data, out_b * row},
                              {(const char *)acc_out, out_b * sizeof(float)}};
        for (const Range &i : in)
            for (const Range &o : out)
                if (i.p < o.p + o.n && o.p < i.p + i.n) return FMHA_ERR_INVALID_ARG;
    }
    if (seqlen == new_seqlen) return FMHA_ERR_INVALID_ARG;      // every CTA of a sequence reads its length
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
    p.row = row;
    p.in_place = in_place ? 1 : 0;
    fmha_evict_select_kernel<<<dim3(H_k, B), kSelThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FMHA_ERR_CUDA;

    // apart from the input, the blocks of a head are spread over CTAs until
    // the SMs hold eight each
    const int block = dt == FMHA_E4M3 ? MoveCfg<128>::BLOCK : MoveCfg<256>::BLOCK;
    const int blocks = (budget + block - 1) / block;
    const int64_t heads = (int64_t)2 * B * H_k;
    int chunks = (int)((8 * (int64_t)sms + heads - 1) / heads);
    if (chunks > blocks) chunks = blocks;
    if (in_place) chunks = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(H_k, B, 2 * chunks);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto move = dt == FMHA_E4M3 ? fmha_evict_move_kernel<128> : fmha_evict_move_kernel<256>;
    if (cudaLaunchKernelEx(&cfg, move, p) != cudaSuccess) return cuda_failed();
    return FMHA_OK;
}
