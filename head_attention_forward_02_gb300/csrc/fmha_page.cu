// fmha_page.cu -- the plan of a step on a paged K/V cache (block tables and
// slot maps from request lengths), and the write of new keys and values into
// pages of e4m3 codes with a scale per page and kv head.
//
// Plan: with P tokens a page, L = seqlen[b] and n = n_new[b], n < 0 drops the
// last -n tokens, and the pages that become empty go onto a stack of free
// ones, in the order of the sequences; n >= 0 needs ceil((L + n) / P) -
// ceil(L / P) pages from its top.  With c_b the running sum of these needs, a
// sequence gets all of them if c_b is at most what the stack holds, else none.
// Sums of whole numbers, so no order of threads shows.
//
// One cluster of up to eight CTAs does it in one launch: every CTA scans all
// sequences for itself (six words each, kept in shared memory), the cluster
// waits until all have read what the call may overwrite in place, and then
// the pages given back, the pages taken, the sequences and the tokens (by fours
// where there are many) are one list of jobs that the threads share out; a job finds its sequence by
// bisection.  What a token's slot needs of pages taken by this call comes from
// the stack, not from the table that other threads write, so there is nothing
// else to wait for.  Bound by latency: 64 sequences of a token each 6.6 us, a launch, two
// dependent reads, a scan, a bisection; 700 sequences with 45000 tokens 15.1, where 24500 jobs on
// 8192 threads are three turns of a bisection, for new pages a second one, and a dependent read
// (18.0 as four lists one after the other, a token a job).
//
// Write: a run of tokens with consecutive slots in one page (some of them
// perhaps left out, by a slot outside the cache); for each kv head
// and of K and V, a = max |x| over it and
//   s = max(scale before, 2^e), e the least with a <= 448 * 2^e
// (a run that begins its page: s = 2^e), rows before the run are rounded again
// to code * (scale before / s) where the scale grew, and the new rows are
// e4m3(x / s).  Scales are powers of two: e4m3 has the same relative step in
// every binade, so a finer scale would not make values more exact, and x / s and
// the old rows' factor are exact, which leaves each value one rounding (a row
// whose scale grows into e4m3's subnormals: two).  A page that another program filled may have
// any scale; then they are rounded once all the same, by way of rounding to odd.
//
// Bound by memory: 2 bytes in and 1 out an element.  A CTA takes the runs that
// begin in 16 tokens, for some heads' K or V, and each of its warps a run of
// up to 16 rows of one of them: two rows a load, all in flight at once, under the
// loads of their slots, and in registers between the maximum and the rounding.
// A longer run (of pages of 32 and more) is spread over two to eight warps, 16
// rows each, the next head's rows fetched under the rounding of this one's.
// 16600 tokens of 8 heads: 21.4 us in pages of 16 tokens, 4.8 TB/s, 70% of the copy
// rate, 22.6 / 24.8 / 28.7 in pages of 32 / 64 / 128 (a long run's pairs follow one another in a
// CTA, with two barriers each, and in pages of 128 the 540 CTAs that have one are 1.2 waves of
// 456); 64 single tokens 4.6 us, a launch and two dependent reads.
#include <cooperative_groups.h>

#include "fmha_cache.cuh"

namespace cg = cooperative_groups;

namespace fmha {
namespace {

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 8192;          // sequences at most: six words each in shared memory

struct PlanParams {
    const int *seqlen, *n_new, *batch_idx, *n_free;
    int *table, *free_list, *n_free_out, *slots, *positions, *cu_new, *new_seqlen;
    int B, N, entries, width, shift, cap;   // cap: pages of the cache, and elements of free_list
    int job;                             // tokens of a job: 1 or 4
};

struct PlanSums {
    long long need, given, tokens;
};

// Exclusive sums over the CTA's threads; total: of all.
__device__ PlanSums plan_scan(PlanSums v, PlanSums &total) {
    __shared__ PlanSums warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PlanSums incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, incl.need, o), b = __shfl_up_sync(0xffffffffu, incl.given, o),
                        c = __shfl_up_sync(0xffffffffu, incl.tokens, o);
        if (lane >= o) {
            incl.need += a;
            incl.given += b;
            incl.tokens += c;
        }
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    PlanSums base = {0, 0, 0};
    total = base;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        const PlanSums s = warp_sum[w];
        if (w < warp) base = PlanSums{base.need + s.need, base.given + s.given, base.tokens + s.tokens};
        total = PlanSums{total.need + s.need, total.given + s.given, total.tokens + s.tokens};
    }
    return PlanSums{base.need + incl.need - v.need, base.given + incl.given - v.given, base.tokens + incl.tokens - v.tokens};
}

// The last of the n ascending values that is at most x (the first is 0).
__device__ __forceinline__ int last_at_most(const int *v, int n, int x) {
    int lo = 0, hi = n;                  // v[lo] <= x; v[hi] > x
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What a request asks for, with everything outside its bounds clamped.
struct PlanRequest {
    int L, n;                            // cached tokens, change (at least -L)
    int entry;                           // its table row, -1: none
    bool fits;                           // its table row holds it
};
__device__ __forceinline__ PlanRequest plan_request(const PlanParams &p, int b, bool report) {
    PlanRequest r;
    const int most = p.width << p.shift;
    r.entry = cache_entry(p.batch_idx, b, p.entries, report);
    r.L = clamped(p.seqlen[b], 0, most, report);
    r.n = clamped(p.n_new[b], -r.L, 0x7fffffff, report);
    r.fits = r.entry >= 0 && r.n <= most - r.L;
    if (r.entry < 0 && r.n < 0) r.n = 0; // no row to take pages from
    if (r.entry >= 0 && !r.fits && report) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
    return r;
}

__global__ void __launch_bounds__(kPlanThreads, 1) fmha_page_plan_kernel(const PlanParams p) {
    extern __shared__ int smem_i[];
    __shared__ int s_granted;
    int *s_len = smem_i, *s_new = s_len + p.B, *s_need = s_new + p.B, *s_given = s_need + p.B, *s_cu = s_given + p.B;
    int *s_entry = s_cu + p.B;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int mask = (1 << p.shift) - 1;
    const bool report = rank == 0;
    if (threadIdx.x == 0) s_granted = 0;
    const int n_free = p.n_free[0];

    // ---- every CTA: the sums of pages needed, pages given back and tokens before each sequence ----
    const int per = (p.B + blockDim.x - 1) / blockDim.x, b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    PlanSums mine = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = plan_request(p, b, report);
        const int had = (r.L + mask) >> p.shift, want = (int)(((long long)r.L + r.n + mask) >> p.shift);
        s_len[b] = r.fits ? r.L : ~r.L;  // a request that cannot fit: the complement
        s_new[b] = r.n;
        s_entry[b] = r.entry;
        if (r.fits && r.n > 0) mine.need += want - had;
        if (r.n < 0) mine.given += had - want;
        mine.tokens += r.n > 0 ? r.n : 0;
    }
    PlanSums total;
    PlanSums at = plan_scan(mine, total);
    const int spare = clamped(n_free, 0, p.cap, report && threadIdx.x == 0);
    const bool over = spare + total.given > p.cap;            // more pages than there are: a page given twice
    const int avail = over ? p.cap : (int)(spare + total.given);
    if (report && threadIdx.x == 0 && (over || total.tokens > p.N)) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
    long long granted = 0;               // the largest sum of needs that the stack holds
    for (int b = b0; b < b1; ++b) {
        const int L = s_len[b] < 0 ? ~s_len[b] : s_len[b], n = s_new[b];
        const int had = (L + mask) >> p.shift, want = (int)(((long long)L + n + mask) >> p.shift);
        s_need[b] = (int)min(at.need, 0x7fffffffll);
        s_given[b] = (int)min(at.given, (long long)avail - spare);
        s_cu[b] = (int)min(at.tokens, (long long)p.N);
        if (s_len[b] >= 0 && n > 0) at.need += want - had;
        if (n < 0) at.given += had - want;
        at.tokens += n > 0 ? n : 0;
        if (at.need <= avail) granted = at.need;
    }
    if (granted > 0) atomicMax(&s_granted, (int)granted);
    // all CTAs have read the lengths and the count that the call may write in place
    cluster.sync();

    const int taken = s_granted, given = avail - spare, tokens = (int)min(total.tokens, (long long)p.N);
    auto row = [&](int b) { return p.table + (int64_t)s_entry[b] * p.width; };
    auto len = [&](int b) { return s_len[b] < 0 ? ~s_len[b] : s_len[b]; };
    auto need = [&](int b) {
        return s_len[b] >= 0 && s_new[b] > 0 ? ((s_len[b] + s_new[b] + mask) >> p.shift) - ((s_len[b] + mask) >> p.shift) : 0;
    };
    auto granted_to = [&](int b) { return s_len[b] >= 0 && (need(b) == 0 || (long long)s_need[b] + need(b) <= taken); };
    // j-th page given back; k-th page taken, from the stack's top down
    auto page_given = [&](int j) {
        const int b = last_at_most(s_given, p.B, j);
        return row(b)[((len(b) + s_new[b] + mask) >> p.shift) + j - s_given[b]];
    };
    auto page_taken = [&](int k) {
        const int i = avail - 1 - k;
        return i < spare ? p.free_list[i] : page_given(i - spare);
    };
    const int quads = p.N / p.job + (p.N % p.job != 0);
    const bool wide = p.job == 4 && ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
    const long long jobs = (long long)given + taken + p.B + quads;
    for (long long x = rank * blockDim.x + threadIdx.x; x < jobs; x += (long long)ranks * blockDim.x) {
        if (x < quads) {
            int pos[4] = {-1, -1, -1, -1}, slot[4] = {-1, -1, -1, -1};
            const int i0 = (int)x * p.job;
            if (i0 < tokens) {
                int b = last_at_most(s_cu, p.B, i0), before = -1, page = -1;
                bool ok = granted_to(b);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= tokens - i0 || k >= p.job) break;
                    const int i = i0 + k;
                    while (b + 1 < p.B && s_cu[b + 1] <= i) {       // the next sequence with tokens
                        ++b;
                        ok = granted_to(b);
                        before = -1;
                    }
                    const int L = len(b);
                    pos[k] = L + i - s_cu[b];
                    if (!ok) continue;
                    const int had = (L + mask) >> p.shift, at = pos[k] >> p.shift;
                    if (at != before) page = at < had ? row(b)[at] : page_taken(s_need[b] + at - had);
                    before = at;
                    if (page >= 0 && page < p.cap) slot[k] = (page << p.shift) + (pos[k] & mask);
                    else atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
                }
            }
            if (wide && p.N - i0 >= 4) {
                *reinterpret_cast<int4 *>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                *reinterpret_cast<int4 *>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < p.job && k < p.N - i0) {
                        p.slots[i0 + k] = slot[k];
                        p.positions[i0 + k] = pos[k];
                    }
            }
            continue;
        }
        const long long y = x - quads;
        if (y < taken) {
            const int k = (int)y, b = last_at_most(s_need, p.B, k);
            row(b)[((s_len[b] + mask) >> p.shift) + k - s_need[b]] = page_taken(k);
        } else if (y < (long long)taken + given) {
            const int j = (int)(y - taken), page = page_given(j);
            if (page < 0 || page >= p.cap) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
            p.free_list[spare + j] = page;
        } else {
            const int b = (int)(y - taken - given);
            p.cu_new[b] = s_cu[b];
            p.new_seqlen[b] = s_new[b] < 0 || granted_to(b) ? len(b) + s_new[b] : len(b);
            if (b == 0) {
                p.n_free_out[0] = avail - taken;
                p.cu_new[p.B] = tokens;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Write
// ---------------------------------------------------------------------------

constexpr int kWriteWarps = 8;
constexpr int kBatchRows = 16;           // tokens of a CTA, and rows that a warp has in registers
constexpr int kLowest = -60, kHighest = 60;   // exponents of the scales

struct WriteParams {
    const uint8_t *x[2];                 // new keys, values: [N, H_k, 128] with strides
    int64_t x_t[2], x_h[2];              // in bytes
    uint8_t *pages[2];                   // [n_pages, H_k, P, 128]
    float *scale[2];                     // [n_pages, H_k]
    const int *slots;                    // [N]
    int N, H_k, shift, slots_end;        // slots_end: n_pages * P
    int pairs;                           // of (head, K or V) that a CTA takes
};

template <bool BF>
__device__ __forceinline__ float2 wide2(uint32_t w) {
    if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <bool BF>
__device__ __forceinline__ float abs_max(uint4 v, float a) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = wide2<BF>(w[i]);
        a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));         // a NaN does not count
    }
    return a;
}
template <bool BF>
__device__ __forceinline__ uint2 codes8(uint4 v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float2 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = wide2<BF>(w[i]);
        x[i].x *= inv;
        x[i].y *= inv;
    }
    return make_uint2(pack4_e4m3(x[0].x, x[0].y, x[1].x, x[1].y), pack4_e4m3(x[2].x, x[2].y, x[3].x, x[3].y));
}

// A scale that this call chooses is a power of two; one that a page had before may be any,
// and its quotients and products have more bits than 32 hold.  To odd: q, the value
// rounded to nearest, with its last bit set towards what is left, so that rounding it again, to
// e4m3, is as rounding the value itself (a tie of q alone is none of the value).
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }
__device__ __forceinline__ float to_odd(float q, float left) {
    const uint32_t u = __float_as_uint(q);
    if ((u & 1u) != 0 || !(left < 0.f || left > 0.f)) return q;      // exact, infinite, NaN
    return __uint_as_float((left < 0.f) == (u >> 31 != 0) ? u + 1 : u - 1);
}
template <bool BF>
__device__ __forceinline__ uint2 codes8_over(uint4 v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = wide2<BF>(w[i]);
        const float a = x.x / s, b = x.y / s;
        y[2 * i] = to_odd(a, fmaf(-a, s, x.x));
        y[2 * i + 1] = to_odd(b, fmaf(-b, s, x.y));
    }
    return make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
}

// The least power of two that brings a to 448 = 1.75 * 2^8 or below it, within
// the bounds.
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kLowest), kHighest);
}

__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// Four codes times a factor, rounded again.
template <bool ANY>
__device__ __forceinline__ uint32_t again4(uint32_t c, float f) {
    const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
    const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    if constexpr (!ANY) return pack4_e4m3(a.x * f, a.y * f, b.x * f, b.y * f);
    auto times = [&](float x) { return to_odd(x * f, fmaf(x, f, -(x * f))); };
    return pack4_e4m3(times(a.x), times(a.y), times(b.x), times(b.y));
}

// Is a token with this slot written?  A slot outside the cache is as a negative one: were
// it the end of a run, two warps would have runs of the same page, in no order.
__device__ __forceinline__ bool written(const WriteParams &p, int slot) { return (unsigned)slot < (unsigned)p.slots_end; }

// A run: tokens [i, i + n) become rows [off, off + n) of a page.
struct Run {
    uint8_t *rows;                       // the page's head: its first row
    float *scale;
    int off;
};
__device__ __forceinline__ Run run_of(const WriteParams &p, int slot, int g, int kv) {
    const int64_t head = (int64_t)(slot >> p.shift) * p.H_k + g;
    return Run{(kv ? p.pages[1] : p.pages[0]) + ((head << p.shift) << 7), (kv ? p.scale[1] : p.scale[0]) + head, slot & ((1 << p.shift) - 1)};
}

// The scale of a run whose largest value is a; old: what it was (rows before).
__device__ __forceinline__ float run_scale(const Run &r, float a, float &old) {
    const float s = __uint_as_float((uint32_t)(scale_exponent(a) + 127) << 23);
    old = r.off > 0 ? *r.scale : 0.f;
    return fmaxf(old, s);
}

// Rows [first, off) of the page by `step` groups of eight lanes, each a row at a time, four in flight.
__device__ __forceinline__ void rescale_rows(const Run &r, float f, int first, int step) {
    uint4 *rows = reinterpret_cast<uint4 *>(r.rows) + (threadIdx.x & 7);
    if (!power_of_two(f)) {
#pragma unroll 1
        for (int j = first; j < r.off; j += step) {
            const uint4 v = rows[j * 8];
            rows[j * 8] = make_uint4(again4<true>(v.x, f), again4<true>(v.y, f), again4<true>(v.z, f), again4<true>(v.w, f));
        }
        return;
    }
    for (int j = first; j < r.off; j += 4 * step) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k * step < r.off) v[k] = rows[(j + k * step) * 8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k * step < r.off)
                rows[(j + k * step) * 8] = make_uint4(again4<false>(v[k].x, f), again4<false>(v[k].y, f), again4<false>(v[k].z, f), again4<false>(v[k].w, f));
    }
}

// Rows [j0, j0 + 16) of a run in a warp's registers, two rows a load; the loads
// are issued whether or not the rows turn out to be written.
struct Batch {
    uint4 v[kBatchRows / 2];
    unsigned live;                       // bit 2 k + half of a lane's half: row 2 k + half is written
};
__device__ __forceinline__ void batch_load(Batch &b, const uint8_t *x, int64_t x_t, int j0, int end) {
    const int half = (threadIdx.x >> 4) & 1;
#pragma unroll
    for (int k = 0; k < kBatchRows / 2; ++k)
        if (j0 + 2 * k + half < end) b.v[k] = *reinterpret_cast<const uint4 *>(x + (j0 + 2 * k + half) * x_t);
}
__device__ __forceinline__ void batch_live(Batch &b, const WriteParams &p, const int *slots, int j0, int n) {
    const int lane = threadIdx.x & 31;
    b.live = __ballot_sync(0xffffffffu, lane < kBatchRows && j0 + lane < n && written(p, slots[j0 + lane])) >> (lane >> 4);
}
template <bool BF>
__device__ __forceinline__ float batch_max(const Batch &b, float a) {
#pragma unroll
    for (int k = 0; k < kBatchRows / 2; ++k)
        if (b.live >> (2 * k) & 1) a = abs_max<BF>(b.v[k], a);
    return a;
}
template <bool BF>
__device__ __forceinline__ void batch_store(const Batch &b, const Run &r, int j0, float inv) {
    const int half = (threadIdx.x >> 4) & 1;
    uint8_t *dst = r.rows + (r.off + j0 + half) * 128 + (threadIdx.x & 15) * 8;
#pragma unroll
    for (int k = 0; k < kBatchRows / 2; ++k)
        if (b.live >> (2 * k) & 1) *reinterpret_cast<uint2 *>(dst + 2 * k * 128) = codes8<BF>(b.v[k], inv);
}
// The same over a scale that is no power of two: the rows are read again, so that the
// usual path keeps its registers.
template <bool BF>
__device__ __forceinline__ void batch_store_over(const uint8_t *x, int64_t x_t, unsigned live, const Run &r, int j0, float s) {
    const int half = (threadIdx.x >> 4) & 1;
    uint8_t *dst = r.rows + (r.off + j0 + half) * 128 + (threadIdx.x & 15) * 8;
#pragma unroll 1
    for (int k = 0; k < kBatchRows / 2; ++k)
        if (live >> (2 * k) & 1)
            *reinterpret_cast<uint2 *>(dst + 2 * k * 128) = codes8_over<BF>(*reinterpret_cast<const uint4 *>(x + (j0 + 2 * k + half) * x_t), s);
}

// How far the run that begins at slots[0] = s goes, at most `room` tokens.
__device__ __forceinline__ int run_length(const WriteParams &p, const int *slots, int s, int room) {
    const int lane = threadIdx.x & 31;
    int n = 1;
    while (n < room) {
        const int j = n + lane, at = j < room ? slots[j] : -1;
        const unsigned stop = __ballot_sync(0xffffffffu, j >= room || (written(p, at) && at != s + j));
        n += stop ? __ffs(stop) - 1 : 32;
        if (stop) break;
    }
    return n;
}

template <bool BF>
__global__ void __launch_bounds__(32 * kWriteWarps, 3) fmha_page_write_kernel(const WriteParams p) {
    __shared__ float s_max[2][kWriteWarps];
    const int c0 = blockIdx.x * kBatchRows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = 1 << p.shift;
    // where runs begin
    const int i = c0 + lane;
    const bool here = lane < kBatchRows && i < p.N;
    const int slot = here ? p.slots[i] : -1, before = here && i > 0 ? p.slots[i - 1] : -1;
    if (warp == 0 && blockIdx.y == 0 && slot >= p.slots_end) atomicCAS(&g_status, FMHA_OK, FMHA_ERR_INVALID_ARG);
    bool begins = written(p, slot);
    for (int j = 1; begins && j <= min(i, slot & (P - 1)); ++j) {
        const int other = j == 1 ? before : p.slots[i - j];
        if (other == slot - j) begins = false;               // of the same run
        else if (written(p, other)) break;
    }
    unsigned starts = __ballot_sync(0xffffffffu, begins);
    if (starts == 0) return;             // the same in every warp
    const int pair0 = blockIdx.y * p.pairs, pairs = min(p.pairs, 2 * p.H_k - pair0);
    // new rows of a pair, from a token on; selected, not indexed: an index would put the parameters into local memory
    auto rows_of = [&](int pair, int t, int64_t &x_t) {
        const int g = pair >> 1, kv = pair & 1;
        x_t = kv ? p.x_t[1] : p.x_t[0];
        return (kv ? p.x[1] + g * p.x_h[1] : p.x[0] + g * p.x_h[0]) + (c0 + t) * x_t + (lane & 15) * 16;
    };
    // the last run is the only one that can have more than 16 rows, which all warps then share
    const int last = 31 - __clz(starts), s_last = __shfl_sync(0xffffffffu, slot, last);
    const int room_last = min(P - (s_last & (P - 1)), p.N - (c0 + last));
    const int n_last = room_last > kBatchRows ? run_length(p, p.slots + c0 + last, s_last, room_last) : 0;
    const bool longer = n_last > kBatchRows;
    if (longer) starts &= ~(1u << last);
    const int items = __popc(starts) * pairs;
    for (int item = warp; item < items; item += kWriteWarps) {
        const int nth = item / pairs, pair = pair0 + item - nth * pairs;
        unsigned rest = starts;
        for (int k = 0; k < nth; ++k) rest &= rest - 1;
        const int t = __ffs(rest) - 1, s = __shfl_sync(0xffffffffu, slot, t);
        const int *slots = p.slots + c0 + t;
        const int room = min(min(P - (s & (P - 1)), p.N - (c0 + t)), kBatchRows);
        const Run r = run_of(p, s, pair >> 1, pair & 1);
        int64_t x_t;
        const uint8_t *x = rows_of(pair, t, x_t);
        Batch b;
        batch_load(b, x, x_t, 0, room);
        batch_live(b, p, slots, 0, run_length(p, slots, s, room));
        float old;
        const float sc = run_scale(r, warp_max(batch_max<BF>(b, 0.f)), old);
        if (r.off > 0 && sc > old) rescale_rows(r, old / sc, lane >> 3, 4);
        if (power_of_two(sc)) batch_store<BF>(b, r, 0, 1.f / sc);
        else batch_store_over<BF>(x, x_t, b.live, r, 0, sc);
        __syncwarp();
        if (lane == 0) *r.scale = sc;
    }
    if (!longer) return;
    // 16 rows a warp: two, four or eight warps a pair, and the other pairs beside it; the next ones' rows are
    // fetched ahead
    const int team = n_last <= 2 * kBatchRows ? 2 : n_last <= 4 * kBatchRows ? 4 : 8;
    const int sub = warp % team, first = warp - sub, j0 = sub * kBatchRows, abreast = kWriteWarps / team;
    Batch b;
    auto fetch = [&](int q) {
        if (q >= pairs) return;
        int64_t x_t;
        const uint8_t *x = rows_of(pair0 + q, last, x_t);
        batch_load(b, x, x_t, j0, n_last);
    };
    fetch(warp / team);
    batch_live(b, p, p.slots + c0 + last, j0, n_last);
    for (int q0 = 0, buf = 0; q0 < pairs; q0 += abreast, buf ^= 1) {
        const int q = q0 + warp / team;
        const bool on = q < pairs;       // the same in every warp of a team
        const Run r = run_of(p, s_last, (pair0 + (on ? q : 0)) >> 1, (pair0 + (on ? q : 0)) & 1);
        float a = warp_max(batch_max<BF>(b, 0.f)), old;
        if (lane == 0) s_max[buf][warp] = a;
        __syncthreads();
        for (int w = 0; w < team; ++w) a = fmaxf(a, s_max[buf][first + w]);
        const float sc = run_scale(r, a, old);
        if (on) {
            if (r.off > 0 && sc > old) rescale_rows(r, old / sc, sub * 4 + (lane >> 3), 4 * team);
            if (power_of_two(sc)) {
                batch_store<BF>(b, r, j0, 1.f / sc);
            } else {
                int64_t x_t;
                const uint8_t *x = rows_of(pair0 + q, last, x_t);
                batch_store_over<BF>(x, x_t, b.live, r, j0, sc);
            }
        }
        fetch(q + abreast);
        __syncthreads();                 // all have read the scale
        if (on && sub == 0 && lane == 0) *r.scale = sc;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int log2_page(int page_size) {
    for (int s = 4; s <= 7; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

}  // namespace

int *page_status_word() { return symbol_address(g_status); }

}  // namespace fmha

using namespace fmha;

extern "C" int fmha_page_plan(const int *seqlen, const int *n_new, const int *batch_idx, int *table, int *free_list,
                              const int *n_free, int *n_free_out, int *slots, int *positions, int *cu_new,
                              int *new_seqlen, int B, int N, int B_table, int max_pages, int n_pages, int page_size,
                              cudaStream_t stream) {
    const int shift = log2_page(page_size);
    if (B < 0 || N < 0 || shift < 0) return FMHA_ERR_INVALID_ARG;
    if (B == 0 && N == 0) return FMHA_OK;
    if (B == 0 || B_table <= 0 || max_pages <= 0 || n_pages <= 0 || max_pages > kMaxCacheRows >> shift ||
        n_pages > 0x7fffffff >> shift)
        return FMHA_ERR_INVALID_ARG;
    if (!seqlen || !n_new || !table || !free_list || !n_free || !n_free_out || !cu_new || !new_seqlen ||
        (N > 0 && (!slots || !positions)))
        return FMHA_ERR_INVALID_ARG;
    for (const void *ptr : {(const void *)seqlen, (const void *)n_new, (const void *)batch_idx, (const void *)table,
                            (const void *)free_list, (const void *)n_free, (const void *)n_free_out, (const void *)slots,
                            (const void *)positions, (const void *)cu_new, (const void *)new_seqlen})
        if (misaligned(ptr, 4)) return FMHA_ERR_INVALID_ARG;
    if (B > kPlanSeqs) return FMHA_ERR_UNSUPPORTED;
    const size_t seqs = (size_t)B * sizeof(int), rows = (size_t)N * sizeof(int);
    const Bytes out[7] = {{table, (size_t)B_table * max_pages * sizeof(int)}, {free_list, (size_t)n_pages * sizeof(int)},
                          {n_free_out, sizeof(int)}, {N ? slots : nullptr, rows}, {N ? positions : nullptr, rows},
                          {cu_new, seqs + sizeof(int)}, {new_seqlen, seqs}};
    // the lengths and the count of free pages may be their own outputs
    const Bytes in[4] = {{n_new, seqs}, {batch_idx, seqs}, {new_seqlen == seqlen ? nullptr : seqlen, seqs},
                         {n_free_out == n_free ? nullptr : n_free, sizeof(int)}};
    if (outputs_clash(out, in)) return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    PlanParams p{};
    p.seqlen = seqlen;
    p.n_new = n_new;
    p.batch_idx = batch_idx;
    p.n_free = n_free;
    p.table = table;
    p.free_list = free_list;
    p.n_free_out = n_free_out;
    p.slots = slots;
    p.positions = positions;
    p.cu_new = cu_new;
    p.new_seqlen = new_seqlen;
    p.B = B;
    p.N = N;
    p.entries = B_table;
    p.width = max_pages;
    p.shift = shift;
    p.cap = n_pages;
    p.job = N > 8 * kPlanThreads ? 4 : 1;
    const int smem = 6 * B * (int)sizeof(int);
    // always to the same: the kernel's limit is the process's, and a smaller call must not lower
    // it between another thread's setting and its launch
    if (smem > 47 * 1024 && cudaFuncSetAttribute(fmha_page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 6 * kPlanSeqs * (int)sizeof(int)) != cudaSuccess)
        return cuda_failed();
    cudaLaunchConfig_t cfg = {};
    // One CTA where every thread has a few jobs at most, of those that the host can count: 64 sequences of a
    // token 6.7 us with one and 6.8 with eight, with 8000 tokens more 18.6 and 8.1.  A cluster would be
    // faster from some 300 jobs on (300 single tokens 10.4 and 8.6), and where many pages come back (200
    // sequences, of which 100 end with up to 512 pages each: 25 and 9.8).
    const int ranks = N > 4 * kPlanThreads || B > kPlanThreads ? 8 : 1;
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fmha_page_plan_kernel, p) != cudaSuccess) return cuda_failed();
    return FMHA_OK;
}

extern "C" int fmha_page_write(fmha_tensor k_new, int64_t k_token_stride, int64_t k_head_stride, fmha_tensor v_new,
                               int64_t v_token_stride, int64_t v_head_stride, const int *slots, void *k_pages,
                               void *v_pages, float *k_scale, float *v_scale, int N, int H_k, int D, int n_pages,
                               int page_size, cudaStream_t stream) {
    const int shift = log2_page(page_size);
    if (N < 0 || H_k <= 0 || H_k > 65535 || D != kD || shift < 0) return FMHA_ERR_INVALID_ARG;
    if (N == 0) return FMHA_OK;
    if (n_pages <= 0 || n_pages > 0x7fffffff >> shift || !slots || !k_scale || !v_scale) return FMHA_ERR_INVALID_ARG;
    if (!k_new.data || !v_new.data || !k_pages || !v_pages) return FMHA_ERR_INVALID_ARG;
    const int dt = k_new.dtype;
    if ((dt != FMHA_F16 && dt != FMHA_BF16) || v_new.dtype != dt)
        return FMHA_ERR_UNSUPPORTED;
    for (const void *ptr : {(const void *)k_new.data, (const void *)v_new.data, (const void *)k_pages, (const void *)v_pages})
        if (misaligned(ptr, 16)) return FMHA_ERR_UNSUPPORTED;
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (s < 0 || s > (int64_t(1) << 40)) return FMHA_ERR_INVALID_ARG;
    // strides that are never stepped along do not count
    if ((N > 1 && (k_token_stride % 8 != 0 || v_token_stride % 8 != 0)) || (H_k > 1 && (k_head_stride % 8 != 0 || v_head_stride % 8 != 0)))
        return FMHA_ERR_UNSUPPORTED;
    if (misaligned(slots, 4) || misaligned(k_scale, 4) || misaligned(v_scale, 4)) return FMHA_ERR_INVALID_ARG;
    const size_t pages = ((size_t)n_pages * H_k << shift) * kD, scales = (size_t)n_pages * H_k * sizeof(float);
    const auto span = [&](int64_t t, int64_t h) { return (size_t)((N - 1) * t + (H_k - 1) * h + kD) * 2; };
    const Bytes out[4] = {{k_pages, pages}, {v_pages, pages}, {k_scale, scales}, {v_scale, scales}};
    const Bytes in[3] = {{k_new.data, span(k_token_stride, k_head_stride)}, {v_new.data, span(v_token_stride, v_head_stride)},
                         {slots, (size_t)N * sizeof(int)}};
    if (outputs_clash(out, in)) return FMHA_ERR_INVALID_ARG;
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    WriteParams p{};
    const fmha_tensor x[2] = {k_new, v_new};
    void *const c[2] = {k_pages, v_pages};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const uint8_t *>(x[i].data);
        p.x_t[i] = 2 * (i ? v_token_stride : k_token_stride);
        p.x_h[i] = 2 * (i ? v_head_stride : k_head_stride);
        p.pages[i] = static_cast<uint8_t *>(c[i]);
        p.scale[i] = i ? v_scale : k_scale;
    }
    p.slots = slots;
    p.N = N;
    p.H_k = H_k;
    p.shift = shift;
    p.slots_end = n_pages << shift;
    // Few tokens: as many CTAs as there are (head, K or V) pairs for every 16 of
    // them (64 single tokens of 8 heads: 4.7 us, two pairs a CTA 7.5, eight 24).  Many: a CTA's
    // warps share out the pairs, or a long run's rows (16600 tokens, 1 / 2 / 4 / 8 pairs: in pages
    // of 16 67 / 40 / 25.1 / 21.0, of 64 48 / 29.0 / 24.7 / 26.5, of 128 41 / 30.4 / 28.6 / 29.4).
    // Between the two the rule is not always the best: 1600 tokens 5.1 with its two pairs, in
    // pages of 16 3.6 with four; 3200 in pages of 128 13.3 with its four, 9.5 with two.
    const int64_t chunks = ((int64_t)N + kBatchRows - 1) / kBatchRows;
    p.pairs = chunks >= 2 * 152 ? (shift >= 6 ? 4 : 8) : chunks >= 152 ? 4 : chunks >= 76 ? 2 : 1;
    const dim3 grid((unsigned)chunks, (2 * H_k + p.pairs - 1) / p.pairs);
    if (grid.y > 65535) return FMHA_ERR_UNSUPPORTED;
    if (dt == FMHA_BF16) fmha_page_write_kernel<true><<<grid, 32 * kWriteWarps, 0, stream>>>(p);
    else fmha_page_write_kernel<false><<<grid, 32 * kWriteWarps, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FMHA_OK : FMHA_ERR_CUDA;
}
