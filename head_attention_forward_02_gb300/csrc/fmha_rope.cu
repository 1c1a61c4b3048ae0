// fmha_rope.cu -- rotary positions of queries and keys, and their gradient.
//
// Operation: the first `rot` elements of a head are rot / 2 pairs (x_a, x_b),
// (a, b) = (i, i + rot / 2) or (2 i, 2 i + 1), and the pair i of a token at
// position t is turned by the angle t * inv_freq[i] and stretched by m:
//   y_a = m (x_a cos - x_b sin),   y_b = m (x_b cos + x_a sin).
// The other elements are copied.  The gradient is the transpose, the turn by
// the opposite angle with the same m.
//
// The angle: what counts is the fraction of a turn t * f / (2 pi) mod 1, which
// fp32 loses for far positions (t = 2^20: half a radian's 2^-4).  f is taken
// apart into its 53-bit integer, multiplied by 2^66 / (2 pi) in 128 bits and
// kept as a 64-bit fraction of a turn, so that t * f mod 1 is one 64-bit
// integer product, off by 2^-31 of a turn at most for any position and any f
// below 2 pi (fp64 arithmetic would do, at two operations a cycle and SM).
//
// Bound by memory: every element is read and written once, and a token's
// rot / 2 sines and cosines serve all its heads, so a CTA takes TOK tokens with
// all heads and computes them once, under the loads of its elements, which
// are all issued first.  4 x 4096 tokens of 32 + 8 heads of 128: 52 us, 6.4 TB/s, 95%
// of the copy rate, to e4m3 46 us, 81%; the gradient of 8 x 2047 tokens of 16 + 16 heads of 64, half of each
// turned, 26 us, 76%; 32 single tokens 2.7 us, a launch.  Heads that cannot be read 16 bytes at a
// time are read element by element: 4 x 4096 tokens of 40 heads of 96, 24 of which are turned, 269 us
// where the bytes take 37 (32 turned: 52).
#include "fmha_cache.cuh"

namespace fmha {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTok = 8;              // tokens of a CTA at most
// items whose loads a thread has in flight: of two 16-byte pieces, or of one
constexpr int rope_batch(bool half) { return half ? 5 : 8; }

struct RopeTensor {
    const uint8_t *in;
    uint8_t *out;
    int64_t in_b, in_t, in_h, out_b, out_t, out_h;   // strides in elements
};

struct RopeParams {
    RopeTensor x[2];                     // q, k
    const int *positions;                // [B, S], or NULL: the token's index in its sequence
    const double *inv_freq;              // [rot / 2]
    int64_t tokens;                      // B * S
    int S, H, heads, D, rot;             // heads: of q and k together
    int chunks;                          // work items of a head
    int tok;                             // tokens of a CTA
    uint32_t magic;                      // i / heads is the high word of i * magic, for 8 * 512 items (one head: 0)
    float magnitude, sign;
    int in_place[2];
};

// 2^64 * (f / (2 pi) mod 1)
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr uint64_t kInv2Pi = 0xA2F9836E4E441529ull;      // floor(2^66 / (2 pi))
    const uint64_t u = (uint64_t)__double_as_longlong(f);
    const int ex = (int)((u >> 52) & 0x7ff);
    const uint64_t m = ex ? (u & 0xfffffffffffffull) | 0x10000000000000ull : 0;   // subnormal: 0
    const int sh = 2 + 1075 - ex;                            // f = m 2^(ex - 1075)
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    uint64_t r;
    if (sh <= 0) r = sh > -64 ? lo << -sh : 0;
    else if (sh < 64) r = (lo >> sh) | (hi << (64 - sh));
    else r = sh < 128 ? hi >> (sh - 64) : 0;
    return u >> 63 ? 0 - r : r;
}

template <bool BF>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Eight elements to the output type
template <bool BF, bool FP8>
__device__ __forceinline__ void store8(uint8_t *dst, const float (&y)[8]) {
    if constexpr (FP8) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
    } else {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<BF>(y[0], y[1]), pack2<BF>(y[2], y[3]), pack2<BF>(y[4], y[5]),
                                                     pack2<BF>(y[6], y[7]));
    }
}

template <bool BF>
__device__ __forceinline__ float load1(const uint8_t *p) {
    const uint32_t w = *reinterpret_cast<const uint16_t *>(p);
    return widen2<BF>(w).x;
}
template <bool BF, bool FP8>
__device__ __forceinline__ void store1(uint8_t *p, float y) {
    if constexpr (FP8) *p = (uint8_t)pack4_e4m3(y, 0.f, 0.f, 0.f);
    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)pack2<BF>(y, 0.f);
}

// VEC: 16-byte accesses.  A work item is then, of one head, eight pairs (HALF:
// eight elements of either half, else four pairs, eight elements in a row) or
// eight elements behind `rot`; without VEC it is one pair or one element.
template <bool BF, bool FP8, bool HALF, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, 3) fmha_rope_kernel(const RopeParams p) {
    constexpr int kBatch = rope_batch(HALF);
    extern __shared__ __align__(16) float2 cs[];             // of the CTA's tokens, cosine and sine of every pair
    __shared__ int pos[kRopeTok];
    __shared__ int64_t base_in[2][kRopeTok], base_out[2][kRopeTok];   // where a token's heads begin, by tensor
    const int64_t first = (int64_t)blockIdx.x * p.tok;
    const int ntok = (int)min((int64_t)p.tok, p.tokens - first);
    const int items = ntok * p.heads, half = p.rot >> 1;
    const int c = threadIdx.x, rows = blockDim.y;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
    constexpr int W = VEC ? 8 : 1, PAIRS = !VEC ? 1 : HALF ? 8 : 4;   // elements, pairs of an item
    const int turned = half / PAIRS;                         // items of a head that are turned
    const bool turn = c < turned;
    const int a = turn ? (HALF || VEC ? c * W : 2 * c) : p.rot + (c - turned) * W;   // first element
    if (tid < ntok) {
        const uint32_t n = (uint32_t)first + tid, b = n / (uint32_t)p.S, s = n - b * p.S;
        pos[tid] = p.positions ? p.positions[n] : (int)s;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            base_in[w][tid] = b * p.x[w].in_b + s * p.x[w].in_t;
            base_out[w][tid] = b * p.x[w].out_b + s * p.x[w].out_t;
        }
    }
    __syncthreads();
    // an item's token, tensor and head
    auto place = [&](int i, int &t, int &h) -> bool {
        t = p.tok == 1 ? 0 : p.magic ? (int)__umulhi(i, p.magic) : i;
        h = i - t * p.heads;
        const bool key = h >= p.H;
        if (key) h -= p.H;
        return key;
    };
    bool ready = false;
    for (int i0 = threadIdx.y; i0 < items || !ready; i0 += kBatch * rows) {
        uint4 u[kBatch], v[kBatch];
        float fu[kBatch], fv[kBatch];
        unsigned todo = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * rows;
            if (i >= items) continue;
            int t, h;
            const bool key = place(i, t, h);
            if ((!turn && (key ? p.in_place[1] : p.in_place[0])) || pos[t] < 0) continue;   // pos < 0: a row without a position
            todo |= 1u << k;
            const uint8_t *src = (key ? p.x[1].in : p.x[0].in) + (base_in[key][t] + h * (key ? p.x[1].in_h : p.x[0].in_h) + a) * 2;
            if constexpr (VEC) {
                u[k] = *reinterpret_cast<const uint4 *>(src);
                if (HALF && turn) v[k] = *reinterpret_cast<const uint4 *>(src + half * 2);
            } else {
                fu[k] = load1<BF>(src);
                if (turn) fv[k] = load1<BF>(src + (HALF ? half * 2 : 2));
            }
        }
        if (!ready) {                                        // under the first loads
            ready = true;
            for (int x = tid; x < ntok * half; x += nthr) {
                const int t = x / half, f = x - t * half;
                const uint64_t phase = (uint64_t)(int64_t)pos[t] * turn_fraction(p.inv_freq[f]);
                float s, co;
                sincospif((float)(int64_t)phase * 0x1p-63f, &s, &co);
                // two pairs of every item side by side, so that a load's threads read a row of them
                const int at = VEC ? (((f % PAIRS) >> 1) * turned + f / PAIRS) * 2 + (f & 1) : f;
                cs[t * half + at] = make_float2(co * p.magnitude, s * p.magnitude * p.sign);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!(todo >> k & 1)) continue;
            int t, h;
            const bool key = place(i0 + k * rows, t, h);
            uint8_t *dst = (key ? p.x[1].out : p.x[0].out) +
                           (base_out[key][t] + h * (key ? p.x[1].out_h : p.x[0].out_h) + a) * (FP8 ? 1 : 2);
            if constexpr (VEC) {
                if (!FP8 && !turn) {     // behind rot: as they are
                    *reinterpret_cast<uint4 *>(dst) = u[k];
                    continue;
                }
                const float4 *w = reinterpret_cast<const float4 *>(cs + t * half) + c;
                const uint32_t uu[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                float y[8], z[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = widen2<BF>(uu[j]);
                    y[2 * j] = x.x;
                    y[2 * j + 1] = x.y;
                }
                if (HALF && turn) {
                    const uint32_t vv[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = widen2<BF>(vv[j]);
                        const float4 cc = w[j * turned];
                        const float y0 = y[2 * j], y1 = y[2 * j + 1];
                        y[2 * j] = y0 * cc.x - x.x * cc.y;
                        z[2 * j] = x.x * cc.x + y0 * cc.y;
                        y[2 * j + 1] = y1 * cc.z - x.y * cc.w;
                        z[2 * j + 1] = x.y * cc.z + y1 * cc.w;
                    }
                    store8<BF, FP8>(dst + half * (FP8 ? 1 : 2), z);
                } else if (turn) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 cc = w[j * turned];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float x0 = y[4 * j + 2 * q], x1 = y[4 * j + 2 * q + 1], co = q ? cc.z : cc.x, s = q ? cc.w : cc.y;
                            y[4 * j + 2 * q] = x0 * co - x1 * s;
                            y[4 * j + 2 * q + 1] = x1 * co + x0 * s;
                        }
                    }
                }
                store8<BF, FP8>(dst, y);
            } else {
                if (turn) {
                    const float2 cc = cs[t * half + c];
                    store1<BF, FP8>(dst, fu[k] * cc.x - fv[k] * cc.y);
                    store1<BF, FP8>(dst + (HALF ? half : 1) * (FP8 ? 1 : 2), fv[k] * cc.x + fu[k] * cc.y);
                } else {
                    store1<BF, FP8>(dst, fu[k]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side: tensors [B, S, heads, D] with strides
// ---------------------------------------------------------------------------

struct Strides {
    int64_t batch, token, head;
};

struct Extent {
    int64_t size, stride;
};

// The tensor's dimensions of more than one element, outermost last.
int extents(const Strides &s, int B, int S, int heads, Extent (&d)[3]) {
    const Extent all[3] = {{heads, s.head}, {S, s.token}, {B, s.batch}};
    int n = 0;
    for (const Extent &e : all) {
        if (e.size <= 1) continue;
        int at = n++;
        for (; at > 0 && d[at - 1].stride > e.stride; --at) d[at] = d[at - 1];
        d[at] = e;
    }
    return n;
}

// No two elements at one place?
bool writable(const Strides &s, int B, int S, int heads, int D) {
    Extent d[3];
    const int n = extents(s, B, S, heads, d);
    int64_t span = D;
    for (int i = 0; i < n; ++i) {
        if (d[i].stride < span) return false;
        span = d[i].stride * (d[i].size - 1) + span;
    }
    return true;
}

int64_t span_elements(const Strides &s, int B, int S, int heads, int D) {
    return (B - 1) * s.batch + (S - 1) * s.token + (heads - 1) * s.head + D;
}

struct View {
    const void *p;
    Strides s;
    int heads, E;                        // E: bytes of an element
};

bool same(const View &a, const View &b, int B, int S) {
    return a.p == b.p && a.E == b.E && a.heads == b.heads && (a.heads == 1 || a.s.head == b.s.head) &&
           (S == 1 || a.s.token == b.s.token) && (B == 1 || a.s.batch == b.s.batch);
}

// May two views share an element?  Apart as a whole, or pieces of the same
// tokens (as of one projection's rows) that lie side by side.
bool may_share(const View &a, const View &b, int B, int S, int D) {
    if (!a.p || !b.p) return false;
    const int64_t na = span_elements(a.s, B, S, a.heads, D) * a.E, nb = span_elements(b.s, B, S, b.heads, D) * b.E;
    if (!overlap(a.p, (size_t)na, b.p, (size_t)nb)) return false;
    if (a.E != b.E) return true;
    const int64_t ts = S > 1 ? a.s.token : B > 1 ? a.s.batch : 0;     // distance of a token's pieces
    if (ts <= 0 || (S > 1 && a.s.token != b.s.token) ||
        (B > 1 && (a.s.batch != b.s.batch || a.s.batch % ts != 0)))
        return true;
    const int64_t ea = (a.heads - 1) * a.s.head + D, eb = (b.heads - 1) * b.s.head + D;
    const int64_t bytes = static_cast<const uint8_t *>(b.p) - static_cast<const uint8_t *>(a.p);
    if (bytes % a.E != 0) return true;
    const int64_t delta = ((bytes / a.E) % ts + ts) % ts;
    return !(delta >= ea && ts - delta >= eb);
}

template <bool BF, bool FP8>
void rope_launch(const RopeParams &p, bool half, bool vec, dim3 grid, dim3 block, int smem, cudaStream_t stream) {
    auto kern = half ? (vec ? fmha_rope_kernel<BF, FP8, true, true> : fmha_rope_kernel<BF, FP8, true, false>)
                     : (vec ? fmha_rope_kernel<BF, FP8, false, true> : fmha_rope_kernel<BF, FP8, false, false>);
    kern<<<grid, block, smem, stream>>>(p);
}

}  // namespace
}  // namespace fmha

using namespace fmha;

extern "C" int fmha_rope(fmha_tensor q, int64_t q_b, int64_t q_t, int64_t q_h, fmha_tensor k, int64_t k_b, int64_t k_t,
                         int64_t k_h, fmha_tensor q_out, int64_t q_out_b, int64_t q_out_t, int64_t q_out_h,
                         fmha_tensor k_out, int64_t k_out_b, int64_t k_out_t, int64_t k_out_h, int B, int S, int H,
                         int H_k, int D, int rot, const int *positions, const double *inv_freq, float magnitude,
                         int layout, int transpose, cudaStream_t stream) {
    if (B < 0 || S < 0 || H < 0 || H_k < 0 || H + (int64_t)H_k > 65535 || D <= 0 || D > FMHA_ROPE_MAX_DIM || rot <= 0 ||
        rot > D || rot % 2 != 0)
        return FMHA_ERR_INVALID_ARG;
    if (layout != FMHA_ROPE_HALF && layout != FMHA_ROPE_PAIRS) return FMHA_ERR_INVALID_ARG;
    if (!(magnitude == magnitude) || magnitude == INFINITY || magnitude == -INFINITY) return FMHA_ERR_INVALID_ARG;
    if (B == 0 || S == 0 || H + H_k == 0) return FMHA_OK;
    if ((int64_t)B * S >= (int64_t(1) << 31) || !inv_freq || misaligned(inv_freq, 8) || misaligned(positions, 4))
        return FMHA_ERR_INVALID_ARG;
    const fmha_tensor in[2] = {q, k}, out[2] = {q_out, k_out};
    const Strides si[2] = {{q_b, q_t, q_h}, {k_b, k_t, k_h}};
    const Strides so[2] = {{q_out_b, q_out_t, q_out_h}, {k_out_b, k_out_t, k_out_h}};
    const int heads[2] = {H, H_k};
    View vi[2] = {}, vo[2] = {};
    RopeParams p{};
    int dt = -1, odt = -1;
    bool vec = D % 8 == 0 && rot % (layout == FMHA_ROPE_HALF ? 16 : 8) == 0;
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        if (!in[i].data || !out[i].data) return FMHA_ERR_INVALID_ARG;
        if (dt < 0) {
            dt = in[i].dtype;
            odt = out[i].dtype;
        }
        if ((dt != FMHA_F16 && dt != FMHA_BF16) || (odt != dt && odt != FMHA_E4M3) || in[i].dtype != dt || out[i].dtype != odt)
            return FMHA_ERR_UNSUPPORTED;
        const int oe = odt == FMHA_E4M3 ? 1 : 2;
        if (misaligned(in[i].data, 2) || misaligned(out[i].data, oe)) return FMHA_ERR_UNSUPPORTED;
        for (const Strides &s : {si[i], so[i]})
            for (int64_t v : {s.batch, s.token, s.head})
                if (v < 0 || v > (int64_t(1) << 40)) return FMHA_ERR_INVALID_ARG;
        if (!writable(so[i], B, S, heads[i], D)) return FMHA_ERR_INVALID_ARG;
        vi[i] = {in[i].data, si[i], heads[i], 2};
        vo[i] = {out[i].data, so[i], heads[i], oe};
        p.in_place[i] = same(vi[i], vo[i], B, S);
        p.x[i] = {static_cast<const uint8_t *>(in[i].data), static_cast<uint8_t *>(out[i].data), si[i].batch, si[i].token,
                  si[i].head, so[i].batch, so[i].token, so[i].head};
        // 16-byte accesses (8-byte stores of e4m3); strides that are never stepped along do not count
        const auto odd = [&](const Strides &s) {
            return (B > 1 && s.batch % 8 != 0) || (S > 1 && s.token % 8 != 0) || (heads[i] > 1 && s.head % 8 != 0);
        };
        vec = vec && !misaligned(in[i].data, 16) && !misaligned(out[i].data, 8 * oe) && !odd(si[i]) && !odd(so[i]);
    }
    // an output is its own input, or apart from everything
    const Bytes lists[2] = {{positions, (size_t)B * S * sizeof(int)}, {inv_freq, (size_t)rot / 2 * sizeof(double)}};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        const size_t n = (size_t)span_elements(so[i], B, S, heads[i], D) * vo[i].E;
        for (const Bytes &l : lists)
            if (overlap(Bytes{vo[i].p, n}, l)) return FMHA_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j) {
            if (heads[j] == 0) continue;
            if (!(i == j && p.in_place[i]) && may_share(vo[i], vi[j], B, S, D)) return FMHA_ERR_INVALID_ARG;
            if (i < j && may_share(vo[i], vo[j], B, S, D)) return FMHA_ERR_INVALID_ARG;
        }
    }
    const int rc = check_device();
    if (rc != FMHA_OK) return rc;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.tokens = (int64_t)B * S;
    p.S = S;
    p.H = H;
    p.heads = H + H_k;
    p.D = D;
    p.rot = rot;
    p.magnitude = magnitude;
    p.sign = transpose ? -1.f : 1.f;
    const bool half = layout == FMHA_ROPE_HALF;
    p.chunks = vec ? (half ? rot / 16 : rot / 8) + (D - rot) / 8 : rot / 2 + (D - rot);
    const dim3 block(p.chunks, p.chunks >= kRopeThreads ? 1 : kRopeThreads / p.chunks);
    // Many tokens: as many a CTA as its threads take in one batch of loads (a CTA
    // of 4 tokens of 32 heads of 64, 16 bytes a thread and item, 4 items, took 27.9 us
    // for 16376 tokens; 16384 of 40 heads of 128, 4 a CTA by this rule, 52 us, one a CTA 71).  Few: a CTA
    // each (32 tokens 2.7 us, two a CTA 3.0, eight 6.3), which from some 500 on is not the best any
    // more (1024 tokens 6.6 us, two a CTA 5.7, four 5.1).
    const int fill = rope_batch(half) * (int)block.y / p.heads;
    p.tok = p.tokens < 4 * 4 * 152 || p.heads > 512 ? 1 : fill < 1 ? 1 : fill > kRopeTok ? kRopeTok : fill;
    p.magic = p.heads > 1 ? (uint32_t)(((uint64_t(1) << 32) + p.heads - 1) / p.heads) : 0;
    const dim3 grid((unsigned)((p.tokens + p.tok - 1) / p.tok));
    const int smem = p.tok * (rot / 2) * (int)sizeof(float2);
    if (dt == FMHA_BF16) {
        if (odt == FMHA_E4M3) rope_launch<true, true>(p, half, vec, grid, block, smem, stream);
        else rope_launch<true, false>(p, half, vec, grid, block, smem, stream);
    } else {
        if (odt == FMHA_E4M3) rope_launch<false, true>(p, half, vec, grid, block, smem, stream);
        else rope_launch<false, false>(p, half, vec, grid, block, smem, stream);
    }
    return cudaGetLastError() == cudaSuccess ? FMHA_OK : FMHA_ERR_CUDA;
}
