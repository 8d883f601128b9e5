// Queries, keys and values of a sparse-attention (QSA) layer on their way to the attention:
// the per-head RMS norm and rotary encoding, written back as rows or straight into the paged
// key/value cache.
//
// Page "ARCHITECTURE PREVIEW / FIELD NOTES", section 01 (24 query heads, 2 key/value heads,
// head dim 256, 64 rotated dims) and section 03 (the attention runs on normalised, partially
// rotated heads).  Per head row x of D values at position p, r rotated dims:
//     n = x / sqrt(mean(x^2) + eps) * w
//     y_j = n_j cos a_j - n_{j+r/2} sin a_j,  y_{j+r/2} = n_{j+r/2} cos a_j + n_j sin a_j,
//     a_j = p theta^(-2j/r),  j < r/2;   y_j = n_j for j >= r
//
//   qsa_norm_rope_kernel  query and key heads, rows in, rows out
//   qsa_kv_append_kernel  key heads (as above) and value heads (copied) into cache pages
//
// Both are bound by memory at length and by latency for single tokens.  A head row is held by
// D / 8 lanes, 8 dims each: a rotated lane has 4 dims of the first half and their 4 partners of
// the second, so that a pair is turned without a shuffle; a warp reads whole 512-byte rows in two
// accesses.  A warp takes one token and several of its query or of its key heads, whose rows are
// in flight together and share the products of the weights with the token's sines and cosines.
#include <math.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace qsa_rows {

// Small blocks start and leave evenly: 8192 tokens 41.6 us (43.7 with 8 warps, 41.4 with 2), fp32 3 x
// 1001 12.0 (12.7, 12.7), append of 8192 tokens 11.4 (11.7, 11.9).
constexpr int kWarps = 4;
constexpr int kMaxPairs = 128;   // rotated pairs of a head: at most 256 / 2
struct Freq {
    double f[kMaxPairs];         // theta^(-2j/r) / (2 pi): turns per position
};

// cos and sin of the token's angles, one pair per lane in turn.  The angle is formed in turns and
// reduced to [-1/2, 1/2] of one in fp64 (positions reach 2^31), then rounded once to fp32.
__device__ __forceinline__ void token_angles(float2 *cs, int64_t pos, const Freq &fr, int half, int lane) {
    for (int j = lane; j < half; j += 32) {
        const double turns = (double)pos * fr.f[j];
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[j] = make_float2(c, s);
    }
}
// a / b and a % b for a >= 0, b > 0 (64-bit division takes some hundred instructions)
__device__ __forceinline__ int64_t div_mod(int64_t a, int b, int &rest) {
    if ((uint64_t)a >> 32 == 0) {
        const uint32_t q = (uint32_t)a / (uint32_t)b;
        rest = (int)((uint32_t)a - q * (uint32_t)b);
        return q;
    }
    rest = (int)(a % b);
    return a / b;
}

// 4 values as loaded, and 4 values stored
__device__ __forceinline__ float4 values(const float4 &r) { return r; }
__device__ __forceinline__ float4 values(const uint2 &r) {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ void st4(float *p, const float4 &x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void st4(bf16 *p, const float4 &x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// head rows of a lane group in flight together, as loaded: 32 (bf16) or 32 (fp32) registers
template <class T> struct In;
template <> struct In<float> {
    using raw = float4;
    static constexpr int ahead = 4;
};
template <> struct In<bf16> {
    using raw = uint2;
    static constexpr int ahead = 8;
};
template <class T> struct Row {
    typename In<T>::raw a, b;
    __device__ __forceinline__ void load(const T *p, int oa, int ob) {
        a = *reinterpret_cast<const typename In<T>::raw *>(p + oa);
        b = *reinterpret_cast<const typename In<T>::raw *>(p + ob);
    }
};

// Where a lane's two groups of 4 dims begin
__device__ __forceinline__ void lane_dims(int gl, int half, int &oa, int &ob) {
    const bool turned = 4 * gl < half;
    oa = turned ? 4 * gl : 8 * gl;
    ob = turned ? half + 4 * gl : 8 * gl + 4;
}
// Products of a lane's weights (1 without `w`) with the token's cosines and sines (1 and 0 for
// dims that are not rotated): y_a = (a ac - b bs) r,  y_b = (b bc + a as) r
struct Coef {
    float ac[4], as[4], bc[4], bs[4];
    __device__ __forceinline__ void set(const float *w, const float2 *cs, int gl, int half, int oa, int ob) {
        const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 a4 = w ? *reinterpret_cast<const float4 *>(w + oa) : one, b4 = w ? *reinterpret_cast<const float4 *>(w + ob) : one;
        const float wa[4] = {a4.x, a4.y, a4.z, a4.w}, wb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = 4 * gl < half ? cs[4 * gl + e] : make_float2(1.f, 0.f);
            ac[e] = wa[e] * t.x;
            as[e] = wa[e] * t.y;
            bc[e] = wb[e] * t.x;
            bs[e] = wb[e] * t.y;
        }
    }
};
// x c + y s with `turn`, else x c (y, which may be infinite or NaN, is another dim's alone)
__device__ __forceinline__ float turn_dim(float x, float c, float y, float s, bool turn) {
    float z = x * c;
    if (turn) z = fmaf(y, s, z);
    return z;
}
// Norm and rotation of one head row held by the D / 8 lanes of a group, of which those with `turn`
// hold rotated dims.  Every lane of the warp takes part.
template <int D>
__device__ __forceinline__ void norm_rope_row(float4 &a, float4 &b, const Coef &k, bool turn, bool norm, float eps) {
    float r = 1.f;
    if (norm) {
        float ss = a.x * a.x, st = b.x * b.x;
        ss = fmaf(a.y, a.y, ss);
        st = fmaf(b.y, b.y, st);
        ss = fmaf(a.z, a.z, ss);
        st = fmaf(b.z, b.z, st);
        ss = fmaf(a.w, a.w, ss) + fmaf(b.w, b.w, st);
#pragma unroll
        for (int o = D / 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss * (1.f / D) + eps);
    }
    const float4 x = a, y = b;
    a = make_float4(turn_dim(x.x, k.ac[0], -y.x, k.bs[0], turn) * r, turn_dim(x.y, k.ac[1], -y.y, k.bs[1], turn) * r,
                    turn_dim(x.z, k.ac[2], -y.z, k.bs[2], turn) * r, turn_dim(x.w, k.ac[3], -y.w, k.bs[3], turn) * r);
    b = make_float4(turn_dim(y.x, k.bc[0], x.x, k.as[0], turn) * r, turn_dim(y.y, k.bc[1], x.y, k.as[1], turn) * r,
                    turn_dim(y.z, k.bc[2], x.z, k.as[2], turn) * r, turn_dim(y.w, k.bc[3], x.w, k.as[3], turn) * r);
}

// ------------------------------------------------------------------ rows to rows
struct NormRopeParams {
    const void *q, *k;
    int64_t q_ld, k_ld;          // elements from one token to the next
    const float *w_q, *w_k;
    const int32_t *pos;
    void *q_out, *k_out;
    int64_t tokens;              // B * Tn
    int Tn, hq, hk, half;
    int per_warp, q_groups, groups;   // heads per warp, warps per token for its query heads and for all
    float eps;
    Freq fr;
};

template <class TI, class TO, int D>
__global__ void __launch_bounds__(32 * kWarps, 6) qsa_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    __shared__ __align__(16) float2 angles[kWarps][kMaxPairs];
    constexpr int G = D / 8, kSub = 32 / G, kAhead = In<TI>::ahead;       // rows a warp holds at once: kAhead * kSub
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (G - 1), sub = lane / G;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    int grp, t;
    const int64_t tok = div_mod(item, p.groups, grp);
    if (tok >= p.tokens) return;                          // whole warps leave together
    const int64_t b = div_mod(tok, p.Tn, t);
    const bool is_q = grp < p.q_groups;                   // uniform
    const int heads = is_q ? p.hq : p.hk, h0 = (is_q ? grp : grp - p.q_groups) * p.per_warp, h1 = min(heads, h0 + p.per_warp);
    const int64_t pos = (int64_t)p.pos[b] + t;
    int oa, ob;
    lane_dims(gl, p.half, oa, ob);
    const TI *in = static_cast<const TI *>(is_q ? p.q : p.k) + tok * (is_q ? p.q_ld : p.k_ld);
    TO *out = static_cast<TO *>(is_q ? p.q_out : p.k_out) + tok * heads * D;
    Row<TI> x[kAhead];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int hh = h + u * kSub + sub;
            if (hh < h1) x[u].load(in + hh * D, oa, ob);
        }
    };
    load(h0);
    const float *w = is_q ? p.w_q : p.w_k;
    token_angles(angles[warp], pos, p.fr, p.half, lane);
    __syncwarp();
    Coef k;
    k.set(w, angles[warp], gl, p.half, oa, ob);
    for (int h = h0;;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u * kSub >= h1) break;                // uniform
            const int hh = h + u * kSub + sub;
            float4 a = values(x[u].a), b = values(x[u].b);
            norm_rope_row<D>(a, b, k, 4 * gl < p.half, w != nullptr, p.eps);
            if (hh < h1) {
                st4(out + hh * D + oa, a);
                st4(out + hh * D + ob, b);
            }
        }
        h += kAhead * kSub;
        if (h >= h1) break;
        load(h);
    }
}

// ------------------------------------------------------------------ rows to cache pages
struct AppendParams {
    const void *k, *v;
    int64_t k_ld, v_ld;
    const float *w_k;
    const int32_t *pos, *n_new, *table;
    bf16 *k_cache, *v_cache;
    int64_t tokens;              // B * Tn
    int Tn, hk, half, max_pages, n_pages, page;
    int per_warp, k_groups, groups;   // heads per warp, warps per token for its key heads and for all
    float eps;
    Freq fr;
};

template <class TI, int D>
__global__ void __launch_bounds__(32 * kWarps, 8) qsa_kv_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ __align__(16) float2 angles[kWarps][kMaxPairs];
    constexpr int G = D / 8, kSub = 32 / G, kAhead = In<TI>::ahead / 2;   // few heads; registers for more warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (G - 1), sub = lane / G;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    int grp, t, slot;
    const int64_t tok = div_mod(item, p.groups, grp);
    if (tok >= p.tokens) return;
    const int64_t b = div_mod(tok, p.Tn, t);
    if (p.n_new && t >= p.n_new[b]) return;               // padding of a ragged batch
    const int64_t pos = (int64_t)p.pos[b] + t;
    if (pos < 0) return;
    const int64_t page = div_mod(pos, p.page, slot);
    if (page >= p.max_pages) return;
    const bool is_k = grp < p.k_groups;                   // uniform
    const int h0 = (is_k ? grp : grp - p.k_groups) * p.per_warp, h1 = min(p.hk, h0 + p.per_warp);
    int oa, ob;
    lane_dims(gl, is_k ? p.half : 0, oa, ob);
    const TI *in = static_cast<const TI *>(is_k ? p.k : p.v) + tok * (is_k ? p.k_ld : p.v_ld);
    Row<TI> x[kAhead];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int hh = h + u * kSub + sub;
            if (hh < h1) x[u].load(in + hh * D, oa, ob);
        }
    };
    load(h0);
    const int pg = p.table[b * p.max_pages + page];
    if (pg < 0 || pg >= p.n_pages) return;                // unmapped
    bf16 *out = (is_k ? p.k_cache : p.v_cache) + ((int64_t)pg * p.hk * p.page + slot) * D;
    Coef k;
    if (is_k) {
        token_angles(angles[warp], pos, p.fr, p.half, lane);
        __syncwarp();
        k.set(p.w_k, angles[warp], gl, p.half, oa, ob);
    }
    for (int h = h0;;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u * kSub >= h1) break;                // uniform
            const int hh = h + u * kSub + sub;
            float4 a = values(x[u].a), c = values(x[u].b);
            if (is_k) norm_rope_row<D>(a, c, k, 4 * gl < p.half, p.w_k != nullptr, p.eps);
            if (hh < h1) {
                st4(out + (int64_t)hh * p.page * D + oa, a);
                st4(out + (int64_t)hh * p.page * D + ob, c);
            }
        }
        h += kAhead * kSub;
        if (h >= h1) break;
        load(h);
    }
}

// An exponential for every 8th frequency, and products by the ratio of neighbours (at most 8
// roundings of 2^-53) in between
static void fill_freq(Freq &fr, int rope, float theta) {
    const double step = rope ? -2.0 / rope * log2((double)theta) : 0.0, ratio = exp2(step);
    for (int j = 0; j < rope / 2; ++j) fr.f[j] = j % 8 ? fr.f[j - 1] * ratio : exp2(j * step) / 6.283185307179586;
}

// Heads per warp: 8 lane groups' rows at length (one load of all, and blocks short enough to fill
// the SMs evenly), fewer when that leaves less than 16 warps per SM.
static int rows_per_warp(int64_t tokens, int rows, int sub) {
    const int64_t want = 148 * 16, per = std::max<int64_t>(1, tokens * rows / want);
    return (int)std::min<int64_t>((per + sub - 1) / sub, 8) * sub;
}

}  // namespace qsa_rows

// ------------------------------------------------------------------ launchers
cudaError_t launch_qsa_norm_rope(const void *q, const void *k, bool in_bf16, int64_t q_ld, int64_t k_ld,
                                 const float *w_q, const float *w_k, const int32_t *pos, int B, int Tn, int hq,
                                 int hk, int d, int rope, float eps, float theta, void *q_out, void *k_out,
                                 bool out_bf16, cudaStream_t s) {
    qsa_rows::NormRopeParams p{};
    p.q = q;
    p.k = k;
    p.q_ld = q_ld;
    p.k_ld = k_ld;
    p.w_q = w_q;
    p.w_k = w_k;
    p.pos = pos;
    p.q_out = q_out;
    p.k_out = k_out;
    p.tokens = (int64_t)B * Tn;
    p.Tn = Tn;
    p.hq = hq;
    p.hk = hk;
    p.half = rope / 2;
    p.eps = eps;
    p.per_warp = qsa_rows::rows_per_warp(p.tokens, hq + hk, 256 / d);
    p.q_groups = (hq + p.per_warp - 1) / p.per_warp;
    p.groups = p.q_groups + (hk + p.per_warp - 1) / p.per_warp;
    qsa_rows::fill_freq(p.fr, rope, theta);
    const int64_t grid = (p.tokens * p.groups + qsa_rows::kWarps - 1) / qsa_rows::kWarps;
    if (grid >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    TraceLaunch tl(s, "qsa_norm_rope");
#define GDN_NR(TI, TO)                                                                                    \
    do {                                                                                                  \
        if (d == 256)                                                                                     \
            qsa_rows::qsa_norm_rope_kernel<TI, TO, 256><<<(unsigned)grid, 32 * qsa_rows::kWarps, 0, s>>>(p); \
        else                                                                                              \
            qsa_rows::qsa_norm_rope_kernel<TI, TO, 128><<<(unsigned)grid, 32 * qsa_rows::kWarps, 0, s>>>(p); \
    } while (0)
    if (in_bf16) { if (out_bf16) GDN_NR(bf16, bf16); else GDN_NR(bf16, float); }
    else         { if (out_bf16) GDN_NR(float, bf16); else GDN_NR(float, float); }
#undef GDN_NR
    return cudaGetLastError();
}

cudaError_t launch_qsa_kv_append(const void *k, const void *v, bool in_bf16, int64_t k_ld, int64_t v_ld,
                                 const float *w_k, const int32_t *pos, const int32_t *n_new, int B, int Tn,
                                 const int32_t *table, int max_pages, int hk, int d, int rope, float eps,
                                 float theta, void *k_cache, void *v_cache, int n_pages, int page, cudaStream_t s) {
    qsa_rows::AppendParams p{};
    p.k = k;
    p.v = v;
    p.k_ld = k_ld;
    p.v_ld = v_ld;
    p.w_k = w_k;
    p.pos = pos;
    p.n_new = n_new;
    p.table = table;
    p.k_cache = static_cast<bf16 *>(k_cache);
    p.v_cache = static_cast<bf16 *>(v_cache);
    p.tokens = (int64_t)B * Tn;
    p.Tn = Tn;
    p.hk = hk;
    p.half = rope / 2;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.page = page;
    p.eps = eps;
    p.per_warp = qsa_rows::rows_per_warp(p.tokens, 2 * hk, 256 / d);
    p.k_groups = (hk + p.per_warp - 1) / p.per_warp;
    p.groups = 2 * p.k_groups;
    qsa_rows::fill_freq(p.fr, rope, theta);
    const int64_t grid = (p.tokens * p.groups + qsa_rows::kWarps - 1) / qsa_rows::kWarps;
    if (grid >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    TraceLaunch tl(s, "qsa_kv_append");
#define GDN_KV(TI)                                                                                        \
    do {                                                                                                  \
        if (d == 256)                                                                                     \
            qsa_rows::qsa_kv_append_kernel<TI, 256><<<(unsigned)grid, 32 * qsa_rows::kWarps, 0, s>>>(p);  \
        else                                                                                              \
            qsa_rows::qsa_kv_append_kernel<TI, 128><<<(unsigned)grid, 32 * qsa_rows::kWarps, 0, s>>>(p);  \
    } while (0)
    if (in_bf16) GDN_KV(bf16); else GDN_KV(float);
#undef GDN_KV
    return cudaGetLastError();
}

}  // namespace gdn
