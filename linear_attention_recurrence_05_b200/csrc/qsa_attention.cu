// Attention of a sparse-attention (QSA) layer over the selected blocks of the paged key/value
// cache: the entry point's launcher, and the kernel for single queries.
//
// Page "ARCHITECTURE PREVIEW / FIELD NOTES", section 03 (exact attention over the selected
// tokens; CAUSAL SPARSE SET) and section 01 (24 query heads, 2 key/value heads, head dim 256,
// budget 512 blocks of 4 tokens).  Query i with heads h reading key/value head h / group:
//     S_i = tokens of its listed complete blocks, then 4 floor((i+1)/4) .. i
//     o_h = sum_{t in S_i} e^{s_ht - m_h} v_t / sum_{t in S_i} e^{s_ht - m_h},  s_ht = scale <q_h, k_t>
// in one pass over S_i with a running reference m_h and sum.
//
// A unit is (query, key/value head): its up to 16 query heads share the gathered rows, and its
// list may be divided over the CTAs of a cluster, which join their partial results over shared
// memory.  The products are taken transposed, so that the many tokens fill the 128 rows of an
// MMA and the few heads are its columns:
//     S^T [128 tokens x 16] = K Q^T,   O^T [D x 16] += V^T P^T.
// Both K (K-major) and V (MN-major) are used in the same shared-memory image, 128-byte rows of
// 64 dims, swizzled, which 16-byte asynchronous copies write straight from cache rows.
//
// One CTA per SM: warps 0-7 softmax and output (warp w: TMEM lanes 32 (w % 4).., one token or
// output dim per thread; column half w / 4), warp 8 issues the MMAs, warps 9-12 gather.
// 32 KB stages (128 tokens x 128 dims of K or V) pass through a ring, ordered K0 K1 V0 K2 V1 ..:
// the scores of tile t + 1 are taken while the softmax of tile t runs.
//
// Bound by latency for a single token (128K tokens, 24 over 2 heads of 256: 9.9 us over 2 x 16 CTAs,
// 12.5 over 2 x 8, of which the launch 2.5; the chain is list, page table, first keys, two products,
// join), by HBM for some rows of a few tokens (16 x 4 at 32K: 39 us, 5 TB/s of distinct rows).  An MMA
// of 16 columns takes 45 clk, not 8; transposed the other way round (heads on the 128 rows) one of 64
// tokens takes as long, so that a tile would take as many again.
#include <algorithm>
#include <array>
#include <cmath>

#include "qsa_attn.cuh"

namespace gdn {
namespace qsa_attn {

constexpr int kTile = 128;                   // tokens per tile (MMA rows)
constexpr int kTileBlocks = kTile / kR;
constexpr int NC = 16, NCW = NC / 2;         // MMA columns: query heads, padded; those of a softmax thread
constexpr int kMaxRing = 6;
constexpr int kMaxSplit = 16;                // CTAs of a cluster (above 8 with the function's consent)
constexpr uint32_t kStage = 32768;           // 128 tokens x 128 dims, bf16
constexpr uint32_t kChunk64 = kTile * 128;   // 128 tokens x 64 dims
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp0 = 9, kLoadWarps = 4;
constexpr int kThreads = 32 * (kLoadWarp0 + kLoadWarps);
constexpr uint32_t kTmemS = 0, kTmemO = 2 * NC, kTmemCols = 64;   // S^T double-buffered, then O^T halves

enum { BAR_FULL = 0, BAR_EMPTY = kMaxRing, BAR_S = 2 * kMaxRing, BAR_P = BAR_S + 2, BAR_PV, BAR_DRAIN, kNumBars };

// Shared memory: the ring, Q [D/64 chunks][16 rows][128 B], P [2 chunks][16 rows][128 B], then
struct Fixed {
    float red[kSoftWarps][NCW];              // column maxima / sums of the warps
    float m[NC], l[NC];                      // the columns' reference and sum (split: read by the cluster's CTAs)
    uint64_t bar[kNumBars];
    uint32_t tmem;
    int abort_flag, len, tail_row;
};
// then the cache row of each listed block, or -1
__host__ __device__ constexpr uint32_t smem_bytes(int D, int ring, int entries) {
    return (uint32_t)ring * kStage + NC * D * 2 + NC * kTile * 2 + (uint32_t)((sizeof(Fixed) + 15) & ~15) +
           (uint32_t)entries * 4;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// fp32 at the same shared-memory offset of CTA `rank` of the cluster
__device__ __forceinline__ float ld_peer(uint32_t saddr, uint32_t rank) {
    float r;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(r) : "r"(saddr), "r"(rank) : "memory");
    return r;
}
// 8 consecutive columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld8(uint32_t a, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) qsa_attention_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(1024) unsigned char sm[];
    constexpr int NST = D / 128;                         // stages per tile of K (and of V)
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);             // (uniform for the compiler)
    const uint32_t unit = p.split > 1 ? blockIdx.x / (uint32_t)p.split : blockIdx.x;
    const int rank = p.split > 1 ? (int)(blockIdx.x % (uint32_t)p.split) : 0;
    const uint32_t rows = (uint32_t)p.B * (uint32_t)p.Qn;
    const int kvh = (int)(unit / rows);                  // key/value head slowest: half the cache at a time in L2
    const int64_t row = unit % rows;
    const int b = (int)row / p.Qn, n = (int)row % p.Qn;
    const int64_t pos = (int64_t)p.qpos[b] + n;
    const bool live = pos >= 0 && (!p.n_query || n < p.n_query[b]);
    const int64_t ncomp = live ? (pos + 1) >> 2 : 0;     // complete blocks; the next one is the tail
    const int tail_n = live && rank == p.split - 1 ? (int)((pos + 1) & 3) : 0;

    unsigned char *sq = sm + (uint32_t)p.ring * kStage, *sp = sq + NC * D * 2;
    Fixed &fx = *reinterpret_cast<Fixed *>(sp + NC * kTile * 2);
    int *tab = reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(&fx) + ((sizeof(Fixed) + 15) & ~15));
    uint64_t *bar = fx.bar;
    volatile int *abort_flag = &fx.abort_flag;

    // this CTA's share of the list (whole tiles); the first entry of each thread and the query heads are
    // on their way while the block starts
    const int32_t *table = p.table + (int64_t)b * p.max_pages, *list = p.blocks + row * p.n_slots;
    const int per = ((p.n_slots + kTileBlocks - 1) / kTileBlocks + p.split - 1) / p.split * kTileBlocks;
    const int s0 = min(p.n_slots, rank * per), s1 = min(p.n_slots, s0 + per);
    int blk = s0 + tid < s1 ? __ldg(list + s0 + tid) : -1;
    constexpr int kQ = NC * (D / 8) / (32 * kSoftWarps);
    uint4 qv[kQ];
    if (warp < kSoftWarps) {
        const __nv_bfloat16 *q = p.q + (row * p.hq + (int64_t)kvh * p.group) * D;
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            const int i = tid + u * 32 * kSoftWarps;
            qv[u] = i / (D / 8) < p.group ? __ldg(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (tid == 0) {
        for (int s = 0; s < p.ring; ++s) {
            mbar_init(&bar[BAR_FULL + s], 32 * kLoadWarps);
            mbar_init(&bar[BAR_EMPTY + s], 1);
        }
        mbar_init(&bar[BAR_S], 1);
        mbar_init(&bar[BAR_S + 1], 1);
        mbar_init(&bar[BAR_P], 32 * kSoftWarps);
        mbar_init(&bar[BAR_PV], 1);
        mbar_init(&bar[BAR_DRAIN], 1);
        fx.abort_flag = 0;
        fx.len = 0;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&fx.tmem, kTmemCols);
        tmem_relinquish();
    }
    __syncthreads();

    // the list as cache rows, skipped entries left as holes; the query heads as the B operand, P's
    // unused rows zero
    {
        int last = 0;
        for (int e = s0 + tid; e < s1; e += kThreads, blk = e < s1 ? __ldg(list + e) : -1) {
            const int r = blk >= 0 && blk < ncomp ? block_row(p, table, (uint32_t)blk, kvh) : -1;
            tab[e - s0] = r;
            if (r >= 0) last = e - s0 + 1;
        }
        if (last) atomicMax(&fx.len, last);
        if (tid == 0) fx.tail_row = tail_n ? block_row(p, table, (uint32_t)ncomp, kvh) : -1;
        if (warp < kSoftWarps) {
#pragma unroll
            for (int u = 0; u < kQ; ++u) {
                const int i = tid + u * 32 * kSoftWarps, r = i / (D / 8), c = i % (D / 8);
                *reinterpret_cast<uint4 *>(sq + (c >> 3) * (NC * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = qv[u];
            }
            for (int i = tid; i < NC * kTile * 2 / 16; i += 32 * kSoftWarps)
                *reinterpret_cast<uint4 *>(sp + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
            fence_smem_to_async();
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, fx.tmem, 0);
    const int len = fx.len, tail_row = fx.tail_row;
    const int nt = __shfl_sync(0xffffffffu, (len + (tail_row >= 0 ? 1 : 0) + kTileBlocks - 1) / kTileBlocks, 0);
    // cache row of token r (0..3) of list entry e, or -1
    auto token_row = [&](int e, int r) {
        const int x = e < len ? tab[e] : e == len && r < tail_n ? tail_row : -1;
        return x < 0 ? -1 : x + r;
    };

    if (warp >= kLoadWarp0) {
        // ================================================================ gather
        // A stage is declared full by its copies themselves (an arrival per thread once they have landed).
        // The copies' shared addresses differ by constants from 4 per lane, and their sources from one per block.
        constexpr int E = kTileBlocks / kLoadWarps;       // blocks of a warp: 32 rows of a tile, two a copy
        const int wl = warp - kLoadWarp0, c = lane & 15, hi = lane >> 4;
        uint32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            at[i] = smem_u32(sm) + (uint32_t)(c >> 3) * kChunk64 + (uint32_t)(wl * 32 + hi) * 128 + (uint32_t)(((c & 7) ^ (2 * i + hi)) << 4);
        int issued = 0, slot = 0;
        uint32_t par = 1;                                 // of the slot's last release
        bool ok = true;
        for (int u = 0; ok && nt > 0 && u < 2 * nt + 2; ++u) {            // K(0) K(1) V(0) K(2) V(1) ..
            const int t = (u >> 1) - (u & 1);
            if (t < 0 || t >= nt) continue;
            const char *src[E];
            int live[E];                                  // tokens of the block that this lane's rows may hold
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = t * kTileBlocks + wl * E + e, x = i < len ? tab[i] : i == len ? tail_row : -1;
                src[e] = reinterpret_cast<const char *>((u & 1 ? p.vc : p.kc) + ((int64_t)max(x, 0) + hi) * D + c * 8);
                live[e] = x < 0 ? 0 : (i < len ? kR : tail_n) - hi;
            }
            for (int st = 0; ok && st < NST; ++st) {
                ok = __all_sync(0xffffffffu, issued < p.ring || wait_abort(&bar[BAR_EMPTY + slot], par, abort_flag));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 16; ++i)              // tile row wl * 32 + 2 i + hi
                    cp_async16_sized(at[i & 3] + (uint32_t)slot * kStage + i * 256, src[i / 2] + st * 256 + (i & 1) * (4 * D),
                                     (i & 1) * 2 < live[i / 2] ? 16 : 0);
                cp_async_arrive(&bar[BAR_FULL + slot]);
                ++issued;
                if (++slot == p.ring) {
                    slot = 0;
                    par ^= 1;
                }
            }
        }
        cp_async_wait_all();
    } else if (warp == kMmaWarp) {
        // ================================================================ MMA issuer
        // the whole warp walks through the tiles (descriptors stay in uniform registers), one lane issues
        constexpr uint32_t id_s = idesc_attn(kTile, NC, false, false), id_o = idesc_attn(128, NC, true, false);
        const uint32_t ring = smem_u32(sm);
        const uint64_t qd = smem_desc(smem_u32(sq), 16, 1024, 2);
        const uint64_t pd = smem_desc(smem_u32(sp), 16, 1024, 2);
        const bool lead = elect_one();
        int slot = 0;
        uint32_t par = 0;
        bool ok = true;
        auto next = [&]() {
            if (lead) mma_commit(&bar[BAR_EMPTY + slot]);
            __syncwarp();
            if (++slot == p.ring) {
                slot = 0;
                par ^= 1;
            }
        };
        auto wait = [&](uint64_t *m, uint32_t phase) {
            ok = __all_sync(0xffffffffu, wait_abort(m, phase, abort_flag));
            return ok;
        };
        for (int t = 0; ok && nt > 0 && t <= nt; ++t) {
            if (t < nt) {
                for (int st = 0; st < NST; ++st, next()) {
                    if (!wait(&bar[BAR_FULL + slot], par)) break;
                    fence_smem_to_async();                // the copies' writes, before the MMAs read them
                    fence_after_sync();
                    const uint64_t a = smem_desc(ring + slot * kStage, 16, 1024, 2);
                    if (lead) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(tmem + kTmemS + (uint32_t)((t & 1) * NC),
                                     a + (uint32_t)((k >> 2) * (kChunk64 >> 4) + (k & 3) * 2),
                                     qd + (uint32_t)((st * 2 + (k >> 2)) * (NC * 8) + (k & 3) * 2), id_s, st > 0 || k > 0);
                    }
                }
                if (!ok) break;
                if (lead) mma_commit(&bar[BAR_S + (t & 1)]);
                __syncwarp();
            }
            if (t > 0) {
                if (!wait(&bar[BAR_P], (uint32_t)(t - 1) & 1)) break;
                for (int st = 0; st < NST; ++st, next()) {
                    if (!wait(&bar[BAR_FULL + slot], par)) break;
                    fence_smem_to_async();                // the copies' writes, before the MMAs read them
                    fence_after_sync();
                    const uint64_t a = smem_desc(ring + slot * kStage, kChunk64, 1024, 2);
                    if (lead) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(tmem + kTmemO + (uint32_t)(NC * st), a + (uint32_t)(k * 128),
                                     pd + (uint32_t)((k >> 2) * (NC * 8) + (k & 3) * 2), id_o, t > 1 || k > 0);
                    }
                }
                if (!ok) break;
                if (lead) mma_commit(&bar[BAR_PV]);
                __syncwarp();
            }
        }
        // the tensor memory is released only after the last issued MMAs have completed
        if (lead) mma_commit(&bar[BAR_DRAIN]);
        __syncwarp();
        mbar_wait(&bar[BAR_DRAIN], 0, kDrainTries);
        __syncwarp();
    } else {
        // ================================================================ softmax, output
        const int wg = warp >> 2, tok = tid & 127, col0 = wg * NCW;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)col0;
        const int chunks = max(0, min(NCW / 4, (p.group + 3) / 4 - wg * (NCW / 4)));   // 4-column chunks in use
        float m[NCW], l[NCW];
#pragma unroll
        for (int c = 0; c < NCW; ++c) {
            m[c] = -INFINITY;
            l[c] = 0.f;
        }
        // once a wait has given up, the remaining tiles run without waits (the warps keep their
        // common barriers) and the output becomes NaN
        bool ok = true;
        for (int t = 0; t < nt; ++t) {
            const bool in = token_row(t * kTileBlocks + (tok >> 2), tok & 3) >= 0;
            ok = __all_sync(0xffffffffu, ok && wait_abort(&bar[BAR_S + (t & 1)], (uint32_t)(t >> 1) & 1, abort_flag));
            fence_after_sync();
            float s[NCW];
            tmem_ld8(lanes + kTmemS + (uint32_t)((t & 1) * NC), s);
            tmem_wait_ld();
            tmem_regs_after_wait(s);
            bool grow = false;
#pragma unroll
            for (int c = 0; c < NCW; ++c) {
                s[c] = in && c < 4 * chunks ? s[c] * p.scale_log2 : -INFINITY;
                grow |= s[c] > m[c] + kGrow;
            }
            // The reference m of a column moves only when a score passes it by 2^8 (weights stay
            // below that, far from fp32's range), so most tiles need no maximum at all: one vote.
            const bool move = any_n(1 + wg, 128, grow);
            if (move) {
#pragma unroll
                for (int c = 0; c < NCW; ++c) {
                    const float x = warp_max(s[c]);
                    if (lane == 0) fx.red[warp][c] = x;
                }
                sync_n(1 + wg, 128);
            }
            // before P and O are written: the last tile's PV product has read and added to them
            if (t > 0) ok = __all_sync(0xffffffffu, ok && wait_abort(&bar[BAR_PV], (uint32_t)(t - 1) & 1, abort_flag));
            if (move) {
                float corr[NCW];
#pragma unroll
                for (int c = 0; c < NCW; ++c) {
                    const float x = fmaxf(fmaxf(fx.red[4 * wg][c], fx.red[4 * wg + 1][c]),
                                          fmaxf(fx.red[4 * wg + 2][c], fx.red[4 * wg + 3][c]));
                    corr[c] = x > m[c] ? ex2(m[c] - x) : 1.f;
                    m[c] = fmaxf(m[c], x);
                    l[c] *= corr[c];
                }
                if (t > 0) {
                    fence_after_sync();
#pragma unroll
                    for (int st = 0; st < NST; ++st) {
                        float o[NCW];
                        tmem_ld8(lanes + kTmemO + NC * st, o);
                        tmem_wait_ld();
                        tmem_regs_after_wait(o);
#pragma unroll
                        for (int c = 0; c < NCW; ++c) o[c] *= corr[c];
                        tmem_st8(lanes + kTmemO + NC * st, o);
                    }
                    tmem_wait_st();
                }
            }
            // P^T operand: row = column, column = token of this tile (bf16: the second product's
            // operand type; a relative error of 2^-8 a term at most, independent between terms, so
            // that a sum's is like the output's own rounding: 0.0018 of the outputs' rms in all for one
            // token at 128K, 0.0017 of it that rounding alone).  A column without a score that compares
            // with its reference (all masked, or NaN) subtracts 0: masked tokens weigh 0, NaN ones NaN.
            unsigned char *pp = sp + (tok >> 6) * (NC * 128) + col0 * 128 + ((tok & 7) << 1);
            const int pc = (tok & 63) >> 3;
#pragma unroll
            for (int c = 0; c < NCW; ++c) {
                if (c < 4 * chunks) {
                    const float x = ex2(s[c] - (m[c] == -INFINITY ? 0.f : m[c]));
                    l[c] += x;
                    *reinterpret_cast<__nv_bfloat16 *>(pp + c * 128 + ((pc ^ (c & 7)) << 4)) = __float2bfloat16_rn(x);
                }
            }
            fence_smem_to_async();
            fence_before_sync();
            arrive(&bar[BAR_P]);
        }
        if (nt > 0) ok = __all_sync(0xffffffffu, ok && wait_abort(&bar[BAR_PV], (uint32_t)(nt - 1) & 1, abort_flag));
        fence_after_sync();
        sync_n(1 + wg, 128);                              // red is free
#pragma unroll
        for (int c = 0; c < NCW; ++c) {
#pragma unroll
            for (int o = 16; o; o >>= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
            if (lane == 0) fx.red[warp][c] = l[c];
        }
        if (tok == 0)
#pragma unroll
            for (int c = 0; c < NCW; ++c) fx.m[col0 + c] = m[c];
        sync_n(1 + wg, 128);
        if (tok < NCW) {
            const float x = fx.red[4 * wg][tok] + fx.red[4 * wg + 1][tok] + fx.red[4 * wg + 2][tok] + fx.red[4 * wg + 3][tok];
            fx.l[col0 + tok] = *abort_flag ? __int_as_float(0x7fc00000) : x;   // a wait that gave up leaves NaN
        }
        sync_n(1 + wg, 128);
#pragma unroll
        for (int st = 0; st < NST; ++st) {
            float o[NCW];
#pragma unroll
            for (int c = 0; c < NCW; ++c) o[c] = 0.f;
            if (nt > 0) {
                tmem_ld8(lanes + kTmemO + NC * st, o);
                tmem_wait_ld();
                tmem_regs_after_wait(o);
            }
#pragma unroll
            for (int c = 0; c < NCW; ++c) {
                const int h = col0 + c;
                if (p.split > 1) {
                    reinterpret_cast<float *>(sm)[h * D + st * 128 + tok] = o[c];   // the ring is idle now
                } else if (h < p.group) {
                    const float lh = fx.l[h];
                    p.out[(row * p.hq + (int64_t)kvh * p.group + h) * D + st * 128 + tok] =
                        __float2bfloat16_rn(lh == 0.f ? 0.f : o[c] / lh);
                }
            }
        }
    }
    __syncwarp();

    if (p.split > 1) {
        // join: m = max m_r, o = sum 2^(m_r - m) o_r / sum 2^(m_r - m) l_r, ranks in order; each
        // CTA of the cluster writes its share of the unit's output
        cluster_sync_all();
        const uint32_t o_at = smem_u32(sm), m_at = smem_u32(fx.m), l_at = smem_u32(fx.l);
        for (int e = rank * kThreads + tid; e < p.group * D; e += p.split * kThreads) {
            const int h = e / D;
            float mm = -INFINITY;
            for (int r = 0; r < p.split; ++r) mm = fmaxf(mm, ld_peer(m_at + 4 * h, r));
            float num = 0.f, den = 0.f;
            for (int r = 0; r < p.split; ++r) {
                const float mr = ld_peer(m_at + 4 * h, r), lr = ld_peer(l_at + 4 * h, r);
                const float w = mr == -INFINITY ? 0.f : ex2(mr - mm);
                num += w * ld_peer(o_at + 4 * e, r);
                den += lr != lr ? lr : w * lr;
            }
            p.out[(row * p.hq + (int64_t)kvh * p.group) * D + e] = __float2bfloat16_rn(den == 0.f ? 0.f : num / den);
        }
        cluster_sync_all();                               // no CTA leaves while a peer reads it
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
static cudaError_t launch_single(AttnParams &p, cudaStream_t s) {
    const int entries = std::max(1, p.n_slots);
    p.ring = kMaxRing;
    while (smem_bytes(D, p.ring, entries) > kMaxSmem) --p.ring;
    const uint32_t smem = smem_bytes(D, p.ring, entries);
    auto kern = qsa_attention_kernel<D>;
    // the same value at every call: host threads share the attribute, and this call's own size would lower it
    // between another thread's setting and its launch
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    if (p.split > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)p.B * p.Qn * p.hkv * p.split;
    if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    if (p.split > 1) {
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)p.split;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
    }
    TraceLaunch tl(s, p.split > 1 ? "qsa_attention_split" : "qsa_attention");
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// q^0.8
static double union_growth(int q) {
    static const auto table = [] {
        std::array<double, 129> t{};
        for (int i = 1; i <= 128; ++i) t[i] = std::pow(i, 0.8);
        return t;
    }();
    return table[q];
}

}  // namespace qsa_attn

cudaError_t launch_qsa_attention(const void *q, const int32_t *blocks, int n_slots, const int32_t *qpos,
                                 const int32_t *n_query, int B, int Qn, const int32_t *table, int max_pages, int hq,
                                 int hkv, int d, const void *k_cache, const void *v_cache, int n_pages, int page,
                                 float scale, void *out, cudaStream_t s) {
    using namespace qsa_attn;
    AttnParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.blocks = blocks;
    p.qpos = qpos;
    p.n_query = n_query;
    p.table = table;
    p.kc = static_cast<const __nv_bfloat16 *>(k_cache);
    p.vc = static_cast<const __nv_bfloat16 *>(v_cache);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.Qn = Qn;
    p.hq = hq;
    p.hkv = hkv;
    p.group = hq / hkv;
    p.n_slots = n_slots;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.page = page;
    p.page_blocks = (uint32_t)(page / kR);
    p.page_inv = 0xffffffffu / p.page_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    // Single queries, the list divided over a cluster while that fills SMs that would stand idle,
    // or tiles of queries that share their lists' union: whichever has the least estimated time,
    // waves of one CTA per SM times (a CTA's 64 KB of keys and values + its start and end), such
    // 64 KB taking a tile 1.27 (D 256) or 1.67 (D 128) times as long.  q queries' lists have about
    // q^0.8 times the tokens of one, at most those of the whole context.  Measured, single queries
    // against tiles in us: 24 over 2 heads of 256 at 64K tokens, 16 queries 15 - 60, 64 30 - 62, 256
    // 111 - 101, 1024 385 - 302; 16 over 4 heads of 128, 64 rows in 16 x 4 42 - 53, 256 queries 123 -
    // 121, 1024 479 - 238; 4 x 200 queries at 4K 300 - 120.
    constexpr int kSms = 148;
    const double known = (double)max_pages * page, list = std::min(known, (double)n_slots * kR + 3.0);
    const double unit_tokens = 16384.0 / d;
    double best = 1e300;
    for (int sp = 1; sp <= kMaxSplit; sp *= 2) {
        const double waves = std::ceil((double)B * Qn * hkv * sp / (sp < 16 ? kSms : 112));   // (clusters of 16: 7 at once)
        const double cost = waves * (std::ceil(list / sp / unit_tokens) + (sp > 1 ? 6.0 : 4.0));
        if (cost < best) {
            best = cost;
            p.split = sp;
            p.qt = 1;
        }
    }
    p.tiles = Qn;
    for (int qt = qsa_tile_queries(Qn, p.group, max_pages, page); qt >= 2; --qt) {
        // as many tiles as the last wave has room for, of nearly equal size
        const int least = (Qn + qt - 1) / qt;
        const double units = (double)B * hkv, waves = std::ceil(units * least / kSms);
        const int tiles = (int)std::min<double>((Qn + 1) / 2, std::max<double>(least, std::floor(waves * kSms / units)));
        const double tokens = std::min(known, union_growth((Qn + tiles - 1) / tiles) * list);
        const double cost = waves * (std::ceil(tokens / unit_tokens) + 8.0) * (d == 256 ? 1.27 : 1.67);
        if (cost < best) {
            best = cost;
            p.split = 1;
            p.tiles = tiles;
            p.qt = (Qn + tiles - 1) / tiles;
        }
    }
    if (p.qt > 1) return launch_qsa_tile(p, d, s);
    return d == 256 ? launch_single<256>(p, s) : launch_single<128>(p, s);
}

}  // namespace gdn
