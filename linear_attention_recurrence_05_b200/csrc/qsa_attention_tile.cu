// Attention of a sparse-attention (QSA) layer over the selected blocks of the paged key/value
// cache.
//
// Page "ARCHITECTURE PREVIEW / FIELD NOTES", section 03 (exact attention over the selected
// tokens; CAUSAL SPARSE SET) and section 01 (24 query heads, 2 key/value heads, head dim 256,
// budget 512 blocks of 4 tokens).  Query i with heads h reading key/value head h / group:
//     S_i = tokens of its listed complete blocks, then 4 floor((i+1)/4) .. i
//     o_h = sum_{t in S_i} e^{s_ht - m_h} v_t / sum_{t in S_i} e^{s_ht - m_h},  s_ht = scale <q_h, k_t>
// in one pass over S_i with a running reference m_h and sum.
//
// Kernel for tiles of queries.  A unit is (tile of consecutive queries, key/value head): its up to
// 128 (query, head) rows are the M rows of the products
//     S [128 x 64 tokens] = Q K^T,   O [128 x D] += P V
// over the tokens of the UNION of the queries' lists, in the order of their positions; a row
// masks the blocks that its own query does not list.  Neighbouring queries share much of their
// lists (q queries with half of their scores' variance in common list about q^0.8 times the
// blocks of one), so each cache row is gathered once for all of them: 2048 queries (24 heads, D
// 256, 512 blocks each) at 64K tokens 1231 us with a unit per query, 591 us in tiles of 10.
//
// The union is a bitmap over the sequence's blocks; a block's place in the list is the number of
// bits below its own, and a second look at the queries' lists sets their masks (a bit per entry).
// A list longer than its room in shared memory is taken in passes.
//
// One CTA per SM: warps 0-3 and 4-7 softmax of the even and of the odd tiles (a row per thread),
// warp 8 issues the MMAs, warps 9-12 gather with 16-byte asynchronous copies straight from cache
// rows into swizzled 128-byte shared-memory rows of 64 dims, which serve K (K-major) and V
// (MN-major) alike.  The weights P and 128 dims of Q are A operands in tensor memory (beside O and
// three tiles of S), the other 128 dims of Q lie in shared memory.  Stages of one tile's K or V
// pass through a ring, ordered K0 K1 K2 V0 K3 V1 ..: the scores run two tiles ahead of the output.
//
// What bounds a tile of 64 tokens at D 256: the MMAs take 1226 clk (a score MMA of 64 columns 45
// clk, not 32), shared memory 1280 (64 KB in, 96 KB out), the gather alone 900 to 1000, the
// exponentials 512; together 1520 clk at 1.6 GHz, the clock that the power limit leaves.  Of the
// start, list and output of a unit (7, 16 and 6 thousand clk beside 256 thousand) nothing overlaps.
#include <algorithm>

#include "qsa_attn.cuh"

namespace gdn {
namespace qsa_attn {
namespace tile {

constexpr int kRows = 128;                   // MMA rows: (query, head) pairs of a unit
constexpr int kN = 64, kTileBlocks = kN / kR;   // tokens of a tile
constexpr uint32_t kChunk = kN * 128;        // bytes of 64 dims of a tile
constexpr uint32_t kRingBytes = 163840;      // stages of one tile's keys or values
constexpr int kMaxRing = 10;                 // D = 128; 5 for 256
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp0 = 9, kLoadWarps = 4;
constexpr int kThreads = 32 * (kLoadWarp0 + kLoadWarps), kWarps = kThreads / 32;
constexpr int kBuf = 3;                      // tiles of S in flight (P in place)
constexpr uint32_t kTmemQ = 0, kTmemS = 64, kTmemO = 256, kTmemCols = 512;   // 128 dims of Q, S, O
__host__ __device__ constexpr uint32_t q_bytes(int D) { return D > 128 ? kRows * 256u : 0u; }   // the other 128, in shared memory
constexpr int kMaxWords = (int)(kRingBytes / 8);   // bitmap words and their prefix sums, in the ring

enum { BAR_FULL = 0, BAR_EMPTY = kMaxRing, BAR_S = 2 * kMaxRing, BAR_P = BAR_S + 2 * kBuf, BAR_PV = BAR_P + kBuf,
       BAR_DRAIN = BAR_PV + kBuf, kNumBars };

// Shared memory: the ring, then
struct Fixed {
    float m[kRows];              // the rows' reference
    float l[2][kRows];           // the rows' sums over even and odd tiles
    int lim[kRows];              // tokens of the list before a query's last one
    uint32_t redo[kRows / 32];   // queries to be taken again alone
    uint64_t bar[kNumBars];
    int wsum[kWarps];
    uint32_t tmem;
    int abort_flag, total, zero_from;
};
// then rows [cap], valid [cap / 32], mask [cap / 32][qt]: the cache row of each listed block (or
// -1), a bit per entry with one, and each query's bits
__host__ __device__ constexpr uint32_t kFixedBytes() { return (uint32_t)((sizeof(Fixed) + 15) & ~15); }
__host__ __device__ constexpr uint32_t smem_bytes(int D, int cap, int qt) {
    return kRingBytes + q_bytes(D) + kFixedBytes() + (uint32_t)cap * 4 + (uint32_t)(cap / 32) * 4 * (uint32_t)(1 + (qt > 1 ? qt : 0));
}

// largest of three (NaN operands do not count); two fp32 operations in one instruction
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
    return unpair(r);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// one MMA, A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)accumulate));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) qsa_attention_tile_kernel(const __grid_constant__ AttnParams p, int cap) {
    extern __shared__ __align__(1024) unsigned char sm[];
    constexpr uint32_t kStage = kN * D * 2;
    constexpr int kRing = kRingBytes / kStage;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);             // (uniform for the compiler)
    const uint32_t unit = blockIdx.x;
    // key/value head slowest (half the cache at a time in L2); late tiles, whose lists are longest
    // in a fresh prompt, first
    const uint32_t per_head = (uint32_t)p.B * (uint32_t)p.tiles;
    const int kvh = (int)(unit / per_head), b = (int)(unit % per_head % (uint32_t)p.B);
    const int tile = p.tiles - 1 - (int)(unit % per_head / (uint32_t)p.B);
    const int n0 = (int)((int64_t)tile * p.Qn / p.tiles), nq = (int)((int64_t)(tile + 1) * p.Qn / p.tiles) - n0;   // <= p.qt
    const int64_t pos0 = (int64_t)p.qpos[b] + n0;
    // live queries: j0 <= j < j1 (positions >= 0, before the row's count, which may be any int32)
    const int j1 = p.n_query ? (int)max((int64_t)0, min((int64_t)nq, (int64_t)p.n_query[b] - n0)) : nq;
    const int j0 = pos0 < 0 ? (int)min((int64_t)j1, -pos0) : 0;
    const int64_t row0 = (int64_t)b * p.Qn + n0;
    const int32_t *table = p.table + (int64_t)b * p.max_pages, *lists = p.blocks + row0 * p.n_slots;

    Fixed &fx = *reinterpret_cast<Fixed *>(sm + kRingBytes + q_bytes(D));
    int *rows = reinterpret_cast<int *>(sm + kRingBytes + q_bytes(D) + kFixedBytes());
    uint32_t *valid = reinterpret_cast<uint32_t *>(rows + cap), *mask = valid + cap / 32;
    uint64_t *bar = fx.bar;
    volatile int *abort_flag = &fx.abort_flag;

    // a tile of padding alone: zeros
    if (j1 <= j0) {
        const int n = nq * p.group * (D / 8);             // 16-byte pieces
        for (int i = tid; i < n; i += kThreads) {
            const int r = i / (D / 8);
            const int64_t at = ((row0 + r / p.group) * p.hq + (int64_t)kvh * p.group + r % p.group) * D + i % (D / 8) * 8;
            *reinterpret_cast<uint4 *>(p.out + at) = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    // the lists on their way to L2 while the block starts
    {
        const char *first = reinterpret_cast<const char *>(lists + (int64_t)j0 * p.n_slots);
        for (int i = tid * 128; i < (j1 - j0) * p.n_slots * 4; i += kThreads * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(first + i));
    }
    if (tid == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&bar[BAR_FULL + s], 32 * kLoadWarps);
            mbar_init(&bar[BAR_EMPTY + s], 1);
        }
        for (int i = 0; i < kBuf; ++i) {
            mbar_init(&bar[BAR_S + i], 1);
            mbar_init(&bar[BAR_S + kBuf + i], 1);
            mbar_init(&bar[BAR_P + i], kSoftWarps / 2);
            mbar_init(&bar[BAR_PV + i], 1);
        }
        mbar_init(&bar[BAR_DRAIN], 1);
        fx.abort_flag = 0;
    }
    if (tid < kRows / 32) fx.redo[tid] = 0;
    if (warp == kMmaWarp) {
        tmem_alloc(&fx.tmem, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, fx.tmem, 0), ring = smem_u32(sm);

    // softmax threads: named barriers of the two warps that share rows (both; the one that waits for the
    // other's reference); this thread's row, its query, its tiles' parity
    const int both_id = 1 + (warp & 3), mine_id = 5 + warp, other_id = 5 + (warp ^ 4);
    const int wg = warp >> 2, row = 32 * (warp & 3) + lane, qj = row / p.group;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int64_t row_at = ((row0 + qj) * p.hq + (int64_t)kvh * p.group + row % p.group) * D;   // in q and out
    if (warp < kSoftWarps) {
        // Q as the first product's A operand, with the scale's sign: dims below 128 in tensor memory
        // (lane = row, column = two dims), the rest in shared memory
        const uint4 *q = reinterpret_cast<const uint4 *>(p.q + row_at + wg * (D / 2));
        uint4 u[D / 16];
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) u[i] = qj < nq ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) u[i].x ^= flip, u[i].y ^= flip, u[i].z ^= flip, u[i].w ^= flip;
        if (D > 128 && wg) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<uint4 *>(sm + kRingBytes + (i >> 3) * (kRows * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4)) = u[i];
            fence_smem_to_async();
        } else {
#pragma unroll
            for (int c = 0; c < D / 4; c += 32) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[4 * i] = __uint_as_float(u[c / 4 + i].x);
                    v[4 * i + 1] = __uint_as_float(u[c / 4 + i].y);
                    v[4 * i + 2] = __uint_as_float(u[c / 4 + i].z);
                    v[4 * i + 3] = __uint_as_float(u[c / 4 + i].w);
                }
                tmem_st32(lanes + kTmemQ + wg * (D / 4) + c, v);
            }
            tmem_wait_st();
        }
    }
    const float scale = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);    // (not 0: a masked score stays -inf)

    // state of the roles that lasts over the unit's passes
    int tile0 = 0;                                        // tiles of earlier passes
    int ld_issued = 0, ld_slot = 0;                       // gather
    uint32_t ld_par = 1;
    int mma_slot = 0;                                     // MMA issuer
    uint32_t mma_par = 0, drain_par = 0;
    bool ok = true;
    uint32_t redo[kRows / 32] = {};

    // The unit's queries together; then, alone and by its own list, each query that lists a block
    // twice (a weight of 2 does not fit a bit) and each whose result is not finite (a NaN or
    // infinite value row that a neighbour lists: its weight 0 does not hide it in the product).
    for (int sub = -1;;) {
        const bool list = sub >= 0;
        const int lj = max(sub, 0);                       // the list's query
        const bool lj_live = lj >= j0 && lj < j1;
        const int64_t lj_comp = lj_live ? (pos0 + lj + 1) >> 2 : 0;     // its complete blocks
        const int lj_tail = lj_live ? (int)((pos0 + lj + 1) & 3) : 0;
        int end = lj_live ? p.n_slots + 1 : 0;            // entries (the list's last is the tail)
        float m = -INFINITY, l = 0.f;
        const int sub0 = tile0;                           // first tile of this sum
        for (int off = 0;; off += cap) {
            // ---------------------------------------------------------------- the pass' entries
            if (list) {
                const int32_t *mine = lists + (int64_t)lj * p.n_slots;
                if (tid == 0) fx.total = 0, fx.zero_from = 0x7fffffff;
                __syncthreads();
                const int n = min(cap, end - off), n32 = (n + 31) & ~31;
                int last = 0;
                for (int i = tid; i < n32; i += kThreads) {               // whole warps
                    const int e = off + i;
                    int r = -1;
                    if (i < n) {
                        int64_t blk = -1;
                        if (e == p.n_slots) {
                            if (lj_tail) blk = lj_comp, fx.zero_from = 4 * i + lj_tail;
                        } else {
                            blk = __ldg(mine + e);
                            if (blk >= lj_comp) blk = -1;
                        }
                        if (blk >= 0) r = block_row(p, table, (uint32_t)blk, kvh);
                    }
                    rows[i] = r;
                    const uint32_t v = __ballot_sync(0xffffffffu, r >= 0);
                    if (lane == 0) valid[i >> 5] = v;
                    if (v) last = (i & ~31) + 32 - __clz(v);
                }
                if (last && lane == 0) atomicMax(&fx.total, last);
                __syncthreads();
            } else {
                // a bit per block of the sequence that any query lists or has as its tail; an
                // entry's place is the number of bits below its own
                uint32_t *bits = reinterpret_cast<uint32_t *>(sm);
                int *before = reinterpret_cast<int *>(sm) + kMaxWords;
                const int64_t known = (int64_t)p.max_pages * p.page / kR;
                const int nb = (int)min(known, ((pos0 + j1) >> 2) + 1), words = (nb + 31) >> 5;
                for (int i = tid; i < words; i += kThreads) bits[i] = 0;
                for (int i = tid; i < cap / 32 * nq; i += kThreads) mask[i] = 0;
                for (int j = tid; j < nq; j += kThreads) fx.lim[j] = 0x7fffffff;
                if (tid == 0) fx.zero_from = 0x7fffffff;
                __syncthreads();
                // f(query, block or -1) for the entries of every live query, by whole warps: -1 for
                // those that are not complete blocks of the query inside the page table
                // (a warp's next 128 entries are on their way while it looks at these)
                constexpr int kAhead = 4;                 // entries of a lane, 32 apart
                auto for_entries = [&](auto f) {
                    const int chunks = (p.n_slots + 32 * kAhead - 1) / (32 * kAhead);
                    int x[kAhead], j = j0, c = warp;
                    auto load = [&](int (&v)[kAhead]) {   // the warp's piece c of query j on, -1 beyond
                        while (c >= chunks && j < j1) c -= chunks, ++j;
                        const int32_t *e = lists + (int64_t)j * p.n_slots;
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) {
                            const int i = 32 * (kAhead * c + u) + lane;
                            v[u] = j < j1 && i < p.n_slots ? __ldg(e + i) : -1;
                        }
                    };
                    for (load(x); j < j1;) {
                        const int jx = j, n = (int)min((int64_t)nb, (pos0 + j + 1) >> 2);
                        int y[kAhead];
                        c += kWarps;
                        load(y);                          // the next piece is on its way meanwhile
                        bool any = false;
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) {
                            if ((uint32_t)x[u] >= (uint32_t)n) x[u] = -1;
                            any |= x[u] >= 0;
                        }
                        if (__any_sync(0xffffffffu, any)) f(jx, x);
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) x[u] = y[u];
                    }
                };
                // query j's tail block, or -1
                auto tail_of = [&](int j) {
                    const int64_t blk = (pos0 + j + 1) >> 2;
                    return ((pos0 + j + 1) & 3) && blk < nb ? (int)blk : -1;
                };
                for_entries([&](int, const int (&blk)[kAhead]) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (blk[u] >= 0) atomicOr(&bits[blk[u] >> 5], 1u << (blk[u] & 31));
                });
                for (int j = j0 + tid; j < j1; j += kThreads) {
                    const int blk = tail_of(j);
                    if (blk >= 0) atomicOr(&bits[blk >> 5], 1u << (blk & 31));
                }
                __syncthreads();
                const int per = (words + kThreads - 1) / kThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
                int sum = 0;
                for (int w = w0; w < w1; ++w) sum += __popc(bits[w]);
                int run = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += x;
                }
                if (lane == 31) fx.wsum[warp] = run;
                __syncthreads();
                int at = run - sum, total = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) at += fx.wsum[w];
                    total += fx.wsum[w];
                }
                end = total;
                const int n = min(cap, end - off);
                // the entries' blocks: few words, which may be full, by a warp each (6 words 1.5 thousand clk, 4.8 by
                // a thread each), many by a thread each (512 words 4.1 thousand clk, 5.0 by a warp each)
                const bool by_warp = words <= 4 * kWarps;
                for (int w = w0; w < w1; ++w) {
                    before[w] = at - off;
                    const uint32_t y = bits[w];
                    if (by_warp) at += __popc(y);
                    else
                        for (uint32_t x = y; x; x &= x - 1, ++at)
                            if (at >= off && at - off < n) rows[at - off] = 32 * w + __ffs(x) - 1;
                }
                __syncthreads();
                for (int w = by_warp ? warp : words; w < words; w += kWarps) {
                    const uint32_t y = bits[w];
                    const int i = before[w] + __popc(y & ((1u << lane) - 1));
                    if (y >> lane & 1 && i >= 0 && i < n) rows[i] = 32 * w + lane;
                }
                if (by_warp) __syncthreads();
                auto place = [&](int blk) { return before[blk >> 5] + __popc(bits[blk >> 5] & ((1u << (blk & 31)) - 1)); };
                for_entries([&](int j, const int (&blk)[kAhead]) {
                    int i[kAhead];
                    uint32_t had[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int x = place(max(blk[u], 0));
                        i[u] = blk[u] >= 0 && x < n ? x : -1;             // (-1 also for entries of earlier passes)
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        had[u] = i[u] >= 0 ? atomicOr(&mask[(i[u] >> 5) * nq + j], 1u << (i[u] & 31)) & 1u << (i[u] & 31) : 0u;
                    if (had[0] | had[1] | had[2] | had[3]) atomicOr(&fx.redo[j >> 5], 1u << (j & 31));
                });
                for (int j = j0 + tid; j < j1; j += kThreads) {
                    const int blk = tail_of(j), i = blk >= 0 ? place(blk) : -1;
                    if (i < 0 || i >= n) continue;
                    atomicOr(&mask[(i >> 5) * nq + j], 1u << (i & 31));
                    fx.lim[j] = 4 * i + (int)((pos0 + j + 1) & 3);
                    if (j == j1 - 1) fx.zero_from = fx.lim[j];           // later tokens are not written yet
                }
                for (int i0 = tid; i0 < ((n + 31) & ~31); i0 += kAhead * kThreads) {
                    int r[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int i = i0 + u * kThreads;
                        r[u] = i < n ? block_row(p, table, (uint32_t)rows[i], kvh) : -1;
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int i = i0 + u * kThreads;
                        const uint32_t v = __ballot_sync(0xffffffffu, r[u] >= 0);
                        if (i < ((n + 31) & ~31)) {       // whole warps
                            rows[i] = r[u];
                            if (lane == 0) valid[i >> 5] = v;
                        }
                    }
                }
                if (tid == 0) fx.total = n;
                __syncthreads();
            }
            fence_smem_to_async();                        // the ring's generic writes before its next copies
            fence_before_sync();
            __syncthreads();
            fence_after_sync();
            const int nt = __shfl_sync(0xffffffffu, (fx.total + kTileBlocks - 1) / kTileBlocks, 0);

            if (warp >= kLoadWarp0) {
                // ============================================================ gather
                // A stage is declared full by its copies themselves (an arrival per thread once they have
                // landed), so that the gather waits for nothing but a free stage.
                // The copies' shared addresses differ by constants from SW ones per lane, and their sources from
                // one per block, so that a copy is one instruction.
                constexpr int RW = kN / kLoadWarps, LPR = D / 8, RPI = 32 / LPR;  // rows of a warp; lanes per row; rows a copy
                constexpr int E = RW / kR, SW = 8 / RPI;                          // blocks of a warp; shared addresses
                static_assert(E == 4, "a warp's blocks are one 16-byte load");
                const int wl = warp - kLoadWarp0, c = lane & (LPR - 1), hi = lane / LPR;
                const int zero_from = fx.zero_from;
                uint32_t at[SW];
#pragma unroll
                for (int i = 0; i < SW; ++i)
                    at[i] = ring + (uint32_t)(c >> 3) * kChunk + (uint32_t)(wl * RW + hi) * 128 + (uint32_t)(((c & 7) ^ (i * RPI + hi)) << 4);
                auto stage = [&](const __nv_bfloat16 *cache, int t) {
                    const int4 x = *reinterpret_cast<const int4 *>(rows + t * kTileBlocks + wl * E);
                    const int row[E] = {x.x, x.y, x.z, x.w};
                    const char *lane_src = reinterpret_cast<const char *>(cache + hi * D + c * 8), *src[E];
                    uint32_t size[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        src[e] = lane_src + (uint64_t)(uint32_t)max(row[e], 0) * (D * 2);
                        size[e] = row[e] >= 0 ? 16u : 0u;
                    }
                    ok = __all_sync(0xffffffffu, ld_issued < kRing || wait_abort(&bar[BAR_EMPTY + ld_slot], ld_par, abort_flag));
                    if (!ok) return;
                    const uint32_t slot = (uint32_t)ld_slot * kStage;
                    const int left = zero_from - t * kN - wl * RW;        // rows before the last query's end
                    if (left >= RW) {
#pragma unroll
                        for (int r = 0; r < RW; r += RPI)
                            cp_async16_sized(at[r / RPI % SW] + slot + r * 128, src[r / kR] + r % kR * (D * 2), size[r / kR]);
                    } else {                              // (the others stay zero)
#pragma unroll
                        for (int r = 0; r < RW; r += RPI)
                            cp_async16_sized(at[r / RPI % SW] + slot + r * 128, src[r / kR] + r % kR * (D * 2),
                                             r + hi < left ? size[r / kR] : 0u);
                    }
                    cp_async_arrive(&bar[BAR_FULL + ld_slot]);
                    ++ld_issued;
                    if (++ld_slot == kRing) {
                        ld_slot = 0;
                        ld_par ^= 1;
                    }
                };
                for (int u = 0; ok && nt > 0 && u < 2 * nt + 4; ++u) {    // K(0) K(1) K(2) V(0) K(3) V(1) ..
                    const int t = (u >> 1) - (u & 1 ? 2 : 0);
                    if (t >= 0 && t < nt) stage(u & 1 ? p.vc : p.kc, t);
                }
                cp_async_wait_all();
            } else if (warp == kMmaWarp) {
                // ============================================================ MMA issuer
                // the whole warp walks through the tiles, so that descriptors stay in uniform registers
                // (issued from a single lane's branch an MMA took 70 clk, more than its run time); one
                // elected lane issues
                const bool lead = elect_one();
                auto next = [&]() {
                    if (lead) mma_commit(&bar[BAR_EMPTY + mma_slot]);
                    __syncwarp();
                    if (++mma_slot == kRing) {
                        mma_slot = 0;
                        mma_par ^= 1;
                    }
                };
                // A wait takes 150 clk also when its phase is over, so each is polled a few MMAs ahead, while
                // the tensor core is busy, and waited for only when that poll came too early.
                auto wait_for = [&](bool polled, uint64_t *m, uint32_t phase) {
                    if (!__all_sync(0xffffffffu, polled)) ok = __all_sync(0xffffffffu, wait_abort(m, phase, abort_flag));
                    return ok;
                };
                const uint64_t qd = smem_desc(ring + kRingBytes, 16, 1024, 2);
                bool k_polled = false;
                for (int t = 0; ok && nt > 0 && t < nt + 2; ++t) {
                    const int T = tile0 + t, U = T - 2;
                    const uint32_t p_phase = (uint32_t)(U / kBuf) & 1;
                    bool p_polled = false, v_polled = false;
                    if (t < nt) {
                        if (!wait_for(k_polled, &bar[BAR_FULL + mma_slot], mma_par)) break;
                        fence_smem_to_async();            // the copies' writes, before the MMAs read them
                        fence_after_sync();
                        const uint64_t kd = smem_desc(ring + mma_slot * kStage, 16, 1024, 2);
                        const uint32_t s_at = tmem + kTmemS + (uint32_t)(T % kBuf * kN);
                        auto scores = [&](int k0, int k1) {
                            if (lead) {
#pragma unroll
                                for (int k = k0; k < k1; ++k) {
                                    const uint64_t kk = kd + (uint32_t)((k >> 2) * (kChunk >> 4) + (k & 3) * 2);
                                    if (k < 8) mma_ts(s_at, tmem + kTmemQ + 8u * k, kk, idesc_attn(kRows, kN, false, false), k > 0);
                                    else mma_bf16(s_at, qd + (uint32_t)(((k >> 2) - 2) * (kRows * 8) + (k & 3) * 2), kk,
                                                  idesc_attn(kRows, kN, false, false), 1u);
                                }
                            }
                            __syncwarp();
                        };
                        scores(0, D / 16 - 4);
                        if (t > 1) {
                            const int v_slot = mma_slot + 1 == kRing ? 0 : mma_slot + 1;
                            p_polled = mbar_try_wait_sleep(&bar[BAR_P + U % kBuf], p_phase, 0);
                            v_polled = mbar_try_wait_sleep(&bar[BAR_FULL + v_slot], v_slot ? mma_par : mma_par ^ 1, 0);
                        }
                        scores(D / 16 - 4, D / 16);
                        next();
                        if (lead) mma_commit(&bar[BAR_S + T % (2 * kBuf)]);
                        __syncwarp();
                    }
                    if (t > 1) {
                        if (!wait_for(p_polled, &bar[BAR_P + U % kBuf], p_phase)) break;
                        if (!wait_for(v_polled, &bar[BAR_FULL + mma_slot], mma_par)) break;
                        fence_smem_to_async();
                        fence_after_sync();
                        const uint64_t vd = smem_desc(ring + mma_slot * kStage, kChunk, 1024, 2);
                        const uint32_t p_at = tmem + kTmemS + (uint32_t)(U % kBuf * kN);
                        auto output = [&](int k0, int k1) {
                            if (lead) {
#pragma unroll
                                for (int k = k0; k < k1; ++k)
                                    mma_ts(tmem + kTmemO, p_at + 8u * k, vd + (uint32_t)(k * 128), idesc_attn(kRows, D, false, true),
                                           U > sub0 || k > 0);
                            }
                            __syncwarp();
                        };
                        output(0, kN / 16 - 1);
                        if (t + 1 < nt) {
                            const int k_slot = mma_slot + 1 == kRing ? 0 : mma_slot + 1;
                            k_polled = mbar_try_wait_sleep(&bar[BAR_FULL + k_slot], k_slot ? mma_par : mma_par ^ 1, 0);
                        }
                        output(kN / 16 - 1, kN / 16);
                        next();
                        if (lead) mma_commit(&bar[BAR_PV + U % kBuf]);
                        __syncwarp();
                    }
                }
                // the pass' products are complete: its ring and list may be written again
                if (lead) mma_commit(&bar[BAR_DRAIN]);
                __syncwarp();
                ok = mbar_wait(&bar[BAR_DRAIN], drain_par, kDrainTries) && ok;   // (also after an abort: no MMA outlives the block)
                drain_par ^= 1;
            } else {
                // ============================================================ softmax
                // Warps 0-3 take the even tiles, 4-7 the odd ones, a row per thread, so that one tile's
                // exponentials run beside the other's maxima.  Only a row's reference passes from tile
                // to tile, as soon as its maximum is known.  Once a wait has given up, the remaining
                // tiles run without waits (the warps keep their common barriers) and the output
                // becomes NaN.
                const bool mine = list ? qj == lj && qj < nq : qj < nq;
                const int lim = list ? fx.zero_from : qj < nq ? fx.lim[qj] : 0;
                const bool warp_live = __any_sync(0xffffffffu, mine);
                for (int t = (tile0 ^ wg) & 1; t < nt; t += 2) {
                    const int T = tile0 + t;
                    ok = __all_sync(0xffffffffu, ok && wait_abort(&bar[BAR_S + T % (2 * kBuf)], (uint32_t)(T / (2 * kBuf)) & 1, abort_flag));
                    fence_after_sync();
                    const uint32_t s_at = lanes + kTmemS + (uint32_t)(T % kBuf * kN);
                    float s[kN];
                    float top = -INFINITY;
                    if (warp_live) {                      // (rows of no query: their P and O are never used)
                        const int e0 = t * kTileBlocks;
                        uint32_t w = mine ? valid[e0 >> 5] : 0u;
                        if (!list && mine) w &= mask[(e0 >> 5) * nq + qj];
                        w >>= e0 & 31;
                        const int left = lim - kR * e0;   // tokens of this tile before the query's end
                        __syncwarp();
                        tmem_ld32(s_at, *reinterpret_cast<float(*)[32]>(&s[0]));
                        tmem_ld32(s_at + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
                        tmem_wait_ld();
                        tmem_regs_after_wait(s);
#pragma unroll
                        for (int i = 0; i < kN; ++i) s[i] = (w >> (i / kR)) & 1 ? s[i] : -INFINITY;
                        if (left < kN) {
#pragma unroll
                            for (int i = 0; i < kN; ++i)
                                if (i >= left) s[i] = -INFINITY;
                        }
                        float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int i = 4; i + 1 < kN; i += 2) tops[(i >> 1) & 3] = max3(tops[(i >> 1) & 3], s[i], s[i + 1]);
                        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
                    }
                    // the row's reference after the tile before
                    __syncwarp();
                    float m_now = -INFINITY;
                    if (T > sub0) {
                        sync_n(mine_id, 64);
                        m_now = fx.m[row];
                    }
                    // The reference moves only when a score passes it by 2^8 (weights stay below that,
                    // far from fp32's range): rarely after a row's first tile.
                    const float m_old = m_now;
                    const bool grow = top > (m_now == -INFINITY ? m_now : m_now + kGrow);
                    if (grow) m_now = top;
                    if (grow || T == sub0) fx.m[row] = m_now;
                    __syncwarp();
                    asm volatile("bar.arrive %0, 64;" ::"r"(other_id) : "memory");
                    if (m != m_now && m_now > -INFINITY) {                // (also moved by the other warp)
                        l *= ex2(m - m_now);
                        m = m_now;
                    }
                    if (__any_sync(0xffffffffu, grow) && T > sub0) {
                        ok = __all_sync(0xffffffffu, ok && wait_abort(&bar[BAR_PV + (T - 1) % kBuf], (uint32_t)((T - 1) / kBuf) & 1, abort_flag));
                        fence_after_sync();
                        const float corr = grow ? ex2(m_old - m_now) : 1.f;
                        __syncwarp();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            tmem_ld16(lanes + kTmemO + c, o);
                            tmem_wait_ld();
                            tmem_regs_after_wait(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= corr;
                            tmem_st16(lanes + kTmemO + c, o);
                        }
                    }
                    __syncwarp();
                    if (warp_live) {
                        // bf16, the second product's operand type: a relative error of 2^-8 a term at
                        // most, independent between terms, so that a sum's is like the output's own
                        // rounding (up to 0.0023 of the outputs' rms in all, 0.0017 of it that
                        // rounding alone); a second product for the rest of the weights would cost a
                        // tile 512 of its 1226 MMA clk again
                        const float m0 = m == -INFINITY ? 0.f : m;
                        const float2 scale2 = make_float2(scale, scale), less = make_float2(-m0, -m0);
                        float2 ls[2] = {};
#pragma unroll
                        for (int h = 0; h < kN; h += 32) {
                            float pw[16];
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 y = fma2(make_float2(s[h + i], s[h + i + 1]), scale2, less);
                                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                                ls[i / 2 & 1] = add2(ls[i / 2 & 1], e);
                                pw[i / 2] = __uint_as_float(pack_bf16(e.x, e.y));
                            }
                            tmem_st16(s_at + h / 2, pw);
                        }
                        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                        tmem_wait_st();
                    }
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive(&bar[BAR_P + T % kBuf]);
                }
            }
            __syncwarp();
            tile0 += nt;
            fence_before_sync();
            __syncthreads();
            fence_after_sync();
            if (off + cap >= end) break;
        }

        // ------------------------------------------------------------------ output
        const bool some = tile0 > sub0;
        const int r0 = list ? lj * p.group : 0, r1 = list ? r0 + p.group : nq * p.group;      // rows of this sum
        if (warp < kSoftWarps) {
            // the last tile's reference is the row's
            if (some && ((tile0 - 1) & 1) != wg) sync_n(mine_id, 64);
            sync_n(both_id, 64);
            const float m_last = some ? fx.m[row] : m;
            fx.l[wg][row] = m == m_last || m == -INFINITY ? l : l * ex2(m - m_last);
            __syncwarp();
            sync_n(both_id, 64);
            const float ls = *abort_flag ? __int_as_float(0x7fc00000) : fx.l[0][row] + fx.l[1][row];
            const float inv = 1.f / ls;
            const bool mine = row >= r0 && row < r1;
            float bad = 0.f;
            if (__any_sync(0xffffffffu, mine)) {
#pragma unroll 1
                for (int c = wg * (D / 2); c < (wg + 1) * (D / 2); c += 32) {
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                    if (some) {
                        tmem_ld32(lanes + kTmemO + c, o);
                        tmem_wait_ld();
                        tmem_regs_after_wait(o);
                    }
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            o[i] = ls == 0.f ? 0.f : o[i] * inv;
                            bad = fmaf(o[i], 0.f, bad);
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(p.out + row_at + c + i) =
                                make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                                           pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7]));
                    }
                    __syncwarp();
                }
            }
            if (!list && bad != 0.f) atomicOr(&fx.redo[qj >> 5], 1u << (qj & 31));
        }
        __syncwarp();
        __syncthreads();
        if (sub < 0) {
#pragma unroll
            for (int w = 0; w < kRows / 32; ++w) redo[w] = fx.redo[w];
        }
        int next = -1;
#pragma unroll
        for (int w = kRows / 32 - 1; w >= 0; --w)
            if (redo[w]) next = 32 * w + __ffs(redo[w]) - 1;
        if (next < 0) break;
#pragma unroll
        for (int w = 0; w < kRows / 32; ++w)
            if (w == next >> 5) redo[w] &= redo[w] - 1;
        sub = next;
    }

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
static cudaError_t launch(const AttnParams &p, int cap, cudaStream_t s) {
    auto kern = qsa_attention_tile_kernel<D>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)p.B * p.tiles * p.hkv;
    if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    TraceLaunch tl(s, "qsa_attention_tile");
    kern<<<(unsigned)ctas, kThreads, smem_bytes(D, cap, p.qt), s>>>(p, cap);
    return cudaGetLastError();
}

}  // namespace tile

int qsa_tile_queries(int Qn, int group, int max_pages, int page) {
    if ((int64_t)max_pages * page / kR > (int64_t)tile::kMaxWords * 32) return 1;
    return std::min(Qn, tile::kRows / group);
}

cudaError_t launch_qsa_tile(const AttnParams &p, int d, cudaStream_t s) {
    // entries of the list held at once: all that there can be, or what fits
    const int64_t known = (int64_t)p.max_pages * p.page / kR, listed = (int64_t)p.qt * (p.n_slots + 1);
    const int64_t entries = (std::max<int64_t>(p.n_slots + 1, std::min(known, listed)) + 31) / 32;
    const int64_t fit = (kMaxSmem - tile::smem_bytes(d, 0, p.qt)) / (tile::smem_bytes(d, 32, p.qt) - tile::smem_bytes(d, 0, p.qt));
    const int cap = (int)std::min(entries, fit) * 32;
    return d == 256 ? tile::launch<256>(p, cap, s) : tile::launch<128>(p, cap, s);
}

}  // namespace qsa_attn
}  // namespace gdn
