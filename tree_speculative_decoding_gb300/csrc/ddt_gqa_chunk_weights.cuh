// ddt_gqa_chunk_weights.cuh -- how much attention every column received: for column j of
// request b, over the counted tokens i and all heads h that see it (ddt_gqa_chunk.cuh),
//   w[j] = decay prev[j] + sum_{i,h} e^{z_ij - lse[i,h]}
// with the scores z and the row sums lse of the chunk attention.
//
// Work.  An item is 256 columns of a request: two tiles of 128 K rows.  Its steps go over
// the K/V heads and, for each, over tiles of NQ rows of q (token-major, the group's heads
// inside a token) of the tokens that see one of the columns.  A step is the transposed
// product S = K q^T of both K tiles with one q tile: a thread of the softmax warps then owns
// a column, and its sum over rows, tiles and heads stays in a register; nothing is added
// atomically.  NQ = 16 where a request has no more rows per K/V head (decode: the loads of K
// bound it), else 128.
// The steps of all items form one line that is dealt to the resident CTAs in equal shares;
// items that were cut leave partial sums (at most two per CTA), which a second kernel adds up
// in the order of the steps.  Everything is fp32 but the products' bf16 inputs; the tensor core truncates
// their sums, which leaves heavy scores low: about half of what the weights are off by (5e-7 with 32 observers;
// the other half is the rounding of the score's factor, which does not average out either).
//
// Measured, D = 128: 32 tokens of 32 requests after 2048..8192, 64 heads on 8, 70 us, 4.7 TB/s (memory, one CTA
// per SM); 32 observers of 32768 columns 41 us; two chunks of 2048 after 4096..8192, 32 heads on 4, 378 us, 730
// TFLOP/s of what is seen, with a cap 602 us.  A step of 128 rows takes ~3100 clk for 1024 of products (whose
// operands both come from shared memory, at its whole rate) and 1024 of exponentials: the sums of 16 rows at a
// time wait for tensor memory and for each other.
//
// Warps: four softmax warps per K tile (eight with NQ = 128: a thread has half of the rows), eight load warps
// (32 K rows and NQ / 8 q rows each), one that issues MMAs.  Scores are double-buffered in tensor memory (2 x 2 x 128 columns).
// Every wait is bounded: on timeout the CTA latches DDT_DEVERR_TIMEOUT, waits for its own
// copies and MMAs and leaves.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "ddt_gqa_chunk.cuh"

namespace ddt {
namespace chunk {
namespace received {

using namespace sm100;

constexpr int kCols = 256;  // columns of an item

struct Params {
    ChunkArgs a;
    WeightArgs w;
    int group;        // query heads per K/V head
    float group_inv;  // 1 / group
    int items_most;   // items of the longest request
    ScoreScale score;
    float cap_most;   // products below this may use CapPoly
    // log2(e) as the rounded factors of a score have it, in two parts: lse and slopes take the same, so that
    // its error counts with z - lse and not with z (capped scores near 36: sums off by 1.1e-6 where 1.6e-6)
    float log2e, log2e_rest;
};

template <int D, int NQ>
struct Cfg {
    static constexpr int kBoxes = D / 64;
    static constexpr int kKBoxBytes = 128 * 128;              // one 128-byte piece of a K tile
    static constexpr int kKBytes = 2 * kBoxes * kKBoxBytes;   // both tiles
    static constexpr int kQBoxBytes = NQ * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;
    static constexpr int kKStages = NQ == 128 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
    static constexpr int kQStages = NQ == 128 ? (D == 128 ? 2 : 4) : 4;
    static constexpr int kRStages = 4;  // of the lists beside the q tiles, which the sums read longer than the products do
    // Warps that share a column.  With 128 rows in a step the sums are what takes the time, and two warps of a
    // scheduler do not fill it: two capped chunks of 2048 take 652 us with one warp, 589 with two.
    static constexpr int kSplit = NQ == 128 ? 2 : 1;
    static constexpr int kSoftWarps = 8 * kSplit, kLoadWarps = 8, kFirstLoad = kSoftWarps, kMmaWarp = kSoftWarps + kLoadWarps,
                         kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kOffK = 0, kOffQ = kOffK + kKStages * kKBytes;
    // per stage NQ each of: -lse, slope, position less the first row's (as a number of either kind); the first position
    static constexpr int kOffRow = kOffQ + kQStages * kQBytes;
    static constexpr int kRowBytes = NQ * 16 + 16;
    static constexpr int kOffBar = kOffRow + kRStages * kRowBytes;
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bQFull = bKEmpty + kKStages, bQEmpty = bQFull + kQStages,
                         bRFull = bQEmpty + kQStages, bREmpty = bRFull + kRStages, bSFull = bREmpty + kRStages, bSEmpty = bSFull + 4, bDrain = bSEmpty + 4, bPair = bDrain + 1, bPairEmpty = bPair + 1,
                         bSegFull = bPairEmpty + 1, bSegEmpty = bSegFull + 2, bCount = bSegEmpty + 2;
    static constexpr int kOffHolder = kOffBar + 8 * bCount;
    static constexpr int kOffWalk = kOffHolder + 8;
    static constexpr int kWalkBytes = 128, kSegBytes = 96;
    static constexpr int kOffPlan = kOffWalk + kWalkBytes + 2 * kSegBytes;
    static constexpr int kOffPair = kOffPlan + 8 * (kThreads / 32);  // the second warps' sums
    static constexpr int kSmemBytes = kOffPair + (kSplit == 2 ? 4 * kCols : 0) + 1024;
    static constexpr int kOffCosts = kOffK;
    static constexpr uint32_t kIdesc = idesc_bf16(128, NQ, 0, 0);
    // Cost of a step and of an item besides; the share that a CTA gets at least.
    static constexpr int kCostStep = 4, kCostItem = 12, kMinShare = 24;
    static_assert(kOffRow % 16 == 0 && kRowBytes % 16 == 0 && kOffBar % 8 == 0 && kOffWalk % 8 == 0 && kOffPlan % 8 == 0, "alignment");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

// ---------------------------------------------------------------- items
struct Owner {
    Request r;
    int prev0, prevs;  // where the columns' earlier sums are, and of how many there are any
};
__device__ __forceinline__ Owner load_owner(const Params &prm, int b, unsigned int *err) {
    Owner o;
    o.r = load_request(prm.a, b, err);
    o.prev0 = o.prevs = 0;
    if (prm.w.prev) {
        if (!prm.w.prev_indptr) {
            o.prev0 = o.r.kv0;
            o.prevs = o.r.N;
        } else {
            o.prev0 = prm.w.prev_indptr[b];
            const int end = prm.w.prev_indptr[b + 1];
            o.prevs = (int)((uint32_t)end - (uint32_t)o.prev0);
            if (o.prev0 < 0 || end < o.prev0 || end > prm.w.total_prev || o.prevs > o.r.N) {
                if (o.r.N > 0) latch(err, DDT_DEVERR_KV_INDPTR);
                o.r.N = o.r.T = 0;
            }
        }
    }
    return o;
}
__device__ __forceinline__ int items_of(const Request &r) { return (int)(((int64_t)r.N + kCols - 1) / kCols); }

// Item n: its first counted token that sees a column, rows from there on, tiles and steps of them.
struct Item {
    int token, rows, tiles, steps;
};
template <int NQ>
__device__ __forceinline__ Item item_of(const Request &r, int n, const Params &prm) {
    const ChunkArgs &a = prm.a;
    const int counted = prm.w.last_rows > 0 ? min(r.T, prm.w.last_rows) : r.T, P = r.N - r.T;
    const int c0 = n * kCols, c1 = min(r.N - c0, kCols) + c0;
    int lo = r.N - counted, hi = r.N - 1;  // positions
    if (c0 >= r.full) {
        lo = max(lo, c0);
        if (a.window > 0) hi = (int)min((int64_t)hi, (int64_t)c1 + a.window - 2);
    }
    Item i;
    i.token = lo - P;
    i.rows = max(0, hi - lo + 1) * prm.group;
    i.tiles = (i.rows + NQ - 1) / NQ;
    i.steps = i.tiles * a.num_kv_heads;
    return i;
}
// units of an item on the line: its steps, or one where there is only something to write
__device__ __forceinline__ int units_of(const Item &i) { return max(1, i.steps); }
template <class C>
__device__ __forceinline__ int64_t item_cost(const Item &i) {
    return C::kCostItem + (int64_t)units_of(i) * C::kCostStep;
}
template <class C>
__device__ __forceinline__ int units_before(int64_t item, int64_t x, int count) {
    const int64_t d = x - (item + C::kCostItem);
    if (d <= 0) return 0;
    const int64_t k = divide(d + C::kCostStep - 1, C::kCostStep);
    return k < count ? (int)k : count;
}

struct Segment {
    int units;      // 0: no more segments
    int k0, steps;  // steps k0 .. k0 + steps - 1 (step k: K/V head k / tiles, tile k % tiles)
    int c0, token, rows, tiles;
    int qo0, kv0, N, P, full, prev0, prevs;
    int part;       // -1: the whole item, else the place of its partial sums
};

template <class C, int NQ>
struct Walk {
    int64_t pos, end;
    Shares shares;
    Owner o;
    int b, n, items, cta;
    int dealt, more;

    __device__ __forceinline__ Segment next(const Params &prm) {
        Segment s;
        s.units = 0;
        while (more && s.units == 0) {
            const Item i = item_of<NQ>(o.r, n, prm);
            const int count = units_of(i);
            const int64_t lo = dealt ? shares.lo(cta) : 0;
            const int k0 = dealt ? units_before<C>(pos, lo, count) : 0;
            const int k1 = dealt ? units_before<C>(pos, end, count) : count;
            s.units = k1 - k0;
            s.k0 = k0;
            s.steps = min(i.steps, k1) - k0;
            s.c0 = n * kCols;
            s.token = i.token;
            s.rows = i.rows;
            s.tiles = max(1, i.tiles);
            s.qo0 = o.r.qo0;
            s.kv0 = o.r.kv0;
            s.N = o.r.N;
            s.P = o.r.N - o.r.T;
            s.full = o.r.full;
            s.prev0 = o.prev0;
            s.prevs = o.prevs;
            s.part = s.units == count ? -1 : 2 * cta + (lo > pos ? 0 : 1);
            if (!dealt) {
                more = 0;
            } else {
                if (s.units > 0 && k0 > 0 && k1 == count) {  // the end of an item that started elsewhere
                    const int first = shares.owner(pos + C::kCostItem);
                    prm.a.notes[cta] = make_int4(b, n, 2 * first + (shares.lo(first) > pos ? 0 : 1), 0);
                }
                pos += item_cost<C>(i);
                ++n;
                while (n >= items && pos < end && ++b < prm.a.batch) {
                    o = load_owner(prm, b, nullptr);
                    items = items_of(o.r);
                    n = 0;
                }
                more = pos < end && b < prm.a.batch;
            }
        }
        return s;
    }
};

// ---------------------------------------------------------------- the sums of one step
// e^(z - lse) of kN rows for the thread's column, summed.  list: -lse (log2 units), slopes and
// positions less the first row's, from the first of these rows on; away: the first row's position
// less the column.  A row sees the column where the distance, unsigned, is at most `most`.
// kFast: the column is seen by all, from no later position where heads have slopes, and capped products are small
// (CapPoly takes three pairs of four).
template <int kScore, bool kFast, int NQ, int kN>
__device__ __forceinline__ float sum_rows(const uint32_t (&s)[kN], const float *list, int away, uint32_t most, const ScoreScale &sc,
                                        const CapPoly &poly) {
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float base = (float)away;
#pragma unroll
    for (int e = 0; e < kN; e += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(list + e);
        float add[4] = {l.x, l.y, l.z, l.w};
        if constexpr (kScore & kBias) {
            const float4 k = *reinterpret_cast<const float4 *>(list + NQ + e), d = *reinterpret_cast<const float4 *>(list + 2 * NQ + e);
            const float ks[4] = {k.x, k.y, k.z, k.w}, ds[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) add[u] = fmaf(-ks[u], kFast ? base + ds[u] : fabsf(base + ds[u]), add[u]);
        }
        int4 r = make_int4(0, 0, 0, 0);
        if (!kFast) r = *reinterpret_cast<const int4 *>(list + 3 * NQ + e);
        const int rs[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
            const float s0 = __uint_as_float(s[e + u]), s1 = __uint_as_float(s[e + u + 1]);
            float2 x = (kScore & kCap) && kFast && (e + u) % 8 != 0 ? score_pair_poly(s0, s1, poly, add[u], add[u + 1])
                                                                   : score_pair<kScore>(s0, s1, sc, add[u], add[u + 1]);
            if (!kFast) {
                x.x = (uint32_t)(away + rs[u]) <= most ? x.x : -INFINITY;
                x.y = (uint32_t)(away + rs[u + 1]) <= most ? x.y : -INFINITY;
            }
            acc[u >> 1] = f2add(acc[u >> 1], make_float2(ex2(x.x), ex2(x.y)));
        }
    }
    return (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
}
// 16 consecutive 32-bit columns of this thread's lane, and the largest of them (kAbs: the largest magnitude)
template <bool kAbs>
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, uint32_t (&r)[16], float &most) {
#define DDT_LD16_MAX(abs)                                                                                                      \
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x16.max" abs ".f32 "                                                      \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"                                        \
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), \
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(most)        \
                 : "r"(taddr))
    if constexpr (kAbs) DDT_LD16_MAX(".abs");
    else DDT_LD16_MAX("");
#undef DDT_LD16_MAX
}

// ---------------------------------------------------------------- the kernel
template <int D, int NQ, int kScore>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1) chunk_weights_kernel(const __grid_constant__ Params prm) {
    using C = Cfg<D, NQ>;
    const ChunkArgs &a = prm.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + C::kOffHolder);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffHolder + 4);
    int64_t *plan = reinterpret_cast<int64_t *>(smem + C::kOffPlan);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = C::kThreads / 32;
    if (warp == C::kMmaWarp && lane == 0) {
        for (int i = 0; i < C::bCount; ++i)
            mbar_init(bar(i), i < C::bKEmpty                          ? 32 * C::kLoadWarps  // load lanes
                              : i >= C::bQFull && i < C::bQEmpty      ? 32 * C::kLoadWarps
                              : i >= C::bRFull && i < C::bREmpty      ? (NQ + 31) / 32
                              : i >= C::bREmpty && i < C::bSFull      ? C::kSoftWarps
                              : i >= C::bSEmpty && i < C::bDrain      ? 4 * C::kSplit
                              : i == C::bPair || i == C::bPairEmpty   ? 8
                              : i >= C::bSegEmpty                     ? C::kSoftWarps + C::kLoadWarps + 1
                                                                      : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait();

    // ---- this CTA's work ----
    const bool dealt = a.num_ctas > 0;
    using W = Walk<C, NQ>;
    W *walk = reinterpret_cast<W *>(smem + C::kOffWalk);
    static_assert(sizeof(W) <= C::kWalkBytes && sizeof(Segment) <= C::kSegBytes, "the walk's room");
    if (dealt) {
        int64_t *costs = reinterpret_cast<int64_t *>(smem + C::kOffCosts);
        for (int b = warp; b < a.batch; b += kWarps) {
            const Owner o = load_owner(prm, b, blockIdx.x == 0 && lane == 0 ? a.err : nullptr);
            const int items = items_of(o.r);
            int64_t sum = 0;
            for (int n = lane; n < items; n += 32) sum += item_cost<C>(item_of<NQ>(o.r, n, prm));
#pragma unroll
            for (int i = 16; i >= 1; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            if (lane == 0) costs[b] = sum;
        }
        if (tid == 0) a.notes[blockIdx.x] = make_int4(-1, 0, 0, 0);
        __syncthreads();
        const int64_t cost = tid < a.batch ? costs[tid] : 0;
        int64_t sum = cost;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, i);
            if (lane >= i) sum += x;
        }
        if (lane == 31) plan[warp] = sum;
        __syncthreads();
        int64_t total = 0, at = sum - cost;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += plan[w];
            total += plan[w];
        }
        const int64_t most = a.forced ? total / C::kCostStep : total / C::kMinShare;
        const int ctas = most < 1 ? 1 : most < a.num_ctas ? (int)most : a.num_ctas;
        if (total == 0 || (int)blockIdx.x >= ctas) return;
        Shares shares;
        shares.q = divide(total, ctas);
        shares.rem = total - shares.q * ctas;
        const int64_t lo = shares.lo(blockIdx.x);
        if (at <= lo && lo < at + cost) {  // the share starts in this thread's request
            walk->shares = shares;
            walk->end = shares.lo(blockIdx.x + 1);
            walk->b = tid;
            walk->cta = blockIdx.x;
            walk->dealt = walk->more = 1;
            walk->pos = at;
        }
        __syncthreads();
        if (warp == C::kFirstLoad) {  // and in which of its items
            const Owner o = load_owner(prm, walk->b, nullptr);
            const int items = items_of(o.r);
            int64_t pos = walk->pos;
            int item = 0;
            for (int n0 = 0; n0 < items; n0 += 32) {
                const int64_t own = n0 + lane < items ? item_cost<C>(item_of<NQ>(o.r, n0 + lane, prm)) : 0;
                int64_t ends = own;
#pragma unroll
                for (int i = 1; i < 32; i <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, ends, i);
                    if (lane >= i) ends += x;
                }
                const uint32_t behind = __ballot_sync(0xffffffffu, n0 + lane < items && pos + ends > lo);
                if (behind) {
                    const int n = __ffs(behind) - 1;
                    pos += __shfl_sync(0xffffffffu, ends - own, n);
                    item = n0 + n;
                    break;
                }
                pos += __shfl_sync(0xffffffffu, ends, 31);
            }
            __syncwarp();
            if (lane == 0) {
                walk->o = o;
                walk->items = items;
                walk->n = item;
                walk->pos = pos;
            }
            __syncwarp();
        }
    } else {
        const Owner o = load_owner(prm, blockIdx.z, blockIdx.x == 0 && tid == 0 ? a.err : nullptr);
        const int items = items_of(o.r);
        if ((int)blockIdx.x >= items) return;
        if (tid == 32 * C::kFirstLoad) {
            walk->o = o;
            walk->items = items;
            walk->b = blockIdx.z;
            walk->n = blockIdx.x;
            walk->cta = walk->dealt = 0;
            walk->more = 1;
        }
    }

    if (warp == C::kMmaWarp) tmem_alloc(smem_u32(holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    pdl_trigger();  // after the wait and the allocation, as in the attention
    volatile uint32_t *ring = reinterpret_cast<volatile uint32_t *>(smem + C::kOffWalk + C::kWalkBytes);
    constexpr int kSegWords = sizeof(Segment) / 4;
    auto read_segment = [&](int n, Segment &s) {
        uint32_t w[kSegWords];
#pragma unroll
        for (int i = 0; i < kSegWords; ++i) w[i] = ring[(n & 1) * (C::kSegBytes / 4) + i];
        memcpy(&s, w, sizeof s);
    };
    auto warp_segment = [&](int n, Segment &s) -> bool {
        if (!warp_wait(bar(C::bSegFull + (n & 1)), (n >> 1) & 1, abort_flag, a.err)) return false;
        read_segment(n, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bSegEmpty + (n & 1)));
        return true;
    };
    Segment sg;

    if (warp >= C::kFirstLoad && warp < C::kFirstLoad + C::kLoadWarps) {
        // ================= K and q rows =================
        constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows an instruction
        const int c = lane % kChunks, sub = lane / kChunks, lw = warp - C::kFirstLoad;
        const int64_t pitch = a.pool_stride * 2;
        int kn = 0, qn = 0;  // stages filled
        bool ok = true;
        auto in_log2 = [&](float x) { return fmaf(x, prm.log2e, x * prm.log2e_rest); };
        auto give_segment = [&](int n) {
            if (lw != 0) return;
            if (n >= 2) ok = warp_wait(bar(C::bSegEmpty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag, a.err);
            if (ok && lane == 0) {
                const Segment s = walk->next(prm);
                uint32_t w[kSegWords];
                memcpy(w, &s, sizeof s);
#pragma unroll
                for (int i = 0; i < kSegWords; ++i) ring[(n & 1) * (C::kSegBytes / 4) + i] = w[i];
                mbar_arrive(bar(C::bSegFull + (n & 1)));
            }
            __syncwarp();
        };
        give_segment(0);
        for (int seg = 0; ok; ++seg) {
            ok = warp_segment(seg, sg);
            if (!ok || sg.units == 0) break;
            give_segment(seg + 1);
            if (!ok) break;
            if (sg.steps <= 0) continue;
            int slot = a.kv_indices[sg.kv0 + min(sg.c0 + 32 * lw + lane, sg.N - 1)];  // past the end: a valid row again
            if (slot < 0 || slot >= a.pool_rows) {
                latch(a.err, DDT_DEVERR_KV_INDEX);
                slot = 0;
            }
            int g = sg.k0 / sg.tiles, tile = sg.k0 - g * sg.tiles;
            for (int k = 0; k < sg.steps; ++k) {
                if (k == 0 || tile == 0) {
                    const int s = kn % C::kKStages, u = kn / C::kKStages;
                    if (u > 0) ok = warp_wait(bar(C::bKEmpty + s), (u - 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    const char *pool = reinterpret_cast<const char *>(a.k_pool) + ((int64_t)g * D + c * 8) * 2;
                    const uint32_t to = sbase + C::kOffK + s * C::kKBytes + (lw >> 2) * (C::kKBytes / 2) + (c >> 3) * C::kKBoxBytes +
                                        (lw & 3) * 32 * 128;
#pragma unroll
                    for (int i = 0; i < 32 / kPer; ++i) {
                        const int r = i * kPer + sub;
                        cp_async_16(to + r * 128 + (((c & 7) ^ (r & 7)) << 4), pool + __shfl_sync(0xffffffffu, slot, r) * pitch);
                    }
                    cp_async_arrive(bar(C::bKFull + s));
                    ++kn;
                }
                const int s = qn % C::kQStages, u = qn / C::kQStages;
                const int rs = qn % C::kRStages, ru = qn / C::kRStages;
                const int first = tile * NQ, last = sg.rows - 1;
                const int t0 = first / prm.group, rem = first - t0 * prm.group;  // the first row's token, and head
                const int64_t row0 = (int64_t)(sg.qo0 + sg.token) * a.num_heads + g * prm.group;
                // this lane's row of the list beside the q tile
                const bool lists = 32 * lw < NQ && 32 * lw + lane < NQ;
                // (behind the last row: that one again, with a sum of infinity, which counts nothing)
                const int own = first + 32 * lw + lane, n = rem + min(own, last) - first;
                const int step = quotient(n, prm.group_inv), token = t0 + step, head = n - step * prm.group;
                float lse = INFINITY, slope = 0.f;
                if (lists && own <= last) {
                    lse = a.lse[row0 + (int64_t)token * a.num_heads + head];
                    if (kScore & kBias) slope = in_log2(a.slopes[g * prm.group + head]);
                }
                if (u > 0) ok = warp_wait(bar(C::bQEmpty + s), (u - 1) & 1, abort_flag, a.err);
                if (!ok) break;
                constexpr int kMine = NQ / C::kLoadWarps;  // q rows of a warp
                const uint32_t to = sbase + C::kOffQ + s * C::kQBytes + (c >> 3) * C::kQBoxBytes;
#pragma unroll
                for (int i = 0; i < (kMine + kPer - 1) / kPer; ++i) {
                    const int r = lw * kMine + i * kPer + sub;
                    if (kMine % kPer != 0 && i * kPer + sub >= kMine) continue;
                    const int m = rem + min(first + r, last) - first, t = quotient(m, prm.group_inv);  // past the end: the last row again
                    cp_async_16(to + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4),
                                a.q + (row0 + (int64_t)(t0 + t) * a.num_heads + m - t * prm.group) * D + c * 8);
                }
                cp_async_arrive(bar(C::bQFull + s));
                if (32 * lw < NQ) {
                    if (ru > 0) ok = warp_wait(bar(C::bREmpty + rs), (ru - 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    float *list = reinterpret_cast<float *>(smem + C::kOffRow + rs * C::kRowBytes);
                    if (lists) {
                        list[32 * lw + lane] = isinf(lse) ? -INFINITY : -in_log2(lse);  // a row that saw nothing counts nothing
                        list[NQ + 32 * lw + lane] = slope;
                        list[2 * NQ + 32 * lw + lane] = (float)(token - t0);
                        reinterpret_cast<int *>(list)[3 * NQ + 32 * lw + lane] = token - t0;
                    }
                    if (lw == 0 && lane == 0) reinterpret_cast<int *>(list)[4 * NQ] = sg.P + sg.token + t0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bRFull + rs));
                }
                ++qn;
                if (++tile == sg.tiles) {
                    tile = 0;
                    ++g;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may land after the CTA has left
    } else if (warp == C::kMmaWarp) {
        // ================= MMA =================
        if (elect_one()) {
            bool ok = true;
            int kn = 0, qn = 0;
            uint32_t tn0 = 0, tn1 = 0;  // score buffers of the two K tiles filled
            for (int seg = 0; ok; ++seg) {
                ok = wait_or_abort(bar(C::bSegFull + (seg & 1)), (seg >> 1) & 1, abort_flag, a.err);
                if (!ok) break;
                read_segment(seg, sg);
                mbar_arrive(bar(C::bSegEmpty + (seg & 1)));
                if (sg.units == 0) break;
                if (sg.steps <= 0) continue;
                int tile = sg.k0 % sg.tiles;
                const bool two = sg.N - sg.c0 > 128;
                for (int k = 0; k < sg.steps && ok; ++k) {
                    if (k == 0 || tile == 0) {
                        ok = wait_or_abort(bar(C::bKFull + kn % C::kKStages), (kn / C::kKStages) & 1, abort_flag, a.err);
                        if (!ok) break;
                        ++kn;
                    }
                    const int ks = (kn - 1) % C::kKStages, qs = qn % C::kQStages;
                    ok = wait_or_abort(bar(C::bQFull + qs), (qn / C::kQStages) & 1, abort_flag, a.err);
                    if (!ok) break;
                    fence_proxy_async_smem();
                    const uint64_t qd = smem_desc(sbase + C::kOffQ + qs * C::kQBytes, 16, 1024);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !two) break;
                        uint32_t &tn = t ? tn1 : tn0;
                        const int buf = 2 * t + (tn & 1);
                        if (tn >= 2) ok = wait_or_abort(bar(C::bSEmpty + buf), ((tn >> 1) - 1) & 1, abort_flag, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kd = smem_desc(sbase + C::kOffK + ks * C::kKBytes + t * (C::kKBytes / 2), 16, 1024);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            mma_ss(tmem + 128 * buf, kd + (((i >> 2) * C::kKBoxBytes + (i & 3) * 32) >> 4),
                                   qd + (((i >> 2) * C::kQBoxBytes + (i & 3) * 32) >> 4), C::kIdesc, i > 0);
                        mma_commit(bar(C::bSFull + buf));
                        ++tn;
                    }
                    if (!ok) break;
                    mma_commit(bar(C::bQEmpty + qs));
                    ++qn;
                    if (++tile == sg.tiles) tile = 0;
                    if (tile == 0 || k == sg.steps - 1) mma_commit(bar(C::bKEmpty + ks));
                }
            }
            mma_commit(bar(C::bDrain));  // every MMA issued has to be done before the exit
            mbar_wait(bar(C::bDrain), 0, kWaitLimit);
        }
        __syncwarp();
    } else if (warp < C::kSoftWarps) {
        // ================= sums (thread = column = TMEM lane of its tile) =================
        const int wq = warp & 3, t = (warp >> 2) & 1, half = warp >> 3;  // half: which rows of a step
        const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
        const ScoreScale sc = prm.score;
        CapPoly poly;
        if constexpr (kScore & kCap) poly.set(sc);
        int qn = 0;
        uint32_t tn = 0;
        bool ok = true;
        for (int seg = 0; ok; ++seg) {
            ok = warp_segment(seg, sg);
            if (!ok || sg.units == 0) break;
            const int j = sg.c0 + 128 * t + 32 * wq + lane;  // the thread's column
            const bool tile_on = sg.c0 + 128 * t < sg.N, full = j < sg.full;
            float total = 0.f;
            int tile = sg.k0 % sg.tiles;
            for (int k = 0; k < sg.steps; ++k) {
                const int qs = qn % C::kRStages;
                const float *list = reinterpret_cast<const float *>(smem + C::kOffRow + qs * C::kRowBytes);
                ok = warp_wait(bar(C::bRFull + qs), (qn / C::kRStages) & 1, abort_flag, a.err);
                if (!ok) break;
                if (tile_on) {
                    const int buf = 2 * t + (tn & 1);
                    const int *ints = reinterpret_cast<const int *>(list);
                    const int away = ints[4 * NQ] - j;                       // the first row's position less the column
                    const int spread = (sg.rows - tile * NQ < NQ) ? -1 : ints[4 * NQ - 1];  // the last one's less the first one's
                    const bool lane_fast = (full || (away >= 0 && (a.window <= 0 || away + spread < a.window))) &&
                                           (!(kScore & kBias) || away >= 0);
                    const bool fast = spread >= 0 && __all_sync(0xffffffffu, lane_fast);
                    const uint32_t most = full ? 0xffffffffu : a.window > 0 ? (uint32_t)a.window - 1u : 0x7fffffffu;
                    ok = warp_wait(bar(C::bSFull + buf), (tn >> 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t col = tmem + lane_off + 128 * buf;
                    float sum = 0.f;
                    // (16 rows at a time, in a loop that is not unrolled: 32 in a go take 9% longer, the next 16
                    // loaded ahead 22% (two capped chunks of 2048): they outgrow the instruction cache)
#pragma unroll 1
                    for (int n = NQ / C::kSplit * half; n < NQ / C::kSplit * (half + 1); n += 16) {
                        uint32_t s[16];
                        float r;
                        tmem_ld16_max<(kScore & kCap) != 0>(col + n, s, r);
                        tmem_wait_ld();
                        bool quick = fast;
                        if constexpr (kScore & kCap) quick = fast && __all_sync(0xffffffffu, r < prm.cap_most);
                        sum += quick ? sum_rows<kScore, true, NQ, 16>(s, list + n, away, most, sc, poly)
                                     : sum_rows<kScore, false, NQ, 16>(s, list + n, away, most, sc, poly);
                    }
                    total += sum;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bSEmpty + buf));
                    ++tn;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bREmpty + qs));
                ++qn;
                if (++tile == sg.tiles) tile = 0;
            }
            if (!ok) break;
            if constexpr (C::kSplit == 2) {
                float *place = reinterpret_cast<float *>(smem + C::kOffPair) + 128 * t + 32 * wq + lane;
                if (half == 1) {
                    if (seg > 0) ok = warp_wait(bar(C::bPairEmpty), (seg - 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    *place = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bPair));
                    continue;
                }
                ok = warp_wait(bar(C::bPair), seg & 1, abort_flag, a.err);
                if (!ok) break;
                total += *place;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bPairEmpty));
            }
            if (sg.part >= 0) {
                a.o_part[(int64_t)sg.part * kCols + 128 * t + 32 * wq + lane] = total;
            } else if (j < sg.N) {
                if (j < sg.prevs) total += prm.w.decay * prm.w.prev[(int64_t)sg.prev0 + j];
                prm.w.weights[(int64_t)sg.kv0 + j] = total;
            }
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The item that ends in a CTA's share: its parts added up in the order of its steps.
template <int NQ>
__global__ void __launch_bounds__(kCols) chunk_weights_join(const __grid_constant__ Params prm) {
    pdl_wait();
    pdl_trigger();
    const int4 note = prm.a.notes[blockIdx.x];
    if (note.x < 0) return;
    const Owner o = load_owner(prm, note.x, nullptr);
    const int64_t j = (int64_t)note.y * kCols + threadIdx.x;
    if (j >= o.r.N) return;
    const int c0 = note.z >> 1, parts = (int)blockIdx.x - c0 + 1;
    float sum = prm.a.o_part[(int64_t)note.z * kCols + threadIdx.x];
    for (int s = 1; s < parts; s += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = s + u < parts ? prm.a.o_part[(int64_t)2 * (c0 + s + u) * kCols + threadIdx.x] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += v[u];
    }
    if (j < o.prevs) sum += prm.w.decay * prm.w.prev[o.prev0 + j];
    prm.w.weights[o.r.kv0 + j] = sum;
}

template <int D, int NQ, int kScore>
cudaError_t launch_weights_one(Params &prm, cudaStream_t s) {
    using C = Cfg<D, NQ>;
    const ChunkArgs &a = prm.a;
    const dim3 grid = a.num_ctas > 0 ? dim3((unsigned)a.num_ctas) : dim3((unsigned)prm.items_most, 1, (unsigned)a.batch);
    cudaError_t e = launch_pdl(chunk_weights_kernel<D, NQ, kScore>, grid, dim3(C::kThreads), C::kSmemBytes, s, prm);
    if (e == cudaSuccess && a.num_ctas > 1)
        e = launch_pdl(chunk_weights_join<NQ>, dim3((unsigned)a.num_ctas), dim3(kCols), 0, s, prm);
    return e;
}
template <int D, int NQ, int kScore>
cudaError_t prepare_weights_one() {
    const cudaError_t e = cudaFuncSetAttribute(chunk_weights_kernel<D, NQ, kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg<D, NQ>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(chunk_weights_kernel<D, NQ, kScore>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                (int)cudaSharedmemCarveoutMaxShared);
}
template <int kScore>
cudaError_t launch_weights_score(Params &prm, int nq, cudaStream_t s) {
    if (prm.a.head_dim == 128) return nq == 16 ? launch_weights_one<128, 16, kScore>(prm, s) : launch_weights_one<128, 128, kScore>(prm, s);
    return nq == 16 ? launch_weights_one<64, 16, kScore>(prm, s) : launch_weights_one<64, 128, kScore>(prm, s);
}
template <int kScore>
cudaError_t prepare_weights_score() {
    cudaError_t e = prepare_weights_one<64, 16, kScore>();
    if (e == cudaSuccess) e = prepare_weights_one<64, 128, kScore>();
    if (e == cudaSuccess) e = prepare_weights_one<128, 16, kScore>();
    if (e == cudaSuccess) e = prepare_weights_one<128, 128, kScore>();
    return e;
}

}  // namespace received
}  // namespace chunk
}  // namespace ddt
