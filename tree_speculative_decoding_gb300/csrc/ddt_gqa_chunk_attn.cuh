// ddt_gqa_chunk_attn.cuh -- attention of a chunk of new tokens over grouped-query K/V
// rows on the sm_103a tensor cores: the kernel, and the joining of split items.
//
// For row (token i of request b, head h), K/V head g = h / group, over the columns j
// that the token sees (ddt_gqa_chunk.cuh has scores and visibility):
//   out[i,h] = sum_j softmax(z)_j v[idx_j][g],  lse = log sum_j e^{z_j}.
//
// Work.  An item is one K/V head of one request and up to kTiles tiles of 128
// consecutive rows (token-major, the group's heads inside a token: the rows that share
// the K/V head).  Its blocks of columns are those that its first or last token sees,
// latest first: the first block then holds what a row weighs most where weights fall
// with distance, and the reference (below) seldom moves.
//   * kTiles = 1: blocks of 64 columns, 256 tensor-memory columns and under half of the
//     shared memory, so two CTAs share an SM (decode, small chunks: the loads bound it).
//   * kTiles = 2: blocks of 128 columns, all of tensor memory; the tensor core works on
//     one tile while the softmax of the other runs.  Where an item's last rows fill one
//     tile only, its blocks alternate between the two tiles' warps and outputs, each with a
//     reference and sum of its own, and the two are joined at the end.
// A CTA takes one item; or the blocks of all items, weighted by what they cost, form one
// line (request, K/V head, rows, columns) that is dealt to the resident CTAs in equal
// shares: a CTA takes the end of one item, whole items, and the start of another.  Every
// CTA finds the cuts from the offsets.  Cut items leave partial results (at most two per
// CTA) in the workspace, and the CTA with an item's end a note for the kernel that joins them.
//
// estimate() weighs the four ways.
//
// Measured, D = 128, 64 heads on 8 but where stated: a prompt of 8192 880 us, 1250 TFLOP/s of what is
// seen; 2048 tokens after 30720, 32 heads on 4, 798 to 830 us by the GPU's clocks (products alone would take 537,
// with loads 575, with the softmax 750), with a cap 1294 us; 64 tokens of 64 requests in windows of 4096
// 171 us, 5.9 TB/s.  Two tiles are bound by a tile's chain (scores, softmax, products): ~3300 clk a
// block where its products take 2048, with the exponentials at 27% and issue at 45% of their rates;
// one tile with few rows by memory.
//
// Score slots: two buffers of one block's scores in tensor memory.  The MMA warp issues
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
// P (bf16) overwrites the scores in place and is the A operand of PV from tensor memory;
// V is read as an MN-major operand from its rows.
//
// The softmax takes weights against the row's reference, the maximum of the first columns it saw
// plus kShift.  The tensor-memory load brings the largest product of every 32 columns with it: only
// where a score could pass the reference by 2^22 the reference moves, and the sums so far are scaled.
// kShift keeps every sum finite: a row's weights sum to 1 at most, so its result is at most the
// largest |v|.
// Statistics, sums and partial results are fp32; the weights are rounded to bf16 for the
// product with V, since the tensor core takes both operands in V's type (2^-8 of each at most).
//
// Infinities and NaN in V: a weight of 0 times NaN is NaN, so a V row that some row of the
// item does not see may not reach the products with such a value.  V rows that no row of the
// item sees are zeros; in those that some see and others do not the load warps replace it by 0 and
// keep the rows that do see it as bits (poison), which are added to the results behind the epilogue.
//
// Every wait is bounded: on timeout the CTA latches DDT_DEVERR_TIMEOUT, waits for its own
// copies and MMAs and leaves.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ddt_gqa_chunk.cuh"

namespace ddt {
namespace chunk {

using namespace sm100;

constexpr int kRows = 128;  // rows per tile (TMEM lanes)
// Cost of an item besides its blocks (Cfg::kCostItem): with 40 instead of 80 the CTAs of a prompt of 8192, dealt,
// end 12% apart, with 120 it takes 893 us where it takes 872.
//
// Weights against the reference: 2^-kShift where the reference was found, 2^-kMost at most, so that
// 2^31 columns sum to 1 at most.  A value's weight loses bits below 2^-126, which for the heaviest
// columns is |v| below 2^-73.
constexpr float kShift = 53.f, kMost = 31.f, kUnshift = 0x1p53f;

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void cp_async_16_or_0(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

struct AttnParams {
    CUtensorMap k_map, v_map;  // the pools as [pool_rows][K/V heads * D], boxes of 16 rows x 64 values
    ChunkArgs a;
    int group;        // query heads per K/V head
    float group_inv;  // 1 / group
    int part_rows;    // rows of a partial result
    int tgs_most;     // items per K/V head of the longest request
    ScoreScale score;
    float cap_most;   // products below this may use it
};

template <int D, int kTiles>
struct Cfg {
    static constexpr int NB = kTiles == 2 ? 128 : 64;    // columns per block
    static constexpr int kPer = kTiles * kRows;          // rows of an item
    static constexpr int kHalves = NB / 64;              // parts of P that PV may start on
    static constexpr int kBoxes = D / 64;                // 128-byte pieces of a row
    static constexpr int kBoxBytes = NB * 128;           // one piece of a block's rows
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
    static constexpr int kQBoxBytes = kRows * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;  // one tile of q
    static constexpr int kKStages = D == 128 ? 2 : 4;
    static constexpr int kVStages = D == 128 ? 2 : 4;
    static constexpr int kUnits = NB / 32;               // 32-row units of a block
    static constexpr int kSoftWarps = 4 * kTiles;
    // two tiles: warps 8..11 load K, 12..15 V, 16 issues MMAs, 17..19 load q; one tile: warp 4
    // issues MMAs, 5..7 load K and V, the softmax warps load their rows of q
    static constexpr int kLoadWarps = kTiles == 2 ? 2 * kUnits : 3;
    static constexpr int kFirstLoad = kTiles == 2 ? kSoftWarps : kSoftWarps + 1;
    static constexpr int kMmaWarp = kTiles == 2 ? kSoftWarps + kLoadWarps : kSoftWarps;
    static constexpr int kQWarps = kTiles == 2 ? 3 : kSoftWarps;
    static constexpr int kThreads = kTiles == 2 ? 640 : 256;
    // registers of the two-tile kernel: a softmax thread's, another's; together no more than at launch
    static constexpr int kSoftRegs = 120, kOtherRegs = 72, kLaunchRegs = 96;
    static_assert(32 * kSoftWarps * kSoftRegs + (640 - 32 * kSoftWarps) * kOtherRegs <= 640 * kLaunchRegs || kTiles == 1, "registers");
    static constexpr uint32_t kTmemCols = kTiles == 2 ? 512 : 256;
    static constexpr uint32_t kColS = 0, kColO = 2 * NB;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTiles * kQBytes;
    static constexpr int kOffV = kOffK + kKStages * kBlockBytes;
    // rows on their way out, 64 bytes of each: with one tile the place of q, which nothing reads then
    static constexpr int kOffStage = kTiles == 2 ? kOffV + kVStages * kBlockBytes : kOffQ;
    static constexpr int kStageBytes = 2048;  // per softmax warp
    static constexpr int kPoisonWords = D * 2 * (kPer / 32);
    static constexpr int kOffPoison = kOffV + kVStages * kBlockBytes + (kTiles == 2 ? kSoftWarps * kStageBytes : 0);
    static constexpr int kOffBar = kOffPoison + 4 * kPoisonWords;
    // barriers
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bVFull = bKEmpty + kKStages,
                         bVEmpty = bVFull + kVStages, bSFull = bVEmpty + kVStages, bPFull = bSFull + 2,
                         bQFull = bPFull + 2 * kHalves, bQEmpty = bQFull + 1, bHalf = bQEmpty + 1, bODone = bHalf + 2, bJoin = bODone + 1,
                         bOFin = bJoin + 1, bDrain = bOFin + 1, bSegDone = bDrain + 1, bSegFull = bSegDone + 2,
                         bSegEmpty = bSegFull + 2, bCount = bSegEmpty + 2;
    static constexpr int kOffHolder = kOffBar + 8 * bCount;  // tensor memory, abort, poison in use, -
    static constexpr int kOffWalk = kOffHolder + 16;
    static constexpr int kWalkBytes = 128, kSegBytes = 96;
    static constexpr int kOffPlan = kOffWalk + kWalkBytes + 2 * kSegBytes;  // a sum per warp; the share's request
    static constexpr int kOffJoin = kOffPlan + 8 * (kThreads / 32) + 32;  // the second tile's references and sums
    static constexpr int kSmemUsed = kOffJoin + (kTiles == 2 ? kRows * 8 : 0);
    static constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for the 1024-byte alignment of swizzle atoms
    static constexpr int kOffCosts = kOffK;  // while the work is dealt: a cost per request
    static constexpr uint32_t kIdescS = idesc_bf16(kRows, NB, 0, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16(kRows, D, 0, 1);
    // Cost of a block with all tiles and with one, in one unit; of an item besides its blocks; the
    // share that a CTA gets at least.
    static constexpr int kCostFull = kTiles == 2 ? 16 : 8, kCostOne = kTiles == 2 ? 11 : 8;
    static constexpr int kCostItem = kTiles == 2 ? 80 : 48, kMinShare = kTiles == 2 ? 56 : 32;
    static_assert(kTiles == 2 || kKStages >= 2, "see the load warps");
    static_assert(kOffPlan % 8 == 0 && kOffWalk % 8 == 0 && kOffBar % 8 == 0, "alignment");
    static_assert(kColO + kTiles * D <= kTmemCols, "tensor memory");
    static_assert(kSmemBytes <= (kTiles == 2 ? 232448 : 115712), "shared memory");
};

// ---------------------------------------------------------------- items
// Item tg of a request's K/V head: rows [tg kPer, ...), its tokens' positions and its blocks.
struct Item {
    int rows, node0, rem0;  // rows; token and head (within the group) of the first one
    int pa, pb;             // positions of its first and last token
    Blocks x;
};
template <class C>
__device__ __forceinline__ int items_of(const Request &r, int group) {
    return (int)(((int64_t)r.T * group + C::kPer - 1) / C::kPer);
}
template <class C>
__device__ __forceinline__ Item item_of(const Request &r, int tg, int group, float group_inv, int window) {
    Item i;
    const int row0 = tg * C::kPer;
    i.rows = min(C::kPer, r.T * group - row0);
    i.node0 = tg == 0 ? 0 : (int)((uint32_t)row0 / (uint32_t)group);
    i.rem0 = row0 - i.node0 * group;
    i.pa = r.N - r.T + i.node0;
    i.pb = i.pa + quotient(i.rem0 + i.rows - 1, group_inv);
    i.x = blocks_of<C::NB>(i.pa, i.pb, window, r.full);
    return i;
}
template <class C>
__device__ __forceinline__ int unit_cost(const Item &i) {
    return C::kPer == 2 * kRows && i.rows <= kRows ? C::kCostOne : C::kCostFull;
}
template <class C>
__device__ __forceinline__ int64_t item_cost(const Item &i) {
    return C::kCostItem + (int64_t)i.x.count * unit_cost<C>(i);
}
// the item's blocks that start before position x (block k starts kCostItem + k unit behind the item)
template <class C>
__device__ __forceinline__ int blocks_before(int64_t item, int64_t x, int unit, int count) {
    const int64_t d = x - (item + C::kCostItem);
    if (d <= 0) return 0;
    // (by constants: a division by a variable takes longer than the rest of the walk's step)
    const uint64_t k = C::kCostOne == C::kCostFull || unit == C::kCostFull ? (uint64_t)(d + C::kCostFull - 1) / C::kCostFull
                                                                           : (uint64_t)(d + C::kCostOne - 1) / C::kCostOne;
    return k < (uint64_t)count ? (int)k : count;
}

// What a CTA does in one go: blocks k0 .. k0 + blocks - 1 of an item.
struct Segment {
    int rows, tiles;  // rows of the item; tiles of 128
    int node0, rem0, pa, pb;
    int g, k0, blocks;
    Blocks x;
    int qo0, kv0, N, full;  // of the request
    int part;               // -1: the whole item, else the place of the partial result
};
// first column of the segment's n-th block
template <class C>
__device__ __forceinline__ int block_column(const Segment &s, int n) {
    const int at = s.x.count - 1 - s.k0 - n;  // latest first
    return (at < s.x.a ? at : s.x.l - s.x.a + at) * C::NB;
}

// The walk over the CTA's segments.  It lives in shared memory: one thread steps it and
// hands the segments to the warps through a ring of two.
template <class C>
struct Walk {
    int64_t pos, end;  // the item's position on the line; the end of the CTA's share
    Shares shares;
    Request r;
    int b, tg, g, cta, tgs;
    int dealt, more;

    // the next segment into `to`; one without blocks when the share is done
    __device__ __forceinline__ void next(const AttnParams &prm, Segment *to) {
        const ChunkArgs &a = prm.a;
        Segment s;
        s.blocks = 0;
        while (more && s.blocks == 0) {
            const Item i = item_of<C>(r, tg, prm.group, prm.group_inv, a.window);
            const int unit = unit_cost<C>(i);
            const int64_t lo = dealt ? shares.lo(cta) : 0;
            const int b0 = dealt ? blocks_before<C>(pos, lo, unit, i.x.count) : 0;
            const int b1 = dealt ? blocks_before<C>(pos, end, unit, i.x.count) : i.x.count;
            s.rows = i.rows;
            s.tiles = (i.rows + kRows - 1) / kRows;
            s.node0 = i.node0;
            s.rem0 = i.rem0;
            s.pa = i.pa;
            s.pb = i.pb;
            s.g = g;
            s.k0 = b0;
            s.blocks = b1 - b0;
            s.x = i.x;
            s.qo0 = r.qo0;
            s.kv0 = r.kv0;
            s.N = r.N;
            s.full = r.full;
            // at most one item of a share starts before it, and at most one ends behind it
            s.part = s.blocks == i.x.count ? -1 : 2 * cta + (lo > pos ? 0 : 1);
            if (!dealt) {
                more = 0;
            } else {
                if (s.blocks > 0 && b0 > 0 && b1 == i.x.count) {  // the end of an item that started elsewhere
                    const int first = shares.owner(pos + C::kCostItem);
                    a.notes[cta] = make_int4(b, g, tg, 2 * first + (shares.lo(first) > pos ? 0 : 1));
                }
                pos += C::kCostItem + (int64_t)i.x.count * unit;
                if (++tg == tgs) {
                    tg = 0;
                    ++g;
                }
                while ((g >= a.num_kv_heads || tgs == 0) && pos < end && ++b < a.batch) {  // the next request with items
                    r = load_request(a, b, nullptr);
                    tgs = items_of<C>(r, prm.group);
                    tg = g = 0;
                }
                more = pos < end && b < a.batch;
            }
        }
        *to = s;
    }
};

// ---------------------------------------------------------------- weights of 64 columns
// The weights of the products s (columns c .. c + 63 of a row at position p) against the reference
// m as bf16 pairs, handed to store(k, pairs) 32 columns at a time.  Returns their sum.
// kFast: all 64 are seen, at columns up to p where `slope` is not 0, and products that are capped
// are small enough for CapPoly (but for kSpecial pairs of 16, which balance the units: 2048 tokens after 30720 take
// 1342, 1312, 1294, 1309 us with 1, 2, 4, 8).
constexpr int kSpecial = 4;
template <int kScore, bool kFast, class Store>
__device__ __forceinline__ float weights_64(const uint32_t (&s)[2][32], uint32_t seen0, uint32_t seen1, int c, int p, float m, float slope,
                                            const ScoreScale &sc, const CapPoly &poly, Store store) {
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float away = (float)(c - p);  // column less position
    // (from the last column, the nearest, on: what is added to it is rounded by the columns' own distances, from the
    // first one on it would be by 63 slope next to the token)
    const float base = (kScore & kBias) && kFast ? fmaf(slope, (float)(c + 63 - p), -m) : -m;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t seen = k ? seen1 : seen0;
        uint32_t pw[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float add0 = base, add1 = base;
            if constexpr (kScore & kBias) {
                const int n = 32 * k + e;
                if (kFast) {
                    add0 = fmaf(slope, (float)(n - 63), base);
                    add1 = fmaf(slope, (float)(n - 62), base);
                } else {
                    add0 = fmaf(-slope, fabsf(away + (float)n), base);
                    add1 = fmaf(-slope, fabsf(away + (float)(n + 1)), base);
                }
            }
            constexpr bool kPoly = (kScore & kCap) && kFast;
            const float s0 = __uint_as_float(s[k][e]), s1 = __uint_as_float(s[k][e + 1]);
            float2 x = kPoly && (e >> 1) % 16 * kSpecial % 16 >= kSpecial ? score_pair_poly(s0, s1, poly, add0, add1)
                                                                        : score_pair<kScore>(s0, s1, sc, add0, add1);
            if (!kFast) {
                x.x = (seen >> e) & 1u ? x.x : -INFINITY;
                x.y = (seen >> (e + 1)) & 1u ? x.y : -INFINITY;
            }
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            acc[(e >> 1) & 1] = f2add(acc[(e >> 1) & 1], make_float2(p0, p1));
            pw[e / 2] = pack_bf16(p0, p1);
        }
        store(k, pw);
    }
    return (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
}
// What a row's largest score is found with: of 64 columns from c on the largest seen product, or
// (where heads have slopes, which change the order) the largest seen score; then the score of that.
template <int kScore>
__device__ __forceinline__ float reach_64(const uint32_t (&s)[2][32], uint32_t seen0, uint32_t seen1, int c, int p, const ScoreScale &sc) {
    float mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        float2 x = make_float2(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1]));
        if constexpr (kScore & kBias)
            x = score_pair<kScore>(x.x, x.y, sc, -sc.slope * fabsf((float)(c + e - p)), -sc.slope * fabsf((float)(c + e + 1 - p)));
        const uint32_t seen = (e < 32 ? seen0 : seen1) >> (e & 31);
        if (seen & 1u) mx = fmaxf(mx, x.x);
        if (seen & 2u) mx = fmaxf(mx, x.y);
    }
    return mx;
}
// The largest score of columns up to p that are all seen.
__device__ __forceinline__ float reach_linear(const uint32_t (&s)[2][32], int c, int p, const ScoreScale &sc) {
    float mx = -INFINITY;
    const float base = sc.slope * (float)(c - p);
#pragma unroll
    for (int e = 0; e < 64; ++e) mx = fmaxf(mx, fmaf(__uint_as_float(s[e >> 5][e & 31]), sc.lin, fmaf(sc.slope, (float)e, base)));
    return mx;
}
template <int kScore>
__device__ __forceinline__ float reached(float mx, bool some, const ScoreScale &sc) {
    if (!some || (kScore & kBias)) return mx;
    return score_pair<kScore>(mx, mx, sc, 0.f, 0.f).x;
}

// halves of a word whose exponent is all ones: bits 15 and 31
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// One row's 8 values of V at `at`, of column j: infinities and NaN become 0, and the rows of the
// item that see the column get them in `poison`, the words of these values (shared-memory addresses).
template <class C>
__device__ __noinline__ void poison_8(uint32_t at, int j, uint32_t poison, int rows_all, int rem0, int pa, float group_inv, int window,
                                      int full, int N) {
    constexpr int kWords = C::kPer / 32;
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
#pragma unroll 1
    for (int w = 0; w < kWords; ++w) {
        uint32_t rows = 0;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            const int r = 32 * w + i;
            const int p = pa + quotient(rem0 + r, group_inv);
            if (r < rows_all && (seen_bits(j, p, window, full, N) & 1u)) rows |= 1u << i;
        }
        if (rows == 0) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t y = (x[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            if ((y & 0x7f80u) != 0x7f80u) continue;
            const bool nan = (y & 0x7fu) != 0, minus = (y >> 15) != 0;
            const uint32_t to = poison + 4 * (2 * e * kWords + w);
            if (nan || !minus) asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(to), "r"(rows) : "memory");
            if (nan || minus) asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(to + 4 * kWords), "r"(rows) : "memory");
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t bad = not_finite(x[e]);
        if (bad & 0x8000u) x[e] &= 0xffff0000u;
        if (bad & 0x80000000u) x[e] &= 0x0000ffffu;
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}

// ---------------------------------------------------------------- the kernel
template <int D, int kTiles, int kScore>
__global__ void __launch_bounds__(Cfg<D, kTiles>::kThreads, kTiles == 2 ? 1 : 2)
chunk_attn_kernel(const __grid_constant__ AttnParams prm) {
    using C = Cfg<D, kTiles>;
    constexpr int NB = C::NB;
    const ChunkArgs &a = prm.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + C::kOffHolder);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffHolder + 4);
    volatile int *poisoned = reinterpret_cast<volatile int *>(smem + C::kOffHolder + 8);  // some segment had poison
    uint32_t *poison = reinterpret_cast<uint32_t *>(smem + C::kOffPoison);  // [value][+, -][rows / 32]
    int64_t *plan = reinterpret_cast<int64_t *>(smem + C::kOffPlan);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kMmaWarp = C::kMmaWarp, kFirstLoad = C::kFirstLoad, kWarps = C::kThreads / 32;
    if (warp == kMmaWarp && lane == 0) {
        for (int i = 0; i < C::bCount; ++i)
            mbar_init(bar(i), i < C::bKEmpty || (i >= C::bVFull && i < C::bVEmpty) ? 32 * C::kUnits  // load lanes
                      : i >= C::bPFull && i < C::bQFull                            ? 4               // row quarters
                      : i == C::bQFull                                             ? C::kQWarps
                      : i == C::bJoin                                              ? 4
                      : i >= C::bSegDone && i < C::bSegFull                        ? C::kSoftWarps
                      : i >= C::bSegEmpty ? C::kSoftWarps + C::kLoadWarps + 1 + (kTiles == 2 ? C::kQWarps : 0)
                                          : 1);
        *abort_flag = 0;
        *poisoned = 0;
        fence_barrier_init();
    }
    for (int i = tid; i < C::kPoisonWords; i += C::kThreads) poison[i] = 0;
    // everything read below may be the previous kernel's output
    pdl_wait();

    // ---- this CTA's work ----
    const bool dealt = a.num_ctas > 0;
    Walk<C> *walk = reinterpret_cast<Walk<C> *>(smem + C::kOffWalk);
    static_assert(sizeof(Walk<C>) <= C::kWalkBytes && sizeof(Segment) <= C::kSegBytes, "the walk's room");
    if (dealt) {
        // a warp sizes a request (lanes take its items in turn), a scan places them on the line
        int64_t *costs = reinterpret_cast<int64_t *>(smem + C::kOffCosts);
        for (int b = warp; b < a.batch; b += kWarps) {
            const Request r = load_request(a, b, blockIdx.x == 0 && lane == 0 ? a.err : nullptr);
            const int tgs = items_of<C>(r, prm.group);
            int64_t sum = 0;
            for (int tg = lane; tg < tgs; tg += 32) sum += item_cost<C>(item_of<C>(r, tg, prm.group, prm.group_inv, a.window));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) costs[b] = sum;
        }
        if (tid == 0) a.notes[blockIdx.x] = make_int4(-1, 0, 0, 0);
        __syncthreads();
        const int64_t head = tid < a.batch ? costs[tid] : 0, cost = head * a.num_kv_heads;
        int64_t sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) plan[warp] = sum;
        fence_proxy_async_smem();  // the costs' place is K's, which tile copies write
        __syncthreads();
        int64_t total = 0, at = sum - cost;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += plan[w];
            total += plan[w];
        }
        // CTAs that take a share: as many as get a few blocks at least
        const int64_t most = a.forced ? total / C::kCostFull : total / C::kMinShare;
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
            walk->g = (int)divide(lo - at, head);
            walk->pos = at + walk->g * head;
        }
        __syncthreads();
        if (warp == kFirstLoad) {  // and in which of its items
            const Request r = load_request(a, walk->b, nullptr);
            const int tgs = items_of<C>(r, prm.group);
            int64_t pos = walk->pos;
            int tg = 0;
            for (int t0 = 0; t0 < tgs; t0 += 32) {
                const int64_t own = t0 + lane < tgs ? item_cost<C>(item_of<C>(r, t0 + lane, prm.group, prm.group_inv, a.window)) : 0;
                int64_t ends = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, ends, o);
                    if (lane >= o) ends += x;
                }
                const uint32_t behind = __ballot_sync(0xffffffffu, t0 + lane < tgs && pos + ends > lo);
                if (behind) {
                    const int n = __ffs(behind) - 1;
                    pos += __shfl_sync(0xffffffffu, ends - own, n);
                    tg = t0 + n;
                    break;
                }
                pos += __shfl_sync(0xffffffffu, ends, 31);
            }
            __syncwarp();
            if (lane == 0) {
                walk->r = r;
                walk->tgs = tgs;
                walk->tg = tg;
                walk->pos = pos;
            }
            __syncwarp();
        }
    } else {
        const int b = blockIdx.z, n = blockIdx.x / a.num_kv_heads;
        const Request r = load_request(a, b, blockIdx.x == 0 && tid == 0 ? a.err : nullptr);
        const int tgs = items_of<C>(r, prm.group);
        if (n >= tgs) return;
        if (tid == 32 * kFirstLoad) {
            walk->r = r;
            walk->b = b;
            walk->tgs = tgs;
            walk->tg = tgs - 1 - n;  // the longest first
            walk->g = blockIdx.x - n * a.num_kv_heads;
            walk->cta = walk->dealt = 0;
            walk->more = 1;
        }
    }

    if (warp == kMmaWarp) tmem_alloc(smem_u32(holder), C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    // After the wait: what starts early behind this kernel sees everything before it.
    // After the allocation: a CTA that starts early cannot take the tensor memory that
    // this one still needs while it waits for this one's end.
    pdl_trigger();
    volatile uint32_t *ring = reinterpret_cast<volatile uint32_t *>(smem + C::kOffWalk + C::kWalkBytes);
    constexpr int kSegWords = sizeof(Segment) / 4;
    // segment n of the CTA; the caller's thread or warp reads it once
    auto read_segment = [&](int n, Segment &s) {
        uint32_t w[kSegWords];
#pragma unroll
        for (int i = 0; i < kSegWords; ++i) w[i] = ring[(n & 1) * (C::kSegBytes / 4) + i];
        memcpy(&s, w, sizeof s);
    };
    auto warp_segment = [&](int n, Segment &s) -> bool {  // false: the wait ran out
        if (!warp_wait(bar(C::bSegFull + (n & 1)), (n >> 1) & 1, abort_flag, a.err)) return false;
        read_segment(n, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bSegEmpty + (n & 1)));
        return true;
    };
    // by one warp: segment n for all of them
    auto give_segment = [&](int n) -> bool {
        if (n >= 2 && !warp_wait(bar(C::bSegEmpty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag, a.err)) return false;
        if (lane == 0) {
            walk->next(prm, reinterpret_cast<Segment *>(smem + C::kOffWalk + C::kWalkBytes + (n & 1) * C::kSegBytes));
            mbar_arrive(bar(C::bSegFull + (n & 1)));
        }
        __syncwarp();
        return true;
    };
    // rows r0, r0 + 32, ... below r1 of the segment's q, one warp, into the swizzled operand layout
    auto load_q = [&](const Segment &s, int r0, int r1, int step) {
        constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows per instruction
        const int c = lane % kChunks, sub = lane / kChunks;
        const uint32_t qb = sbase + C::kOffQ + (c >> 3) * C::kQBoxBytes;
        const uint16_t *q = a.q + ((int64_t)(s.qo0 + s.node0) * a.num_heads + s.g * prm.group) * D + c * 8;
        const int end = min(r1, s.rows);
        for (int r = r0; r < end; r += step) {
#pragma unroll 4
            for (int i = 0; i < 32 / kPer; ++i) {
                const int rr = r + i * kPer + sub, rt = rr & (kRows - 1);
                if (rr < end) {
                    const int n = s.rem0 + rr, node = quotient(n, prm.group_inv), hg = n - node * prm.group;
                    cp_async_16(qb + (rr / kRows) * C::kQBytes + (rt >> 3) * 1024 + (rt & 7) * 128 + (((c & 7) ^ (rt & 7)) << 4),
                                q + ((int64_t)node * a.num_heads + hg) * D);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bQFull));
    };
    // What a wait until the softmax warps have left segment n waits for, and its parity.  Two barriers in turn: the
    // ring hands segment n + 1 out once all have left n - 2, so of n's barrier the phase before n's is
    // over, and the one behind it cannot end without who waits.  (With one barrier a wait in segment n + 1 would also
    // pass while n - 1 is still being left.)
    auto seg_done = [&](int n) { return bar(C::bSegDone + (n & 1)); };
    auto seg_parity = [](int n) { return (uint32_t)(n >> 1) & 1u; };
    Segment sg;

    if (warp >= C::kSoftWarps) {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp >= kFirstLoad && warp < kFirstLoad + C::kLoadWarps) {
            // ================= K and V rows =================
            // A unit is 32 rows of a block of K or V.  Two-tile kernel: a warp has the same
            // unit of every block of K, or of V.  One-tile kernel: three warps take the units
            // in turn in the order K(0) K(1) V(0) K(2) V(1) ... V(blocks - 1).
            //
            // An "empty" wait goes by the phase's parity, so a warp may not reach a use of a
            // stage while the use two before is still to be read.  Where a warp has a unit of
            // every block its own last wait excludes that.  In the one-tile order the unit
            // before one of V(j) is of K(j) at the earliest (whose wait implies PV(j - 4) is
            // done, with two stages), the one before K(j) of V(j - 3) (S(j - 4) done, since
            // S(w + 1) is issued before PV(w)).
            constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows an instruction
            const int c = lane % kChunks, sub = lane / kChunks;
            const int64_t pitch = a.pool_stride * 2;
            int base = 0;  // blocks of the segments before
            bool ok = true;
            constexpr bool kWalks = kTiles == 1;  // the first load warp does, between its units
            if (kWalks && warp == kFirstLoad) ok = give_segment(0);
            for (int seg = 0; ok; ++seg) {
                ok = warp_segment(seg, sg);
                if (!ok || sg.blocks == 0) break;
                bool gives = kWalks && warp == kFirstLoad;
                const int64_t at = ((int64_t)sg.g * D + c * 8) * 2;
                const char *kp = reinterpret_cast<const char *>(a.k_pool) + at, *vp = reinterpret_cast<const char *>(a.v_pool) + at;
                const int32_t *slots = a.kv_indices + sg.kv0;
                constexpr bool kApart = kTiles == 2;
                const int lw = warp - kFirstLoad;
                const bool v_warp = kApart && lw >= C::kLoadWarps / 2;
                const int last = 2 * sg.blocks - 1, end = (kApart ? 1 : 2) * sg.blocks * C::kUnits;
                const int step = kApart ? C::kLoadWarps / 2 : C::kLoadWarps;
                // block of unit n, and whether it is its V
                auto block_of = [&](int n, bool &is_v) {
                    const int q = n / C::kUnits;
                    if constexpr (kApart) {
                        is_v = v_warp;
                        return q;
                    }
                    is_v = q == last || (q > 0 && !(q & 1));
                    return q == last ? sg.blocks - 1 : is_v ? q / 2 - 1 : (q + 1) / 2;
                };
                auto column_of = [&](int n) {
                    bool is_v;
                    const int j = block_of(n, is_v);
                    return block_column<C>(sg, j) + 32 * (n % C::kUnits);
                };
                auto fetch = [&](int n) { return slots[min(column_of(n) + lane, sg.N - 1)]; };  // past the end: a valid row again
                int n = v_warp ? lw - C::kLoadWarps / 2 : lw;
                int ahead = n < end ? fetch(n) : 0;
                const int first_units = n + 2 * step;  // in flight before the walk goes on
                for (; n < end; n += step) {
                    if (kWalks && gives && n >= first_units) {
                        ok = give_segment(seg + 1);
                        if (!ok) break;
                        gives = false;
                    }
                    int slot = ahead;
                    if (slot < 0 || slot >= a.pool_rows) {
                        latch(a.err, DDT_DEVERR_KV_INDEX);
                        slot = 0;
                    }
                    if (n + step < end) ahead = fetch(n + step);
                    bool is_v;
                    const int j = base + block_of(n, is_v);
                    const int s = is_v ? j % C::kVStages : j % C::kKStages, u = is_v ? j / C::kVStages : j / C::kKStages;
                    if (u > 0) ok = warp_wait(bar((is_v ? C::bVEmpty : C::bKEmpty) + s), (u - 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    const uint32_t to = (is_v ? C::kOffV : C::kOffK) + s * C::kBlockBytes + (c >> 3) * C::kBoxBytes +
                                        (n % C::kUnits) * 32 * 128;
                    const uint32_t full = bar((is_v ? C::bVFull : C::bKFull) + s);
                    const char *pool = is_v ? vp : kp;
                    // Columns that no row of the item sees (behind the last one, or outside its window) are zeros:
                    // the products of their weights, which are 0, then are too.
                    const int col = column_of(n);
                    uint32_t some = 0xffffffffu, every = 0xffffffffu;
                    if (!all_see(col, 32, sg.pa, sg.pb, a.window, sg.full)) {
                        const int mine = col + lane;
                        const bool in_full = mine < sg.full;
                        some = __ballot_sync(0xffffffffu, in_full || (mine <= sg.pb && (a.window <= 0 || mine > sg.pa - a.window)));
                        every = __ballot_sync(0xffffffffu, in_full || (mine <= sg.pa && (a.window <= 0 || mine > sg.pb - a.window)));
                    }
                    // 16 slots in a row (a page, or rows taken in order) are one tile copy for each 64 values,
                    // which takes few issue slots; others 16 bytes a lane.
                    if (every == 0xffffffffu && __all_sync(0xffffffffu, slot == __shfl_sync(0xffffffffu, slot, lane & 16) + (lane & 15))) {
                        if (lane == 0) mbar_arrive_expect_tx(full, 32 * D * 2);
                        else mbar_arrive(full);
                        if ((lane & 15) == 0) {
                            const uint32_t at = sbase + (is_v ? C::kOffV : C::kOffK) + s * C::kBlockBytes + ((n % C::kUnits) * 32 + lane) * 128;
#pragma unroll
                            for (int x = 0; x < C::kBoxes; ++x)
                                tma_load_2d(at + x * C::kBoxBytes, is_v ? &prm.v_map : &prm.k_map, sg.g * D + 64 * x, slot, full);
                        }
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 32 / kPer; ++i) {
                        const int k = i * kPer + sub;
                        cp_async_16_or_0(sbase + to + k * 128 + (((c & 7) ^ (k & 7)) << 4), pool + __shfl_sync(0xffffffffu, slot, k) * pitch,
                                         (some >> k) & 1u);
                    }
                    if (!is_v || some == every) {
                        cp_async_arrive(full);
                        continue;
                    }
                    // rows of V that some row sees and another does not
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    uint32_t bad = 0;
#pragma unroll
                    for (int i = 0; i < 32 / kPer; ++i) {
                        const int k = i * kPer + sub;
                        const uint4 x = *reinterpret_cast<const uint4 *>(smem + to + k * 128 + (((c & 7) ^ (k & 7)) << 4));
                        if (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) bad |= 1u << i;
                    }
                    if (__any_sync(0xffffffffu, bad)) {
                        // the poison is the segment's own: the one before has to be through with it
                        if (seg > 0) ok = warp_wait(seg_done(seg - 1), seg_parity(seg - 1), abort_flag, a.err);
                        if (!ok) break;
                        for (; bad; bad &= bad - 1) {
                            const int k = (__ffs(bad) - 1) * kPer + sub;
                            poison_8<C>(sbase + to + k * 128 + (((c & 7) ^ (k & 7)) << 4), col + k,
                                        sbase + C::kOffPoison + 4 * (c * 8) * 2 * (C::kPer / 32), sg.rows, sg.rem0, sg.pa,
                                        prm.group_inv, a.window, sg.full, sg.N);
                        }
                        __syncwarp();
                        if (lane == 0) *poisoned = 1;
                        __syncwarp();
                    }
                    mbar_arrive(full);
                }
                if (ok && gives) ok = give_segment(seg + 1);
                base += sg.blocks;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may land after the CTA has left
            // (nor a tile copy, which only the MMA warp waits for: where it gave up, they have this long)
            if (!ok)
                for (int i = 0; i < 1000; ++i) __nanosleep(1000);
        } else if (warp == kMmaWarp) {
            // ================= MMA =================
            if (elect_one()) {
                const uint64_t q0 = smem_desc(sbase + C::kOffQ, 16, 1024), k0 = smem_desc(sbase + C::kOffK, 16, 1024),
                               v0 = smem_desc(sbase + C::kOffV, C::kBoxBytes, 1024);  // + bytes >> 4
                bool ok = true;
                int ks = 0, vs = 0;
                uint32_t kph = 0, vph = 0, pph[2] = {0, 0};
                // The tensor pipe is idle while this thread waits or computes: the loop is
                // unrolled over tiles and slots and keeps its stages and phases in counters.
                auto run = [&](auto tile_count, int items) {
                    constexpr int A = decltype(tile_count)::value;  // tiles of the segment
                    constexpr int kOuts = kTiles;                   // outputs that work units alternate between
                    int w = 0;
                    auto issue_s = [&](int slot, int n) {
                        const int t = A == 2 ? slot : 0;
                        if (t == 0) {
                            ok = wait_or_abort(bar(C::bKFull + ks), kph, abort_flag, a.err);
                            if (!ok) return;
                            fence_proxy_async_smem();  // written by cp.async, read by the tensor core
                        }
                        tc_fence_after();
                        const uint64_t qd = q0 + t * (C::kQBytes >> 4), kd = k0 + (uint32_t)ks * (C::kBlockBytes >> 4);
                        const uint32_t d = tmem + C::kColS + NB * slot;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            mma_ss(d, qd + (((i >> 2) * C::kQBoxBytes + (i & 3) * 32) >> 4),
                                   kd + (((i >> 2) * C::kBoxBytes + (i & 3) * 32) >> 4), C::kIdescS, i > 0);
                        mma_commit(bar(C::bSFull + slot));
                        if (t == A - 1) {
                            mma_commit(bar(C::bKEmpty + ks));
                            if (++ks == C::kKStages) {
                                ks = 0;
                                kph ^= 1;
                            }
                        }
                        if (kTiles == 2 && n == items - 1) mma_commit(bar(C::bQEmpty));
                    };
                    auto issue_pv = [&](int slot) {
                        const int t = A == 2 ? slot : 0;
                        if (t == 0) {
                            ok = wait_or_abort(bar(C::bVFull + vs), vph, abort_flag, a.err);
                            if (!ok) return;
                            fence_proxy_async_smem();
                        }
                        const uint64_t vd = v0 + (uint32_t)vs * (C::kBlockBytes >> 4);
                        const uint32_t p = tmem + C::kColS + NB * slot, d = tmem + C::kColO + D * (kOuts == 2 ? slot : 0);
                        const uint32_t later = w >= kOuts;  // an output's first product overwrites
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h) {
                            ok = wait_or_abort(bar(C::bPFull + C::kHalves * slot + h), pph[slot], abort_flag, a.err);
                            if (!ok) return;
                            tc_fence_after();
#pragma unroll
                            for (int i = 4 * h; i < 4 * h + 4; ++i)
                                mma_ts(d, p + 8 * i, vd + i * (2048 >> 4), C::kIdescPV, i > 0 ? 1u : later);
                            if (h + 1 < C::kHalves) mma_commit(bar(C::bHalf + slot));
                        }
                        pph[slot] ^= 1;
                        if (kOuts == 1) mma_commit(bar(C::bODone));
                        if (t == A - 1) {
                            mma_commit(bar(C::bVEmpty + vs));
                            if (++vs == C::kVStages) {
                                vs = 0;
                                vph ^= 1;
                            }
                        }
                    };
#pragma unroll
                    for (int slot = 0; slot < 2; ++slot)
                        if (ok && slot < items) issue_s(slot, slot);
                    while (ok && w < items) {
#pragma unroll
                        for (int slot = 0; slot < 2; ++slot) {
                            if (!ok || w >= items) break;
                            issue_pv(slot);
                            if (ok && w + 2 < items) issue_s(slot, w + 2);
                            ++w;
                        }
                    }
                };
                bool was_lone = false;
                for (int seg = 0; ok; ++seg) {
                    ok = wait_or_abort(bar(C::bSegFull + (seg & 1)), (seg >> 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    read_segment(seg, sg);
                    mbar_arrive(bar(C::bSegEmpty + (seg & 1)));
                    if (sg.blocks == 0) break;
                    ok = wait_or_abort(bar(C::bQFull), seg & 1, abort_flag, a.err);
                    if (!ok) break;
                    if constexpr (kTiles == 2) {
                        // A lone tile's second output is read by the first tile's warps, which the second
                        // tile's do not wait for.
                        if (was_lone) ok = wait_or_abort(seg_done(seg - 1), seg_parity(seg - 1), abort_flag, a.err);
                        if (!ok) break;
                        was_lone = sg.tiles == 1;
                        if (sg.tiles == 2) run(std::integral_constant<int, 2>{}, 2 * sg.blocks);
                        else run(std::integral_constant<int, 1>{}, sg.blocks);
                        // Of a lone tile's single block the second tile's warps have no part: they may not have read
                        // bOFin's phase of the segment before yet, which this one's would hide from them.
                        if (ok && seg > 0 && sg.tiles == 1 && sg.blocks == 1)
                            ok = wait_or_abort(seg_done(seg - 1), seg_parity(seg - 1), abort_flag, a.err);
                        if (!ok) break;
                    } else {
                        run(std::integral_constant<int, 1>{}, sg.blocks);
                    }
                    mma_commit(bar(C::bOFin));  // completes when the segment's MMAs have
                }
                mma_commit(bar(C::bDrain));  // every MMA issued has to be done before the exit
                mbar_wait(bar(C::bDrain), 0, kWaitLimit);
            }
            __syncwarp();
        } else if (kTiles == 2) {
            // ================= q, a segment ahead; the first warp walks =================
            const bool walks = warp == kMmaWarp + 1;
            if (walks) give_segment(0);
            for (int seg = 0;; ++seg) {
                if (!warp_segment(seg, sg) || sg.blocks == 0) break;
                if (walks && !give_segment(seg + 1)) break;
                if (seg > 0 && !warp_wait(bar(C::bQEmpty), (seg - 1) & 1, abort_flag, a.err)) break;
                load_q(sg, 32 * (warp - kMmaWarp - 1), kTiles * kRows, 32 * C::kQWarps);
            }
        }
    } else {
        // ================= softmax (thread = row = TMEM lane of its tile) =================
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        const int t = warp >> 2, wq = warp & 3;
        const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
        ScoreScale sc = prm.score;
        CapPoly poly;
        if constexpr (kScore & kCap) poly.set(sc);
        uint32_t uses0 = 0, uses1 = 0;  // of the slots, in the segments before
        uint32_t done = 0, joins = 0;           // blocks, and joins, so far
        bool ok = true;
        for (int seg = 0; ok; ++seg) {
            ok = warp_segment(seg, sg);
            if (!ok || sg.blocks == 0) break;
            const bool lone = kTiles == 2 && sg.tiles == 1;          // one tile, served by both tiles' warps
            const int first = (lone ? 0 : t * kRows) + 32 * wq;      // the warp's first row in the item
            const int j0 = lone ? t : 0, step = lone ? 2 : 1;        // its blocks
            if constexpr (kTiles == 1) load_q(sg, first, first + 32, 32);
            const bool warp_on = first < sg.rows;  // the warp has rows
            const bool row_on = first + lane < sg.rows;
            const int rn = sg.rem0 + min(first + lane, sg.rows - 1);  // (lanes behind the last row repeat it)
            const int node = quotient(rn, prm.group_inv);
            const int p = sg.pa + node;
            if constexpr (kScore & kBias) sc.slope = a.slopes[sg.g * prm.group + rn - node * prm.group] * kLog2e;
            float m_ref = -INFINITY, l = 0.f;  // the reference in log2 units, the sum against it
            for (int j = j0; warp_on && j < sg.blocks; j += step) {
                const int slot = kTiles == 2 ? t : j & 1;
                const uint32_t phase = ((slot ? uses1 : uses0) + (lone || kTiles == 1 ? j >> 1 : j)) & 1;
                const uint32_t col = tmem + lane_off + C::kColS + NB * slot;
                const int c0 = block_column<C>(sg, j);
                const bool lane_fast = all_see(c0, NB, p, p, a.window, sg.full) && (!(kScore & kBias) || c0 + NB - 1 <= p);
                const bool fast = __all_sync(0xffffffffu, lane_fast);
                ok = warp_wait(bar(C::bSFull + slot), phase, abort_flag, a.err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1  // (unrolled, the loop outgrows the instruction cache: 1142 us where this takes 981)
                for (int h = 0; h < C::kHalves; ++h) {
                    const int c = c0 + 64 * h;
                    uint32_t s[2][32];  // the products
                    float r[2];         // and the largest of each 32
                    tmem_ld32_max<(kScore & kCap) != 0>(col + 64 * h, s[0], r[0]);
                    tmem_ld32_max<(kScore & kCap) != 0>(col + 64 * h + 32, s[1], r[1]);
                    uint32_t seen0 = 0xffffffffu, seen1 = 0xffffffffu;
                    if (!fast) {
                        seen0 = seen_bits(c, p, a.window, sg.full, sg.N);
                        seen1 = seen_bits(c + 32, p, a.window, sg.full, sg.N);
                    }
                    tmem_wait_ld();
                    // How far the scores reach: at most (seen whole, or no cap), or exactly.
                    float top;
                    bool quick = fast;  // the weights do not look at what is seen
                    if constexpr (kScore & kCap) {
                        quick = fast && __all_sync(0xffffffffu, fmaxf(r[0], r[1]) < prm.cap_most);
                        if (fast) top = reached<kCap>(fmaxf(r[0], r[1]), true, sc);
                        else top = reached<kScore>(reach_64<kScore>(s, seen0, seen1, c, p, sc), (seen0 | seen1) != 0, sc);
                    } else {
                        if (!fast) {  // products of columns that the row does not see: their weights are 0 whatever is added
                            r[0] = r[1] = -INFINITY;
                            // The distance, too, goes off the products: the weights' slope (j - p) is slope |p - j| up to
                            // the row's own position alone, and columns behind it (of a prefix that all see) are here.
                            const float less = (kScore & kBias) ? -sc.slope / sc.lin : 0.f;
#pragma unroll
                            for (int e = 0; e < 64; ++e) {
                                if constexpr (kScore & kBias)
                                    s[e >> 5][e & 31] = __float_as_uint(fmaf(less, fabsf((float)(c - p) + (float)e), __uint_as_float(s[e >> 5][e & 31])));
                                s[e >> 5][e & 31] = ((e < 32 ? seen0 : seen1) >> (e & 31)) & 1u ? s[e >> 5][e & 31] : 0xff800000u;
                                r[e & 1] = fmaxf(r[e & 1], __uint_as_float(s[e >> 5][e & 31]));
                            }
                            quick = true;
                        }
                        top = reached<0>(fmaxf(r[0], r[1]), true, sc);
                    }
                    // less the nearest column's distance (or, of a slope below 0, the farthest's)
                    if ((kScore & kBias) && fast) top += fmaxf(sc.slope * (float)(c - p), sc.slope * (float)(c + 63 - p));
                    if (__any_sync(0xffffffffu, row_on && top > m_ref - kMost)) {
                        // The reference moves to the largest of these scores, and what was summed against
                        // the old one shrinks.
                        if (kScore == kBias && fast) top = reach_linear(s, c, p, sc);
                        else if ((kScore & kCap) && fast) top = reached<kScore>(reach_64<kScore>(s, seen0, seen1, c, p, sc), (seen0 | seen1) != 0, sc);
                        const bool up = row_on && top > m_ref - kMost;
                        if (__any_sync(0xffffffffu, up)) {
                            const float alpha = up ? ex2(m_ref - (top + kShift)) : 1.0f;
                            if (up) m_ref = top + kShift;
                            l *= alpha;
                            // The products so far have to be done before the output is scaled: of this
                            // block's first half; or of the output's last block (with two outputs S(w) was
                            // issued behind it, so it is done).
                            if (h > 0) ok = warp_wait(bar(C::bHalf + slot), phase, abort_flag, a.err);
                            else if (kTiles == 1 && j > 0) ok = warp_wait(bar(C::bODone), (done + j - 1) & 1, abort_flag, a.err);
                            if (!ok) break;
                            if (h > 0 || j > j0) {
                                tc_fence_after();
                                const uint32_t oc = tmem + lane_off + C::kColO + D * t;
#pragma unroll 1
                                for (int q = 0; q < D / 8; ++q) {
                                    uint32_t o8[8];
                                    tmem_ld8(oc + 8 * q, o8);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 8; ++e) o8[e] = __float_as_uint(__uint_as_float(o8[e]) * alpha);
                                    tmem_st8(oc + 8 * q, o8);
                                }
                            }
                        }
                    }
                    const float m = m_ref == -INFINITY ? 0.f : m_ref;  // nothing seen yet: the weights are 0
                    auto store = [&](int k, const uint32_t (&pw)[16]) {  // over products that have been read
                        tmem_st16(col + 32 * h + 16 * k, pw);
                    };
                    float sum = 0.f;
                    if (quick) {
                        sum = weights_64<kScore, true>(s, seen0, seen1, c, p, m, fast ? sc.slope : 0.f, sc, poly, store);
                    } else if ((kScore & kCap) && (fast || __any_sync(0xffffffffu, (seen0 | seen1) != 0))) {
                        sum = weights_64<kScore, false>(s, seen0, seen1, c, p, m, sc.slope, sc, poly, store);
                    } else {  // no row of the warp sees any
                        const uint32_t none[16] = {};
                        store(0, none);
                        store(1, none);
                    }
                    l += sum;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bPFull + C::kHalves * slot + h));
                }
                if (!ok) break;
            }
            // a tile's warps without rows hand their part of the weights on as it is: its rows go nowhere
            for (int j = j0; ok && !warp_on && j < sg.blocks; j += step) {
                const int slot = kTiles == 2 ? t : j & 1;
                ok = warp_wait(bar(C::bSFull + slot), ((slot ? uses1 : uses0) + (lone || kTiles == 1 ? j >> 1 : j)) & 1, abort_flag, a.err);
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    if (lane == 0) mbar_arrive(bar(C::bPFull + C::kHalves * slot + h));
            }
            if (!ok) break;
            uses0 += lone || kTiles == 1 ? (sg.blocks + 1) >> 1 : sg.blocks;
            uses1 += lone || kTiles == 1 ? sg.blocks >> 1 : sg.blocks;
            done += sg.blocks;
            // ---- epilogue ----
            ok = warp_wait(bar(C::bOFin), seg & 1, abort_flag, a.err);
            if (!ok) break;
            const bool poisoned_now = *poisoned != 0;
            if (lone) {
                // (the wait above: the first tile's warps have left the segment before, so these places are free)
                volatile float *place = reinterpret_cast<volatile float *>(smem + C::kOffJoin) + 2 * (32 * wq + lane);
                if (t == 1) {
                    place[0] = m_ref;
                    place[1] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bJoin));
                } else {
                    ok = warp_wait(bar(C::bJoin), joins & 1, abort_flag, a.err);
                    if (!ok) break;
                    const float m1 = place[0], l1 = place[1], m = fmaxf(m_ref, m1);
                    // what the two outputs count (without a reference the sum is 0, or NaN)
                    const float keep0 = m_ref == -INFINITY ? l : ex2(m_ref - m), keep1 = m1 == -INFINITY ? l1 : ex2(m1 - m);
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < D / 8; ++q) {
                        uint32_t o0[8], o1[8];
                        tmem_ld8(tmem + lane_off + C::kColO + 8 * q, o0);
                        tmem_ld8(tmem + lane_off + C::kColO + D + 8 * q, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o0[e] = __float_as_uint((keep0 != 0.f ? __uint_as_float(o0[e]) * keep0 : 0.f) +
                                                    (keep1 != 0.f ? __uint_as_float(o1[e]) * keep1 : 0.f));
                        tmem_st8(tmem + lane_off + C::kColO + 8 * q, o0);
                    }
                    tmem_wait_st();
                    l = (keep0 != 0.f ? l * keep0 : 0.f) + (keep1 != 0.f ? l1 * keep1 : 0.f);
                    m_ref = m;
                }
                ++joins;
            }
            if (warp_on && !(lone && t == 1)) {
                tc_fence_after();
                const int64_t row = (int64_t)(sg.qo0 + sg.node0 + node) * a.num_heads + sg.g * prm.group + rn - node * prm.group;
                const bool part = sg.part >= 0;
                const int64_t prow = (int64_t)sg.part * prm.part_rows + first;  // of the warp's first row
                const bool none = l == 0.f;
                const float inv = 1.f / l;
                // The rows leave through shared memory: a thread writes its row's next 64 bytes there,
                // and four lanes write each row's to global memory.
                uint8_t *stage = smem + C::kOffStage + (kTiles == 2 ? warp : 2 * warp) * C::kStageBytes;
                auto put = [&](int c, uint4 v) {  // chunk c of this lane's row
                    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v;
                };
                auto flush = [&](int piece, auto row_start) {  // row_start: row of the warp -> its bytes' place
                    __syncwarp();
                    uint4 v[4];
                    const int c = lane & 3;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rw = 8 * i + (lane >> 2);
                        v[i] = *reinterpret_cast<const uint4 *>(stage + rw * 64 + ((c ^ ((rw >> 1) & 3)) << 4));
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rw = 8 * i + (lane >> 2);
                        if (first + rw < sg.rows) reinterpret_cast<uint4 *>(row_start(rw))[4 * piece + c] = v[i];
                    }
                };
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t t32[32];
                    tmem_ld32(tmem + lane_off + C::kColO + D * t + 32 * q, t32);
                    tmem_wait_ld();
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(t32[e]);
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                    if (part) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                put(e, make_uint4(__float_as_uint(o[16 * h + 4 * e]), __float_as_uint(o[16 * h + 4 * e + 1]),
                                                  __float_as_uint(o[16 * h + 4 * e + 2]), __float_as_uint(o[16 * h + 4 * e + 3])));
                            flush(2 * q + h, [&](int rw) { return a.o_part + (prow + rw) * D; });
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            put(e, make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                              pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7])));
                        flush(q, [&](int rw) {
                            const int n = sg.rem0 + first + rw, nd = quotient(n, prm.group_inv);
                            return a.out + ((int64_t)(sg.qo0 + sg.node0 + nd) * a.num_heads + sg.g * prm.group + n - nd * prm.group) * D;
                        });
                    }
                }
                if (row_on) {
                    // (the shift goes before the logarithm, as a power of two: -53 + log2 would be rounded by 53's size)
                    const float lse = none ? -INFINITY : ((m_ref - kShift) + log2f(l * kUnshift)) * kLn2;
                    if (part) a.lse_part[prow + lane] = lse;
                    else if (a.lse) a.lse[row] = lse;
                }
                if (poisoned_now) {  // rows that have left get what their columns of V held
                    __syncwarp();
#pragma unroll 1
                    for (int e = 0; e < D; ++e) {
                        uint32_t *w = poison + 2 * e * (C::kPer / 32) + first / 32;
                        const bool plus = (w[0] >> lane) & 1u, minus = (w[C::kPer / 32] >> lane) & 1u;
                        __syncwarp();
                        if (lane == 0) w[0] = w[C::kPer / 32] = 0;
                        if (!plus && !minus) continue;
                        const float x = plus ? minus ? NAN : INFINITY : -INFINITY;
                        if (part) {
                            a.o_part[(prow + lane) * D + e] += x;
                        } else {
                            __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(a.out) + row * D + e;
                            *o = __float2bfloat16_rn(__bfloat162float(*o) + x);
                        }
                    }
                }
            }
            tc_fence_before();  // the outputs have been read before the next segment's first products
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_done(seg));
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// out = sum_s e^{lse_s - LSE} o_s over the parts s of a cut item, LSE = log sum_s e^{lse_s}.
// CTA (c, y) has 8 rows of the item that ends in CTA c's share, a warp each: its lanes hold
// the weights of 32 parts at a time, then sum D / 32 values of every part.
constexpr int kCombineWarps = 8;

template <int D, int kTiles>
__global__ void __launch_bounds__(32 * kCombineWarps) chunk_combine_kernel(const __grid_constant__ AttnParams prm) {
    using C = Cfg<D, kTiles>;
    constexpr int E = D / 32, kFlight = 8;  // values of a lane; parts in flight
    const ChunkArgs &a = prm.a;
    const int lane = threadIdx.x & 31, cta = blockIdx.x;
    const int first_row = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int4 note = a.notes[cta];
    if (note.x < 0) return;
    const Request r = load_request(a, note.x, nullptr);
    const Item it = item_of<C>(r, note.z, prm.group, prm.group_inv, a.window);
    if (first_row >= it.rows) return;
    const int c0 = note.w >> 1, parts = cta - c0 + 1;
    auto place = [&](int s) { return (int64_t)(s == 0 ? note.w : 2 * (c0 + s)) * prm.part_rows + first_row; };
    // weights of 2^-9 at most: those of DDT_GQA_MAX_CTAS parts sum to 1, and finite parts to a finite value
    constexpr float kLess = 9.f, kMore = 512.f;
    static_assert(DDT_GQA_MAX_CTAS <= 512, "parts of a row");
    float m = -INFINITY, den = 0.f;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s0 = 0; s0 < parts; s0 += 32) {
        const float ls = s0 + lane < parts ? a.lse_part[place(s0 + lane)] : -INFINITY;
        float mg = fmaxf(m, ls);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
        const float keep = m == -INFINITY ? 0.f : ex2((m - mg) * kLog2e);
        const float w = ls == -INFINITY ? 0.f : ex2((ls - mg) * kLog2e - kLess);  // NaN stays
        float sum = w;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        den = den * keep + sum;
        m = mg;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= keep;
        const int n = min(32, parts - s0);
        for (int s = 0; s < n; s += kFlight) {
            float v[kFlight][E];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (s + u >= n) break;
                const float *o = a.o_part + place(s0 + s + u) * D + lane * E;
                if constexpr (E == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(o);
                    v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(o);
                    v[u][0] = x.x; v[u][1] = x.y;
                }
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (s + u >= n) break;
                const float ws = __shfl_sync(0xffffffffu, w, s + u);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(ws, v[u][e], acc[e]);
            }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den, lse = den == 0.f ? -INFINITY : m + log2f(den * kMore) * kLn2;
    const int n = it.rem0 + first_row, node = quotient(n, prm.group_inv);
    const int64_t row = (int64_t)(r.qo0 + it.node0 + node) * a.num_heads + note.y * prm.group + n - node * prm.group;
    uint16_t *dst = a.out + row * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0) a.lse[row] = lse;
}

template <int D, int kTiles, int kScore>
cudaError_t launch_attn(AttnParams &prm, cudaStream_t s) {
    using C = Cfg<D, kTiles>;
    const ChunkArgs &a = prm.a;
    const dim3 grid = a.num_ctas > 0 ? dim3((unsigned)a.num_ctas)
                                     : dim3((unsigned)(prm.tgs_most * a.num_kv_heads), 1, (unsigned)a.batch);
    cudaError_t e = launch_pdl(chunk_attn_kernel<D, kTiles, kScore>, grid, dim3(C::kThreads), C::kSmemBytes, s, prm);
    if (e == cudaSuccess && a.num_ctas > 1)
        e = launch_pdl(chunk_combine_kernel<D, kTiles>,
                       dim3((unsigned)a.num_ctas, (unsigned)((prm.part_rows + kCombineWarps - 1) / kCombineWarps)),
                       dim3(32 * kCombineWarps), 0, s, prm);
    return e;
}

template <int D, int kTiles, int kScore>
cudaError_t prepare_attn() {
    if (kTiles == 2) {  // the softmax warps would wait for registers that the launch does not have
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, chunk_attn_kernel<D, kTiles, kScore>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < Cfg<D, kTiles>::kLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    const cudaError_t e = cudaFuncSetAttribute(chunk_attn_kernel<D, kTiles, kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg<D, kTiles>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(chunk_attn_kernel<D, kTiles, kScore>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                (int)cudaSharedmemCarveoutMaxShared);
}

// one translation unit per kScore: they compile side by side
template <int kScore>
cudaError_t launch_attn_score(AttnParams &prm, cudaStream_t s) {
    const bool two = prm.a.tiles == 2;
    if (prm.a.head_dim == 128) return two ? launch_attn<128, 2, kScore>(prm, s) : launch_attn<128, 1, kScore>(prm, s);
    return two ? launch_attn<64, 2, kScore>(prm, s) : launch_attn<64, 1, kScore>(prm, s);
}
template <int kScore>
cudaError_t prepare_attn_score() {
    cudaError_t e = prepare_attn<64, 1, kScore>();
    if (e == cudaSuccess) e = prepare_attn<64, 2, kScore>();
    if (e == cudaSuccess) e = prepare_attn<128, 1, kScore>();
    if (e == cudaSuccess) e = prepare_attn<128, 2, kScore>();
    return e;
}

}  // namespace chunk
}  // namespace ddt
