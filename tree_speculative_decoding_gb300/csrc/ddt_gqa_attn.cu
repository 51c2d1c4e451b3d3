// ddt_gqa_attn.cu -- tree-verify attention over grouped-query K/V rows on the
// sm_103a tensor cores.
//
// For row (tree node i of request b, head h), K/V head g = h / group, over the
// columns j that mask row i makes visible:
//   s_j = scale <q[i,h], k[idx_j][g]>,  out[i,h] = sum_j softmax(s)_j v[idx_j][g],
//   lse = log sum_j e^{s_j}
// in one pass over the columns with a running reference and sum.
//
// Work.  An item is one K/V head of one request and up to kTiles tiles of 128
// consecutive rows (node-major, the group's heads inside a node: the rows that
// share the K/V head); its K and V rows are gathered once for all its tiles, a
// block of columns at a time.
//   * kTiles = 1: blocks of 64 columns, 256 tensor-memory columns and under half
//     of the shared memory, so two CTAs share an SM: one's prologue, softmax and
//     epilogue run under the other's loads.  The only choice when a request's rows
//     per K/V head fit one tile (decode, small trees): the loads bound it.
//   * kTiles = 2: blocks of 128 columns, all of tensor memory; the tensor core
//     works on one tile while the softmax of the other runs, and K and V are read
//     half as often.  An item's last rows may fill one tile only: its blocks then
//     alternate between the two tiles' warps and outputs, each with a reference and
//     sum of its own, and the two are joined at the end.
// A CTA takes one item; or the blocks of all items, weighted by what they cost,
// form one line (request, K/V head, rows, columns) that is dealt to the resident
// CTAs in equal shares: a CTA takes the end of one item, whole items, and the
// start of another, whatever the requests' lengths are.  Items that were cut leave
// partial results (at most two per CTA) in the workspace for the combine kernel,
// and a note of where they are.  Every CTA finds the same cuts from the offsets.
// estimate() weighs the four ways.
//
// Measured with the combine kernel, D = 128: 64 requests of one token after
// 1024..16384, 64 heads on 8: 345 us, 6.6 TB/s, bound by memory.  32 requests of
// 17..33 tokens after 2048..8192, 32 heads on 4: 99 us, 3.7 TB/s and 735 TFLOP/s;
// 65 tokens after 131072, 64 heads on 8: 272 us, 1025 TFLOP/s, in short runs, 300 us
// and 930 TFLOP/s held for seconds under the power limit: a block of two tiles takes
// ~2700 clk where its products take 2048.  A tile's next scores wait for its softmax
// and its products (tensor memory is full; a third slot at D = 64, where it fits,
// measured 6% slower), and the gather takes issue slots from the softmax: with a
// sixteenth of the copies (timing only) the long one took 227 us where it took 291,
// the 32 requests 83 where they took 104.  Of the 99 us, 8 fill the first pipeline,
// 6 to 10 each go to a CTA's change of item, 9 to the combine.
//
// Score slots: two buffers of one block's scores in tensor memory.  Work unit w
// of a segment (block-major, tiles inside a block) uses slot w mod 2.  The MMA
// warp issues
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
// so the scores of w + 1 are being computed, or done, while the softmax of w
// runs.  P (bf16) overwrites the scores in place and is the A operand of PV
// from tensor memory; V is read as an MN-major operand from its gathered rows.
//
// Warps: four softmax warps per tile (thread = row = TMEM lane), one warp that
// issues MMAs, and load warps that copy row pieces with 16-byte cp.async into the
// 128-byte-swizzled layout of the MMA descriptors.  (A TMA row gather costs its
// warp ~57 clk for 512 bytes and measured half the rate.)
//
// The softmax does not look for a block's maximum: the weights of 64 columns are
// taken against the row's reference, the maximum of the first columns it saw.
// Only where their sum passes 2^40 (or the row had seen nothing) the maximum is
// found, the reference moves, and the sums so far are scaled.  Statistics, sums and
// partial results are fp32.  The weights are rounded to bf16 for the product with V,
// since the tensor core takes both operands in V's type: 2^-8 of each at most, at any
// scale, which adds up to 2^-8 sum p|v| to the result (0.0023 of the largest value
// against 0.0017 for weights in fp32, both with the output's own rounding); their sum
// is taken before that.  Sums against the reference overflow where |v| is above ~2^67
// (at a million columns): such a row is computed again, as below.
//
// Columns that a row does not see get p = 0, but 0 * NaN is NaN: a V row that
// holds NaN or infinities reaches the output rows that do not see it.  Rows whose
// output is not finite are therefore computed again over their visible columns only,
// after the CTA's last segment (rows_again): 16 rows at a time on the warps' own
// products, K and V read from global memory in place of the pipeline.
//
// Every wait is bounded: on timeout the CTA latches DDT_DEVERR_TIMEOUT, waits
// for its own copies and MMAs and leaves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ddt_gqa.cuh"
#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace {

using namespace sm100;

constexpr int kRows = 128;  // rows per tile (TMEM lanes)
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kSumLimit = 1099511627776.0f;  // 2^40: weights of 64 columns that sum to more move the reference
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct GqaParams {
    GqaArgs a;
    int group;        // query heads per K/V head
    float group_inv;  // 1 / group
    int part_rows;  // rows of a partial result
    int tgs_most;   // items per K/V head of the longest request
};

// n / group for 0 <= n < 128 * 128, 1 <= group <= 128 by the reciprocal: (n + 1/2) /
// group is at least 1/256 from a whole number, and off by less than 16384.5 * 2^-22.
__device__ __forceinline__ int quotient(int n, float group_inv) { return (int)(((float)n + 0.5f) * group_inv); }

template <int D, int kTiles>
struct Cfg {
    static constexpr int NB = kTiles == 2 ? 128 : 64;    // columns per block
    static constexpr int kHalves = NB / 64;              // parts of P that PV may start on
    static constexpr int kBoxes = D / 64;                // 128-byte pieces of a row
    static constexpr int kBoxBytes = NB * 128;           // one piece of a block's rows
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
    static constexpr int kQBoxBytes = kRows * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;  // one tile of q
    static constexpr int kKStages = D == 128 ? 2 : 4;
    static constexpr int kVStages = D == 128 ? (kTiles == 2 ? 3 : 2) : 4;  // V waits for the softmax, K does not
    static constexpr int kUnits = NB / 32;               // 32-row units of a block
    static constexpr int kSoftWarps = 4 * kTiles;
    // two tiles: warps 8..11 load K, 12..15 V, 16 issues MMAs (its warpgroup's others
    // are idle); one tile: warp 4 issues MMAs, 5..7 load
    static constexpr int kLoadWarps = kTiles == 2 ? 2 * kUnits : 3;
    static constexpr int kFirstLoad = kTiles == 2 ? kSoftWarps : kSoftWarps + 1;
    static constexpr int kMmaWarp = kTiles == 2 ? kSoftWarps + kLoadWarps : kSoftWarps;
    static constexpr int kThreads = kTiles == 2 ? 640 : 256;
    // Registers of the two-tile kernel: a softmax thread's, another's; together no more than at
    // launch.  65 tokens after 131072, and 8 requests of 33 after 1024..16384: 272 and 118 us with
    // 120 / 72, 273 and 121 us with 128 / 72, 281 and 124 us with 136 / 64, 291 and 127 us with
    // 112 / 80.
    static constexpr int kSoftRegs = 120, kOtherRegs = 72, kLaunchRegs = 96;
    static_assert(32 * kSoftWarps * kSoftRegs + (640 - 32 * kSoftWarps) * kOtherRegs <= 640 * kLaunchRegs || kTiles == 1, "registers");
    static constexpr uint32_t kTmemCols = kTiles == 2 ? 512 : 256;
    static constexpr uint32_t kColS = 0, kColO = 2 * NB;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTiles * kQBytes;
    static constexpr int kOffV = kOffK + kKStages * kBlockBytes;
    static constexpr int kOffBar = kOffV + kVStages * kBlockBytes;
    // barriers
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bVFull = bKEmpty + kKStages,
                         bVEmpty = bVFull + kVStages, bSFull = bVEmpty + kVStages, bPFull = bSFull + 2,
                         bQFull = bPFull + 2 * kHalves, bHalf = bQFull + 1, bODone = bHalf + 2, bOFin = bODone + 1, bJoin = bOFin + 1, bDrain = bJoin + 1,
                         bSegFull = bDrain + 1, bSegEmpty = bSegFull + 2, bCount = bSegEmpty + 2;
    static constexpr int kOffHolder = kOffBar + 8 * bCount;
    static constexpr int kOffWalk = kOffHolder + 16;  // 128 bytes: the walk; 2 x 48: the segments it has given
    static constexpr int kOffPlan = kOffWalk + 128 + 2 * 48;  // a sum per warp, then where the CTA's share starts
    static constexpr int kOffJoin = kOffPlan + 8 * (kThreads / 32);  // the second tile's references and sums
    static constexpr int kSmemUsed = kOffJoin + (kTiles == 2 ? kRows * 8 : 0);
    static constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for the 1024-byte alignment of swizzle atoms
    static constexpr uint32_t kIdescS = idesc_bf16(kRows, NB, 0, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16(kRows, D, 0, 1);
    // Cost of a block with all tiles and with one, in one unit; of an item besides its
    // blocks: a CTA that goes on to another one writes the last one's rows, loads q and
    // fills its pipeline anew, 6 to 10 us (two tiles) or 2 to 3 us; and the share that a CTA
    // gets at least.  Measured with D = 128, 64 heads on 8.  An item at 80 / 48 (two tiles / one):
    // 8 requests of 33 tokens after 1024..16384 take 119 us, one token after 4096 14.1 us; at 24 /
    // 24 137 and 14.4 us, at 160 / 96 125 and 14.6 us.  Shares of 56 / 32: one request of 33 after
    // 1024 14.5 us, one token after 600 11.9 us; of 28 / 16 16.2 and 10.8 us (and one token after
    // 4096 16.0 us); of 120 / 80 18.7 and 15.6 us.
    static constexpr int kCostFull = kTiles == 2 ? 16 : 8, kCostOne = kTiles == 2 ? 11 : 8;
    static constexpr int kCostItem = kTiles == 2 ? 80 : 48, kMinShare = kTiles == 2 ? 56 : 32;
    static_assert(kTiles == 2 || (kKStages >= 2 && kKStages <= kVStages), "see the load warps");
    static_assert(kOffPlan % 8 == 0, "alignment");
    static_assert(kColO + kTiles * D <= kTmemCols, "tensor memory");
    static_assert(kSmemBytes <= (kTiles == 2 ? 232448 : 115712), "shared memory");
};

// The waits try the barrier first: the abort flag is read only where the phase
// is still open.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *err) {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    latch(err, DDT_DEVERR_TIMEOUT);
    return false;
}
// The same for a whole warp: it succeeds for every lane or for none, so the warp
// stays converged for the warp-collective instructions after it.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *err) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, err));
}

// ---------------------------------------------------------------- the deal
// A request's offsets, checked, and the size of its items.
struct Request {
    int qo0, T, kv0, N, m0;
    int tgs;        // tile groups: items per K/V head (0: nothing to do)
    int blocks;     // blocks of columns
    bool last_one;  // the last tile group has one tile of two
};

template <class C>
__device__ __forceinline__ int64_t item_cost(const Request &r, int tg) {
    return C::kCostItem + (int64_t)r.blocks * (tg == r.tgs - 1 && r.last_one ? C::kCostOne : C::kCostFull);
}
// of the items of one K/V head
template <class C>
__device__ __forceinline__ int64_t head_cost(const Request &r) {
    return r.tgs > 0 ? (r.tgs - 1) * (C::kCostItem + (int64_t)r.blocks * C::kCostFull) + item_cost<C>(r, r.tgs - 1) : 0;
}
template <class C>
__device__ __forceinline__ int64_t request_cost(const Request &r, int num_kv_heads) {
    return head_cost<C>(r) * num_kv_heads;
}

// kTiles: tiles of an item.  err: where a bad request is reported, or null.
template <class C, int kTiles>
__device__ __forceinline__ Request load_request(const GqaArgs &a, int group, int b, unsigned int *err) {
    Request r;
    r.qo0 = a.qo_indptr[b];
    const int qo1 = a.qo_indptr[b + 1];
    r.kv0 = a.kv_indptr[b];
    const int kv1 = a.kv_indptr[b + 1];
    r.m0 = a.mask_indptr[b];
    const int m1 = a.mask_indptr[b + 1];
    // Differences of broken offsets wrap, which is why their order counts; the words of a long
    // request do not fit 32 bits.
    r.T = (int)((uint32_t)qo1 - (uint32_t)r.qo0);
    r.N = (int)((uint32_t)kv1 - (uint32_t)r.kv0);
    const bool bad_qo = r.T < 0 || r.T > a.max_q_len || r.qo0 < 0 || qo1 > a.total_q || qo1 < r.qo0;
    const bool bad_kv = r.N < r.T || r.N > a.max_kv_len || r.kv0 < 0 || kv1 > a.total_kv || kv1 < r.kv0;
    const bool bad_mask =
        !bad_qo && !bad_kv && (r.m0 < 0 || (int64_t)m1 - r.m0 != (int64_t)r.T * ((r.N + 31) >> 5) || m1 > a.total_mask_words);
    if (bad_qo || bad_kv || bad_mask) {
        latch(err, (bad_qo ? DDT_DEVERR_QO_INDPTR : 0u) | (bad_kv ? DDT_DEVERR_KV_INDPTR : 0u) |
                       (bad_mask ? DDT_DEVERR_MASK_INDPTR : 0u));
        r.T = 0;
    }
    const int rows = r.T * group, per = kTiles * kRows;
    r.tgs = (rows + per - 1) / per;
    r.blocks = r.tgs > 0 ? (r.N + C::NB - 1) / C::NB : 0;
    r.last_one = kTiles == 2 && rows - (r.tgs - 1) * per <= kRows;
    return r;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // a, b >= 0; nearly always small enough for 32 bits
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// the item's blocks that start before position x (block k starts kCostItem + k unit behind the item)
template <class C>
__device__ __forceinline__ int blocks_before(int64_t item, int64_t x, int unit, int blocks) {
    const int64_t d = x - (item + C::kCostItem);
    if (d <= 0) return 0;
    const int64_t k = unit == C::kCostFull ? (d + C::kCostFull - 1) / C::kCostFull : (d + C::kCostOne - 1) / C::kCostOne;
    return k < blocks ? (int)k : blocks;
}

// What a CTA does in one go: `blocks` blocks of an item, from column c_begin on.
struct Segment {
    int row0, rows, tiles;  // rows of the request from row0 on; tiles of 128
    int g, c_begin, c_end, blocks;
    int qo0, kv0, m0, W;    // of the request
    int part;               // -1: the whole item, else the place of the partial result
};

// The walk over the CTA's segments.  It lives in shared memory: one thread steps
// it and hands the segments to the warps through a ring of two.
template <class C, int kTiles>
struct Walk {
    int64_t pos, lo, hi;  // the item's position on the line; the CTA's share of it
    Request r;
    int b, tg, g, cta;
    int dealt, more;
    int first_b;          // the request that the share starts in, and its position
    int64_t first_pos;

    // one item, whole
    __device__ __forceinline__ void start_item(const Request &req, int b_, int tg_, int g_) {
        r = req;
        b = b_;
        tg = tg_;
        g = g_;
        pos = lo = hi = 0;
        cta = 0;
        dealt = 0;
        more = 1;
    }
    // share [lo_, hi_), which starts inside request b_, whose items start at pos_
    __device__ __forceinline__ void start_share(const Request &req, int cta_, int b_, int64_t pos_, int64_t lo_, int64_t hi_) {
        r = req;
        cta = cta_;
        b = b_;
        lo = lo_;
        hi = hi_;
        first_b = b_;
        first_pos = pos_;
        dealt = more = 1;
        const int64_t head = head_cost<C>(r), full = C::kCostItem + (int64_t)r.blocks * C::kCostFull;
        g = (int)divide(lo - pos_, head);
        pos = pos_ + g * head;
        tg = min((int)divide(lo - pos, full), r.tgs - 1);
        pos += tg * full;
    }
    // back to the first segment
    __device__ __forceinline__ void restart(const GqaArgs &a, int group) {
        if (dealt) start_share(load_request<C, kTiles>(a, group, first_b, nullptr), cta, first_b, first_pos, lo, hi);
        else more = 1;
    }
    // the next segment; one without blocks when the share is done
    __device__ __forceinline__ Segment next(const GqaArgs &a, int group, int tgs_most) {
        Segment s;
        s.blocks = 0;
        while (more && s.blocks == 0) {
            const int unit = tg == r.tgs - 1 && r.last_one ? C::kCostOne : C::kCostFull;
            const int b0 = dealt ? blocks_before<C>(pos, lo, unit, r.blocks) : 0;
            const int b1 = dealt ? blocks_before<C>(pos, hi, unit, r.blocks) : r.blocks;
            s.row0 = tg * kTiles * kRows;
            s.rows = min(kTiles * kRows, r.T * group - s.row0);
            s.tiles = (s.rows + kRows - 1) / kRows;
            s.g = g;
            s.c_begin = b0 * C::NB;
            s.c_end = min(r.N, b1 * C::NB);
            s.blocks = b1 - b0;
            s.qo0 = r.qo0;
            s.kv0 = r.kv0;
            s.m0 = r.m0;
            s.W = (r.N + 31) >> 5;
            // at most one item of a share starts before it, and at most one ends behind it
            s.part = s.blocks == r.blocks ? -1 : 2 * cta + (lo > pos ? 0 : 1);
            if (!dealt) {
                more = 0;
            } else {
                // for the combine: the place of the item's first part (the later ones are at 2 CTA) and
                // the CTA that has its last
                if (s.blocks > 0) {
                    int2 &note = a.notes[((int64_t)b * a.num_kv_heads + g) * tgs_most + tg];
                    if (b0 == 0) note.x = s.part;
                    if (b1 == r.blocks) note.y = cta;
                }
                pos += item_cost<C>(r, tg);
                if (++tg == r.tgs) {
                    tg = 0;
                    ++g;
                }
                while ((g >= a.num_kv_heads || r.tgs == 0) && pos < hi && ++b < a.batch) {  // the next request with items
                    r = load_request<C, kTiles>(a, group, b, nullptr);
                    tg = g = 0;
                }
                more = pos < hi && b < a.batch;
            }
        }
        return s;
    }
};

// ---------------------------------------------------------------- rows that are not finite
// 16 rows of a segment (from row16 on) and 32 of the values (from e0 on), by one warp: where
// the output written for a row holds an infinity or NaN, it is computed again over the
// columns that the row sees.  In V infinities and NaN are replaced by 0 in the products; which
// values they belong in, and with which sign, is kept as bits: kinds[e] has four for a pair of
// rows (r, r + 8): seen as +inf by either, as -inf by either (NaN: both).  The weights are
// taken against the running maximum and 2^31 below it, so that the sums stay finite: a row
// has no 2^31 columns.  Bound by the latency of a block's slots, rows and products (few
// warps, little in flight): one request of 33 tokens after 4096, 64 heads on 8, takes 0.39 ms
// with a NaN in a prefix row, 0.06 without; 32 such requests with one NaN 4.2 ms, 0.24 without
// (72 ms with one row and column at a time).  Pieces of 32 values, and a loop over the scores that
// is not unrolled, keep the registers below what the softmax needs: with 64 values and the loop
// unrolled this takes 2.4 ms, and the kernels lose 3 to 12% where nothing is computed again.
constexpr int kKindWords = 32;

template <int D>
__device__ __forceinline__ void rows_again_16(const GqaParams &prm, const Segment &sg, int row16, int e0, uint32_t *kinds) {
    constexpr uint32_t kAll = 0xffffffffu, kRow0 = 0x11111111u;
    const GqaArgs &a = prm.a;
    const int lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
    // the lane's rows r8 and r8 + 8: query, mask words, and its 8 of the 32 outputs
    const uint16_t *q[2];
    const uint32_t *words[2];
    void *out[2];
    bool bad[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int ri = row16 + r8 + 8 * i, rr = sg.row0 + min(ri, sg.rows - 1), node = quotient(rr, prm.group_inv);
        const int64_t row = (int64_t)(sg.qo0 + node) * a.num_heads + sg.g * prm.group + rr - node * prm.group;
        q[i] = a.q + row * D + 8 * c4;
        words[i] = a.mask + sg.m0 + (int64_t)node * sg.W;
        uint32_t high = 0;  // an exponent of ones among the values
        if (sg.part >= 0) {
            float *o = a.o_part + ((int64_t)sg.part * prm.part_rows + min(ri, sg.rows - 1)) * D + e0 + 8 * c4;
            out[i] = o;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 x = reinterpret_cast<const uint4 *>(o)[k];
                const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) high |= (v[e] & 0x7f800000u) == 0x7f800000u;
            }
        } else {
            uint16_t *o = a.out + row * D + e0 + 8 * c4;
            out[i] = o;
            const uint4 x = *reinterpret_cast<const uint4 *>(o);
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) high |= (v[e] & 0x7f80u) == 0x7f80u || (v[e] & 0x7f800000u) == 0x7f800000u;
        }
        bad[i] = ((__ballot_sync(kAll, high != 0 && ri < sg.rows) >> (4 * r8)) & 15u) != 0;
    }
    if (!__any_sync(kAll, bad[0] || bad[1])) return;
    kinds[lane] = 0;
    __syncwarp();

    const float sc = a.scale * kLog2e;
    float acc[4][4], ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    const uint16_t *kp = a.k_pool + (int64_t)sg.g * D + 8 * c4, *vp = a.v_pool + (int64_t)sg.g * D + e0 + 4 * r8;
    auto slot_of = [&](int c) {  // of column c + lane % 16
        const int s = a.kv_indices[sg.kv0 + min(c + (lane & 15), sg.c_end - 1)];
        return s < 0 || s >= a.pool_rows ? 0 : s;  // latched by the load warps
    };
    int ahead = slot_of(sg.c_begin);
    for (int c = sg.c_begin; c < sg.c_end; c += 16) {
        const int slot = ahead;
        if (c + 16 < sg.c_end) ahead = slot_of(c + 16);
        // the lane's columns: c + 2 c4, + 1, + 8, + 9
        uint32_t seen[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w = (words[i][c >> 5] >> (c & 31)) & 0xffffu;
            if (sg.c_end - c < 16) w &= (1u << (sg.c_end - c)) - 1u;
            seen[i] = w >> (2 * c4);
        }
        if (!__any_sync(kAll, ((seen[0] | seen[1]) & 0x303u) != 0)) continue;
        uint2 v[4];  // 4 values from e0 + 4 r8 on of the lane's columns
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = *reinterpret_cast<const uint2 *>(vp + __shfl_sync(kAll, slot, 2 * c4 + (k & 1) + 8 * (k >> 1)) * a.pool_stride);
        const uint16_t *k0 = kp + __shfl_sync(kAll, slot, r8) * a.pool_stride, *k1 = kp + __shfl_sync(kAll, slot, r8 + 8) * a.pool_stride;
        // Scores.  A lane has 8 values in a row of each 32 of q and of K: any order will do, as
        // long as it is the same in both.
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
            const uint4 q0 = *reinterpret_cast<const uint4 *>(q[0] + d), q1 = *reinterpret_cast<const uint4 *>(q[1] + d);
            const uint4 x0 = *reinterpret_cast<const uint4 *>(k0 + d), x1 = *reinterpret_cast<const uint4 *>(k1 + d);
            mma_16x8x16(s[0], q0.x, q1.x, q0.y, q1.y, x0.x, x0.y);
            mma_16x8x16(s[1], q0.x, q1.x, q0.y, q1.y, x1.x, x1.y);
            mma_16x8x16(s[0], q0.z, q1.z, q0.w, q1.w, x0.z, x0.w);
            mma_16x8x16(s[1], q0.z, q1.z, q0.w, q1.w, x1.z, x1.w);
        }
        uint32_t high = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x[2] = {v[k].x, v[k].y};
#pragma unroll
            for (int e = 0; e < 2; ++e) high |= (x[e] & 0x7f80u) == 0x7f80u || (x[e] & 0x7f800000u) == 0x7f800000u;
        }
        if (__any_sync(kAll, high != 0)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // the 16 rows that see column k of the lane, at bits 4 r (+ 1 for r + 8); those whose
                // weight there is 0 because the score is -inf: 0 times infinity is NaN
                const int j = k >> 1, bit = (k & 1) + 8 * j;
                uint32_t rows = 0, zero = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool sees = (seen[i] >> bit) & 1u;
                    rows |= ((__ballot_sync(kAll, sees) >> c4) & kRow0) << i;
                    zero |= ((__ballot_sync(kAll, sees && s[j][2 * i + (k & 1)] == -INFINITY) >> c4) & kRow0) << i;
                }
                uint32_t x[2] = {v[k].x, v[k].y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t y = (x[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                    if ((y & 0x7f80u) != 0x7f80u) continue;
                    const bool nan = (y & 0x7fu) != 0, minus = (y >> 15) != 0;
                    const uint32_t plus_rows = nan || !minus ? rows : zero, minus_rows = nan || minus ? rows : zero;
                    if (rows) atomicOr(&kinds[4 * r8 + e], plus_rows | minus_rows << 2);
                    x[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
                }
                v[k] = make_uint2(x[0], x[1]);
            }
        }
        uint32_t p[2][2];  // weights of the lane's columns: [c or c + 8][row]
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[4], mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = (seen[i] >> ((k & 1) + 8 * (k >> 1))) & 1u ? s[k >> 1][2 * i + (k & 1)] * sc : -INFINITY;
                mx = fmaxf(mx, x[k]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2)) + 31.f;
            if (mx > ref[i]) {
                const float alpha = ex2(ref[i] - mx);
                ref[i] = mx;
                l[i] *= alpha;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    acc[n][2 * i] *= alpha;
                    acc[n][2 * i + 1] *= alpha;
                }
            }
            const float m = ref[i] == -INFINITY ? 0.f : ref[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = ex2(x[k] - m);
                l[i] += x[k];
            }
            p[0][i] = pack_bf16(x[0], x[1]);
            p[1][i] = pack_bf16(x[2], x[3]);
        }
        const uint32_t w[4][2] = {{v[0].x, v[0].y}, {v[1].x, v[1].y}, {v[2].x, v[2].y}, {v[3].x, v[3].y}};
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // column r8 of this product is value 4 r8 + n
            const uint32_t pick = n & 1 ? 0x7632u : 0x5410u;
            mma_16x8x16(acc[n], p[0][0], p[0][1], p[1][0], p[1][1], __byte_perm(w[0][n >> 1], w[1][n >> 1], pick),
                        __byte_perm(w[2][n >> 1], w[3][n >> 1], pick));
        }
    }
    __syncwarp();  // kinds is complete
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
        if (!bad[i]) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float y[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                y[n] = acc[n][2 * i + j] * inv;
                const uint32_t kind = (kinds[4 * (2 * c4 + j) + n] >> (4 * r8 + i)) & 5u;
                if (kind) y[n] += kind == 1 ? INFINITY : kind == 4 ? -INFINITY : __uint_as_float(0x7fffffffu);
            }
            if (sg.part >= 0) {
                reinterpret_cast<float4 *>(out[i])[j] = make_float4(y[0], y[1], y[2], y[3]);
            } else {
                reinterpret_cast<uint2 *>(out[i])[j] = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            }
        }
    }
    __syncwarp();  // kinds is read
}

// All segments of the CTA once more, after the last: each softmax warp takes its share of
// the groups of rows.  Here nothing waits for it but the CTA's end.  room: shared memory that
// nothing else uses any more; done: the CTA's walk, which has come to its end.
template <class C, int D, int kTiles>
__device__ __forceinline__ void rows_again(const GqaParams &prm, const Walk<C, kTiles> *done, uint8_t *room, int warp) {
    constexpr int kRoom = 1024;
    static_assert(sizeof(Walk<C, kTiles>) + sizeof(Segment) + 4 * kKindWords <= kRoom && C::kSoftWarps * kRoom <= C::kBlockBytes, "room");
    room += warp * kRoom;
    uint32_t *kinds = reinterpret_cast<uint32_t *>(room);
    Walk<C, kTiles> *walk = reinterpret_cast<Walk<C, kTiles> *>(room + 4 * kKindWords);
    Segment *place = reinterpret_cast<Segment *>(room + 4 * kKindWords + sizeof(Walk<C, kTiles>));
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        *walk = *done;
        walk->restart(prm.a, prm.group);
    }
    while (true) {
        if (lane == 0) *place = walk->next(prm.a, prm.group, prm.tgs_most);
        __syncwarp();
        const Segment sg = *place;
        __syncwarp();
        if (sg.blocks == 0) return;
        const int units = (sg.rows + 15) / 16 * (D / 32);
#pragma unroll 1
        for (int u = warp; u < units; u += C::kSoftWarps)
            rows_again_16<D>(prm, sg, u / (D / 32) * 16, u % (D / 32) * 32, kinds);
    }
}

template <int D, int kTiles>
__global__ void __launch_bounds__(Cfg<D, kTiles>::kThreads, kTiles == 2 ? 1 : 2)
gqa_attn_kernel(const __grid_constant__ GqaParams prm) {
    using C = Cfg<D, kTiles>;
    constexpr int NB = C::NB;
    const GqaArgs &a = prm.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + C::kOffHolder);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffHolder + 4);
    volatile int *not_finite = reinterpret_cast<volatile int *>(smem + C::kOffHolder + 8);  // a row of the CTA was not
    int64_t *plan = reinterpret_cast<int64_t *>(smem + C::kOffPlan);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kMmaWarp = C::kMmaWarp, kFirstLoad = C::kFirstLoad;
    if (warp == kMmaWarp && lane == 0) {
        for (int i = 0; i < C::bCount; ++i)
            mbar_init(bar(i), i < C::bKEmpty || (i >= C::bVFull && i < C::bVEmpty) ? 32 * C::kUnits  // load lanes
                      : i >= C::bPFull && i < C::bQFull                            ? 4               // row quarters
                      : i == C::bQFull                                             ? C::kSoftWarps
                      : i == C::bJoin                                              ? 4
                      : i >= C::bSegEmpty                                          ? C::kSoftWarps + C::kLoadWarps + 1
                                                                                   : 1);
        *abort_flag = 0;
        *not_finite = 0;
        fence_barrier_init();
    }
    // everything read below may be the previous kernel's output (q, the appended rows, the mask)
    pdl_wait();

    // ---- this CTA's work ----
    const bool dealt = a.num_ctas > 0;
    Walk<C, kTiles> *walk = reinterpret_cast<Walk<C, kTiles> *>(smem + C::kOffWalk);
    static_assert(sizeof(Walk<C, kTiles>) <= 128 && sizeof(Segment) <= 48, "the walk's room");
    if (dealt) {  // batch <= kThreads: thread i sizes request i, and a scan places it on the line
        constexpr int kWarps = C::kThreads / 32;
        Request req;
        int64_t cost = 0;
        if (tid < a.batch) {
            req = load_request<C, kTiles>(a, prm.group, tid, blockIdx.x == 0 ? a.err : nullptr);
            cost = request_cost<C>(req, a.num_kv_heads);
        }
        int64_t sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) plan[warp] = sum;
        __syncthreads();
        int64_t total = 0, at = sum - cost;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += plan[w];
            total += plan[w];
        }
        // CTAs that take a share: as many as get a few blocks at least; CTA c has the
        // positions [c q + min(c, rem), ...) of the line
        const int64_t most = a.forced ? total / C::kCostFull : total / C::kMinShare;
        const int ctas = most < 1 ? 1 : most < a.num_ctas ? (int)most : a.num_ctas;
        if (total == 0 || (int)blockIdx.x >= ctas) return;
        const int64_t q = divide(total, ctas), rem = total - q * ctas, c = blockIdx.x;
        const int64_t lo = c * q + min(c, rem), hi = (c + 1) * q + min(c + 1, rem);
        if (at <= lo && lo < at + cost) walk->start_share(req, blockIdx.x, tid, at, lo, hi);
    } else {
        const int b = blockIdx.z, tg = blockIdx.x / a.num_kv_heads;
        const Request req = load_request<C, kTiles>(a, prm.group, b, blockIdx.x == 0 && tid == 0 ? a.err : nullptr);
        if (tg >= req.tgs) return;
        if (tid == 0) walk->start_item(req, b, tg, blockIdx.x - tg * a.num_kv_heads);
    }

    if (warp == kMmaWarp) tmem_alloc(smem_u32(holder), C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    // After the wait: what starts early behind this kernel sees everything before
    // it.  After the allocation: a CTA that starts early cannot take the tensor
    // memory that this one still needs while it waits for this one's end.
    pdl_trigger();
    volatile Segment *ring = reinterpret_cast<volatile Segment *>(smem + C::kOffWalk + 128);
    // segment n of the CTA (its fields, or blocks = 0 behind the last); the caller's thread or warp
    // reads it once
    auto read_segment = [&](int n, Segment &s) {
        volatile Segment &x = ring[n & 1];
        s.row0 = x.row0;
        s.rows = x.rows;
        s.tiles = x.tiles;
        s.g = x.g;
        s.c_begin = x.c_begin;
        s.c_end = x.c_end;
        s.blocks = x.blocks;
        s.qo0 = x.qo0;
        s.kv0 = x.kv0;
        s.m0 = x.m0;
        s.W = x.W;
        s.part = x.part;
    };
    auto warp_segment = [&](int n, Segment &s) -> bool {  // false: the wait ran out
        if (!warp_wait(bar(C::bSegFull + (n & 1)), (n >> 1) & 1, abort_flag, a.err)) return false;
        read_segment(n, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bSegEmpty + (n & 1)));
        return true;
    };
    Segment sg;

    if (warp >= C::kSoftWarps) {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));  // one instruction for each warpgroup
        if (warp >= kFirstLoad && warp < kFirstLoad + C::kLoadWarps) {
            // ================= gather =================
            // A unit is 32 rows of a block of K or V.  Two-tile kernel: a warp has the same
            // unit of every block of K, or of V.
            // One-tile kernel: three warps take the units in turn in the order K(0) K(1)
            // V(0) K(2) V(1) ... V(blocks - 1).  A unit's fixed cost (its waits) and its
            // copies overlap those of the other warps' units.  A copy instruction moves
            // 512 bytes; the next unit's slots are loaded while this one's rows are copied.
            //
            // An "empty" wait goes by the phase's parity, so a warp may not reach a use of
            // a stage while the use two before is still to be read.  Where a warp has a
            // unit of every block its own last wait excludes that.  In the one-tile order
            // the unit before one of V(j) is of K(j) at the earliest (whose wait implies
            // PV(j - 4) is done, with two stages), the one before K(j) of V(j - 3) (S(j - 4)
            // done, since S(w + 1) is issued before PV(w)).
            constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows an instruction
            const int c = lane % kChunks, sub = lane / kChunks;
            const int64_t pitch = a.pool_stride * 2;
            int base = 0;  // blocks of the segments before
            bool ok = true;
            auto give_segment = [&](int n) {  // by the first load warp
                if (warp != kFirstLoad) return;
                if (n >= 2) ok = warp_wait(bar(C::bSegEmpty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag, a.err);
                if (ok && lane == 0) {
                    const Segment s = walk->next(a, prm.group, prm.tgs_most);
                    const_cast<Segment &>(ring[n & 1]) = s;
                    mbar_arrive(bar(C::bSegFull + (n & 1)));
                }
                __syncwarp();
            };
            give_segment(0);
            for (int seg = 0; ok; ++seg) {
                ok = warp_segment(seg, sg);
                if (!ok || sg.blocks == 0) break;
                give_segment(seg + 1);
                if (!ok) break;
                const int64_t at = ((int64_t)sg.g * D + c * 8) * 2;
                const char *kp = reinterpret_cast<const char *>(a.k_pool) + at, *vp = reinterpret_cast<const char *>(a.v_pool) + at;
                const int32_t *slots = a.kv_indices + sg.kv0 + sg.c_begin;
                const int cols = sg.c_end - sg.c_begin;
                constexpr bool kApart = kTiles == 2;
                const int lw = warp - kFirstLoad;
                const bool v_warp = kApart && lw >= C::kUnits;
                const int last = 2 * sg.blocks - 1, end = (kApart ? 1 : 2) * sg.blocks * C::kUnits;
                const int step = kApart ? C::kUnits : C::kLoadWarps;
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
                auto fetch = [&](int n) {
                    bool is_v;
                    const int j = block_of(n, is_v);
                    return slots[min(j * NB + 32 * (n % C::kUnits) + lane, cols - 1)];  // past the end: a valid row again
                };
                int n = v_warp ? lw - C::kUnits : lw;
                int ahead = n < end ? fetch(n) : 0;
                for (; n < end; n += step) {
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
                    const uint32_t to = sbase + (is_v ? C::kOffV : C::kOffK) + s * C::kBlockBytes +
                                        (c >> 3) * C::kBoxBytes + (n % C::kUnits) * 32 * 128;
                    const char *pool = is_v ? vp : kp;
#pragma unroll
                    for (int i = 0; i < 32 / kPer; ++i) {
                        const int k = i * kPer + sub;
                        cp_async_16(to + k * 128 + (((c & 7) ^ (k & 7)) << 4), pool + __shfl_sync(0xffffffffu, slot, k) * pitch);
                    }
                    cp_async_arrive(bar((is_v ? C::bVFull : C::bKFull) + s));
                }
                base += sg.blocks;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may land after the CTA has left
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
                    auto issue_s = [&](int slot) {
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
                        if (ok && slot < items) issue_s(slot);
                    while (ok && w < items) {
#pragma unroll
                        for (int slot = 0; slot < 2; ++slot) {
                            if (!ok || w >= items) break;
                            issue_pv(slot);
                            if (ok && w + 2 < items) issue_s(slot);
                            ++w;
                        }
                    }
                };
                for (int seg = 0; ok; ++seg) {
                    ok = wait_or_abort(bar(C::bSegFull + (seg & 1)), (seg >> 1) & 1, abort_flag, a.err);
                    if (!ok) break;
                    read_segment(seg, sg);
                    mbar_arrive(bar(C::bSegEmpty + (seg & 1)));
                    if (sg.blocks == 0) break;
                    ok = wait_or_abort(bar(C::bQFull), seg & 1, abort_flag, a.err);
                    if (!ok) break;
                    if constexpr (kTiles == 2) {
                        if (sg.tiles == 2) run(std::integral_constant<int, 2>{}, 2 * sg.blocks);
                        else run(std::integral_constant<int, 1>{}, sg.blocks);
                    } else {
                        run(std::integral_constant<int, 1>{}, sg.blocks);
                    }
                    mma_commit(bar(C::bOFin));  // completes when the segment's MMAs have
                }
                mma_commit(bar(C::bDrain));  // every MMA issued has to be done before the exit
                mbar_wait(bar(C::bDrain), 0, kWaitLimit);
            }
            __syncwarp();
        }
    } else {
        // ================= softmax (thread = row = TMEM lane of its tile) =================
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        const int t = warp >> 2, wq = warp & 3;
        const int r = 32 * wq + lane;  // row within the tile
        const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
        const float sc = a.scale * kLog2e;
        // parity of the uses of the slots that this warp serves (two tiles: its own one); its blocks, and joins, so far
        uint32_t phases = 0, done = 0, joins = 0;
        bool ok = true;
        for (int seg = 0; ok; ++seg) {
            ok = warp_segment(seg, sg);
            if (!ok || sg.blocks == 0) break;
            const bool lone = kTiles == 2 && sg.tiles == 1;  // one tile, served by both tiles' warps
            const int first = lone ? 0 : t * kRows;          // the tile's first row in the item
            const int rows_t = sg.rows - first;
            // ---- q rows of this warp into the swizzled operand layout ----
            if (32 * wq < rows_t && !(lone && t == 1)) {
                constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows per step
                const int c = lane % kChunks, sub = lane / kChunks;
                const uint32_t qb = sbase + C::kOffQ + t * C::kQBytes + (c >> 3) * C::kQBoxBytes;
                const uint16_t *q = a.q + ((int64_t)sg.qo0 * a.num_heads + sg.g * prm.group) * D + c * 8;
#pragma unroll 4
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int rt = 32 * wq + i * kPer + sub;
                    if (rt < rows_t) {
                        const int rr = sg.row0 + first + rt;
                        const int node = quotient(rr, prm.group_inv), hg = rr - node * prm.group;
                        cp_async_16(qb + (rt >> 3) * 1024 + (rt & 7) * 128 + (((c & 7) ^ (rt & 7)) << 4),
                                    q + ((int64_t)node * a.num_heads + hg) * D);
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bQFull));
            const bool warp_on = 32 * wq < rows_t;  // the warp has rows
            const bool row_on = r < rows_t;
            const int rr = sg.row0 + (row_on ? first + r : 0);
            const int node = quotient(rr, prm.group_inv);
            const uint32_t *words = a.mask + sg.m0 + (int64_t)node * sg.W;
            float m_ref = -INFINITY, l = 0.f;  // the reference in log2 units, the sum against it
            constexpr int kW = NB / 32;
            const int j0 = lone ? t : 0, step = lone ? 2 : 1;
            const uint32_t *at = words + ((sg.c_begin + j0 * NB) >> 5);  // the next block's mask words,
            int left = sg.c_end - sg.c_begin - j0 * NB;                  // and the columns from it on
            auto mask_words = [&](uint32_t (&mw)[kW]) {
                if (left >= NB) {
#pragma unroll
                    for (int k = 0; k < kW; ++k) mw[k] = at[k];
                } else {
#pragma unroll
                    for (int k = 0; k < kW; ++k) {
                        mw[k] = 32 * k < left ? at[k] : 0u;
                        if (32 * k < left && left - 32 * k < 32) mw[k] &= (1u << (left - 32 * k)) - 1u;
                    }
                }
                at += step * kW;
                left -= step * NB;
            };
            uint32_t mnext[kW];
            if (warp_on && j0 < sg.blocks) mask_words(mnext);
            uint32_t own = 0;  // this warp's blocks in the segment
            for (int j = j0; j < sg.blocks; j += step, ++own) {
                const int slot = kTiles == 2 ? t : j & 1;
                const uint32_t phase = (phases >> slot) & 1;
                const uint32_t col = tmem + lane_off + C::kColS + NB * slot;
                uint32_t mw[kW];
                if (warp_on) {
#pragma unroll
                    for (int k = 0; k < kW; ++k) mw[k] = mnext[k];
                    if (j + step < sg.blocks) mask_words(mnext);
                }
                ok = warp_wait(bar(C::bSFull + slot), phase, abort_flag, a.err);
                if (!ok) break;
                if (warp_on) {
                    tc_fence_after();
                    uint32_t all = mw[0];
#pragma unroll
                    for (int k = 1; k < kW; ++k) all &= mw[k];
                    const bool whole = __all_sync(0xffffffffu, all == 0xffffffffu);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h) {
                        // The one-tile kernel keeps the 64 scores until the weights are sure and stores
                        // these as it goes; the two-tile kernel, short of registers, reads the scores
                        // again when the reference moves and stores the weights at the end (the other
                        // way round measured 2% and 12% slower).
                        constexpr bool kKeep = kTiles == 1;
                        uint32_t s[2][32];  // the scores
                        auto take = [&]() {
                            tmem_ld32(col + 64 * h, s[0]);
                            tmem_ld32(col + 64 * h + 32, s[1]);
                            tmem_wait_ld();
                            if (!whole) {  // unseen columns at -inf; a branch, not selects: most blocks are seen whole
                                asm volatile("");
#pragma unroll
                                for (int e = 0; e < 64; ++e)
                                    s[e >> 5][e & 31] = ((mw[2 * h + (e >> 5)] >> (e & 31)) & 1u) ? s[e >> 5][e & 31] : 0xff800000u;
                            }
                        };
                        if (kKeep) take();
                        uint32_t pw[2][16];  // the weights as bf16 pairs
                        float sum;
                        while (true) {
                            if (!kKeep) take();
                            const float m = m_ref == -INFINITY ? 0.f : m_ref;  // nothing seen: every weight is 0
                            const float2 scv = make_float2(sc, sc), nmv = make_float2(-m, -m);
                            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 x = f2fma(make_float2(__uint_as_float(s[k][e]), __uint_as_float(s[k][e + 1])), scv, nmv);
                                    const float p0 = ex2(x.x), p1 = ex2(x.y);
                                    acc = f2add(acc, make_float2(p0, p1));
                                    pw[k][e / 2] = pack_bf16(p0, p1);
                                }
                                if (kKeep) tmem_st16(col + 32 * h + 16 * k, pw[k]);  // over scores that have been read
                            }
                            sum = acc.x + acc.y;
                            const bool moves = row_on && (sum > kSumLimit || (m_ref == -INFINITY && (mw[2 * h] | mw[2 * h + 1])));
                            if (!__any_sync(0xffffffffu, moves)) break;
                            // The reference moves to the largest of these scores, and what was summed
                            // against the old one shrinks; then the weights are taken again.
                            float mx = -INFINITY;
                            if (kKeep) {
#pragma unroll
                                for (int e = 0; e < 64; ++e) mx = fmaxf(mx, __uint_as_float(s[e >> 5][e & 31]));
                            } else {
#pragma unroll 1
                                for (int q = 0; q < 8; ++q) {
                                    uint32_t o8[8];
                                    tmem_ld8(col + 64 * h + 8 * q, o8);
                                    tmem_wait_ld();
                                    const uint32_t seen = (q < 4 ? mw[2 * h] : mw[2 * h + 1]) >> (8 * (q & 3));
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        if ((seen >> e) & 1u) mx = fmaxf(mx, __uint_as_float(o8[e]));
                                }
                            }
                            mx *= sc;
                            const bool up = moves && mx > m_ref;
                            if (!__any_sync(0xffffffffu, up)) break;  // scores of -inf or NaN move nothing
                            if (kKeep) tmem_wait_st();  // the next weights go to the same columns: stores have no order
                            const float alpha = up ? ex2(m_ref - mx) : 1.0f;
                            if (up) m_ref = mx;
                            l *= alpha;
                            // The products so far have to be done before the output is scaled: of this
                            // block's first half; or of the output's last block (with two outputs S(w)
                            // was issued behind it, so it is done).
                            if (h > 0) ok = warp_wait(bar(C::bHalf + slot), phase, abort_flag, a.err);
                            else if (kTiles == 1 && own > 0) ok = warp_wait(bar(C::bODone), (done + own - 1) & 1, abort_flag, a.err);
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
                        if (!ok) break;
                        l += sum;
                        if (!kKeep) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) tmem_st16(col + 32 * h + 16 * k, pw[k]);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::bPFull + C::kHalves * slot + h));
                    }
                    if (!ok) break;
                } else {
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        if (lane == 0) mbar_arrive(bar(C::bPFull + C::kHalves * slot + h));
                }
                phases ^= 1u << slot;
            }
            if (!ok) break;
            done += own;
            // ---- epilogue ----
            ok = warp_wait(bar(C::bOFin), seg & 1, abort_flag, a.err);
            float keep0 = 1.f, keep1 = 0.f;  // what the two outputs of a lone tile count
            if (ok && lone) {
                // The wait above: the first tile's warps have left the segment before (its q is
                // theirs), so these places are free.
                volatile float *place = reinterpret_cast<volatile float *>(smem + C::kOffJoin) + 2 * r;
                if (t == 1) {
                    place[0] = m_ref;
                    place[1] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bJoin));
                } else {
                    ok = warp_wait(bar(C::bJoin), joins & 1, abort_flag, a.err);
                    const float m1 = place[0], l1 = place[1], m = fmaxf(m_ref, m1);
                    keep0 = m_ref == -INFINITY ? l : ex2(m_ref - m);  // without a reference the sum is 0, or NaN
                    keep1 = m1 == -INFINITY ? l1 : ex2(m1 - m);
                    l = (keep0 != 0.f ? l * keep0 : 0.f) + (keep1 != 0.f ? l1 * keep1 : 0.f);
                    m_ref = m;
                }
                ++joins;
            }
            if (ok && warp_on && !(lone && t == 1)) {
                tc_fence_after();
                const int head = sg.g * prm.group + rr - node * prm.group;
                const int64_t row = (int64_t)(sg.qo0 + node) * a.num_heads + head;
                const bool part = sg.part >= 0;
                const int64_t prow = (int64_t)sg.part * prm.part_rows + first + r;  // (of lanes without a row: not used)
                const float inv = 1.f / l;
                const bool none = l == 0.f;
                float check = 0.f;
                // The rows leave through the tile's place for q, which nothing reads any more: a
                // thread writes its row's next 128 bytes there, and eight lanes write each row's to
                // global memory (a thread's own 16-byte stores, a row apart, measured 5.8 us a tile).
                uint8_t *stage = smem + C::kOffQ + t * C::kQBytes + wq * 4096;
                auto put = [&](int piece, int c, uint4 v) {  // chunk c of this lane's row
                    *reinterpret_cast<uint4 *>(stage + (piece % C::kBoxes) * C::kQBoxBytes + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
                };
                auto flush = [&](int piece, auto row_start) {  // row_start: row of the warp -> its bytes' place
                    __syncwarp();
                    uint4 v[8];
                    const int c = lane & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rw = 4 * i + (lane >> 3);
                        v[i] = *reinterpret_cast<const uint4 *>(stage + (piece % C::kBoxes) * C::kQBoxBytes + rw * 128 +
                                                                ((c ^ (rw & 7)) << 4));
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rw = 4 * i + (lane >> 3);
                        if (32 * wq + rw < rows_t) reinterpret_cast<uint4 *>(row_start(rw))[8 * piece + c] = v[i];
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
                    if (lone) {
                        tmem_ld32(tmem + lane_off + C::kColO + D + 32 * q, t32);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = (keep0 != 0.f ? o[e] * keep0 : 0.f) + (keep1 != 0.f ? __uint_as_float(t32[e]) * keep1 : 0.f);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        check = fmaf(o[e], 0.f, check);  // NaN from the first infinity or NaN on
                        o[e] = none ? 0.f : o[e] * inv;
                    }
                    if (part) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            put(q, e, make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                                                 __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3])));
                        flush(q, [&](int rw) { return a.o_part + (prow - lane + rw) * D; });
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            put(q >> 1, 4 * (q & 1) + e,
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7])));
                        if (q & 1)
                            flush(q >> 1, [&](int rw) {
                                const int n = sg.row0 + first + 32 * wq + rw, nd = quotient(n, prm.group_inv);
                                return a.out + ((int64_t)(sg.qo0 + nd) * a.num_heads + sg.g * prm.group + n - nd * prm.group) * D;
                            });
                    }
                }
                if (row_on) {
                    const float lse = none ? -INFINITY : (m_ref + log2f(l)) * kLn2;
                    if (part) a.lse_part[prow] = lse;
                    else if (a.lse) a.lse[row] = lse;
                }
                // (a NaN sum stays one whatever V holds)
                if (row_on && check != check && l > 0.f) *not_finite = 1;
                tc_fence_before();  // the output has been read before the next segment's first product
            }
        }
        // ---- rows that are not finite ----
        named_barrier(1, 32 * C::kSoftWarps);  // every row of the CTA is written; its products have left shared memory
        if (*not_finite && !*abort_flag) rows_again<C, D, kTiles>(prm, walk, smem + C::kOffK, warp);
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// out = sum_s e^{lse_s - LSE} o_s over the parts s of a cut item, LSE = log sum_s
// e^{lse_s}.  A CTA has 8 kRowsOfWarp rows of an item and leaves at once where one
// CTA did the item whole; a warp joins kRowsOfWarp rows at a time: 32 / kRowsOfWarp
// lanes hold the weights of that many parts of each, then all lanes sum D / 32
// values of every row.
constexpr int kCombineWarps = 8;

template <int D, int kTiles, int kRowsOfWarp>
__global__ void __launch_bounds__(32 * kCombineWarps) gqa_combine_kernel(const GqaParams prm) {
    using C = Cfg<D, kTiles>;
    constexpr int E = D / 32, R = kRowsOfWarp, L = 32 / R;  // lanes of a row's parts
    constexpr int kFlight = 8 / R;                          // parts in flight
    const GqaArgs &a = prm.a;
    const int lane = threadIdx.x & 31;
    const int bg = blockIdx.x / prm.tgs_most, tg = blockIdx.x - bg * prm.tgs_most;
    const int b = bg / a.num_kv_heads, g = bg - b * a.num_kv_heads;
    const int first = (blockIdx.y * kCombineWarps + (threadIdx.x >> 5)) * R;  // of the item's rows
    pdl_wait();
    pdl_trigger();
    const int2 note = a.notes[blockIdx.x];
    const Request r = load_request<C, kTiles>(a, prm.group, b, nullptr);
    if (tg >= r.tgs || note.x < 0) return;  // no such item, or one CTA did it whole
    if (note.y >= a.num_ctas) return;       // nobody wrote it: the kernel before gave up (a timeout is latched)
    const int row0 = tg * kTiles * kRows, rows = min(kTiles * kRows, r.T * prm.group - row0);
    if (first >= rows) return;
    const int c0 = note.x >> 1, parts = note.y - c0 + 1;
    // row i of the warp; lanes of rows that are not there repeat the last one
    auto place = [&](int s, int i) { return (int64_t)(s == 0 ? note.x : 2 * (c0 + s)) * prm.part_rows + min(first + i, rows - 1); };
    // weights of 2^-9 at most: those of DDT_GQA_MAX_CTAS parts sum to 1, and finite parts to a finite value
    constexpr float kShift = 9.f;
    static_assert(DDT_GQA_MAX_CTAS <= 512, "parts of a row");
    float m = -INFINITY, den = 0.f;  // of the lane's row (lane / L)
    float acc[R][E];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
    for (int s0 = 0; s0 < parts; s0 += L) {
        const int mine = s0 + lane % L;
        const float ls = mine < parts ? a.lse_part[place(mine, lane / L)] : -INFINITY;
        float mg = fmaxf(m, ls);
#pragma unroll
        for (int o = L / 2; o >= 1; o >>= 1) mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
        const float keep = m == -INFINITY ? 0.f : ex2((m - mg) * kLog2e);
        const float w = ls == -INFINITY ? 0.f : ex2((ls - mg) * kLog2e - kShift);  // NaN stays
        float sum = w;
#pragma unroll
        for (int o = L / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        den = den * keep + sum;
        m = mg;
        if (s0 > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float k = __shfl_sync(0xffffffffu, keep, i * L);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[i][e] *= k;
            }
        }
        const int n = min(L, parts - s0);
        for (int s = 0; s < n; s += kFlight) {
            float v[kFlight][R][E];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (s + u >= n) break;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float *o = a.o_part + place(s0 + s + u, i) * D + lane * E;
                    if constexpr (E == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(o);
                        v[u][i][0] = x.x; v[u][i][1] = x.y; v[u][i][2] = x.z; v[u][i][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2 *>(o);
                        v[u][i][0] = x.x; v[u][i][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (s + u >= n) break;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float ws = __shfl_sync(0xffffffffu, w, i * L + s + u);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[i][e] = fmaf(ws, v[u][i][e], acc[i][e]);
                }
            }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den, lse = den == 0.f ? -INFINITY : m + (log2f(den) + kShift) * kLn2;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float k = __shfl_sync(0xffffffffu, inv, i * L), ls = __shfl_sync(0xffffffffu, lse, i * L);
        if (first + i >= rows) break;
        const int rr = row0 + first + i, node = quotient(rr, prm.group_inv);
        const int64_t row = (int64_t)(r.qo0 + node) * a.num_heads + g * prm.group + rr - node * prm.group;
        uint16_t *dst = a.out + row * D + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(acc[i][0] * k, acc[i][1] * k), pack_bf16(acc[i][2] * k, acc[i][3] * k));
        else
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16(acc[i][0] * k, acc[i][1] * k);
        if (a.lse && lane == 0) a.lse[row] = ls;
    }
}

template <int D, int kTiles>
cudaError_t launch(GqaParams &prm, int num_sms, cudaStream_t s) {
    using C = Cfg<D, kTiles>;
    GqaArgs &a = prm.a;
    const dim3 grid = a.num_ctas > 0 ? dim3((unsigned)a.num_ctas)
                                     : dim3((unsigned)(prm.tgs_most * a.num_kv_heads), 1, (unsigned)a.batch);
    cudaError_t e = launch_pdl(gqa_attn_kernel<D, kTiles>, grid, dim3(C::kThreads), C::kSmemBytes, s, prm);
    if (e == cudaSuccess && a.num_ctas > 0) {
        // four rows of a warp at once where there are many: 8448 rows (4 requests of 33 x 64)
        // 40.1 us with the attention against 42.2 us, 25600 rows 113 against 121, 2112 rows 31.8 against 30.2
        const int R = (int64_t)a.total_q * a.num_heads > 32LL * num_sms ? 4 : 1;
        const dim3 items((unsigned)(a.batch * a.num_kv_heads * prm.tgs_most),
                         (unsigned)((prm.part_rows + kCombineWarps * R - 1) / (kCombineWarps * R)));
        e = launch_pdl(R == 4 ? gqa_combine_kernel<D, kTiles, 4> : gqa_combine_kernel<D, kTiles, 1>, items,
                       dim3(32 * kCombineWarps), 0, s, prm);
    }
    return e;
}

template <int D, int kTiles>
cudaError_t prepare() {
    if (kTiles == 2) {  // the softmax warps would wait for registers that the launch does not have
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, gqa_attn_kernel<D, kTiles>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < Cfg<D, kTiles>::kLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    const cudaError_t e = cudaFuncSetAttribute(gqa_attn_kernel<D, kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg<D, kTiles>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(gqa_attn_kernel<D, kTiles>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                (int)cudaSharedmemCarveoutMaxShared);
}

}  // namespace

cudaError_t gqa_prepare_device() {
    cudaError_t e = prepare<64, 1>();
    if (e == cudaSuccess) e = prepare<64, 2>();
    if (e == cudaSuccess) e = prepare<128, 1>();
    if (e == cudaSuccess) e = prepare<128, 2>();
    return e;
}

int gqa_tiles(int max_q_len, int group) { return max_q_len * group > kRows ? 2 : 1; }

int gqa_part_rows(int tiles, int max_q_len, int group) { return std::min(max_q_len * group, tiles * kRows); }

int gqa_tile_groups(int tiles, int max_q_len, int group) {
    return (max_q_len * group + tiles * kRows - 1) / (tiles * kRows);
}

size_t gqa_layout(GqaArgs &a, void *base) {
    const int group = a.num_heads / a.num_kv_heads;
    const size_t rows = (size_t)2 * a.num_ctas * gqa_part_rows(a.tiles, a.max_q_len, group);
    const size_t items = (size_t)a.batch * a.num_kv_heads * gqa_tile_groups(a.tiles, a.max_q_len, group);
    auto align = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t notes = align(items * sizeof(int2)), o = align(rows * a.head_dim * sizeof(float));
    if (base) {
        char *p = static_cast<char *>(base);
        a.notes = reinterpret_cast<int2 *>(p);
        a.o_part = reinterpret_cast<float *>(p + notes);
        a.lse_part = reinterpret_cast<float *>(p + notes + o);
    }
    return notes + o + align(rows * sizeof(float));
}

namespace {

bool may_deal(int batch, int max_kv_len) { return batch <= kGqaMaxDealtBatch && max_kv_len > 256; }
int slots(int tiles, int num_sms) { return std::min(num_sms * (tiles == 2 ? 1 : 2), DDT_GQA_MAX_CTAS); }

// Microseconds that a call takes, roughly: with its blocks dealt to `ctas` CTAs, or
// (ctas = 0) with a CTA per item, which the hardware hands out as others end.  Dealing
// costs the plan, cut items and the combine kernel, and evens out long or few items;
// two tiles halve the reads of K and V, one tile starts and ends faster.  The constants
// are fitted to 224 shapes measured dealt and undealt, above 128 rows with one tile and
// two (1 to 64 requests, 500 to 16000 columns even and ragged, 1 to 33 tokens, 4 to 16
// K/V heads): each way within 10%.  The choice costs 1% over the best of these on average and
// 20% at most (29% over some 100 other shapes, prompt chunks among them), where one fixed way
// (two tiles above 128 rows, dealt) cost 17% and 100%.  The sizes are means over the call: one
// long request among many short ones, and a kv_indices longer than its requests, are weighed
// as an even batch of them.  64
// requests of 33 tokens x 64 heads after 1000 take 230 us dealt with two tiles, 130 us
// undealt with one; 4 of them after 16000 120 us dealt and 217 us undealt; 16 of 32
// tokens after 8000 122 us undealt with two tiles, 140 us with one.
double estimate(const GqaArgs &a, int tiles, int ctas, int num_sms) {
    const double rows = std::min((double)a.total_q / a.batch, (double)a.max_q_len) * (a.num_heads / a.num_kv_heads);
    const double columns = std::min((double)a.total_kv / a.batch, (double)a.max_kv_len);
    const double items = (double)a.batch * a.num_kv_heads * std::ceil(rows / (tiles * kRows));
    const double width = 0.6 + 0.4 * a.head_dim / 128, block = 64.0 * tiles;
    if (ctas > 0) {
        const double all = rows * a.batch * a.num_kv_heads / 1000;
        return tiles == 1 ? 12.5 + items * (2.9 + 1.44 * width * columns / block) / ctas + 0.22 * all
                          : 17.5 + items * (8.9 + 1.97 * width * columns / block) / ctas + 0.16 * all;
    }
    const double start = tiles == 1 ? 3.2 : 8.6, tail = tiles == 1 ? 0.68 : 0.8;
    // one tile: two CTAs on an SM slow each other down
    const double per_block = width * (tiles == 1 ? 0.73 + 0.39 * std::min(std::max(items / num_sms - 1, 0.0), 1.0) : 1.6);
    const double longest = start + per_block * a.max_kv_len / block, mean = start + per_block * columns / block;
    const double waves = items / (num_sms * (tiles == 1 ? 2 : 1));
    return 4 + (waves <= 1 ? longest : std::max(longest, (waves + tail) * mean));
}

}  // namespace

int gqa_most_ctas(int batch, int num_heads, int num_kv_heads, int max_q_len, int max_kv_len, int num_sms) {
    return may_deal(batch, max_kv_len) ? slots(gqa_tiles(max_q_len, num_heads / num_kv_heads), num_sms) : 0;
}

void gqa_choose(GqaArgs &a, size_t workspace_bytes, int num_sms) {
    const int most_tiles = gqa_tiles(a.max_q_len, a.num_heads / a.num_kv_heads);
    int best_tiles = 1, best_ctas = 0;
    double best = 0;
    for (int tiles = 1; tiles <= most_tiles; ++tiles) {
        a.tiles = tiles;
        a.num_ctas = may_deal(a.batch, a.max_kv_len) ? slots(tiles, num_sms) : 0;
        while (a.num_ctas > 0 && gqa_layout(a, nullptr) > workspace_bytes) --a.num_ctas;
        for (int dealt = a.num_ctas > 0; dealt >= 0; --dealt) {
            const int ctas = dealt ? a.num_ctas : 0;
            const double us = estimate(a, tiles, ctas, num_sms);
            if (best == 0 || us < best) {
                best = us;
                best_tiles = tiles;
                best_ctas = ctas;
            }
        }
    }
    a.tiles = best_tiles;
    a.num_ctas = best_ctas;
}

cudaError_t launch_gqa_attn(const GqaArgs &a, int num_sms, cudaStream_t s) {
    GqaParams prm;
    prm.a = a;
    prm.group = a.num_heads / a.num_kv_heads;
    prm.group_inv = 1.0f / (float)prm.group;
    prm.part_rows = gqa_part_rows(a.tiles, a.max_q_len, prm.group);
    prm.tgs_most = gqa_tile_groups(a.tiles, a.max_q_len, prm.group);
    const bool two = a.tiles == 2;
    if (a.head_dim == 128) return two ? launch<128, 2>(prm, num_sms, s) : launch<128, 1>(prm, num_sms, s);
    return two ? launch<64, 2>(prm, num_sms, s) : launch<64, 1>(prm, num_sms, s);
}

}  // namespace ddt
