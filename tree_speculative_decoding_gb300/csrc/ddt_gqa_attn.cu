// ddt_gqa_attn.cu -- tree-verify attention over grouped-query K/V rows on the
// sm_103a tensor cores.
//
// For row (tree node i of request b, head h), K/V head g = h / group, over the
// columns j that mask row i makes visible:
//   s_j = scale <q[i,h], k[idx_j][g]>,  out[i,h] = sum_j softmax(s)_j v[idx_j][g],
//   lse = log sum_j e^{s_j}
// in one pass over the columns with a running maximum and sum.
//
// Work of a CTA: one K/V head of one request, one split of its columns, and up
// to kTiles tiles of 128 consecutive rows (node-major, the group's heads inside
// a node: the rows that share the K/V head).  The K and V rows of a block are
// gathered once for all its tiles.
//   * kTiles = 1: blocks of 64 columns, 256 tensor-memory columns and under half
//     of the shared memory, so two CTAs share an SM: one's prologue, softmax and
//     epilogue run under the other's loads.  Taken when a request's rows per K/V
//     head fit one tile (decode, small trees): the loads bound it.
//   * kTiles = 2: blocks of 128 columns, all of tensor memory; the tensor core
//     works on one tile while the softmax of the other runs.
// Score slots: two buffers of one block's scores in tensor memory.  Work item w
// (block-major, tiles inside a block) uses slot w mod 2: with two tiles each has
// its own, with one tile blocks alternate.  The MMA warp issues
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
// so the scores of w + 1 are being computed, or done, while the softmax of w
// runs.  P (bf16) overwrites the scores in place and is the A operand of PV
// from tensor memory; V is read as an MN-major operand from its gathered rows.
//
// Warps: four softmax warps per tile (thread = row = TMEM lane), one that issues
// MMAs, one that gathers rows by TMA (tile::gather4: four 128-byte row pieces an
// instruction, 128-byte swizzle, the layout the MMA descriptors expect).
//
// Columns that a row does not see get p = 0, but 0 * NaN is NaN: a V row that
// holds NaN or infinities reaches the output rows that do not see it.  A row
// whose output is not finite is therefore computed again on the CUDA cores over
// its visible columns only (the running maximum and sum stand: the scores were
// selected before they were used).
//
// Every wait is bounded: on timeout the CTA latches DDT_DEVERR_TIMEOUT, waits
// for its own copies and MMAs and leaves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "ddt_gqa.cuh"
#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace {

using namespace sm100;

constexpr int kRows = 128;      // rows per tile (TMEM lanes)
constexpr int kSplitUnit = 128; // a split is a whole number of these columns
constexpr uint32_t kWaitLimit = 1u << 22;
// Lazy rescale: the running maximum (log2 units) moves only when a block's
// exceeds it by more than this, so p <= 2^48; the fp32 sums stay finite for
// |v| below ~2^59 at a million columns, and bf16 weights keep their relative
// precision at any scale.
constexpr float kRescaleLog2 = 48.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct GqaParams {
    GqaArgs a;
    int group;     // query heads per K/V head
};

template <int D, int kTiles>
struct Cfg {
    static constexpr int NB = kTiles == 2 ? 128 : 64;    // columns per block
    static constexpr int kBoxes = D / 64;                // 128-byte pieces of a row
    static constexpr int kBoxBytes = NB * 128;           // one piece of a block's rows
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
    static constexpr int kQBoxBytes = kRows * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;  // one tile of q
    static constexpr int kKStages = D == 128 ? (kTiles == 2 ? 3 : 2) : 4;
    static constexpr int kVStages = D == 128 ? 2 : 4;
    static constexpr int kHalves = NB / 64;              // parts of P that PV may start on
    static constexpr int kUnits = NB / 32;               // 32-row units of a block
    static constexpr int kLoadWarps = 4 * kTiles - 1;    // with the MMA warp: whole warpgroups
    static constexpr int kThreads = 256 * kTiles;
    static constexpr uint32_t kTmemCols = kTiles == 2 ? 512 : 256;
    static constexpr uint32_t kColS = 0, kColO = 2 * NB;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTiles * kQBytes;
    static constexpr int kOffV = kOffK + kKStages * kBlockBytes;
    static constexpr int kOffBar = kOffV + kVStages * kBlockBytes;
    // barriers
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bVFull = bKEmpty + kKStages,
                         bVEmpty = bVFull + kVStages, bSFull = bVEmpty + kVStages, bPFull = bSFull + 2,
                         bQFull = bPFull + 2 * kHalves, bODone = bQFull + 1, bOFin = bODone + 1, bCount = bOFin + 1;
    static constexpr int kOffHolder = kOffBar + 8 * bCount;
    static constexpr int kSmemUsed = kOffHolder + 8;
    static constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for the 1024-byte alignment of swizzle atoms
    static constexpr uint32_t kIdescS = idesc_bf16(kRows, NB, 0, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16(kRows, D, 0, 1);
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

// Output of one row over its visible columns of [c_begin, c_end), by the whole
// warp: lane l keeps values [l D / 32, (l + 1) D / 32).  m is the row's running
// maximum in log2 units.
template <int D>
__device__ __forceinline__ void row_again(const GqaArgs &a, const uint16_t *q, const uint32_t *words, int kv0, int c_begin,
                                       int c_end, int g, float m, float (&o)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = __uint_as_float((uint32_t)q[lane * E + e] << 16);
        o[e] = 0.f;
    }
    for (int j = c_begin; j < c_end; ++j) {
        if (!((words[j >> 5] >> (j & 31)) & 1u)) continue;
        int64_t slot = a.kv_indices[kv0 + j];
        if (slot < 0 || slot >= a.pool_rows) slot = 0;
        const int64_t at = slot * a.pool_stride + (int64_t)g * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(x[e], __uint_as_float((uint32_t)a.k_pool[at + e] << 16), s);
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float p = ex2(s * (a.scale * kLog2e) - m);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, __uint_as_float((uint32_t)a.v_pool[at + e] << 16), o[e]);
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

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kMmaWarp = 4 * kTiles, kFirstLoad = kMmaWarp + 1;
    // everything read below may be the previous kernel's output (q, the appended rows, the mask)
    pdl_wait();

    // ---- the CTA's work: K/V head g of request b, rows [row0, row0 + rows), columns [c_begin, c_end) ----
    const int g = blockIdx.x % a.num_kv_heads, tile_group = blockIdx.x / a.num_kv_heads;
    const int split = blockIdx.y, b = blockIdx.z;
    const int qo0 = a.qo_indptr[b], qo1 = a.qo_indptr[b + 1];
    const int kv0 = a.kv_indptr[b], kv1 = a.kv_indptr[b + 1];
    const int m0 = a.mask_indptr[b], m1 = a.mask_indptr[b + 1];
    const int T = qo1 - qo0, N = kv1 - kv0, W = (N + 31) >> 5;
    const bool bad_qo = T < 0 || T > a.max_q_len || qo0 < 0 || qo1 > a.total_q;
    const bool bad_kv = N < T || N > a.max_kv_len || kv0 < 0 || kv1 > a.total_kv;
    const bool bad_mask = !bad_qo && !bad_kv && (m0 < 0 || m1 - m0 != T * W || m1 > a.total_mask_words);
    if (bad_qo || bad_kv || bad_mask) {
        if (tid == 0)
            latch(a.err, (bad_qo ? DDT_DEVERR_QO_INDPTR : 0u) | (bad_kv ? DDT_DEVERR_KV_INDPTR : 0u) |
                             (bad_mask ? DDT_DEVERR_MASK_INDPTR : 0u));
        return;
    }
    const int row0 = tile_group * kTiles * kRows;
    const int rows = min(kTiles * kRows, T * prm.group - row0);
    const int c_begin = split * a.split_cols;
    const int c_end = min(N, c_begin + a.split_cols);
    if (rows <= 0 || c_begin >= c_end) return;  // the combine knows which splits of a request exist
    const int nblk = (c_end - c_begin + NB - 1) / NB;
    const int tiles = (rows + kRows - 1) / kRows;  // 1 .. kTiles
    const int items = nblk * tiles;

    // ---- barriers and tensor memory ----
    if (warp == kMmaWarp && lane == 0) {
        // P of a slot: one arrival per softmax warp that has rows in the slot's tile
        const int w0 = (min(rows, kRows) + 31) >> 5, w1 = tiles == 2 ? (rows - kRows + 31) >> 5 : w0;
        for (int i = 0; i < C::bCount; ++i)
            mbar_init(bar(i), i < C::bKFull + C::kKStages || (i >= C::bVFull && i < C::bVFull + C::kVStages) ? 32 * C::kUnits
                      : i >= C::bPFull && i < C::bPFull + C::kHalves ? w0 : i >= C::bPFull + C::kHalves && i < C::bQFull ? w1 : i == C::bQFull ? (tiles == 2 ? w0 + w1 : w0) : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == kMmaWarp) tmem_alloc(smem_u32(holder), C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    // After the wait: what starts early behind this kernel sees everything before
    // it.  After the allocation: a CTA that starts early cannot take the tensor
    // memory that this one still needs while it waits for this one's end.
    pdl_trigger();
    // Registers of the two-tile kernel: 512 threads x 128 at launch = 256 x 184 (softmax: a block's
    // scores of a row) + 256 x 72.
    if (warp >= kMmaWarp) {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");  // one instruction for the warpgroup
        if (warp >= kFirstLoad) {
            // ================= gather =================
            // The warps take units of 32 rows in turn, in the order K(0) K(1) V(0)
            // K(2) V(1) ... V(nblk - 1): a unit's fixed cost (its waits) and its copies
            // overlap those of the other warps' units.  A copy instruction moves 512
            // bytes; the next unit's slots are loaded while this one's rows are copied.
            constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows an instruction
            const int c = lane % kChunks, sub = lane / kChunks;
            const int64_t at = ((int64_t)g * D + c * 8) * 2, pitch = a.pool_stride * 2;
            const char *kp = reinterpret_cast<const char *>(a.k_pool) + at, *vp = reinterpret_cast<const char *>(a.v_pool) + at;
            const int last = 2 * nblk - 1, end = 2 * nblk * C::kUnits;
            // block of the sequence's group q, and whether it is its V
            auto block_of = [&](int q, bool &is_v) {
                is_v = q == last || (q > 0 && !(q & 1));
                return q == last ? nblk - 1 : is_v ? q / 2 - 1 : (q + 1) / 2;
            };
            auto fetch = [&](int n) {
                bool is_v;
                const int j = block_of(n / C::kUnits, is_v);
                return a.kv_indices[kv0 + min(c_begin + j * NB + 32 * (n % C::kUnits) + lane, c_end - 1)];  // past the end: a valid row again
            };
            int n = warp - kFirstLoad;
            int ahead = n < end ? fetch(n) : 0;
            for (; n < end; n += C::kLoadWarps) {
                int slot = ahead;
                if (slot < 0 || slot >= a.pool_rows) {
                    latch(a.err, DDT_DEVERR_KV_INDEX);
                    slot = 0;
                }
                if (n + C::kLoadWarps < end) ahead = fetch(n + C::kLoadWarps);
                bool is_v;
                const int j = block_of(n / C::kUnits, is_v);
                const int s = is_v ? j % C::kVStages : j % C::kKStages, u = is_v ? j / C::kVStages : j / C::kKStages;
                if (u > 0 && !warp_wait(bar((is_v ? C::bVEmpty : C::bKEmpty) + s), (u - 1) & 1, abort_flag, a.err)) break;
                const uint32_t to = sbase + (is_v ? C::kOffV : C::kOffK) + s * C::kBlockBytes + (c >> 3) * C::kBoxBytes +
                                    (n % C::kUnits) * 32 * 128;
                const char *pool = is_v ? vp : kp;
#pragma unroll
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int k = i * kPer + sub;
                    cp_async_16(to + k * 128 + (((c & 7) ^ (k & 7)) << 4), pool + __shfl_sync(0xffffffffu, slot, k) * pitch);
                }
                cp_async_arrive(bar((is_v ? C::bVFull : C::bKFull) + s));
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may land after the CTA has left
        } else {
            // ================= MMA =================
            if (elect_one()) {
                const uint64_t q0 = smem_desc(sbase + C::kOffQ, 16, 1024), k0 = smem_desc(sbase + C::kOffK, 16, 1024),
                               v0 = smem_desc(sbase + C::kOffV, C::kBoxBytes, 1024);  // + bytes >> 4
                bool ok = wait_or_abort(bar(C::bQFull), 0, abort_flag, a.err);
                // The tensor pipe is idle while this thread waits or computes: the loop is
                // unrolled over the two slots and keeps its stages and phases in counters.
                auto run = [&](auto tile_count) {
                    constexpr int A = decltype(tile_count)::value;  // tiles of the CTA
                    int ks = 0, vs = 0, w = 0;
                    uint32_t kph = 0, vph = 0, pph = 0;
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
                        const uint32_t p = tmem + C::kColS + NB * slot, d = tmem + C::kColO + D * t;
                        const uint32_t later = w >= A;  // the first block's product overwrites
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h) {
                            ok = wait_or_abort(bar(C::bPFull + C::kHalves * slot + h), pph, abort_flag, a.err);
                            if (!ok) return;
                            tc_fence_after();
#pragma unroll
                            for (int i = 4 * h; i < 4 * h + 4; ++i)
                                mma_ts(d, p + 8 * i, vd + i * (2048 >> 4), C::kIdescPV, i > 0 ? 1u : later);
                        }
                        if (A == 1) mma_commit(bar(C::bODone));
                        if (t == A - 1) {
                            mma_commit(bar(C::bVEmpty + vs));
                            if (++vs == C::kVStages) {
                                vs = 0;
                                vph ^= 1;
                            }
                        }
                    };
                    if (ok) issue_s(0);
                    if (ok && items > 1) issue_s(1);
                    while (ok && w < items) {
#pragma unroll
                        for (int slot = 0; slot < 2; ++slot) {
                            if (!ok || w >= items) break;
                            issue_pv(slot);
                            if (ok && w + 2 < items) issue_s(slot);
                            ++w;
                        }
                        pph ^= 1;
                    }
                };
                if constexpr (kTiles == 2) {
                    if (tiles == 2) run(std::integral_constant<int, 2>{});
                    else run(std::integral_constant<int, 1>{});
                } else {
                    run(std::integral_constant<int, 1>{});
                }
                // completes when every MMA issued has: the epilogue (and, after a timeout, the exit) waits for it
                mma_commit(bar(C::bOFin));
                mbar_wait(bar(C::bOFin), 0, kWaitLimit);
            }
            __syncwarp();
        }
    } else {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ================= softmax (thread = row = TMEM lane of its tile) =================
        const int t = warp >> 2, wq = warp & 3;
        const int r = 32 * wq + lane;  // row within the tile
        const int rows_t = rows - t * kRows;
        const bool warp_on = t < tiles && 32 * wq < rows_t;
        if (warp_on) {
            const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
            // ---- q rows of this warp into the swizzled operand layout ----
            {
                constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows per step
                const int c = lane % kChunks, sub = lane / kChunks;
                const uint32_t qb = sbase + C::kOffQ + t * C::kQBytes;
#pragma unroll 8
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int rt = 32 * wq + i * kPer + sub;
                    if (rt < rows_t) {
                        const int rr = row0 + t * kRows + rt;
                        const int node = rr / prm.group, hg = rr - node * prm.group;
                        const uint4 v = reinterpret_cast<const uint4 *>(
                            a.q + ((int64_t)(qo0 + node) * a.num_heads + g * prm.group + hg) * D)[c];
                        const uint32_t at = qb + (c >> 3) * C::kQBoxBytes + (rt >> 3) * 1024 + (rt & 7) * 128 +
                                            (((c & 7) ^ (rt & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                                     "r"(v.w)
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bQFull));
            }
            const bool row_on = r < rows_t;
            const int rr = row0 + t * kRows + (row_on ? r : 0);
            const int node = rr / prm.group, head = g * prm.group + rr - node * prm.group;
            const uint32_t *words = a.mask + m0 + (int64_t)node * W;
            const float sc = a.scale * kLog2e;
            float m_ref = -INFINITY, l = 0.f;
            constexpr int kW = NB / 32;
            auto mask_words = [&](int j, uint32_t (&mw)[kW]) {
#pragma unroll
                for (int k = 0; k < kW; ++k) {
                    const int c0 = c_begin + j * NB + 32 * k;
                    uint32_t x = c0 < c_end ? words[c0 >> 5] : 0u;
                    if (c0 < c_end && c_end - c0 < 32) x &= (1u << (c_end - c0)) - 1u;
                    mw[k] = x;
                }
            };
            uint32_t mw[kW], mnext[kW];
            mask_words(0, mnext);
            bool ok = true;
            for (int j = 0; j < nblk; ++j) {
                const int w = j * tiles + t, slot = w & 1;
                const uint32_t col = tmem + lane_off + C::kColS + NB * slot;
#pragma unroll
                for (int k = 0; k < kW; ++k) mw[k] = mnext[k];
                if (j + 1 < nblk) mask_words(j + 1, mnext);
                ok = warp_wait(bar(C::bSFull + slot), (w >> 1) & 1, abort_flag, a.err);
                if (!ok) break;
                tc_fence_after();
                uint32_t all = mw[0];
#pragma unroll
                for (int k = 1; k < kW; ++k) all &= mw[k];
                float sv[NB];
                {
                    uint32_t t32[kW][32];
#pragma unroll
                    for (int k = 0; k < kW; ++k) tmem_ld32(col + 32 * k, t32[k]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < NB; ++k) sv[k] = __uint_as_float(t32[k >> 5][k & 31]);
                }
                if (all != 0xffffffffu) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) sv[k] = ((mw[k >> 5] >> (k & 31)) & 1u) ? sv[k] : -INFINITY;
                }
                float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                for (int k = 4; k < NB; k += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = k + 4 + e < NB ? fmaxf(fmaxf(mx[e], sv[k + e]), sv[k + 4 + e]) : fmaxf(mx[e], sv[k + e]);
                }
                const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                float alpha = 1.0f;
                if (mb > m_ref + kRescaleLog2) {  // also the first visible block (m_ref = -inf)
                    alpha = ex2(m_ref - mb);
                    l *= alpha;
                    m_ref = mb;
                }
                // The output so far shrinks before PV(w).  With two tiles S(w) was issued behind
                // this tile's last PV, so that is done; with one it has to be waited for.
                if (j > 0 && __any_sync(0xffffffffu, row_on && alpha != 1.0f)) {
                    if (tiles == 1 && !warp_wait(bar(C::bODone), (j - 1) & 1, abort_flag, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t oc = tmem + lane_off + C::kColO + D * t;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t t32[32];
                        tmem_ld32(oc + 32 * q, t32);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) t32[e] = __float_as_uint(__uint_as_float(t32[e]) * alpha);
                        tmem_st32(oc + 32 * q, t32);
                    }
                }
                const float mref = m_ref == -INFINITY ? 0.f : m_ref;  // nothing seen yet: every p is 0
                const float2 scv = make_float2(sc, sc), nmv = make_float2(-mref, -mref);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < NB / 64; ++h) {
                    uint32_t pw[32];
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        const float2 x = f2fma(make_float2(sv[64 * h + k], sv[64 * h + k + 1]), scv, nmv);
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        acc = f2add(acc, make_float2(p0, p1));
                        pw[k / 2] = pack_bf16(p0, p1);
                    }
                    tmem_st32(col + 32 * h, pw);  // over scores that have been read
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::bPFull + C::kHalves * slot + h));
                }
                l += acc.x + acc.y;
            }
            // ---- epilogue ----
            ok = ok && warp_wait(bar(C::bOFin), 0, abort_flag, a.err) && *abort_flag == 0;
            if (__all_sync(0xffffffffu, ok)) {
                tc_fence_after();
                const int64_t row = (int64_t)(qo0 + node) * a.num_heads + head;
                const int64_t all_rows = (int64_t)a.total_q * a.num_heads;
                const bool part = a.num_splits > 1;
                float *op = part ? a.o_part + ((int64_t)split * all_rows + row) * D : nullptr;
                uint16_t *ob = a.out + row * D;
                const float inv = 1.f / l;
                const bool none = l == 0.f;
                bool finite = true;
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t t32[32];
                    tmem_ld32(tmem + lane_off + C::kColO + D * t + 32 * q, t32);
                    tmem_wait_ld();
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        finite = finite && (t32[e] & 0x7f800000u) != 0x7f800000u;
                        o[e] = none ? 0.f : __uint_as_float(t32[e]) * inv;
                    }
                    if (row_on && part) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<float4 *>(op)[8 * q + e] =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else if (row_on) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(ob)[4 * q + e] =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                }
                if (row_on) {
                    const float lse = none ? -INFINITY : (m_ref + log2f(l)) * kLn2;
                    if (part) a.lse_part[(int64_t)split * all_rows + row] = lse;
                    else if (a.lse) a.lse[row] = lse;
                }
                // rows that something unseen may have reached (a NaN sum stays one whatever V holds)
                uint32_t again = __ballot_sync(0xffffffffu, row_on && !finite && l > 0.f);
                while (again) {
                    const int from = __ffs(again) - 1;
                    again &= again - 1;
                    const int n2 = __shfl_sync(0xffffffffu, node, from);
                    const int64_t row2 = __shfl_sync(0xffffffffu, (long long)row, from);
                    const float m2 = __shfl_sync(0xffffffffu, m_ref, from), inv2 = __shfl_sync(0xffffffffu, inv, from);
                    float o[D / 32];
                    row_again<D>(a, a.q + row2 * D, a.mask + m0 + (int64_t)n2 * W, kv0, c_begin, c_end, g, m2, o);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const float x = o[e] * inv2;
                        if (part) {
                            a.o_part[((int64_t)split * all_rows + row2) * D + lane * (D / 32) + e] = x;
                        } else {
                            const __nv_bfloat16 y = __float2bfloat16_rn(x);
                            a.out[row2 * D + lane * (D / 32) + e] = *reinterpret_cast<const uint16_t *>(&y);
                        }
                    }
                }
            }
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

// out = sum_s e^{lse_s - LSE} o_s over the splits that the row's request has
// (columns [s * split_cols, ...) below its length), LSE = log sum_s e^{lse_s}.
// One warp per (token, head) row: lane s, s + 32, ... holds split s's weight,
// then the lanes sum D / 32 values each.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) gqa_combine_kernel(const GqaArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x, h = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (h >= a.num_heads) return;
    const int b = find_request(a.qo_indptr, a.batch, t, lane);
    if (b >= a.batch) return;
    const int qo0 = a.qo_indptr[b], T = a.qo_indptr[b + 1] - qo0;
    const int kv0 = a.kv_indptr[b], N = a.kv_indptr[b + 1] - kv0;
    const int m0 = a.mask_indptr[b], m1 = a.mask_indptr[b + 1];
    // a request that the attention refused has no partial results
    if (T < 1 || T > a.max_q_len || qo0 < 0 || qo0 + T > a.total_q || t - qo0 >= T || N < T || N > a.max_kv_len || kv0 < 0 ||
        kv0 + N > a.total_kv || m0 < 0 || m1 - m0 != T * ((N + 31) >> 5) || m1 > a.total_mask_words)
        return;
    const int splits = min(a.num_splits, (N + a.split_cols - 1) / a.split_cols);
    const int64_t rows = (int64_t)a.total_q * a.num_heads, row = (int64_t)t * a.num_heads + h;
    constexpr int kL = DDT_MAX_SPLITS / 32;
    float ls[kL], m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kL; ++k) {
        const int s = lane + 32 * k;
        ls[k] = s < splits ? a.lse_part[(int64_t)s * rows + row] : -INFINITY;
        m = fmaxf(m, ls[k]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < kL; ++k) {
        ls[k] = ls[k] == -INFINITY ? 0.f : ex2((ls[k] - m) * kLog2e);  // now the split's weight (NaN stays)
        den += ls[k];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kL; ++k) {
        const int left = min(32, splits - 32 * k);
#pragma unroll 4
        for (int s = 0; s < left; ++s) {
            const float wgt = __shfl_sync(0xffffffffu, ls[k], s);
            const float *o = a.o_part + ((int64_t)(32 * k + s) * rows + row) * D + lane * E;
            float v[E];
            if constexpr (E == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(o);
                v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(o);
                v[0] = x.x; v[1] = x.y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wgt, v[e], acc[e]);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) w[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint16_t *dst = a.out + row * D + lane * E;
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(dst) = w[0];
    if (a.lse && lane == 0) a.lse[row] = den == 0.f ? -INFINITY : m + log2f(den) * kLn2;
}

int tiles_per_cta(int max_q_len, int group) { return max_q_len * group > kRows ? 2 : 1; }

template <int D, int kTiles>
cudaError_t launch_partial(const GqaParams &prm, cudaStream_t s) {
    const GqaArgs &a = prm.a;
    const int groups = (a.max_q_len * prm.group + kTiles * kRows - 1) / (kTiles * kRows);
    const dim3 grid((unsigned)(groups * a.num_kv_heads), (unsigned)a.num_splits, (unsigned)a.batch);
    return launch_pdl(gqa_attn_kernel<D, kTiles>, grid, dim3(Cfg<D, kTiles>::kThreads), Cfg<D, kTiles>::kSmemBytes, s, prm);
}

template <int D, int kTiles>
cudaError_t prepare() {
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

int gqa_choose_splits(int batch, int num_heads, int num_kv_heads, int max_q_len, int max_kv_len, int num_sms,
                      int max_splits) {
    const int group = num_heads / num_kv_heads;
    const int tiles = tiles_per_cta(max_q_len, group);
    const long long ctas = (long long)batch * num_kv_heads * ((max_q_len * group + tiles * kRows - 1) / (tiles * kRows));
    const long long slots = (long long)num_sms * (tiles == 2 ? 1 : 2);
    const long long units = ((long long)max_kv_len + kSplitUnit - 1) / kSplitUnit;
    long long want = (2 * slots + ctas - 1) / ctas;
    if (want > (units + 1) / 2) want = (units + 1) / 2;
    if (want > max_splits) want = max_splits;
    return want < 1 ? 1 : (int)want;
}

void gqa_split_layout(int max_kv_len, int requested, int *split_cols, int *splits) {
    const int64_t want = requested < 1 ? 1 : requested;
    int64_t cols = (max_kv_len + want - 1) / want;
    cols = (cols + kSplitUnit - 1) / kSplitUnit * kSplitUnit;
    *splits = (int)((max_kv_len + cols - 1) / cols);
    *split_cols = *splits <= 1 ? max_kv_len : (int)cols;
    if (*splits < 1) *splits = 1;
}

cudaError_t launch_gqa_attn(const GqaArgs &a, cudaStream_t s) {
    GqaParams prm;
    prm.a = a;
    prm.group = a.num_heads / a.num_kv_heads;
    const int tiles = tiles_per_cta(a.max_q_len, prm.group);
    cudaError_t e = a.head_dim == 128 ? (tiles == 2 ? launch_partial<128, 2>(prm, s) : launch_partial<128, 1>(prm, s))
                                      : (tiles == 2 ? launch_partial<64, 2>(prm, s) : launch_partial<64, 1>(prm, s));
    if (e == cudaSuccess && a.num_splits > 1) {
        const dim3 grid((unsigned)a.total_q, (unsigned)((a.num_heads + kCombineWarps - 1) / kCombineWarps));
        e = a.head_dim == 128 ? launch_pdl(gqa_combine_kernel<128>, grid, dim3(32 * kCombineWarps), 0, s, a)
                              : launch_pdl(gqa_combine_kernel<64>, grid, dim3(32 * kCombineWarps), 0, s, a);
    }
    return e;
}

}  // namespace ddt
