// ddt_cache.cu -- rows of the cache in every layer's pool at once: copies,
// the commit of accepted nodes, and compaction.
//
// All three move whole rows, 16 bytes a thread and several loads in flight
// before the first store, and are bound by memory: a copy of 16384 rows of 2 KB
// in 32 pools (2.1 GB read and written) takes 312 us, 6.9 TB/s; the commit of 64
// requests' paths in 64 pools of 2 KB rows 7.1 us; the compaction of 16 pools of
// 65536 rows of 2 KB, half of them named (1.1 GB), 169 us, 6.4 TB/s.  None of the kernels
// announces its end early: the calls that may follow (ddt_verify_attn among
// them) read pool rows before they wait for the previous kernel, so these
// have to be complete when the next one starts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ddt_internal.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // 16-byte pieces in flight per thread
constexpr int kChunkBytes = kThreads * kUnroll * 16;

// rows of one CTA's chunk: about kChunkBytes, at least one row
inline int chunk_rows(int64_t row_bytes) { return row_bytes >= kChunkBytes ? 1 : (int)(kChunkBytes / row_bytes); }

// Pieces of `rows` rows: row k goes from src + from(k) * vecs to dst + to(k) *
// vecs; a pair that is none skips the row.
template <typename Pair>
__device__ __forceinline__ void move_rows(const uint4 *src, uint4 *dst, uint32_t rows, uint32_t vecs, Pair pair) {
    const uint64_t pieces = (uint64_t)rows * vecs;
    for (uint64_t e0 = threadIdx.x; e0 < pieces; e0 += kThreads * kUnroll) {
        uint4 v[kUnroll];
        int64_t to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t e = e0 + u * kThreads;
            to[u] = -1;
            if (e < pieces) {
                const uint32_t k = rows == 1 ? 0u : (uint32_t)e / vecs;  // a chunk of several rows is small
                const int64_t c = (int64_t)(e - (uint64_t)k * vecs);
                int64_t from, dest;
                if (pair(k, from, dest)) {
                    v[u] = src[from * vecs + c];
                    to[u] = dest * vecs + c;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] >= 0) dst[to[u]] = v[u];
    }
}

// ---------------------------------------------------------------- copy
__global__ void __launch_bounds__(kThreads)
cache_copy_kernel(const uint8_t *src_slab, int64_t src_pool_bytes, int64_t src_rows, uint8_t *dst_slab,
                  int64_t dst_pool_bytes, int64_t dst_rows, int num_pools, uint32_t vecs, int rows_per_cta,
                  const int32_t *src, const int32_t *dst, int n, unsigned int *err) {
    pdl_wait();
    const int64_t i0 = (int64_t)blockIdx.x * rows_per_cta;
    const uint32_t rows = (uint32_t)min((int64_t)rows_per_cta, n - i0);
    for (int p = blockIdx.y; p < num_pools; p += gridDim.y)
        move_rows(reinterpret_cast<const uint4 *>(src_slab + p * src_pool_bytes),
                  reinterpret_cast<uint4 *>(dst_slab + p * dst_pool_bytes), rows, vecs,
                  [&](uint32_t k, int64_t &from, int64_t &to) {
                      from = src[i0 + k];
                      to = dst[i0 + k];
                      const bool ok = from >= 0 && from < src_rows && to >= 0 && to < dst_rows;
                      if (!ok) latch(err, DDT_DEVERR_KV_INDEX);
                      return ok;
                  });
}

// ---------------------------------------------------------------- commit
// One thread owns one 16-byte column of the request's rows: it reads the
// column of all accepted rows, then writes it, so a row that is both source
// and destination moves its value from before the call without any exchange
// between threads.
constexpr int kCommitThreads = 128;
constexpr int kPath = DDT_MAX_DEPTH + 1;

__global__ void __launch_bounds__(kCommitThreads)
cache_commit_kernel(uint8_t *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools, uint32_t vecs,
                    const int32_t *kv_indices, const int32_t *kv_indptr, const int32_t *qo_indptr,
                    const int32_t *accept_len, const int32_t *accepted_nodes, int total_kv, int max_depth,
                    int32_t *new_len, unsigned int *err) {
    __shared__ int64_t s_src[kPath], s_dst[kPath];
    __shared__ int s_n;
    const int b = blockIdx.z;
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;  // the CTA that reports
    pdl_wait();
    if (threadIdx.x < 32) {  // lane k checks and resolves path entry k
        const int lane = threadIdx.x;
        const unsigned full = 0xffffffffu;
        const int width = max_depth + 1;
        const int64_t T = (int64_t)qo_indptr[b + 1] - qo_indptr[b];  // broken offsets do not fit 32 bits
        const int64_t kv0 = kv_indptr[b], kv1 = kv_indptr[b + 1];
        const int n = accept_len[b];
        const int ak = lane < width ? accepted_nodes[(int64_t)b * width + lane] : 0;
        const int aprev = __shfl_up_sync(full, ak, 1);
        const int64_t P = kv1 - kv0 - T;
        const bool bad_entry = lane < n && (lane == 0 ? ak != 0 : (ak <= aprev || ak >= T));
        bool ok = T >= 0 && P >= 0 && kv0 >= 0 && kv1 <= total_kv && n <= width && n <= T && n >= (T > 0 ? 1 : 0) &&
                  !__any_sync(full, bad_entry);
        unsigned int bit = DDT_DEVERR_ACCEPTED;
        int64_t sr = 0, dr = 0;
        if (ok && lane < n) {
            sr = kv_indices[kv0 + P + ak];
            dr = kv_indices[kv0 + P + lane];
        }
        const bool bad_row = ok && lane < n && (sr < 0 || sr >= pool_rows || dr < 0 || dr >= pool_rows);
        if (__any_sync(full, bad_row)) {
            bit = DDT_DEVERR_KV_INDEX;
            ok = false;
        }
        if (lane < kPath) {
            s_src[lane] = sr;
            s_dst[lane] = dr;
        }
        if (lane == 0) {
            s_n = ok ? n : 0;
            if (first && !ok) latch(err, bit);
            if (first && ok && new_len) new_len[b] = (int32_t)(P + n);
        }
    }
    __syncthreads();
    const int n = s_n;
    int64_t from[kPath], to[kPath];
#pragma unroll
    for (int k = 0; k < kPath; ++k) {
        const bool moves = k < n && s_src[k] != s_dst[k];
        from[k] = moves ? s_src[k] * vecs : -1;
        to[k] = s_dst[k] * vecs;
    }
    for (int p = blockIdx.y; p < num_pools; p += gridDim.y) {
        uint4 *pool = reinterpret_cast<uint4 *>(slab + p * pool_bytes);
        for (uint32_t c = blockIdx.x * kCommitThreads + threadIdx.x; c < vecs; c += gridDim.x * kCommitThreads) {
            uint4 v[kPath];
#pragma unroll
            for (int k = 0; k < kPath; ++k)
                if (from[k] >= 0) v[k] = pool[from[k] + c];
#pragma unroll
            for (int k = 0; k < kPath; ++k)
                if (from[k] >= 0) pool[to[k] + c] = v[k];
        }
    }
}

// ---------------------------------------------------------------- compact
// Workspace: a header, one bit per row (named or not), the number of named
// rows before each word of bits, and the two lists of the move, both
// ascending: hole k takes the row of mover k.
constexpr int kPlanThreads = 1024;
constexpr int kAloneSlots = 32768;
struct CompactHeader {
    int32_t live;    // n: named rows
    int32_t below;   // named rows below row n: they stay
    int32_t moves;   // holes below n = named rows at or above n
};
struct CompactWs {
    CompactHeader *head;
    uint32_t *bits;
    uint32_t *before;
    int32_t *holes;
    int32_t *movers;
};
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline size_t compact_layout(int64_t rows, void *base, CompactWs *w) {
    const size_t words = (size_t)((rows + 31) / 32), half = (size_t)(rows / 2 + 1);
    uint8_t *p = static_cast<uint8_t *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return at;
    };
    const size_t head = take(sizeof(CompactHeader)), bits = take(words * 4), before = take(words * 4),
                 holes = take(half * 4), movers = take(half * 4);
    if (w) {
        w->head = reinterpret_cast<CompactHeader *>(p + head);
        w->bits = reinterpret_cast<uint32_t *>(p + bits);
        w->before = reinterpret_cast<uint32_t *>(p + before);
        w->holes = reinterpret_cast<int32_t *>(p + holes);
        w->movers = reinterpret_cast<int32_t *>(p + movers);
    }
    return off;
}

__global__ void __launch_bounds__(kThreads)
compact_mark_kernel(const int32_t *indices, int total, int64_t pool_rows, uint32_t *bits, unsigned int *err) {
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const int r = indices[i];
    if (r < 0 || r >= pool_rows) {
        latch(err, DDT_DEVERR_KV_INDEX);
        return;
    }
    atomicOr(&bits[r >> 5], 1u << (r & 31));
}

__device__ __forceinline__ uint32_t block_sum(uint32_t x, uint32_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if (lane == 0) scratch[warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, scratch[lane]);
}

// CTA c plans words [1024 c, 1024 c + 1024), one per thread.  Every CTA counts
// all the bits itself (n has to be known before a row can be called a hole or
// a mover): the bits of a pool of 65536 rows are 8 KB, so that costs less than
// another launch or an exchange between CTAs.  It grows with the square of the pool: half
// of the rows named, rows of 16 bytes, the call takes 14 us for 2^16 rows, 22 us for 2^20, 58 us for
// 2^22 and 316 us for 2^24.
// kAlone: one CTA has all the words and marks them itself, in shared memory, in
// place of the two launches before (the clearing and the marking).
template <bool kAlone>
__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(CompactWs w, int words, int32_t *live_out, const int32_t *indices, int total, int64_t pool_rows,
                    unsigned int *err) {
    __shared__ uint32_t scratch[32], warp_sum[32], s_bits[kAlone ? kPlanThreads : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * kPlanThreads;
    pdl_wait();
    if (kAlone) {
        s_bits[tid] = 0;
        __syncthreads();
        for (int i = tid; i < total; i += kPlanThreads) {
            const int r = indices[i];
            if (r < 0 || r >= pool_rows) latch(err, DDT_DEVERR_KV_INDEX);
            else atomicOr(&s_bits[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        if (tid < words) w.bits[tid] = s_bits[tid];
    }
    const uint32_t *bits = kAlone ? s_bits : w.bits;
    uint32_t all = 0, ahead = 0;
    for (int i = tid; i < words; i += kPlanThreads) {
        const uint32_t c = __popc(bits[i]);
        all += c;
        if (i < first) ahead += c;
    }
    const int n = (int)block_sum(all, scratch);
    ahead = block_sum(ahead, scratch);
    uint32_t stay = 0;  // named rows below n
    for (int i = tid; i < words && i <= (n >> 5); i += kPlanThreads) {
        const uint32_t x = bits[i];
        stay += __popc(i < (n >> 5) ? x : x & ((1u << (n & 31)) - 1u));
    }
    stay = block_sum(stay, scratch);
    // named rows before this thread's word
    const int i = first + tid;
    const uint32_t x = i < words ? bits[i] : 0u;
    uint32_t sum = __popc(x);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    uint32_t before = ahead + sum - __popc(x);
    for (int k = 0; k < warp; ++k) before += warp_sum[k];
    if (i < words) w.before[i] = before;
    // The words' unnamed rows below n, and their named ones from n on, are consecutive
    // places of the lists: a warp writes its 32 words' one after another, a lane per row
    // (16000 slots of 32768 rows 13.0 us; a thread per word, its rows in turn, 17.9 us;
    // with a test that skips words without either 14.5 us).
    for (int k = 0; k < 32 && i - lane + k < words; ++k) {
        const uint32_t xk = __shfl_sync(0xffffffffu, x, k);
        const int base = 32 * (i - lane + k), ahead_k = (int)__shfl_sync(0xffffffffu, before, k);
        const int low = min(32, max(0, n - base));  // the word's rows below n
        const uint32_t lower = (1u << lane) - 1u;
        const bool named = (xk >> lane) & 1u;
        if (!named && lane < low) w.holes[base - ahead_k + __popc(~xk & lower)] = base + lane;
        if (named && lane >= low) w.movers[ahead_k + __popc(xk & lower) - (int)stay] = base + lane;
    }
    if (blockIdx.x == 0 && tid == 0) {
        w.head->live = n;
        w.head->below = (int32_t)stay;
        w.head->moves = n - (int32_t)stay;
        *live_out = n;
    }
}

// The slots first (a share for every CTA), then chunks of movers in every pool:
// the number of movers is known on the device only, so the CTAs stride over them.
__global__ void __launch_bounds__(kThreads)
compact_move_kernel(CompactWs w, uint8_t *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools,
                    uint32_t vecs, int rows_per_cta, const int32_t *indices, int total, int32_t *new_indices) {
    pdl_wait();
    const int n = w.head->live, stay = w.head->below, moves = w.head->moves;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int r = indices[i];
        int to = r;
        if (r >= n && r < pool_rows) {
            const uint32_t below = w.bits[r >> 5] & ((1u << (r & 31)) - 1u);
            to = w.holes[w.before[r >> 5] + __popc(below) - stay];
        }
        new_indices[i] = to;
    }
    const int chunks = (moves + rows_per_cta - 1) / rows_per_cta;
    for (int64_t u = blockIdx.x; u < (int64_t)chunks * num_pools; u += gridDim.x) {
        const int chunk = (int)(u / num_pools), p = (int)(u - (int64_t)chunk * num_pools), k0 = chunk * rows_per_cta;
        uint4 *pool = reinterpret_cast<uint4 *>(slab + p * pool_bytes);
        move_rows(pool, pool, (uint32_t)min(rows_per_cta, moves - k0), vecs,
                  [&](uint32_t k, int64_t &from, int64_t &to) {
                      from = w.movers[k0 + k];
                      to = w.holes[k0 + k];
                      return true;
                  });
    }
}

}  // namespace

cudaError_t launch_cache_copy(const void *src_slab, int64_t src_pool_bytes, int64_t src_rows, void *dst_slab,
                              int64_t dst_pool_bytes, int64_t dst_rows, int num_pools, int64_t row_bytes,
                              const int32_t *src, const int32_t *dst, int n, unsigned int *err, cudaStream_t s) {
    const int per = chunk_rows(row_bytes);
    const dim3 grid((unsigned)((n + per - 1LL) / per), (unsigned)(num_pools < 65535 ? num_pools : 65535));
    return launch_pdl(cache_copy_kernel, grid, dim3(kThreads), 0, s, static_cast<const uint8_t *>(src_slab),
                      src_pool_bytes, src_rows, static_cast<uint8_t *>(dst_slab), dst_pool_bytes, dst_rows, num_pools,
                      (uint32_t)(row_bytes / 16), per, src, dst, n, err);
}

cudaError_t launch_cache_commit(void *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools, int64_t row_bytes,
                                const int32_t *kv_indices, const int32_t *kv_indptr, const int32_t *qo_indptr,
                                const int32_t *accept_len, const int32_t *accepted_nodes, int batch, int total_kv,
                                int max_depth, int32_t *new_len, int num_sms, unsigned int *err, cudaStream_t s) {
    const uint32_t vecs = (uint32_t)(row_bytes / 16);
    const unsigned cols = (vecs + kCommitThreads - 1) / kCommitThreads;
    // A CTA resolves its request's path once and walks the pools: as many CTAs
    // per request as fill the SMs (16 CTAs of 128 threads each).
    int64_t per = (16LL * num_sms + (int64_t)batch * cols - 1) / ((int64_t)batch * cols);
    if (per > num_pools) per = num_pools;
    for (int b0 = 0; b0 < batch; b0 += 65535) {
        const int nb = batch - b0 < 65535 ? batch - b0 : 65535;
        const dim3 grid(cols < 1024 ? cols : 1024, (unsigned)(per < 65535 ? per : 65535), (unsigned)nb);
        const cudaError_t e = launch_pdl(
            cache_commit_kernel, grid, dim3(kCommitThreads), 0, s, static_cast<uint8_t *>(slab), pool_bytes, pool_rows,
            num_pools, vecs, kv_indices, kv_indptr + b0, qo_indptr + b0, accept_len + b0,
            accepted_nodes + (int64_t)b0 * (max_depth + 1), total_kv, max_depth, new_len ? new_len + b0 : nullptr, err);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

size_t cache_compact_workspace(int64_t pool_rows) { return compact_layout(pool_rows, nullptr, nullptr); }

cudaError_t launch_cache_compact(void *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools, int64_t row_bytes,
                                 const int32_t *kv_indices, int total, int32_t *new_indices, int32_t *live,
                                 void *workspace, int num_sms, unsigned int *err, cudaStream_t s) {
    CompactWs w;
    compact_layout(pool_rows, workspace, &w);
    const int words = (int)((pool_rows + 31) / 32);
    // One CTA plans a small pool alone, two launches less: 1500 slots of 4096 rows 6.8 us
    // against 10.4 us, 32000 of 32768 14.8 us against 16.5 us.
    const bool alone = words <= kPlanThreads && total <= kAloneSlots;
    cudaError_t e = alone ? cudaSuccess : cudaMemsetAsync(w.bits, 0, (size_t)words * 4, s);
    if (e == cudaSuccess && total > 0 && !alone)
        e = launch_pdl(compact_mark_kernel, dim3((unsigned)((total + kThreads - 1LL) / kThreads)), dim3(kThreads), 0, s,
                       kv_indices, total, pool_rows, w.bits, err);
    if (e == cudaSuccess)
        e = launch_pdl(alone ? compact_plan_kernel<true> : compact_plan_kernel<false>,
                       dim3((unsigned)((words + kPlanThreads - 1) / kPlanThreads)), dim3(kPlanThreads), 0, s, w, words,
                       live, kv_indices, total, pool_rows, err);
    // A CTA's steps do not overlap, so many CTAs with a few steps each: 1 GB of moves
    // took 169 us with 64 CTAs per SM, 10 us more with the 8 that fit at once.  No more
    // than the most steps there can be (half of the rows move at most).
    const int per = chunk_rows(row_bytes);
    const int64_t most_moves = total < pool_rows / 2 ? total : pool_rows / 2;
    int64_t ctas = (most_moves + per - 1) / per * num_pools, slots = (total + kThreads - 1LL) / kThreads;
    if (ctas < slots) ctas = slots;
    if (ctas > 64LL * num_sms) ctas = 64LL * num_sms;
    if (ctas < 1) ctas = 1;
    if (e == cudaSuccess)
        e = launch_pdl(compact_move_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, s, w, static_cast<uint8_t *>(slab),
                       pool_bytes, pool_rows, num_pools, (uint32_t)(row_bytes / 16), per, kv_indices, total, new_indices);
    return e;
}

}  // namespace ddt
