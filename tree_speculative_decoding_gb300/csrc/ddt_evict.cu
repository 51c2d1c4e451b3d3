// ddt_evict.cu -- a cache cut down to the columns that received most.
//
// Request b keeps min(N_b, budget_b) of its columns: in the order of their keys (the
// first `sinks` and the last `recent` columns and +inf on top, NaN with -inf at the
// bottom), ties to the lower column.  What stays keeps its order.
//
// A request has a cluster of CTAs, each with an equal run of its columns, whose weights it
// keeps as ordered 32-bit keys in shared memory (and reads again where they are written).  The smallest key that stays is
// found by its bytes, highest first: a histogram of the keys that agree so far, summed over
// the cluster through distributed shared memory, and the byte at which the count reaches what
// is to stay.  Columns above that key stay, and of those with the key as many of the first
// ones as are left.  A count of both per warp, scanned over the CTA and the cluster, then gives
// every column its place.  Nothing depends on the order of atomics (they count).
//
// Measured back to back: 4097 columns 8.4 us, 64 requests of 1024..16384 15 us, 8 of 131072 24 us.
// Bound by latency: a launch, one pass over 4 bytes a column, up to four histograms with a cluster
// barrier each, one pass over 8 bytes a column that writes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace {

using namespace sm100;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kAhead = 4;            // loads in flight of a thread
constexpr int kMostKeys = 45056;     // of a CTA in shared memory; further ones are read again
// A cluster grows up to 8 CTAs to keep a CTA's columns below.  (Of 16 the SMs that share a cluster hold one at a
// time: 8 requests of 131072 take 37 us, with 8 CTAs 25.)
constexpr int kColumnsOfCta = 8192;
constexpr uint32_t kTop = 0xff800000u;  // key of +inf
constexpr uint32_t kAll = 0xffffffffu;

struct EvictParams {
    EvictArgs a;
    int cluster;  // CTAs of a request
    int keys;     // of a CTA, in shared memory
};

// Floats as integers of the same order: -0 is 0, NaN is -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x != x ? -INFINITY : x);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t remote_u32(uint32_t local, uint32_t cta) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(local, cta)) : "memory");
    return v;
}
// columns of request b, or -1 where its offsets are broken
__device__ __forceinline__ int columns_of(const EvictArgs &a, int b) {
    const int kv0 = a.kv_indptr[b], kv1 = a.kv_indptr[b + 1];
    const int n = (int)((uint32_t)kv1 - (uint32_t)kv0);
    return kv0 < 0 || kv1 < kv0 || kv1 > a.total_kv || n > a.max_kv_len ? -1 : n;
}

__global__ void __launch_bounds__(kThreads, 1) evict_kernel(const __grid_constant__ EvictParams prm) {
    const EvictArgs &a = prm.a;
    extern __shared__ uint32_t keys[];
    __shared__ uint4 copies[256];  // a histogram, four counts for each byte
    __shared__ uint32_t counts[4][256], sums[256];
    __shared__ uint32_t above[kWarps], equal[kWarps], totals[2], found[3], before[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = prm.cluster, b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    auto sync_all = [&]() {  // and what the cluster's CTAs wrote is seen
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    if (tid < 256) copies[tid] = make_uint4(0, 0, 0, 0);
    if (tid < 2) before[tid] = 0;
    pdl_wait();
    pdl_trigger();

    // ---- the request, and its columns' keys ----
    const int checked = columns_of(a, b), N = max(checked, 0);
    if (checked < 0 && rank == 0 && tid == 0) latch(a.err, DDT_DEVERR_KV_INDPTR);
    const int kept = min(N, max(a.budget[b], 0)), kv0 = a.kv_indptr[b];
    const int per = (int)((((int64_t)N + cluster - 1) / cluster + 31) & ~31);
    const int c0 = (int)min((int64_t)N, (int64_t)rank * per), n = min(per, N - c0);  // the CTA's columns
    const float *w = a.weights + kv0 + c0;
    const int recent_from = N - min(a.recent, N);
    auto make_key = [&](int i) {
        const int j = c0 + i;
        return j < a.sinks || j >= recent_from ? kTop : key_of(w[i]);
    };
    auto key = [&](int i) { return i < prm.keys ? keys[i] : make_key(i); };
    const int here = min(n, prm.keys);
    for (int i0 = tid; i0 < here; i0 += kAhead * kThreads) {
        uint32_t k[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) k[e] = i0 + e * kThreads < here ? make_key(i0 + e * kThreads) : 0u;
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            if (i0 + e * kThreads < here) keys[i0 + e * kThreads] = k[e];
    }
    __syncthreads();
    // what the requests before this one keep, and leave (sums of broken offsets may wrap: every place is checked)
    uint32_t stay = 0, go = 0;
    for (int i = tid; i < b; i += kThreads) {
        const int m = max(columns_of(a, i), 0), k = min(m, max(a.budget[i], 0));
        stay += k;
        go += m - k;
    }
    if (b > 32 * warp) {
        stay = __reduce_add_sync(kAll, stay);
        go = __reduce_add_sync(kAll, go);
        if (lane == 0) {
            atomicAdd(&before[0], stay);
            atomicAdd(&before[1], go);
        }
    }

    // ---- the smallest key that stays, and how many columns that have it do ----
    uint32_t prefix = 0, mask = 0, left = kept;
    if (kept == N || kept == 0) {
        prefix = kept ? 0u : kAll;  // below and above every key
        left = 0;
    } else {
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix) atomicAdd(&reinterpret_cast<uint32_t *>(copies)[((k >> shift) & 255u) * 4 + (lane & 3)], 1u);
            }
            __syncthreads();
            if (cluster > 1) {
                if (tid < 256) {
                    const uint4 v = copies[tid];
                    counts[pass][tid] = (v.x + v.y) + (v.z + v.w);
                }
                cluster_sync();
                uint32_t v[2];  // thread (byte, q) adds those of CTAs q and q + 4
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int from = (tid >> 8) + 4 * r;
                    v[r] = from < cluster ? remote_u32(smem_u32(&counts[pass][tid & 255]), from) : 0u;
                }
                reinterpret_cast<uint32_t *>(copies)[(tid & 255) * 4 + (tid >> 8)] = v[0] + v[1];
                __syncthreads();
            }
            if (warp < 8) {
                const uint4 v = copies[tid];
                sums[255 - tid] = (v.x + v.y) + (v.z + v.w);  // the highest byte first
                copies[tid] = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
            if (warp == 0) {  // lane l has the bytes 255 - 8 l and the 7 below
                const uint4 lo = reinterpret_cast<const uint4 *>(sums)[2 * lane], hi = reinterpret_cast<const uint4 *>(sums)[2 * lane + 1];
                const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                uint32_t mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine += v[i];
                uint32_t upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(kAll, upto, o);
                    if (lane >= o) upto += x;
                }
                if (upto >= left && upto - mine < left) {
                    uint32_t sum = upto - mine;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (sum < left && sum + v[e] >= left) {
                            found[0] = 255 - 8 * lane - e;
                            found[1] = left - sum;
                            found[2] = v[e] == left - sum;
                        }
                        sum += v[e];
                    }
                }
            }
            __syncthreads();
            prefix |= found[0] << shift;
            mask |= 255u << shift;
            left = found[1];
            if (found[2]) {  // all that agree so far stay: nothing is left to find
                prefix -= 1;
                left = 0;
                break;
            }
        }
    }

    // ---- places ----
    // a warp has a run of the CTA's columns, which it goes through in order
    const int run = ((n + kWarps - 1) / kWarps + 31) & ~31, r0 = min(n, warp * run), r1 = min(n, r0 + run);
    uint32_t up = 0, same = 0;
    for (int i = r0 + lane; i < r1; i += 32) {
        const uint32_t k = key(i);
        up += k > prefix;
        same += k == prefix;
    }
    up = __reduce_add_sync(kAll, up);
    same = __reduce_add_sync(kAll, same);
    if (lane == 0) {
        above[warp] = up;
        equal[warp] = same;
    }
    __syncthreads();
    uint32_t up_before = __reduce_add_sync(kAll, lane < warp ? above[lane] : 0u);
    uint32_t same_before = __reduce_add_sync(kAll, lane < warp ? equal[lane] : 0u);
    if (cluster > 1) {
        if (tid == kThreads - 32) {  // the last warp knows the sums
            totals[0] = up_before + up;
            totals[1] = same_before + same;
        }
        cluster_sync();
        const uint32_t u = lane < rank ? remote_u32(smem_u32(&totals[0]), lane) : 0u;
        const uint32_t s = lane < rank ? remote_u32(smem_u32(&totals[1]), lane) : 0u;
        up_before += __reduce_add_sync(kAll, u);
        same_before += __reduce_add_sync(kAll, s);
    }
    const uint32_t base = before[0], gone = before[1];
    if (rank == 0 && tid == 0) {
        if (b == 0) a.new_indptr[0] = 0;
        a.new_indptr[b + 1] = (int)(base + kept);
        if (base + kept > (uint32_t)a.total_new || (a.evicted && gone + (N - kept) > (uint32_t)a.total_evicted)) latch(a.err, DDT_DEVERR_KV_INDPTR);
    }
    const uint32_t lanes = (1u << lane) - 1u;
#pragma unroll 2
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < r1;
        const int slot = in ? a.kv_indices[kv0 + c0 + i] : 0;
        const float x = in ? w[i] : 0.f;
        const uint32_t k = in ? key(i) : 0u;
        const uint32_t ups = __ballot_sync(kAll, in && k > prefix), sames = __ballot_sync(kAll, in && k == prefix);
        const uint32_t u = up_before + __popc(ups & lanes), s = same_before + __popc(sames & lanes);
        const uint32_t stayed = u + min(s, left);  // of the request's columns before this one
        if (in && (k > prefix || (k == prefix && s < left))) {
            const uint32_t to = base + stayed;
            if (to < (uint32_t)a.total_new) {
                a.new_indices[to] = slot;
                if (a.new_weights) a.new_weights[to] = x;
            }
        } else if (in && a.evicted) {
            const uint32_t to = gone + c0 + i - stayed;
            if (to < (uint32_t)a.total_evicted) a.evicted[to] = slot;
        }
        up_before += __popc(ups);
        same_before += __popc(sames);
    }
    if (cluster > 1) cluster_sync();  // no CTA leaves while another one reads its counts
}

int cluster_of(int max_kv_len) {
    int c = 1;
    while (c < 8 && (int64_t)c * kColumnsOfCta < max_kv_len) c *= 2;
    return c;
}

}  // namespace

cudaError_t evict_prepare_device() {
    return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
}

cudaError_t launch_cache_evict(const EvictArgs &a, cudaStream_t s) {
    EvictParams prm;
    prm.a = a;
    prm.cluster = cluster_of(a.max_kv_len);
    const int64_t per = (((int64_t)a.max_kv_len + prm.cluster - 1) / prm.cluster + 31) & ~31;
    prm.keys = (int)std::min<int64_t>(per, kMostKeys);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(prm.cluster * a.batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)prm.keys * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)prm.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = prm.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, prm);
}

}  // namespace ddt
